"""What the projection's work call says of workspaces and limits, on the CPU."""
import ctypes

import pytest

import krylov_solvers_adjoint_amd as K

lib = K._lib
P = 256  # an address that is never followed


def sizes(rows, inner, outer, kind, act):
    f, n = K._I64(), K._I64()
    assert lib.sla_linear_work(rows, inner, outer, kind, act, ctypes.byref(f),
                               ctypes.byref(n)) == K.OK
    return f.value, n.value


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("inner, outer", [(4096, 1024), (4096, 4096), (200000, 64), (64, 64)])
def test_few_rows_ask_for_no_split_sums(inner, outer, kind):
    """Up to 64 rows are one launch that keeps its sums on the chip."""
    for rows in (1, 4, 16, 33, 64):
        assert sizes(rows, inner, outer, kind, 3)[0] == 0
    assert sizes(65, 200000, 64, kind, 3)[0] > 0


def test_the_last_rows_below_2_to_the_31():
    """A launch of 2^32 threads does not exist: the work call refuses what the launch would."""
    rows = 2 ** 31 - 128
    assert sizes(rows, 8, 16, 2, 0)[1] > 0 and sizes(rows, 96, 16, 2, 0)[1] > rows
    for more in (rows + 1, 2 ** 31 - 1):
        assert lib.sla_linear_work(more, 8, 16, 2, 0, None, None) == K.ERR_ARG
        assert lib.sla_last_error().decode().startswith("sla_linear_work: rows")
        assert lib.sla_linear(P, 8, P, None, 2, None, 0, more, 8, 16, 2, 0, P, P, 1 << 60,
                              None) == K.ERR_ARG
