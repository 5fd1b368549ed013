"""What the projection's work call says of workspaces and limits, on the CPU."""
import ctypes

import pytest

import krylov_solvers_adjoint_amd as K

lib = K._lib


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
