"""The orthogonalised update on tiles of 128, with split sums and their join, and
the one-workgroup kernels, against 64 bits with a tolerance that sees a lost part.

Relative to the result's norm, five default steps.  Each factor is rounded to 22
bits; in an emulation with exact sums (64 x 128 to 870 x 2070) all of that leaves
2^-20.3, the roundings' own 2^-23.8 (half a step of 22 bits over sqrt 3) ten times.
fp32's sums add 3 K / 32 terms, half a step each and independent: at most
sqrt(3 * 4096 / 32) 2^-24 = 2^-19.7 of a product, ten times that is 2^-16.4 at the
end.  Both together stay below 2^-16 (the emulation without one of the three
products of parts: 2^-12.8 at least).  16-bit results add half a step."""
import pytest
import torch

import net_refs as R
from test_gpu_net_ortho import TRIPLE, matrices

pytestmark = pytest.mark.gpu
TOL = 2.0 ** -16


def wanted(m, triples):
    """In 64 bits, where m lies."""
    x = m.double()
    x = x / x.square().sum((-1, -2), keepdim=True).sqrt()
    tall = x.shape[-2] > x.shape[-1]
    x = x.transpose(-1, -2).contiguous() if tall else x
    for a, b, c in triples:
        gram = x @ x.transpose(-1, -2).contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(-1, -2) if tall else x


def near(m, got, triples):
    for one, x in zip(m, got):
        assert R.rel(x, wanted(one, triples)) < TOL + R.half_step(m.dtype)


@pytest.mark.parametrize("count, rows, cols", [
    (3, 870, 2070), (3, 2070, 870),     # A on tiles of 128 in three splits; X at odd edges
    (1, 1024, 4096), (1, 4096, 1024),   # seven splits, of unlike lengths
    (20, 520, 520), (20, 600, 520),     # all three on tiles of 128, without splits
    (1, 2500, 2500),                    # 210 lower tiles, mirrored
    (2, 1403, 515), (1, 96, 4096), (1, 4096, 96), (1, 320, 4096), (5, 129, 130)])
@pytest.mark.parametrize("kind", ["fp32", "fp16", "bf16"])
def test_large_matrices(count, rows, cols, kind):
    import krylov_solvers_adjoint_amd as K
    m = matrices(count, rows, cols, R.TYPES[kind]).cuda()
    got = K.orthogonalise(m)
    near(m, got, [TRIPLE] * 5)
    assert torch.equal(K.orthogonalise(m), got)


@pytest.mark.parametrize("rows, cols", [(1024, 4096), (4096, 1024), (1300, 1300)])
def test_large_matrices_one_step_and_other_coefficients(rows, cols):
    """A single step, whose terms are not yet damped by those that follow."""
    import krylov_solvers_adjoint_amd as K
    m = matrices(1, rows, cols, torch.float32).cuda()
    for triples in ([TRIPLE], [(3.0, -3.5, 1.4), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]):
        near(m, K.orthogonalise(m, len(triples), triples), triples)


@pytest.mark.parametrize("rows, cols", [(128, 128), (100, 127), (127, 100), (64, 512), (512, 64),
                                        (128, 64), (64, 128), (20, 400), (400, 20), (513, 64),
                                        (64, 513), (16, 16), (33, 70)])
def test_one_workgroup_and_its_neighbours(rows, cols):
    import krylov_solvers_adjoint_amd as K
    m = matrices(3, rows, cols, torch.float32).cuda()
    got = K.orthogonalise(m)
    near(m, got, [TRIPLE] * 5)
    assert torch.equal(K.orthogonalise(m), got)


def test_large_views_graphs_and_streams():
    """Rows further apart than they are long; replayed beside another call of the same size."""
    import krylov_solvers_adjoint_amd as K
    base = matrices(1, 1024, 4200, torch.bfloat16).cuda()
    m = base[:, :, 9:4105]
    want = K.orthogonalise(m.contiguous())
    assert torch.equal(K.orthogonalise(m), want)
    other = matrices(1, 1024, 4096, torch.bfloat16, seed=3).cuda()
    beside_want = K.orthogonalise(other)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        K.orthogonalise(m)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = K.orthogonalise(m)
    for k in range(3):
        base.copy_(matrices(1, 1024, 4200, torch.bfloat16, seed=10 + k))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            beside = K.orthogonalise(other)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, K.orthogonalise(m)) and torch.equal(beside, beside_want)


def test_a_large_matrix_that_is_not_finite_leaves_the_others():
    import krylov_solvers_adjoint_amd as K
    m = matrices(3, 870, 2070, torch.float32).cuda()
    want = K.orthogonalise(m)
    m[1, 869, 2069] = float("nan")
    got = K.orthogonalise(m)
    assert got[1].isnan().all()
    assert torch.equal(got[0], want[0]) and torch.equal(got[2], want[2])
