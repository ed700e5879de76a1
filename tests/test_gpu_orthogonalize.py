"""gnn_orthogonalize against the steps in 64 bits.

Tolerance: the kernels keep X, A = X X^T and Q = a I + b A + c A^2 in fp16 planes (11 bits for bf16
updates, 22 for fp32) and sum in fp32.  The same steps on the host, with matrix products in fp32 and
X, A, Q rounded to such planes, are some distance from the 64-bit result; the kernels' roundings are
others of the same size, so their distance (2-norm over the matrix) is allowed three times that, and
the rounding of the result to its type (eps / 2) on top."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")

F32, BF16 = torch.float32, torch.bfloat16
QUINTIC = (3.4445, -4.7750, 2.0315)


def steps64(g, steps, coefs=QUINTIC, eps=1e-7):
    x = g.double().cpu()
    x = x / (x.norm() + eps)
    wide = x.shape[0] <= x.shape[1]
    x = x if wide else x.T
    for _ in range(steps):
        a = x @ x.T
        x = coefs[0] * x + (coefs[1] * a + coefs[2] * a @ a) @ x
    return x if wide else x.T


def planes(x, count):
    up = x.double() * 4096
    hi = up.half()
    kept = hi.double()
    if count == 2:
        kept = kept + (up - kept).half().double()
    return (kept / 4096).float()


def rounded_steps(g, steps, coefs=QUINTIC, eps=1e-7):
    count = 2 if g.dtype == F32 else 1
    x = g.double().cpu()
    x = (x / (x.norm() + eps)).float()
    x = x if x.shape[0] <= x.shape[1] else x.T
    for _ in range(steps):
        x = planes(x, count)
        a = planes(x @ x.T, count)
        q = planes(coefs[0] * torch.eye(len(a)) + coefs[1] * a + coefs[2] * (a @ a), count)
        x = q @ x
    return (x if g.shape[0] <= g.shape[1] else x.T).double()


def run(g, steps=5, out=None, **kw):
    b = g.shape[0] if g.dim() == 3 else 1
    m, n = g.shape[-2:]
    ws = torch.full((gm.gnn_orthogonalize_workspace_size(b, m, n, g.dtype),), 0xFF,
                    dtype=torch.uint8, device="cuda")      # NaN everywhere
    out = torch.empty_like(g) if out is None else out
    gm.gnn_orthogonalize(g, out, ws, steps=steps, **kw)
    return out


def check(g, got, steps=5, scale=1.0, coefs=QUINTIC, eps=1e-7):
    for x, y in zip(g.reshape(-1, *g.shape[-2:]), got.reshape(-1, *g.shape[-2:])):
        want = steps64(x, steps, coefs, eps) * scale
        near = rounded_steps(x, steps, coefs, eps) * scale
        tol = 3 * (near - want).norm() + torch.finfo(g.dtype).eps / 2 * want.norm()
        off = (y.double().cpu() - want).norm()
        assert off <= tol, (float(off), float(tol), float(want.norm()))


def gaussian(*shape, seed=0, dtype=F32, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(*shape, generator=g)).to(dtype).cuda()


SHAPES = [(1, 1, 1), (1, 1, 7), (2, 5, 1), (1, 3, 3), (3, 17, 40), (1, 64, 64), (2, 65, 63),
          (1, 130, 200), (1, 200, 130), (1, 256, 256), (4, 128, 300), (1, 300, 1000),
          (1, 1411, 1300), (3, 1025, 700)]


@pytest.mark.parametrize("b,m,n", SHAPES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_steps(b, m, n, dtype):
    g = gaussian(b, m, n, seed=m * n, dtype=dtype, size=1e-3)
    check(g, run(g))


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_number_of_steps_and_scale(steps, dtype):
    g = gaussian(96, 160, seed=steps, dtype=dtype)
    check(g, run(g, steps=steps, scale=0.2), steps=steps, scale=0.2)


@pytest.mark.parametrize("m,n", [(1600, 223), (223, 2400), (960, 160), (320, 1920)])
def test_long_matrices_keep_their_size(m, n):
    """Their eigenvalues are alike, so that rounded factors would scale the result: with 22 bits by some
    2^-21 a step, which the steps' slopes (below 4 each) can make 2^-11 at most; the rounding of the
    result is of either sign."""
    k = n // 8 if n < m else m // 8
    strong = gaussian(m, k, seed=m) @ gaussian(k, n, seed=n)
    g = (strong / math.sqrt(k) + gaussian(m, n, seed=m + n)).to(BF16)
    got, want = run(g).double().cpu(), steps64(g, 5)
    assert abs(float((got * want).sum() / want.square().sum()) - 1) < 1e-4
    check(g, run(g))


def test_low_rank_and_strong_directions():
    a, b = gaussian(200, 4, seed=1), gaussian(4, 333, seed=2)
    g = a @ b + 1e-3 * gaussian(200, 333, seed=3)
    for x in (g, g.to(BF16), (a @ b)):
        check(x, run(x))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [1e-30, 1e-12, 1e25])
def test_size_does_not_matter(size, dtype):
    """The update's size drops out (eps = 0), over the exponents of either type."""
    g = gaussian(70, 90, seed=5, dtype=dtype, size=size)
    check(g, run(g, eps=0.0), eps=0.0)


def test_eps():
    g = gaussian(40, 50, seed=6, size=1e-4)
    check(g, run(g, eps=float(g.norm())), eps=float(g.norm()))


def test_converging_coefficients_orthogonalise():
    """3/2 s - 1/2 s^3 goes to 1 on (0, 1]: the rows become orthonormal."""
    g = gaussian(60, 400, seed=7)
    out = run(g, steps=16, coefs=(1.5, -0.5, 0.0))
    eye = out.double() @ out.double().T
    # singular values of a 60 x 400 Gaussian lie within a factor of 3 of each other and above
    # 1/25 of its norm: ten steps of growth by 3/2 and six of quadratic convergence
    assert float((eye - torch.eye(60, device="cuda")).abs().max()) < 1e-4
    check(g, out, steps=16, coefs=(1.5, -0.5, 0.0))


def test_zero_and_not_finite():
    for dtype in (F32, BF16):
        g = gaussian(3, 50, 70, seed=8, dtype=dtype)
        g[0] = 0
        g[2, 3, 4] = math.inf
        out = run(g)
        assert torch.all(out[0] == 0) and torch.isnan(out[2]).all()
        check(g[1], out[1])
        g[2, 3, 4] = math.nan
        assert torch.isnan(run(g)[2]).all()
        assert torch.all(run(g, eps=0.0)[0] == 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strides_and_in_place(dtype):
    whole = gaussian(3, 33, 101, seed=9, dtype=dtype)
    g = whole[:, 1:30, 2:75]
    into = torch.full((3, 40, 80), 7.0, dtype=dtype, device="cuda")
    out = into[:, 2:31, 3:76]
    want = run(g.contiguous())
    run(g, out=out)
    assert torch.equal(out, want)
    outside = torch.ones(3, 40, 80, dtype=torch.bool)
    outside[:, 2:31, 3:76] = False
    assert torch.all(into.cpu()[outside] == 7.0)
    same = g.contiguous()
    run(same, out=same)
    assert torch.equal(same, want)


def test_batch_equals_single():
    g = gaussian(5, 64, 200, seed=10)
    out = run(g)
    for i in range(5):
        assert torch.equal(run(g[i].contiguous()), out[i])


def test_on_another_stream_and_in_a_graph():
    g = gaussian(2, 150, 260, seed=11, dtype=BF16)
    want = run(g)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    out = torch.empty_like(g)
    ws = torch.empty(gm.gnn_orthogonalize_workspace_size(2, 150, 260, BF16), dtype=torch.uint8,
                     device="cuda")
    gm.gnn_orthogonalize(g, out, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gm.gnn_orthogonalize(g, out, ws)
    for turn in range(3):
        g.copy_(gaussian(2, 150, 260, seed=20 + turn, dtype=BF16))
        want = run(g)
        out.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
