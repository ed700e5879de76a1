"""The learned operators at the ends of their documented ranges: offsets past 2^31 elements, the widest
rows, the longest sequences, the largest matrices."""
import math

import pytest
import torch

from tests.test_gpu_attention import BF16, F32, U

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")


def room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def grad_ws(n, rows, d):
    return torch.empty(gm.gnn_embedding_grad_workspace_size(n, rows, d), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("d", [2 ** 24, 2 ** 24 - 3])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_widest_rows(d, dtype):
    """Sums of at most two values are exact to one rounding, whatever their order."""
    table = torch.randn(2, d, device="cuda", dtype=dtype)
    ids = torch.tensor([1, 0, 1], dtype=torch.int32, device="cuda")
    out = torch.full((3, d), math.nan, device="cuda", dtype=dtype)
    gm.gnn_embedding_lookup(table, ids, 2.0, out)
    assert torch.equal(out, 2 * table[ids.long()])
    dout = torch.randn(3, d, device="cuda", dtype=dtype)
    want = torch.stack([dout[1].float(), dout[0].float() + dout[2].float()])
    grad = torch.full((2, d), math.nan, device="cuda")
    gm.gnn_embedding_grad(ids, dout, 1.0, grad, grad_ws(3, 2, d))
    assert torch.equal(grad, want)
    grad.fill_(math.nan)
    uniq = torch.empty(2, dtype=torch.int32, device="cuda")
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    gm.gnn_embedding_grad_rows(ids, dout, 1.0, 2, uniq, count, grad, grad_ws(3, 2, d))
    assert torch.equal(grad, want) and uniq.tolist() == [0, 1] and count.item() == 2


@pytest.mark.parametrize("n", [40, 20_000])
def test_gradients_of_a_large_table(n):
    """Rows past 2^31 elements, written and added to."""
    rows, d = 17_000_001, 128
    room(12)
    ids = torch.randint(rows, (n,), dtype=torch.int32, device="cuda")
    ids[:3] = torch.tensor([rows - 1, 0, rows - 1], dtype=torch.int32)
    dout = torch.randn(n, d, device="cuda", dtype=BF16)
    grad = torch.full((rows, d), math.nan, dtype=BF16, device="cuda")
    ws = grad_ws(n, rows, d)
    gm.gnn_embedding_grad(ids, dout, 1.0, grad, ws)
    named, place, count = torch.unique(ids.long(), return_inverse=True, return_counts=True)
    want = torch.zeros(len(named), d, dtype=torch.float64, device="cuda").index_add_(0, place, dout.double())
    size = torch.zeros_like(want).index_add_(0, place, dout.double().abs())
    got = grad[named].double()
    assert torch.all((got - want).abs() <= (count[:, None] + 2) * U * size + 2.0 ** -8 * want.abs() * 1.001)
    grad[named] = 0
    assert all(not torch.any(part) for part in grad.split(1_000_000))
    gm.gnn_embedding_grad(ids, dout, 1.0, grad, ws, accumulate=True)
    assert torch.equal(grad[named].double(), got)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_sequence_of_some_million_states(dtype):
    """17 million states of 128: offsets past 2^31 elements.  All scores are zero but of a few states near
    the end, in the middle and at the start, which take all weight: exp(-60) of the others is nothing."""
    nk, d = 17_000_123, 128
    room(30)
    k = torch.zeros(nk, 1, d, device="cuda", dtype=dtype)
    v = torch.ones(nk, 1, d, device="cuda", dtype=dtype)
    at = torch.tensor([0, 1, 8_500_000, 16_777_217, nk - 1], device="cuda")
    k[at, 0, 0] = 60.0
    v[at] = torch.randn(5, 1, d, device="cuda").to(dtype)
    q = torch.zeros(3, 1, d, device="cuda", dtype=dtype)
    q[:, 0, 0] = 1.0
    q[2] = 0
    qp, kp = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (3, nk))
    ws = torch.empty(gm.gnn_cross_attention_workspace_size(1, 3, nk, 3, nk, 1, 1, d, dtype, True),
                     dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty(3, 1, device="cuda")
    gm.gnn_cross_attention(q, k, v, qp, kp, 3, nk, 1.0, out, ws, lse=lse)
    half = torch.finfo(dtype).eps / 2
    # five equal weights of 1/5 (a rounding each, and of five sums); the others' 17e6 exp(-60) is below u
    want = v[at, 0].double().mean(0)
    tol = (half + 16 * U) * v[at, 0].double().abs().mean(0) + half * want.abs()
    assert torch.all((out[:2, 0].double() - want).abs() <= tol)
    assert torch.all((lse[:2, 0].double() - (60 + math.log(5))).abs() <= 8 * U * 64)
    # equal weights of everything: the splits' sums are of 2^18 ones at most each, exact, and v is one
    # but for five rows
    want = (nk - 5 + v[at, 0].double().sum(0)) / nk
    assert torch.all((out[2, 0].double() - want).abs() <= half * 1.01 + 2.0 ** -12)
    assert abs(float(lse[2, 0]) - math.log(nk)) <= 2.0 ** -12
    dout = torch.randn(3, 1, d, device="cuda").to(dtype)
    dout[2] = 0
    dq, dk, dv = torch.empty_like(q), torch.full_like(k, math.nan), torch.full_like(v, math.nan)
    gm.gnn_cross_attention_backward(q, k, v, qp, kp, 3, nk, 1.0, out, lse, dout, dq, dk, dv, ws)
    want = dout[:2, 0].double().sum(0) / 5
    tol = 1.1 * ((2.0 ** -16 + 2 * 64 * 16 * U) * dout[:2, 0].double().abs().sum(0) / 5 + half * want.abs())
    assert torch.all((dv[at, 0].double() - want).abs() <= tol)
    dv[at] = 0
    assert float(dv.abs().max()) <= 1e-20 and not torch.isnan(dk).any()


def test_largest_matrices():
    """32768 x 32768, one step, some columns against 64 bits: (c0 I + c1 A + c2 A^2) Y of X's columns Y by
    products with X.  The norm is a sum over everything."""
    room(60)
    s = 32768
    c = (3.4445, -4.7750, 2.0315)
    # singular values that matter: some strong directions
    g = torch.randn(s, 16, device="cuda") @ torch.randn(16, s, device="cuda")
    g += 0.1 * torch.randn(s, s, device="cuda")
    out = torch.empty_like(g)
    ws = torch.empty(gm.gnn_orthogonalize_workspace_size(1, s, s, F32), dtype=torch.uint8, device="cuda")
    gm.gnn_orthogonalize(g, out, ws, steps=1)
    del ws
    norm = sum(float(part.double().square().sum()) for part in g.split(1024)) ** 0.5 + 1e-7
    columns = torch.tensor([0, 1, 63, 64, 16384, 20000, s - 2, s - 1], device="cuda")

    def times(transposed, y):         # X y or X^T y
        if transposed:
            return sum(part.double().T.contiguous() @ y[i * 1024:(i + 1) * 1024]
                       for i, part in enumerate(g.split(1024))) / norm
        return torch.cat([part.double() @ y for part in g.split(1024)]) / norm

    y = g[:, columns].double() / norm
    ay = times(False, times(True, y))
    want = c[0] * y + c[1] * ay + c[2] * times(False, times(True, ay))
    off = (out[:, columns].double() - want).norm()
    # 22 bits of X, A and Q, and sums of 2^15 terms in 32 bits (2^7.5 u on average), of three products
    assert off <= (3 * 8 * 2.0 ** -22 + 3 * 8 * 2.0 ** 7.5 * U) * float(want.norm())
