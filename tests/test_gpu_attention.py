"""gnn_cross_attention and its backward pass against the formulas in 64 bits.

Tolerances are first-order bounds of the roundings, element by element, with u = 2^-24 and r the
half step of bf16 (2^-8; 0 for fp32).  A score is off by e = (d + 6) u scale sum |q||k| (the dot
product, the scale, the exponent's argument); a weight P by its own share of eta = 2 e + (n + 8) u,
and r where it is rounded to multiply v; dP by (d + 1) u sum |dout||v|; D by what the stored out is
off, times |dout|; dS by all of them and r; and every sum of m terms by m u of its terms' sizes.
Numbers below 2^-126 are zeros in 32 bits: a weight is off by that much whatever its size, which the
bounds in relative terms alone would deny."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")

F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24
TINY = 2.0 ** -126


def formulas(q, k, v, dout, scale, r):
    """One sequence and one state head in float64: q, dout [m, d] (the rows of all heads that share the
    states), k, v [n, d].  Returns {name: (value, bound before the last rounding)}."""
    m, d = q.shape
    n = k.shape[0]
    if n == 0:
        zero = torch.zeros(m, d, dtype=torch.float64)
        res = {"out": (zero, zero), "lse": (torch.full((m,), -math.inf).double(), torch.zeros(m).double())}
        if dout is not None:
            none = torch.zeros(0, d, dtype=torch.float64)
            res.update(dq=(zero, zero), dk=(none, none), dv=(none, none))
        return res
    s = scale * (q @ k.T)
    size = abs(scale) * (q.abs() @ k.abs().T)
    e = (d + 6) * U * size.amax(1, keepdim=True)
    lse = torch.logsumexp(s, 1, keepdim=True)
    p = torch.exp(s - lse)
    eta = 2 * e + (n + 8) * U
    out = p @ v
    out_err = ((eta + r) * (p @ v.abs()) + TINY * (1 + v.abs().sum(0))) * 1.1
    lse_err = (e + (n + 4) * U + 4 * U * lse.abs()) * 1.1
    res = {"out": (out, out_err), "lse": (lse[:, 0], lse_err[:, 0])}
    if dout is None:
        return res
    stored = out_err + out.abs() * (r + U)
    dd = (dout * out).sum(1, keepdim=True)
    dd_err = (dout.abs() * stored).sum(1, keepdim=True) + (d + 1) * U * (dout * out).abs().sum(1, keepdim=True)
    dp = dout @ v.T
    dp_err = (d + 1) * U * (dout.abs() @ v.abs().T)
    eta = eta + lse_err
    ds = p * (dp - dd)
    ds_err = (eta + r + 2 * U) * ds.abs() + p * (dp_err + dd_err) + TINY * (1 + (dp - dd).abs())
    a = abs(scale)
    res["dq"] = (scale * ds @ k, 1.1 * a * (ds_err @ k.abs() + (n + 2) * U * (ds.abs() @ k.abs())))
    res["dk"] = (scale * ds.T @ q, 1.1 * a * (ds_err.T @ q.abs() + (m + 2) * U * (ds.abs().T @ q.abs())))
    p_err = (eta + r) * p + TINY
    res["dv"] = (p.T @ dout, 1.1 * (p_err.T @ dout.abs() + (m + 2) * U * (p.T @ dout.abs())))
    return res


def tensor(rows, heads, d, dtype, seed, size=1.0):
    g = torch.Generator().manual_seed(seed)
    return (size * torch.randn(rows, heads, d, generator=g)).to(dtype)


def indptr(lengths):
    return torch.tensor([0] + list(lengths)).cumsum(0).to(torch.int32)


class Call:
    """Inputs on the host, and what the kernels give for them."""

    def __init__(self, nq, nk, heads, kv, d, dtype, scale=None, size=1.0, count=None, seed=0):
        self.nq, self.nk, self.heads, self.kv, self.d, self.dtype = nq, nk, heads, kv, d, dtype
        self.scale = d ** -0.5 if scale is None else scale
        self.q = tensor(sum(nq), heads, d, dtype, seed + 1, size)
        self.k = tensor(sum(nk), kv, d, dtype, seed + 2, size)
        self.v = tensor(sum(nk), kv, d, dtype, seed + 3)
        self.dout = tensor(sum(nq), heads, d, dtype, seed + 4)
        self.count = count

    def run(self, backward=True, stream=None, max_q=None, max_k=None):
        c = lambda t: t.cuda()
        q, k, v, g = c(self.q), c(self.k), c(self.v), c(self.dout)
        qp, kp = c(indptr(self.nq)), c(indptr(self.nk))
        mq = max(self.nq + [0]) if max_q is None else max_q
        mk = max(self.nk + [0]) if max_k is None else max_k
        count = None if self.count is None else torch.tensor(self.count, device="cuda")
        ws = torch.full((gm.gnn_cross_attention_workspace_size(
            len(self.nq), len(q), len(k), mq, mk, self.heads, self.kv, self.d, self.dtype,
            backward),), 0xFF, dtype=torch.uint8, device="cuda")
        nan = lambda t: torch.full_like(t, math.nan)
        out, lse = nan(q), torch.full((len(q), self.heads), math.nan, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        common = dict(k_count=count, d_status=status, stream=stream)
        torch.cuda.synchronize()
        gm.gnn_cross_attention(q, k, v, qp, kp, mq, mk, self.scale, out, ws, lse=lse, **common)
        res = {"out": out, "lse": lse}
        if backward:
            dq, dk, dv = nan(q), nan(k), nan(v)
            gm.gnn_cross_attention_backward(q, k, v, qp, kp, mq, mk, self.scale, out, lse, g, dq, dk,
                                            dv, ws, **common)
            res.update(dq=dq, dk=dk, dv=dv)
        torch.cuda.synchronize()
        self.status = int(status.item())
        return {x: y.cpu() for x, y in res.items()}

    def check(self, got, backward=True):
        r = torch.finfo(BF16).eps / 2 if self.dtype == BF16 else 0.0
        half = torch.finfo(self.dtype).eps / 2
        qp, kp = indptr(self.nq).tolist(), indptr(self.nk).tolist()
        group = self.heads // self.kv
        scale = float(torch.tensor(self.scale, dtype=F32))
        for b in range(len(self.nq)):
            i = slice(qp[b], qp[b + 1])
            n = self.nk[b] if self.count is None else min(max(self.count[b], 0), self.nk[b])
            j, rest = slice(kp[b], kp[b] + n), slice(kp[b] + n, kp[b + 1])
            for h in range(self.kv):
                hs = slice(h * group, (h + 1) * group)
                rows = lambda t: t[i, hs].double().reshape(-1, self.d)
                ref = formulas(rows(self.q), self.k[j, h].double(), self.v[j, h].double(),
                               rows(self.dout) if backward else None, scale, r)
                for name, (want, bound) in ref.items():
                    if name == "lse":
                        have, step = got["lse"][i, hs].double().reshape(-1), 0.0
                    elif name in ("dk", "dv"):
                        have, step = got[name][j, h].double(), half
                        assert torch.all(got[name][rest, h] == 0), (b, h, name)
                    else:
                        have, step = got[name][i, hs].double().reshape(-1, self.d), half
                    if name == "lse" and n == 0:
                        assert torch.all(have == -math.inf)
                        continue
                    tol = bound + step * (want.abs() + bound)
                    bad = ~((have - want).abs() <= tol)
                    assert not bad.any(), (b, h, name, int(bad.sum()), float((have - want).abs().max()),
                                           float(tol.max()))


CASES = [
    ([1], [1], 1, 1, 8), ([1], [0], 2, 1, 16), ([0, 3], [5, 0], 2, 2, 24),
    ([3, 0, 1, 7], [33, 64, 1, 0], 4, 2, 32), ([31, 33, 32], [63, 65, 64], 2, 1, 64),
    ([1, 1, 1], [700, 1, 2049], 8, 2, 128), ([5], [1500], 12, 2, 80), ([130, 257], [129, 40], 4, 4, 72),
    ([128], [128], 4, 1, 128), ([300, 2], [31, 900], 6, 3, 40), ([700], [20], 8, 1, 104),
    ([1], [5000], 1, 1, 120), ([2] * 40, [17, 3] * 20, 4, 4, 48),
]


@pytest.mark.parametrize("nq,nk,heads,kv,d", CASES)
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_forward_and_backward(nq, nk, heads, kv, d, dtype):
    c = Call(nq, nk, heads, kv, d, dtype, seed=d)
    got = c.run()
    assert c.status == gm.GNN_OK
    c.check(got)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [1e-3, 8.0])
def test_flat_and_peaked_weights(size, dtype):
    """Nearly equal weights, and scores of some hundreds, where one state takes all."""
    c = Call([40, 3], [300, 70], 4, 2, 64, dtype, size=size, seed=7)
    c.check(c.run())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_other_scales(dtype):
    for scale in (0.0, -0.3, 1.0):
        c = Call([20], [90], 2, 2, 16, dtype, scale=scale, seed=9)
        c.check(c.run())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nq", [[9, 9, 9, 9], [90, 90, 90, 90]])
def test_counts_leave_states_out(nq, dtype):
    """States past the count hold infinities and NaN; counts of zero, negative and too large."""
    c = Call(nq, [100, 64, 40, 300], 4, 2, 64, dtype, count=[61, 0, -3, 10 ** 12], seed=11)
    at = indptr(c.nk).tolist()
    for lo, hi in ((at[0] + 61, at[1]), (at[1], at[2]), (at[2], at[3])):
        c.k[lo:hi], c.v[lo:hi] = math.nan, math.inf
    got = c.run()
    assert c.status == gm.GNN_OK
    c.check(got)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_neighbours_do_not_leak(dtype):
    """A sequence of NaN and infinities leaves the sequences beside it as they are."""
    clean = Call([4, 5, 6], [70, 50, 90], 4, 2, 64, dtype, seed=13)
    bad = Call([4, 5, 6], [70, 50, 90], 4, 2, 64, dtype, seed=13)
    bad.k[70:120], bad.v[70:120] = math.nan, math.inf
    bad.q[4:9], bad.dout[4:9] = math.inf, math.nan
    a, b = clean.run(), bad.run()
    for name in a:
        lo, hi = (70, 120) if name in ("dk", "dv") else (4, 9)
        assert torch.equal(a[name][:lo], b[name][:lo]) and torch.equal(a[name][hi:], b[name][hi:]), name


def test_minus_infinity_scores():
    """A state whose score is -inf has no weight; a row whose scores all are has no weights at all."""
    c = Call([2], [40], 1, 1, 16, F32, scale=1.0, seed=15)
    c.q[:] = 0.0
    c.q[:, 0, 0] = 1.0
    c.k[3, 0, 0] = -math.inf
    got = c.run()
    assert torch.isfinite(got["out"]).all()
    c.k[:, 0, 0] = -math.inf
    got = c.run()
    assert torch.all(got["out"] == 0) and torch.all(got["lse"] == -math.inf)
    assert torch.all(got["dv"] == 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nq", [3, 200])
def test_all_scores_far_below_zero(nq, dtype):
    """lse near -600: what lies past a sequence's end has a score of zero, far above it."""
    c = Call([nq, nq], [45, 7], 2, 1, 32, dtype, scale=1.0, seed=31)
    c.q[:, :, 0], c.k[:, :, 0] = 25.0, -25.0
    c.check(c.run())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_infinite_states_stay_in_their_rows_and_gradients(dtype):
    """A state of -inf scores (its weight is zero), with a row count that ends inside a tile."""
    c = Call([5], [70], 1, 1, 16, dtype, scale=1.0, seed=33)
    c.q[:, 0, 0] = 1.0
    c.k[9, 0, 0] = -math.inf
    got = c.run()
    assert torch.isfinite(got["out"]).all() and torch.isfinite(got["dv"]).all()
    assert torch.all(got["dv"][9] == 0)
    assert torch.isfinite(got["dk"]).all() and torch.all(got["dk"][9] == 0)


def test_same_bits_every_time_and_other_bounds():
    c = Call([1, 60], [3000, 1200], 8, 2, 64, BF16, seed=17)
    a, b = c.run(), c.run()
    for x in a:
        assert torch.equal(a[x], b[x]), x
    c.check(c.run(max_q=500, max_k=10_000))       # looser host bounds: another plan


def test_strided_rows():
    """k and v as halves of one projection, q and out as columns of wider rows."""
    c = Call([7, 40], [90, 33], 4, 2, 32, BF16, seed=19)
    want = c.run()
    kv = torch.empty(123, 4, 32, dtype=BF16, device="cuda")
    kv[:, :2], kv[:, 2:] = c.k.cuda(), c.v.cuda()
    q = torch.full((47, 6, 32), math.nan, dtype=BF16, device="cuda")
    q[:, 1:5] = c.q.cuda()
    out = torch.full((47, 5, 32), 3.0, dtype=BF16, device="cuda")
    qp, kp = indptr(c.nq).cuda(), indptr(c.nk).cuda()
    ws = torch.empty(gm.gnn_cross_attention_workspace_size(2, 47, 123, 40, 90, 4, 2, 32, BF16, True),
                     dtype=torch.uint8, device="cuda")
    lse = torch.empty(47, 4, device="cuda")
    gm.gnn_cross_attention(q[:, 1:5], kv[:, :2], kv[:, 2:], qp, kp, 40, 90, c.scale, out[:, :4], ws,
                           lse=lse)
    assert torch.equal(out[:, :4].cpu(), want["out"]) and torch.all(out[:, 4] == 3.0)
    dkv = torch.empty_like(kv)
    dq = torch.full_like(out, 5.0)
    gm.gnn_cross_attention_backward(q[:, 1:5], kv[:, :2], kv[:, 2:], qp, kp, 40, 90, c.scale,
                                    out[:, :4], lse, c.dout.cuda(), dq[:, :4], dkv[:, :2], dkv[:, 2:], ws)
    assert torch.equal(dq[:, :4].cpu(), want["dq"]) and torch.all(dq[:, 4] == 5.0)
    assert torch.equal(dkv[:, :2].cpu(), want["dk"]) and torch.equal(dkv[:, 2:].cpu(), want["dv"])


def test_bad_indptr_and_bounds_are_reported():
    c = Call([6, 6], [50, 50], 2, 1, 32, F32, seed=21)
    c.run(max_q=5)
    assert c.status == gm.GNN_ERR_CAPACITY
    c.run(max_k=49)
    assert c.status == gm.GNN_ERR_CAPACITY
    q, k = c.q.cuda(), c.k.cuda()
    out, lse = torch.zeros_like(q), torch.empty(12, 2, device="cuda")
    ws = torch.empty(gm.gnn_cross_attention_workspace_size(2, 12, 100, 12, 100, 2, 1, 32, F32),
                     dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for qp, kp in (([0, 7, 6], [0, 50, 100]), ([0, 6, 13], [0, 50, 100]), ([-1, 6, 12], [0, 50, 100]),
                   ([0, 6, 12], [0, 101, 100]), ([0, 6, 12], [-5, 50, 100])):
        status.zero_()
        gm.gnn_cross_attention(q, k, k, torch.tensor(qp, dtype=torch.int32, device="cuda"),
                               torch.tensor(kp, dtype=torch.int32, device="cuda"), 12, 100, 1.0, out,
                               ws, lse=lse, d_status=status)
        assert status.item() == gm.GNN_ERR_OUT_OF_RANGE, (qp, kp)


def test_rows_of_no_sequence_stay():
    c = Call([4, 4], [30, 30], 2, 2, 16, F32, seed=23)
    q, k, v = c.q.cuda(), c.k.cuda(), c.v.cuda()
    qp = torch.tensor([2, 4, 6], dtype=torch.int32, device="cuda")
    kp = torch.tensor([10, 30, 50], dtype=torch.int32, device="cuda")
    out, lse = torch.full_like(q, 7.0), torch.full((8, 2), 7.0, device="cuda")
    dq, dk, dv = torch.full_like(q, 7.0), torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    ws = torch.empty(gm.gnn_cross_attention_workspace_size(2, 8, 60, 2, 20, 2, 2, 16, F32, True),
                     dtype=torch.uint8, device="cuda")
    gm.gnn_cross_attention(q, k, v, qp, kp, 2, 20, 0.25, out, ws, lse=lse)
    gm.gnn_cross_attention_backward(q, k, v, qp, kp, 2, 20, 0.25, out, lse, q, dq, dk, dv, ws)
    for t, lo, hi in ((out, 2, 6), (lse, 2, 6), (dq, 2, 6), (dk, 10, 50), (dv, 10, 50)):
        assert torch.all(t[:lo] == 7.0) and torch.all(t[hi:] == 7.0) and not torch.any(t[lo:hi] == 7.0)


@pytest.mark.parametrize("which", ["q", "k", "v"])
def test_gradient_against_differences(which):
    """(f(x + h e) - f(x - h e)) / 2h of f = sum out * dout by the kernels, against their gradient.
    The truncation is what the same difference of the formulas in 64 bits shows; each f is a sum of
    values that are off by at most the forward pass's bound."""
    h = 2.0 ** -6
    c = Call([5, 30], [40, 70], 4, 2, 32, F32, seed=25)
    grad = c.run()["d" + which].double()
    x = getattr(c, which).clone()
    e = tensor(*x.shape, F32, 99)
    exact, seen, slack = [], [], 0.0
    group = 2
    for sign in (1, -1):
        setattr(c, which, (x.double() + sign * h * e.double()).float())
        out = c.run(backward=False)["out"].double()
        seen.append(float((out * c.dout.double()).sum()))
        f = 0.0
        qp, kp = indptr(c.nq).tolist(), indptr(c.nk).tolist()
        for b in range(2):
            i, j = slice(qp[b], qp[b + 1]), slice(kp[b], kp[b + 1])
            for s in range(2):
                hs = slice(s * group, (s + 1) * group)
                rows = lambda t: t[i, hs].double().reshape(-1, 32)
                value, err = formulas(rows(c.q), c.k[j, s].double(), c.v[j, s].double(), None,
                                      float(torch.tensor(c.scale, dtype=F32)), 0.0)["out"]
                f += float((value * rows(c.dout)).sum())
                slack += float(((err + U * value.abs()) * rows(c.dout).abs()).sum())
        exact.append(f)
    setattr(c, which, x)
    along = float((grad * e.double()).sum())
    truth = (exact[0] - exact[1]) / (2 * h)
    # the gradient of the formulas along e
    ref = 0.0
    for b in range(2):
        i, j = slice(qp[b], qp[b + 1]), slice(kp[b], kp[b + 1])
        for s in range(2):
            hs = slice(s * group, (s + 1) * group)
            rows = lambda t: t[i, hs].double().reshape(-1, 32)
            value, err = formulas(rows(c.q), c.k[j, s].double(), c.v[j, s].double(), rows(c.dout),
                                  float(torch.tensor(c.scale, dtype=F32)), 0.0)["d" + which]
            d = rows(e) if which == "q" else e[j, s].double()
            ref += float((value * d).sum())
            slack += 2 * h * float(((err + U * value.abs()) * d.abs()).sum())
    assert abs((seen[0] - seen[1]) / (2 * h) - along) <= abs(truth - ref) + slack / (2 * h)


def test_on_another_stream_and_in_a_graph():
    c = Call([1, 40, 3], [900, 200, 77], 4, 2, 64, BF16, seed=27)
    want = c.run()
    got = c.run(stream=torch.cuda.Stream())
    for x in want:
        assert torch.equal(want[x], got[x]), x
    q, k, v, g = c.q.cuda(), c.k.cuda(), c.v.cuda(), c.dout.cuda()
    qp, kp = indptr(c.nq).cuda(), indptr(c.nk).cuda()
    ws = torch.empty(gm.gnn_cross_attention_workspace_size(3, 44, 1177, 40, 900, 4, 2, 64, BF16, True),
                     dtype=torch.uint8, device="cuda")
    lse = torch.empty(44, 4, device="cuda")
    out, dq, dk, dv = (torch.empty_like(t) for t in (q, q, k, v))

    def step():
        gm.gnn_cross_attention(q, k, v, qp, kp, 40, 900, c.scale, out, ws, lse=lse)
        gm.gnn_cross_attention_backward(q, k, v, qp, kp, 40, 900, c.scale, out, lse, g, dq, dk, dv, ws)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for turn in range(3):
        q.copy_(tensor(44, 4, 64, BF16, 50 + turn))
        step()
        want = [t.clone() for t in (out, lse, dq, dk, dv)]
        for t in (out, lse, dq, dk, dv):
            t.fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((out, lse, dq, dk, dv), want):
            assert torch.equal(x, y)
