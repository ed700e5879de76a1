"""Gradients of gnn_cross_attention over few states, where P (dP - D) is a small difference of large
numbers.  Helpers and notation as in test_gpu_attention.py; u = 2^-24."""
import math

import pytest
import torch

from tests.test_gpu_attention import BF16, F32, U, Call, formulas, indptr

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nq,heads,kv,d", [([1], 1, 1, 8), ([5, 2, 9], 4, 2, 64), ([1, 1, 1, 1], 8, 2, 40),
                                           ([300, 130, 40], 8, 8, 128), ([33] * 40, 8, 8, 72)])
def test_a_single_state_has_no_gradient_of_its_score(nq, heads, kv, d, dtype):
    """P is 1 whatever q and k are: dq and dk are zero, not roundings of dP - D."""
    c = Call(nq, [1] * len(nq), heads, kv, d, dtype, seed=d)
    got = c.run()
    c.check(got)
    assert torch.all(got["dq"] == 0) and torch.all(got["dk"] == 0)
    assert torch.any(got["dv"] != 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_single_state_beside_others(dtype):
    """By length, and by a count that leaves one state."""
    c = Call([4, 7, 3, 6], [1, 90, 30, 0], 4, 2, 32, dtype, count=[1, 90, 1, 0], seed=41)
    got = c.run()
    c.check(got)
    q, k = indptr(c.nq).tolist(), indptr(c.nk).tolist()
    for b in (0, 2):
        assert torch.all(got["dq"][q[b]:q[b + 1]] == 0) and torch.all(got["dk"][k[b]:k[b + 1]] == 0)
    assert torch.any(got["dq"][q[1]:q[2]] != 0) and torch.any(got["dk"][k[1]:k[2]] != 0)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_single_state_still_shows_what_is_not_finite(dtype):
    c = Call([3], [1], 2, 1, 16, dtype, seed=43)
    c.dout[1, 0, 3] = math.nan
    got = c.run()
    assert torch.isnan(got["dq"][1, 0]).all() and torch.isnan(got["dk"]).all()
    assert torch.all(got["dq"][0] == 0) and torch.all(got["dq"][1, 1] == 0)


@pytest.mark.parametrize("nk", [2, 3, 17, 31, 32])
@pytest.mark.parametrize("nq", [3, 70])
def test_scores_gradients_add_up_to_zero(nq, nk):
    """Where all states have one k, dq = scale k sum_j dS_j = 0.  v is the same up to 2^-12, so dS is far
    smaller than dP and D, whose own roundings (of d products) must drop out of the sum: what may be
    left of it is (n + 8) u of the terms' sizes, twice (the sum, and its correction's), and what the
    weights' sum is off 1 of the correction."""
    d = 64
    c = Call([nq, nq], [nk, nk], 2, 1, d, F32, seed=nk)
    c.k[:] = c.k[:1]
    c.v = 1 + 2.0 ** -12 * c.v
    got = c.run()
    c.check(got)
    scale = c.scale
    for b in range(2):
        q = c.q[b * nq:(b + 1) * nq].double()
        g = c.dout[b * nq:(b + 1) * nq].double()
        k, v = c.k[b * nk:(b + 1) * nk, 0].double(), c.v[b * nk:(b + 1) * nk, 0].double()
        dp = g @ v.T                                     # [nq, heads, nk]
        ds = (dp - dp.mean(2, keepdim=True)).abs().sum(2) / nk
        dp_err = (d + 1) * U * (g.abs() @ v.abs().T).amax(2)
        e = (d + 6) * U * scale * (q.abs() @ k[0].abs())
        eta = 4 * e + (2 * nk + 16) * U
        bound = 2 * (nk + 8) * U * (ds + 2 * dp_err) + eta * 3 * dp_err
        tol = 1.1 * scale * bound[:, :, None] * k[0].abs() + 2.0 ** -126
        assert torch.all(got["dq"][b * nq:(b + 1) * nq].double().abs() <= tol)


def short_formulas(q, k, v, dout, scale):
    """{name: (value, bound before the last rounding)} of one sequence's gradients in bf16 where P and dS
    are multiplied as two bf16 (2^-8 of 2^-8 off): as formulas(), with D from the stored out, or over
    up to 32 states from P dP itself."""
    n, d = k.shape
    m = q.shape[0]
    forward = formulas(q, k, v, None, scale, 2.0 ** -8)
    out, out_err = forward["out"]
    lse_err = forward["lse"][1][:, None]
    s = scale * (q @ k.T)
    size = abs(scale) * (q.abs() @ k.abs().T)
    p = torch.softmax(s, 1)
    r = 2.0 ** -16
    eta = 2 * (d + 6) * U * size.amax(1, keepdim=True) + (n + 8) * U + lse_err
    dp, dp_err = dout @ v.T, (d + 1) * U * (dout.abs() @ v.abs().T)
    dd = (p * dp).sum(1, keepdim=True)
    ds = p * (dp - dd)
    dd_err = (dout.abs() * (out_err + out.abs() * (2.0 ** -8 + U))).sum(1, keepdim=True) + \
        (d + 1) * U * (dout * out).abs().sum(1, keepdim=True)
    if n <= 32:
        dd_err = (p * dp_err).sum(1, keepdim=True) + U * dd.abs() + \
            (eta + (n + 2) * U) * (ds.abs().sum(1, keepdim=True) + dd_err)
    ds_err = (eta + r + 3 * U) * ds.abs() + p * (dp_err + dd_err) + 2.0 ** -126
    p_err = (eta + r) * p + 2.0 ** -126
    a = abs(scale)
    return {"dq": (scale * ds @ k, 1.1 * a * (ds_err @ k.abs() + (n + 2) * U * (ds.abs() @ k.abs()))),
            "dk": (scale * ds.T @ q, 1.1 * a * (ds_err.T @ q.abs() + (m + 2) * U * (ds.abs().T @ q.abs()))),
            "dv": (p.T @ dout, 1.1 * (p_err.T @ dout.abs() + (m + 2) * U * (p.T @ dout.abs())))}


@pytest.mark.parametrize("d", [32, 80, 128])
@pytest.mark.parametrize("nq,nk,heads,kv,max_k", [
    ([3, 40, 600, 9, 300], [5, 60, 700, 300, 31], 4, 2, None),      # beside a long sequence
    ([300] * 40, [31, 2, 17, 32, 7] * 8, 4, 2, 10_000),             # under a loose bound
    ([130] * 20 + [700], [45, 3, 66, 32, 12] * 4 + [520], 32, 16, None)])
def test_precision_goes_by_the_sequence_itself(nq, nk, heads, kv, max_k, d):
    """The gradients of a sequence of few rows or states carry two bf16 of P and dS, whatever else is in
    the call and however loose its bounds are."""
    c = Call(nq, nk, heads, kv, d, BF16, seed=d)
    got = c.run(max_k=max_k)
    c.check(got)
    group, scale = heads // kv, float(torch.tensor(c.scale, dtype=F32))
    q, k = indptr(nq).tolist(), indptr(nk).tolist()
    for b in range(len(nq)):
        if nk[b] >= 512 and nq[b] * group >= 512:
            continue
        i, j = slice(q[b], q[b + 1]), slice(k[b], k[b + 1])
        for h in range(kv):
            rows = lambda t: t[i, h * group:(h + 1) * group].double().reshape(-1, d)
            ref = short_formulas(rows(c.q), c.k[j, h].double(), c.v[j, h].double(), rows(c.dout), scale)
            for name, (want, bound) in ref.items():
                have = rows(got[name]) if name == "dq" else got[name][j, h].double()
                tol = bound + 2.0 ** -8 * (want.abs() + bound)
                bad = ~((have - want).abs() <= tol)
                assert not bad.any(), (b, h, name, int(bad.sum()), float((have - want).abs().max()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("nq", [1, 5, 33, 64, 70])
def test_infinite_gradients_of_the_output(nq, dtype):
    """dv = P^T dout is infinite where a row of dout is, with the number of rows inside a tile or not, and
    finite in its other columns; the row is the first of a tile.  (bf16: P is the sum of two, of which the
    lower may be zero or negative, and zero times infinity is NaN.)"""
    c = Call([nq], [40], 1, 1, 16, dtype, seed=nq)
    for row in (0, 32, 64):
        if row < nq:
            c.dout[row, 0, 3], c.dout[row, 0, 5] = math.inf, -math.inf
    got = c.run()
    if dtype == F32:
        assert torch.all(got["dv"][:, 0, 3] == math.inf) and torch.all(got["dv"][:, 0, 5] == -math.inf)
    assert not torch.isfinite(got["dv"][:, 0, [3, 5]]).any()
    rest = [x for x in range(16) if x not in (3, 5)]
    assert torch.isfinite(got["dv"][:, 0, rest]).all()
