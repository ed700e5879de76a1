"""Embedding lookup with scaling and its gradient by sorted ids, against the definitions in 64 bits.

Tolerances: a lookup rounds the fp32 product (2^-24) and then to the output's type (eps / 2).  A sum
of c terms in fp32, in any order, is off by at most (c - 1) 2^-24 times the sum of their magnitudes;
the scale adds one fp32 rounding and the store eps / 2 of the result."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")

F32, BF16 = torch.float32, torch.bfloat16
ULP = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def make_ids(kind, n, rows, seed):
    rng = np.random.default_rng(seed)
    if kind == "one":
        ids = np.full(n, rows - 1)
    elif kind == "skewed":
        ids = np.minimum(rows * rng.random(n) ** 6, rows - 1).astype(np.int64)
    elif kind == "distinct":
        ids = rng.permutation(rows)[:n]
    else:
        ids = rng.integers(0, rows, n)
    return torch.from_numpy(np.ascontiguousarray(ids, dtype=np.int32))


def padded(rows, d, extra, dtype, value=None, seed=0):
    """[rows, d] inside wider rows; the columns beyond d hold NaN."""
    g = torch.Generator().manual_seed(seed)
    t = torch.full((max(rows, 1), d + extra), math.nan, dtype=dtype)
    t[:, :d] = torch.randn(max(rows, 1), d, generator=g).to(dtype) if value is None else value
    return t.cuda()[:rows, :d]


def ws_for(n, rows, d):
    return torch.empty(gm.gnn_embedding_grad_workspace_size(n, rows, d), dtype=torch.uint8,
                       device="cuda")


def reference(ids, dout, rows, scale, pad):
    """(sums, tolerance without the last rounding, counts) in float64 on the host."""
    x = dout.double().cpu()
    keep = ids != pad if pad >= 0 else torch.ones_like(ids, dtype=torch.bool)
    at = ids[keep].long()
    total = torch.zeros(rows, x.shape[1], dtype=torch.float64).index_add_(0, at, x[:len(ids)][keep])
    size = torch.zeros_like(total).index_add_(0, at, x[:len(ids)][keep].abs())
    count = torch.bincount(at, minlength=rows)
    return total * scale, abs(scale) * size * (count[:, None] + 2) * ULP, count


LOOKUPS = [(0, 5, 4), (1, 1, 1), (1, 9, 3), (5, 7, 8), (1000, 333, 7), (777, 50, 100), (64, 10, 602),
           (2049, 1000, 12), (300, 99, 515), (40_000, 5000, 129)]


@pytest.mark.parametrize("n,rows,d", LOOKUPS)
@pytest.mark.parametrize("tt,ot", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_lookup(n, rows, d, tt, ot):
    ids = make_ids("uniform", n, rows, n + d)
    pad = 0 if d % 2 else -1
    extra = d % 3
    table = padded(rows, d, extra, tt, seed=d)
    out = padded(n + 3, d, extra, ot, value=5.0)
    scale = math.sqrt(d)
    gm.gnn_embedding_lookup(table, ids.cuda(), scale, out, pad_id=pad)
    want = table.double().cpu()[ids.long()] * float(np.float32(scale))
    if pad >= 0:
        want[ids == pad] = 0
    got = out.double().cpu()
    tol = want.abs() * (half_step(ot) * (1 + ULP) + ULP)
    assert torch.all((got[:n] - want).abs() <= tol)
    assert torch.all(got[n:] == 5.0)
    if extra:      # the columns beyond d stay as they were
        whole = torch.as_strided(out, (n + 3, extra), (d + extra, 1), d)
        assert torch.isnan(whole).all()


def test_lookup_count_and_bad_ids():
    table = torch.arange(40, dtype=F32, device="cuda").reshape(10, 4)
    ids = torch.tensor([3, 10, -1, 2, 9, 9], dtype=torch.int32, device="cuda")
    out = torch.full((6, 4), 7.0, device="cuda")
    n = torch.tensor([5], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gm.gnn_embedding_lookup(table, ids, 2.0, out, d_n=n, d_status=status)
    want = torch.zeros(6, 4)
    t = table.cpu() * 2
    want[0], want[3], want[4], want[5] = t[3], t[2], t[9], 7.0
    assert torch.equal(out.cpu(), want)
    assert status.item() == gm.GNN_ERR_OUT_OF_RANGE


def test_lookup_not_finite():
    """Infinities and NaN pass through; a padding id's row is zero whatever the table holds there."""
    table = torch.tensor([[math.nan] * 8, [math.inf] * 8, [-math.inf, math.nan] * 4, [1e38] * 8],
                         device="cuda")
    ids = torch.tensor([0, 1, 2, 3], dtype=torch.int32, device="cuda")
    out = torch.empty(4, 8, dtype=BF16, device="cuda")
    gm.gnn_embedding_lookup(table, ids, 1.0, out, pad_id=0)
    got = out.float().cpu()
    assert torch.all(got[0] == 0) and torch.all(got[1] == math.inf)
    assert torch.equal(got[2].isnan(), torch.tensor([False, True] * 4))


def test_lookup_large_table_offsets():
    """Row offsets past 2^31 elements."""
    rows, d = 17_000_001, 128
    table = torch.empty(rows, d, dtype=BF16, device="cuda")
    ids = torch.tensor([rows - 1, 0, rows - 2, 16_777_217], dtype=torch.int32, device="cuda")
    table[ids.long()] = torch.randn(4, d, device="cuda").to(BF16)
    out = torch.empty(4, d, dtype=BF16, device="cuda")
    gm.gnn_embedding_lookup(table, ids, 1.0, out)
    assert torch.equal(out, table[ids.long()])


GRADS = [(1, 1, 1, "one", -1), (7, 3, 5, "uniform", -1), (64, 64, 8, "one", -1), (65, 9, 9, "uniform", 2),
         (1000, 40, 64, "uniform", -1), (1024, 10_000, 64, "uniform", -1), (4000, 20_000, 100, "distinct", -1),
         (8192, 300, 12, "skewed", 0), (8193, 70_000, 3, "skewed", -1), (9000, 9000, 515, "skewed", 0),
         (20_000, 3, 33, "one", -1), (100_000, 2_000_003, 16, "skewed", 5), (60_000, 500, 257, "skewed", -1)]


@pytest.mark.parametrize("n,rows,d,kind,pad", GRADS)
@pytest.mark.parametrize("dt,gt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_grad_dense(n, rows, d, kind, pad, dt, gt):
    ids = make_ids(kind, n, rows, n)
    extra = d % 3
    dout = padded(n, d, extra, dt, seed=n)
    scale = 0.37
    want, tol, _ = reference(ids, dout, rows, float(np.float32(scale)), pad)
    for accumulate in (False, True):
        grad = padded(rows, d, extra, gt, value=None if accumulate else math.nan, seed=3)
        old = grad.double().cpu() if accumulate else torch.zeros(rows, d, dtype=torch.float64)
        gm.gnn_embedding_grad(ids.cuda(), dout, scale, grad, ws_for(n, rows, d), pad_id=pad,
                              accumulate=accumulate)
        got, total = grad.double().cpu(), want + old
        bound = tol * (1 + half_step(gt)) + total.abs() * (half_step(gt) * 1.001 + ULP) + old.abs() * ULP
        bad = (got - total).abs() > bound
        assert not bad.any() and not got.isnan().any(), (accumulate, int(bad.sum()))


BUCKETS = [(2048, 1, 9, "one", -1), (2049, 65, 5, "uniform", 0), (5000, 3, 1030, "skewed", -1),
           (8192, 20_000, 260, "skewed", 1), (12_000, 191_999, 31, "uniform", -1),
           (12_000, 192_000, 31, "uniform", -1), (16_384, 262_143, 128, "skewed", -1),
           (16_384, 1, 7, "one", -1), (16_384, 2_000_003, 8, "skewed", 0), (16_385, 5000, 64, "skewed", -1)]


@pytest.mark.parametrize("n,rows,d,kind,pad", BUCKETS)
@pytest.mark.parametrize("dt,gt", [(F32, F32), (F32, BF16), (BF16, F32), (BF16, BF16)])
def test_grad_dense_of_some_thousand_positions(n, rows, d, kind, pad, dt, gt):
    test_grad_dense(n, rows, d, kind, pad, dt, gt)
    # the same bits every time, and ids out of range and positions past the count have no part in them
    ids, dout = make_ids(kind, n, rows, n), padded(n, d, 1, dt, seed=n)
    first, again = torch.empty(rows, d, dtype=gt, device="cuda"), torch.empty(rows, d, dtype=gt, device="cuda")
    ids[n // 3] = pad
    d_n = torch.tensor([n - 5], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gm.gnn_embedding_grad(ids.cuda(), dout, 1.0, first, ws_for(n, rows, d), pad_id=pad, d_n=d_n)
    ids[n // 3] = rows
    dout[n // 3], dout[n - 5:] = math.nan, math.nan
    gm.gnn_embedding_grad(ids.cuda(), dout, 1.0, again, ws_for(n, rows, d), pad_id=pad, d_n=d_n,
                          d_status=status)
    assert torch.equal(first, again) and not first.isnan().any()
    assert status.item() == gm.GNN_ERR_OUT_OF_RANGE


@pytest.mark.parametrize("n,rows,d,kind,pad", GRADS)
def test_grad_rows(n, rows, d, kind, pad):
    ids = make_ids(kind, n, rows, n)
    dout = padded(n, d, d % 3, BF16, seed=n)
    want, tol, count = reference(ids, dout, rows, 1.0, pad)
    nodes = torch.nonzero(count).squeeze(1)
    cap = len(nodes) + 2
    uniq = torch.full((cap,), -7, dtype=torch.int32, device="cuda")
    number = torch.full((1,), -7, dtype=torch.int64, device="cuda")
    grad = torch.full((cap, d), 9.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = ws_for(n, rows, d)
    gm.gnn_embedding_grad_rows(ids.cuda(), dout, 1.0, rows, uniq, number, grad, ws, pad_id=pad,
                               d_status=status)
    assert number.item() == len(nodes) and status.item() == gm.GNN_OK
    assert torch.equal(uniq.cpu()[:-2].long(), nodes) and torch.all(uniq[-2:] == -7)
    got = grad.double().cpu()
    assert torch.all(got[-2:] == 9.0)
    assert torch.all((got[:-2] - want[nodes]).abs() <= tol[nodes] + want[nodes].abs() * ULP)
    # the same bits every time
    again = torch.full_like(grad, 9.0)
    gm.gnn_embedding_grad_rows(ids.cuda(), dout, 1.0, rows, uniq, number, again, ws, pad_id=pad)
    assert torch.equal(grad, again)
    # a list that is too short: reported, and nothing past it is written
    if len(nodes) > 1:
        short = torch.full((len(nodes),), -7, dtype=torch.int32, device="cuda")
        rows_short = torch.full((len(nodes), d), 9.0, device="cuda")
        gm.gnn_embedding_grad_rows(ids.cuda(), dout, 1.0, rows, short[:-1], number, rows_short, ws,
                                   pad_id=pad, d_status=status)
        assert status.item() == gm.GNN_ERR_CAPACITY and number.item() == len(nodes)
        assert short[-1].item() == -7 and torch.all(rows_short[-1] == 9.0)
        assert torch.equal(rows_short[:-1], grad[:len(nodes) - 1])


def test_grad_many_tiles():
    """More sort tiles than one workgroup sums by itself, three digits."""
    n, rows, d = 2_200_000, 100_000, 4
    ids = make_ids("skewed", n, rows, 5)
    dout = padded(n, d, 0, F32, seed=1)
    want, tol, count = reference(ids, dout, rows, 1.0, -1)
    grad = torch.empty(rows, d, device="cuda")
    gm.gnn_embedding_grad(ids.cuda(), dout, 1.0, grad, ws_for(n, rows, d))
    assert torch.all((grad.double().cpu() - want).abs() <= tol + want.abs() * ULP)


@pytest.mark.parametrize("n", [50, 20_000])
def test_grad_bad_ids_and_count(n):
    ids = make_ids("uniform", n, 100, 1)
    ids[3], ids[n // 2] = 100, -2
    act = n - 7
    dout = padded(n, 12, 0, F32, seed=2)
    dout[act:] = math.nan         # beyond the count: not read
    good = ids.clone()
    good[3] = good[n // 2] = 100
    good[act:] = 100
    want, tol, count = reference(good, torch.nan_to_num(dout), 101, 1.0, 100)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    grad = torch.empty(100, 12, device="cuda")
    d_n = torch.tensor([act], device="cuda")
    gm.gnn_embedding_grad(ids.cuda(), dout, 1.0, grad, ws_for(n, 100, 12), d_n=d_n, d_status=status)
    assert status.item() == gm.GNN_ERR_OUT_OF_RANGE
    assert torch.all((grad.double().cpu() - want[:100]).abs() <= (tol + want.abs() * ULP)[:100])


def test_grad_of_nothing():
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    dout = torch.empty(0, 8, device="cuda")
    for rows in (3, 1000):
        grad = torch.full((rows, 8), math.nan, device="cuda")
        gm.gnn_embedding_grad(none, dout, 1.0, grad, ws_for(0, rows, 8))
        assert torch.all(grad == 0)
        gm.gnn_embedding_grad(none, dout, 1.0, grad, ws_for(0, rows, 8), accumulate=True)
        assert torch.all(grad == 0)
    number = torch.full((1,), 5, dtype=torch.int64, device="cuda")
    gm.gnn_embedding_grad_rows(none, dout, 1.0, 10, none, number, dout, ws_for(0, 10, 8))
    assert number.item() == 0
    # every position is padding
    ids = torch.full((100,), 4, dtype=torch.int32, device="cuda")
    grad = torch.full((10, 8), math.nan, device="cuda")
    gm.gnn_embedding_grad(ids, torch.full((100, 8), math.nan, device="cuda"), 1.0, grad,
                          ws_for(100, 10, 8), pad_id=4)
    assert torch.all(grad == 0)


def test_grad_not_finite_stays_in_its_row():
    ids = make_ids("uniform", 3000, 50, 9)
    dout = padded(3000, 16, 0, F32, seed=4)
    first = int((ids == 7).nonzero()[0])
    dout[first, 3] = math.nan
    dout[int((ids == 8).nonzero()[0]), 4] = math.inf
    grad = torch.empty(50, 16, device="cuda")
    gm.gnn_embedding_grad(ids.cuda(), dout, 1.0, grad, ws_for(3000, 50, 16))
    fine = torch.isfinite(grad).cpu()
    assert not fine[7, 3] and not fine[8, 4] and int((~fine).sum()) == 2


def test_grad_is_the_lookups_derivative():
    """<lookup(T + h E) - lookup(T - h E), dout> / 2h = <grad, E>: the lookup is linear in the table,
    so differences are exact up to rounding."""
    n, rows, d = 500, 60, 24
    ids = make_ids("skewed", n, rows, 11).cuda()
    table, e = padded(rows, d, 0, F32, seed=5), padded(rows, d, 0, F32, seed=6)
    dout = padded(n, d, 0, F32, seed=7)
    up, down = torch.empty(n, d, device="cuda"), torch.empty(n, d, device="cuda")
    gm.gnn_embedding_lookup(table + 0.5 * e, ids, 1.5, up, pad_id=1)
    gm.gnn_embedding_lookup(table - 0.5 * e, ids, 1.5, down, pad_id=1)
    grad = torch.empty(rows, d, device="cuda")
    gm.gnn_embedding_grad(ids, dout, 1.5, grad, ws_for(n, rows, d), pad_id=1)
    left = float(((up.double() - down.double()) * dout.double()).sum())
    right = float((grad.double() * e.double()).sum())
    # every term of either side carries a few roundings of values below 20
    assert abs(left - right) <= 8 * ULP * 20 * 20 * n * d


def test_on_another_stream_and_in_a_graph():
    n, rows, d = 12_000, 700, 40
    s = torch.cuda.Stream()
    ids, dout = make_ids("skewed", n, rows, 2).cuda(), padded(n, d, 0, BF16, seed=8)
    table = padded(rows, d, 0, F32, seed=9)
    grad, out = torch.empty(rows, d, device="cuda"), torch.empty(n, d, device="cuda")
    ws = ws_for(n, rows, d)
    want_grad, want_out = torch.empty_like(grad), torch.empty_like(out)
    gm.gnn_embedding_grad(ids, dout, 1.0, want_grad, ws)
    gm.gnn_embedding_lookup(table, ids, 3.0, want_out)
    torch.cuda.synchronize()
    gm.gnn_embedding_grad(ids, dout, 1.0, grad, ws, stream=s)
    gm.gnn_embedding_lookup(table, ids, 3.0, out, stream=s)
    s.synchronize()
    assert torch.equal(grad, want_grad) and torch.equal(out, want_out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gm.gnn_embedding_lookup(table, ids, 3.0, out)
        gm.gnn_embedding_grad(ids, dout, 1.0, grad, ws)
    for turn in range(3):
        ids.copy_(make_ids("skewed", n, rows, 20 + turn))
        gm.gnn_embedding_grad(ids, dout, 1.0, want_grad, ws)
        gm.gnn_embedding_lookup(table, ids, 3.0, want_out)
        grad.fill_(math.nan)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(grad, want_grad) and torch.equal(out, want_out)
