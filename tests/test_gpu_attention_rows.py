"""gnn_cross_attention and its gradients where sequences have many rows: tiles of 128 rows, a wavefront
each 32 of them, which the library takes from 256 tiles on (sequences times state heads times tiles of
rows).  Against the formulas in 64 bits, with the bounds of test_gpu_attention.py."""
import math

import pytest
import torch

from tests.test_gpu_attention import BF16, F32, Call, indptr

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")


def tiles(c):
    return len(c.nq) * c.kv * -(-max(c.nq) * (c.heads // c.kv) // 128)


EDGES = [63, 64, 65, 127, 128, 129, 0, 1, 2, 31, 32, 33, 90, 95, 96, 97]


@pytest.mark.parametrize("d", [8, 24, 40, 72, 80, 96, 104, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_many_sequences_of_some_rows(d, dtype):
    """Each query head over states of its own; rows that end inside a tile of 128, none among them."""
    nq = ([64, 70, 33, 0, 127, 128, 129, 5] * 5)[:40]
    c = Call(nq, (EDGES * 3)[:40], 8, 8, d, dtype, seed=d)
    assert tiles(c) >= 256
    got = c.run()
    assert c.status == gm.GNN_OK
    c.check(got)


@pytest.mark.parametrize("d", [32, 64, 80, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_grouped_heads_and_counts(d, dtype):
    """Four heads over one of states, and counts that end inside tiles; what lies past them is not finite."""
    count = [200, 64, 65, 0, -3, 63, 1, 129, 90, 17, 10 ** 12, 127, 128, 2, 33, 96]
    c = Call([130, 1, 60, 128] * 4, [200, 130] * 8, 32, 8, d, dtype, count=count, seed=d)
    assert tiles(c) >= 256
    k = indptr(c.nk).tolist()
    for b, n in enumerate(count):
        n = min(max(n, 0), c.nk[b])
        c.k[k[b] + n:k[b + 1]], c.v[k[b] + n:k[b + 1]] = math.nan, math.inf
    got = c.run()
    assert c.status == gm.GNN_OK
    c.check(got)


@pytest.mark.parametrize("d", [32, 80, 96, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_long_sequences(d, dtype):
    """Sums of more than 512 terms, where one bf16 of P and dS is multiplied, and states split among
    workgroups beside them."""
    c = Call([300, 257, 256], [700, 513, 1100], 64, 32, d, dtype, seed=d)
    assert tiles(c) >= 256
    c.check(c.run())
    c = Call([300, 140], [1500, 640], 4, 1, d, dtype, seed=d + 1)
    assert tiles(c) < 256
    c.check(c.run())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("size", [1e-3, 8.0])
def test_flat_and_peaked_weights(size, dtype):
    c = Call([130] * 18, EDGES + [300, 257], 16, 8, 64, dtype, size=size, seed=7)
    assert tiles(c) >= 256
    c.check(c.run())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_all_scores_far_below_zero(dtype):
    """lse near -600: what lies past a sequence's end has a score of zero, far above it."""
    c = Call([70] * 40, (EDGES * 3)[:40], 8, 8, 32, dtype, scale=1.0, seed=31)
    c.q[:, :, 0], c.k[:, :, 0] = 25.0, -25.0
    assert tiles(c) >= 256
    c.check(c.run())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_neighbours_do_not_leak(dtype):
    nq, nk = [70] * 40, [90, 65, 33, 128] * 10
    clean, bad = (Call(nq, nk, 8, 8, 40, dtype, seed=13) for _ in range(2))
    q, k = indptr(nq).tolist(), indptr(nk).tolist()
    bad.k[k[5]:k[6]], bad.v[k[5]:k[6]] = math.nan, math.inf
    bad.q[q[5]:q[7]], bad.dout[q[5]:q[7]] = math.inf, math.nan
    a, b = clean.run(), bad.run()
    for name in a:
        lo, hi = (k[5], k[7]) if name in ("dk", "dv") else (q[5], q[7])
        assert torch.equal(a[name][:lo], b[name][:lo]) and torch.equal(a[name][hi:], b[name][hi:]), name


def test_same_bits_every_time():
    c = Call([130, 90] * 8, [200, 61] * 8, 32, 8, 128, BF16, seed=17)
    a, b = c.run(), c.run()
    for x in a:
        assert torch.equal(a[x], b[x]), x
