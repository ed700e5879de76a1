"""gnn_orthogonalize where its products take tiles of 128 and 192, which overhang planes padded to 64:
large matrices and batches of middling ones.  Against the steps in 64 bits, every matrix of the batch,
with the tolerance of test_gpu_orthogonalize.py (three times what the same roundings cost on plain
products, and the rounding of the result)."""
import pytest
import torch

from tests.test_gpu_orthogonalize import BF16, F32, QUINTIC, gaussian, run

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")


def wide(x):
    return (x if x.shape[0] <= x.shape[1] else x.T).contiguous()


def steps64(g, steps=5):
    x = g.double()
    x = wide(x / (x.norm() + 1e-7))
    for _ in range(steps):
        a = torch.mm(x, x.T.contiguous())
        x = QUINTIC[0] * x + torch.mm(QUINTIC[1] * a + QUINTIC[2] * torch.mm(a, a), x)
    return x


def planes(x, count):
    up = x.double() * 4096
    kept = up.half().double()
    if count == 2:
        kept = kept + (up - kept).half().double()
    return kept / 4096


def rounded_steps(g, steps=5):
    """The products in 64 bits, so that X, A and Q are rounded as planes and nothing else is."""
    count = 2 if g.dtype == F32 else 1
    x = g.double()
    x = wide(x / (x.norm() + 1e-7))
    eye = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    for _ in range(steps):
        x = planes(x, count)
        a = planes(torch.mm(x, x.T.contiguous()), count)
        x = torch.mm(planes(QUINTIC[0] * eye + QUINTIC[1] * a + QUINTIC[2] * torch.mm(a, a), count), x)
    return x


def check(g, got):
    # sums of k products in 32 bits: k 2^-24 of their sizes at most, k^1/2 of it on average; three
    # products a step, whose errors the steps' slopes (at most 3.5 a step) carry on
    for x, y in zip(g.reshape(-1, *g.shape[-2:]), got.reshape(-1, *g.shape[-2:])):
        want = steps64(x)
        near = rounded_steps(x)
        sums = max(x.shape) ** 0.5 * 2.0 ** -24 * 3 * sum(3.5 ** i for i in range(5)) if g.dtype == F32 else 0.0
        tol = 3 * (near - want).norm() + (torch.finfo(g.dtype).eps / 2 + sums) * want.norm()
        off = (wide(y).double() - want).norm()
        assert off <= tol, (float(off), float(tol), float(want.norm()))
        # and nowhere far off: a tile that is missing or misplaced shows at single places
        # (a place is off by the root mean square times 10 where some ten million are looked at)
        far = (wide(y).double() - want).abs().max()
        assert far <= 10 * tol / want.numel() ** 0.5 + torch.finfo(g.dtype).eps / 2 * want.abs().max()


# the tiles that the library takes: 192 and 192, 128 and 192, 128 and 128 (bf16; fp32 128 and 64 at most)
@pytest.mark.parametrize("b,m,n", [(8, 1100, 1400), (8, 1400, 1100), (16, 1100, 1100), (32, 700, 740),
                                   (32, 740, 700), (64, 450, 500), (64, 500, 450), (2, 2571, 1030),
                                   (1, 1990, 2300), (1, 2300, 1990)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_tiles(b, m, n, dtype):
    g = gaussian(b, m, n, seed=m + n, dtype=dtype, size=1e-3)
    check(g, run(g))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_strided_output_of_large_tiles(dtype):
    into = torch.full((8, 1103, 1408), 7.0, dtype=dtype, device="cuda")
    g = gaussian(8, 1100, 1400, seed=3, dtype=dtype)
    out = into[:, 1:1101, 3:1403]
    run(g, out=out)
    assert torch.equal(out, run(g))
    into[:, 1:1101, 3:1403] = 7.0
    assert torch.all(into == 7.0)
