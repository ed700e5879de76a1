"""The scale of orthogonalised bf16 updates whose singular values are alike: there the diagonals of A and
Q are alike too, and a rounding common to all of them would scale the whole result.

Bound on the scale: the diagonals are kept in fp32, so that what is left are the roundings of X's
entries, up to 2^-12 of either sign.  Entries that have only the 128 mantissas of bf16 share them: their
mean stays below 2^-12 / 128^(1/2) a step, and the steps carry a relative error on by a factor of up to
about 5, five times: below 2^-11, an eighth of the half step of bf16.  (One rounding of 2^-12 common to
the diagonal of A alone moves Q, with slopes 4.8 and 4.1, by 2^-9.)  The distance is bounded as in
test_gpu_orthogonalize.py."""
import math

import pytest
import torch

from tests.test_gpu_orthogonalize import BF16, QUINTIC, check, gaussian, run, steps64

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")


def update(kind, s, l):
    if kind == "gaussian":
        g = gaussian(s, l, seed=s)
    elif kind == "signs":
        g = gaussian(s, l, seed=s).sign()
    elif kind == "orthonormal rows":
        g = torch.linalg.qr(gaussian(l, s, seed=s).double())[0].T.contiguous().float()
    else:
        k = max(1, s // 8)
        g = gaussian(s, k, seed=s) @ gaussian(k, l, seed=l) / math.sqrt(k) + gaussian(s, l, seed=s + l)
    return g.to(BF16)


SHAPES = [(16, 4096), (48, 4096), (144, 3000), (223, 2400), (321, 4000), (400, 4000)]


@pytest.mark.parametrize("kind", ["gaussian", "signs", "orthonormal rows", "strong directions"])
@pytest.mark.parametrize("s,l", SHAPES)
def test_scale(s, l, kind):
    g = update(kind, s, l)
    if s == 223:
        g = g.T.contiguous()
    got, want = run(g), steps64(g, 5)
    y = got.double().cpu()
    assert abs(float((y * want).sum() / want.square().sum()) - 1) < 2.0 ** -11
    check(g, got)


@pytest.mark.parametrize("coefs,steps", [((1.5, -0.5, 0.0), 5), ((2.0, -1.5, 0.5), 8), (QUINTIC, 1), (QUINTIC, 3)])
def test_scale_with_other_steps(coefs, steps):
    """(Their slopes are no larger.)"""
    for s, l in ((321, 4000), (144, 3000)):
        g = update("orthonormal rows", s, l)
        got, want = run(g, steps=steps, coefs=coefs), steps64(g, steps, coefs)
        y = got.double().cpu()
        assert abs(float((y * want).sum() / want.square().sum()) - 1) < 2.0 ** -11, (s, l)
        check(g, got, steps=steps, coefs=coefs)


def test_scale_of_large_tiles():
    """Tiles of 192, whose products read what the planes leave of the diagonals in other places."""
    g = torch.stack([update("orthonormal rows", 1100, 1400)] * 8)
    got, want = run(g), steps64(g[0], 5)
    for y in got:
        assert abs(float((y.double().cpu() * want).sum() / want.square().sum()) - 1) < 2.0 ** -11
        assert torch.equal(y, got[0])


def test_square_multiples_of_the_identity_and_constant_updates():
    """All of their entries are alike, X's too: three common roundings of 2^-12 a step, whose slopes the
    steps carry on, are within two steps of bf16 of the result (its own rounding, common too, is up to
    half of one)."""
    for g in (torch.eye(144, 3000), torch.eye(512, 512), torch.ones(48, 4096), torch.ones(512, 4096)):
        g = g.to(BF16).cuda()
        y, want = run(g).double().cpu(), steps64(g, 5)
        assert float((y - want).abs().max()) <= 2 * 2.0 ** -7 * float(want.abs().max())


@pytest.mark.parametrize("b,m,n", [(4, 3290, 138), (3, 2529, 167), (7, 144, 2562)])
def test_long_sums_in_fp32(b, m, n):
    """A's diagonal is a sum of k squares: k / 16 additions of a sum of sixteen, each rounded by up to 2^-24
    of the sum so far, by 2.5e-8 of it in the root mean square over the mantissas, 2.5e-8 (k / 48)^(1/2) of
    the whole in all.  A step's Q moves by up to 1.8 of that (where s^2 = 1.4), and the later steps'
    slopes carry it on by up to 5, so 9 at most and, for the other terms' part, 12 here; the planes add some
    2e-7."""
    k = max(m, n)
    tol = 12 * 2.5e-8 * (k / 48) ** 0.5 + 2e-7
    g = torch.stack([gaussian(m, min(m, n) // 8, seed=i) @ gaussian(min(m, n) // 8, n, seed=9 + i) /
                     math.sqrt(min(m, n) // 8) + gaussian(m, n, seed=20 + i) for i in range(b)])
    for x, y in zip(g, run(g)):
        want = steps64(x, 5)
        assert float((y.double().cpu() - want).norm() / want.norm()) <= tol
