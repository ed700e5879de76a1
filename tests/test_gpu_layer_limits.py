"""The norm and the dense layers where values are extreme: far arguments, infinities, rows far from zero."""
import pytest
import torch

from . import layers as ref
from .test_gpu_dense import B, F, normal, space

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("name", ref.ACTS)
def test_activations_of_the_farthest_arguments(name, dtype):
    """act and act' up to the type's largest number: z, 1 or 0, the functions' limits there."""
    top = torch.finfo(dtype).max
    z = torch.tensor([[s * v] for v in (1e5, 1e10, 1e19, 1e20, 1e30, top) for s in (1, -1)], device="cuda", dtype=dtype)
    one = torch.ones(1, 1, device="cuda", dtype=dtype)
    out, dx = torch.empty_like(z), torch.empty_like(z)
    n = z.shape[0]
    gm.gnn_linear(z, one, out, space(gm.gnn_linear_workspace_size, n, 1, 1, dtype), activation=name)
    gm.gnn_linear_backward(z, one, torch.ones_like(z), space(gm.gnn_linear_workspace_size, n, 1, 1, dtype, True),
                           activation=name, pre=z, dx=dx)
    up = z > 0
    if name == "none":
        want, slope = z, torch.ones_like(z)
    elif name == "sigmoid":
        want, slope = up.to(dtype), torch.zeros_like(z)
    else:
        want, slope = torch.where(up, z, 0.0), up.to(dtype)
    assert torch.equal(out, want) and torch.equal(dx, slope)


def signs(t):
    return t.float().sign() * float("inf")


@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape", [(1, 300, 40), (6, 70, 50), (20, 70, 50), (33, 1030, 72), (40, 200, 520), (300, 64, 640),
                                   (511, 136, 257), (600, 136, 72), (600, 72, 520), (2000, 40, 300)])
def test_an_infinite_input_or_weight(shape, dtype, bad):
    """An infinity of x reaches its column's line of dw with the sign of dz, one of w its line's column of dx; a NaN
    stays NaN there; all else is what it is without it.  (Sums of one and of two planes of dz, whole and split.)"""
    n, i, o = shape
    g = torch.Generator(device="cuda").manual_seed(n + i)
    x, w, dout = normal(n, i, dtype=dtype, gen=g), normal(i, o, dtype=dtype, gen=g), normal(n, o, dtype=dtype, gen=g)
    pre = normal(n, o, dtype=dtype, gen=g).abs()      # slopes above 0, of full precision
    ws = space(gm.gnn_linear_workspace_size, n, i, o, dtype, True)

    def gradients():
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(o, device="cuda", dtype=dtype)
        gm.gnn_linear_backward(x, w, dout, ws, activation="gelu", pre=pre, dx=dx, dw=dw, dbias=db)
        return dx, dw, db

    clean = gradients()
    row, col, line, at = n // 2, i // 3, i - 1, o - 2
    x[row, col], w[line, at] = bad, bad
    dx, dw, db = gradients()
    gone = torch.full((1,), float("nan"), device="cuda")
    want_dw = signs(dout[row]) * (1 if bad > 0 else -1) if bad == bad else gone.expand(o)
    want_dx = signs(dout[:, at]) * (1 if bad > 0 else -1) if bad == bad else gone.expand(n)
    torch.testing.assert_close(dw[col].float(), want_dw, rtol=0, atol=0, equal_nan=True)
    torch.testing.assert_close(dx[:, line].float(), want_dx, rtol=0, atol=0, equal_nan=True)
    lines = torch.arange(i, device="cuda")
    assert torch.equal(dw[lines != col], clean[1][lines != col]) and torch.equal(db, clean[2])
    assert torch.equal(dx[:, lines != line], clean[0][:, lines != line])


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("n, i, o, count", [(12, 70, 50, 12), (5, 300, 136, 4), (70, 300, 130, 65), (300, 520, 250, 300),
                                            (700, 200, 328, 300), (700, 64, 96, 700), (2500, 136, 200, 511)])
def test_an_infinite_input_or_weight_of_a_pair(n, i, o, count, dtype):
    """The same of the gated pair, whose dx sums both projections' planes, under a device count."""
    g = torch.Generator(device="cuda").manual_seed(n + i + 1)
    x, dout, up = (normal(n, c, dtype=dtype, gen=g) for c in (i, o, o))
    wg, wu = (normal(i, o, dtype=dtype, gen=g) for _ in range(2))
    gate = 0.1 + normal(n, o, dtype=dtype, gen=g).abs()      # act and its slope above 0
    d_n = torch.tensor([count], device="cuda")
    ws = space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype, True)

    def gradients():
        dx, dwg, dwu = torch.zeros_like(x), torch.empty_like(wg), torch.empty_like(wu)
        gm.gnn_gated_linear_backward(x, wg, wu, gate, up, dout, ws, activation="gelu_tanh", dx=dx, dw_gate=dwg,
                                     dw_up=dwu, d_n=d_n)
        return dx[:count], dwg, dwu

    clean = gradients()
    row, col, first, second = count // 2, i // 3, i - 1, i // 2
    x[row, col], wg[first, 3], wu[second, o - 1] = float("inf"), float("inf"), -float("inf")
    dx, dwg, dwu = gradients()
    assert torch.equal(dwg[col].float(), signs(dout[row].float() * up[row].float()))
    assert torch.equal(dwu[col].float(), signs(dout[row]))
    assert torch.equal(dx[:, first].float(), signs(dout[:count, 3].float() * up[:count, 3].float()))
    assert torch.equal(dx[:, second].float(), -signs(dout[:count, o - 1]))
    lines = torch.arange(i, device="cuda")
    for a, b in zip((dwg, dwu), clean[1:]):
        assert torch.equal(a[lines != col], b[lines != col])
    keep = (lines != first) & (lines != second)
    assert torch.equal(dx[:, keep], clean[0][:, keep])


@pytest.mark.parametrize("dtype", [F, B])
def test_a_workspace_of_the_largest_batch_serves_smaller_ones(dtype):
    """One workspace, sized once, for a batch that shrinks to a row; results as with a workspace of their own."""
    i, o, most = 520, 1032, 1100
    g = torch.Generator(device="cuda").manual_seed(3)
    x, w, wu, dout = (normal(*s, dtype=dtype, gen=g) for s in ((most, i), (i, o), (i, o), (most, o)))
    calls = (gm.gnn_linear_workspace_size, gm.gnn_gated_linear_workspace_size)
    shared = [space(c, most, i, o, dtype, b) for c in calls for b in (False, True)]
    for n in (1100, 1000, 768, 500, 200, 64, 8, 1, 0):
        results = []
        for ws in (shared, [space(c, n, i, o, dtype, b) for c in calls for b in (False, True)]):
            out, gate, up, y = torch.empty(4, n, o, device="cuda", dtype=dtype)
            dx, dw, dx2, dwg, dwu = (torch.empty(s, device="cuda", dtype=dtype) for s in ((n, i), (i, o), (n, i), (i, o), (i, o)))
            gm.gnn_linear(x[:n], w, y, ws[0])
            gm.gnn_linear_backward(x[:n], w, dout[:n], ws[1], dx=dx, dw=dw)
            gm.gnn_gated_linear(x[:n], w, wu, out, ws[2], gate=gate, up=up)
            gm.gnn_gated_linear_backward(x[:n], w, wu, gate, up, dout[:n], ws[3], dx=dx2, dw_gate=dwg, dw_up=dwu)
            results.append((out, gate, up, y, dx, dw, dx2, dwg, dwu))
        assert all(torch.equal(a, b) for a, b in zip(*results)), n


def offset_bounds(x, eps):
    """(out, its bound, rstd, its bound) of fp32 rows far from zero, without parameters.  A row's mean is off by em at
    first; the differences from it are exact (numbers within a factor of two of each other), their own mean puts it
    right, so that what is left of the error is that sum's, of the differences' size."""
    u, rows = ref.U, ref.ROW
    m = x.mean(1, keepdim=True)
    c = x - m
    em = rows * u * x.abs().mean(1, keepdim=True)
    ec = (rows + 4) * u * (c.abs().mean(1, keepdim=True) + em) + 2 * u * (c.abs() + em)
    v = (c * c).mean(1, keepdim=True)
    ev = (rows + 8) * u * (v + em * em) + 2 * em * (rows + 4) * u * (c.abs().mean(1, keepdim=True) + em)
    r = (v + eps) ** -0.5
    er = r * (0.5 * ev / (v + eps) + 4 * u)
    y = c * r
    return y, (ec * (r + er) + c.abs() * er + 3 * u * y.abs()) * (1 + u), r[:, 0], er[:, 0]


@pytest.mark.parametrize("value", [0.1, -1000.1, 12345.678, 3.0e7])
@pytest.mark.parametrize("d", [3, 7, 100, 300, 768, 1000, 1025, 4095, 5000, 16383])
def test_rows_of_one_value(d, value):
    """Whatever the value and the width, its mean is the value, and the row's result is the bias."""
    x = torch.full((9, d), value, device="cuda")
    b = torch.randn(d, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    out, mean, rstd = torch.empty_like(x), *torch.empty(2, 9, device="cuda")
    gm.gnn_layer_norm(x, None, b, 1e-5, out, mean=mean, rstd=rstd)
    y, ey, r, er = offset_bounds(x.double(), 1e-5)
    assert torch.equal(mean, x[:, 0])
    ref.close(out, (b.double().expand_as(x), ey + ref.U * (b.double().abs() + ey)))
    ref.close(rstd, (r, er))
    assert float((out - b).abs().max()) < 1e-4


@pytest.mark.parametrize("d", [64, 100, 768, 2500, 5000, 16384])
@pytest.mark.parametrize("shift, scale", [(1000.0, 0.01), (-3.0e4, 1.0), (0.0, 1.0)])
def test_rows_far_from_zero(d, shift, scale):
    """What the mean's own rounding takes from rows far from zero is given back."""
    g = torch.Generator(device="cuda").manual_seed(2)
    x = normal(33, d, dtype=F, gen=g, scale=scale) + shift
    out, mean, rstd = torch.empty_like(x), *torch.empty(2, 33, device="cuda")
    gm.gnn_layer_norm(x, None, None, 0.0, out, mean=mean, rstd=rstd)
    y, ey, r, er = offset_bounds(x.double(), 0.0)
    if shift:
        ref.close(out, (y, ey), "out")
        ref.close(rstd, (r, er), "rstd")
        exact = x.double().mean(1)
        ref.close(mean, (exact, ref.U * exact.abs() + ey.mean(1) / r), "mean")
    else:      # differences from a mean near zero are rounded
        want = ref.norm(x.double(), None, None, 0.0, F)
        for got, bound in zip((out, mean, rstd), want):
            ref.close(got, bound)


def test_the_mean_of_a_row_that_is_not_finite():
    x = torch.ones(4, 200, device="cuda")
    x[0, 3], x[1, 4], x[2, 5] = float("inf"), -float("inf"), float("nan")
    out, mean, rstd = torch.empty_like(x), *torch.empty(2, 4, device="cuda")
    gm.gnn_layer_norm(x, None, None, 1e-5, out, mean=mean, rstd=rstd)
    assert mean[0] == float("inf") and mean[1] == -float("inf") and torch.isnan(mean[2]) and mean[3] == 1
    assert torch.isnan(out[:3]).all() and torch.isnan(rstd[:3]).all() and (out[3] == 0).all()


@pytest.mark.parametrize("dtype", [F, B])
def test_small_means_keep_their_digits(dtype):
    """Rows spread around zero whose sums are exact: multiples of 2^-10 below 8, of which 4000 add up below 2^24 of them
    in any order.  The mean is their quotient, which the differences' own roundings must not get into."""
    g = torch.Generator(device="cuda").manual_seed(4)
    x = normal(500, 4000, dtype=F, gen=g).clamp(-7, 7) + 0.02 * normal(500, 1, dtype=F, gen=g)
    x = ((x * 1024).round() / 1024).to(dtype)
    out, mean, rstd = torch.empty_like(x), *torch.empty(2, 500, device="cuda")
    gm.gnn_layer_norm(x, None, None, 1e-5, out, mean=mean, rstd=rstd)
    assert torch.equal(mean, (x.double().sum(1) / 4000).float())
