"""The layer norm and the dense layers in 64 bits, with bounds on what the kernels may be off by.

u is half a step of fp32 at 1 (2^-24), h half a step of the result's type relative to the value.
"""
import math

import torch

U = 2.0 ** -24
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"]


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def act(name, z):
    """act(z), act'(z) of a float64 z."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        return torch.relu(z), (z > 0).double()
    if name == "gelu":
        phi = torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
        return z * torch.special.ndtr(z), torch.special.ndtr(z) + z * phi
    if name == "gelu_tanh":
        c = math.sqrt(2 / math.pi)
        t = torch.tanh(c * (z + 0.044715 * z ** 3))
        return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    if name == "sigmoid":
        return s, s * (1 - s)
    return z * s, s * (1 + z * (1 - s))


def act_error(dtype):
    """Of act (relative) and act' (absolute).  fp32: up to some thirty roundings of values of at most 1.2; the
    bf16 layers' exponentials and reciprocals and the fit of erfc: 1.3e-5 < 2^-16 of values up to 1.2."""
    return 2.0 ** -19 if dtype == torch.float32 else 2.0 ** -15


def product(x, w):
    """x w, and the error of a sum of fp32 products in any order: one step (a sum may be cut, not rounded) of
    2 u for each addition, of the sum of the terms' sizes."""
    return x @ w, 2 * U * (x.shape[1] + 8) * (x.abs() @ w.abs())


def linear(x, w, bias, name, residual, dtype):
    """(out, its bound, pre, its bound); the arguments in float64."""
    z, ez = product(x, w)
    if bias is not None:
        z = z + bias
        ez = ez + 2 * U * (z.abs() + bias.abs())
    y, _ = act(name, z)
    ey = 1.2 * ez + (act_error(dtype) * y.abs() if name != "none" else 0)
    if residual is not None:
        y = y + residual
        ey = ey + 2 * U * (y.abs() + residual.abs())
    h = half_step(dtype)
    return y, ey + h * (y.abs() + ey), z, ez + h * (z.abs() + ez)


def gated(x, wg, wu, bg, bu, name, dtype):
    """[(out, bound), (gate, bound), (up, bound)]"""
    h = half_step(dtype)
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    if bg is not None:
        g, eg = g + bg, eg + 2 * U * ((g + bg).abs() + bg.abs())
    if bu is not None:
        u, eu = u + bu, eu + 2 * U * ((u + bu).abs() + bu.abs())
    a, _ = act(name, g)
    ea = 1.2 * eg + act_error(dtype) * a.abs()
    y = a * u
    ey = ea * u.abs() + eu * a.abs() + ea * eu + 2 * U * y.abs()
    return [(y, ey + h * (y.abs() + ey)), (g, eg + h * (g.abs() + eg)), (u, eu + h * (u.abs() + eu))]


def _gradients(x, parts, dtype, rounded):
    """parts: (w, dz, bound of dz in fp32) of each projection; [(dx, bound), then (dw, bound), (db, bound) of
    each].  rounded: dz is not an input and is rounded to dtype, to two planes for short sums."""
    h = half_step(dtype)
    terms = sum(w.shape[1] for w, _, _ in parts)

    def plane(short):
        if dtype == torch.float32 or not rounded:
            return 0.0
        return 2.0 ** -17 if short else h

    dx, edx = 0, 0
    for w, dz, e in parts:
        p, ep = product(dz, w.t().contiguous())
        dx, edx = dx + p, edx + ep + (e + plane(terms < 512) * dz.abs()) @ w.abs().t()
    edx = edx + 2 * U * dx.abs()
    out = [(dx, edx + h * (dx.abs() + edx))]
    xt = x.t().contiguous()
    for w, dz, e in parts:
        dw, edw = product(xt, dz)
        edw = edw + xt.abs() @ (e + plane(x.shape[0] < 512) * dz.abs())
        db = dz.sum(0)
        edb = e.sum(0) + U * (x.shape[0] + 8) * dz.abs().sum(0)
        out += [(dw, edw + h * (dw.abs() + edw)), (db, edb + h * (db.abs() + edb))]
    return out


def linear_gradients(x, w, dout, name, pre, dtype):
    """[(dx, bound), (dw, bound), (dbias, bound)]"""
    if name == "none":
        return _gradients(x, [(w, dout, torch.zeros_like(dout))], dtype, False)
    dz = dout * act(name, pre)[1]
    e = act_error(dtype) * dout.abs() + 4 * U * dz.abs()
    return _gradients(x, [(w, dz, e)], dtype, True)


def gated_gradients(x, wg, wu, dout, name, g, u, dtype):
    """[(dx, bound), (dw_gate, ..), (dbias_gate, ..), (dw_up, ..), (dbias_up, ..)]"""
    a, slope = act(name, g)
    dg, du = dout * u * slope, dout * a
    eg = act_error(dtype) * (dout * u).abs() + 4 * U * dg.abs()
    eu = act_error(dtype) * du.abs() + 4 * U * du.abs()
    return _gradients(x, [(wg, dg, eg), (wu, du, eu)], dtype, True)


# A row's sums: pieces of 8 in a tree, up to 8 pieces, 6 exchanges and up to 16 wavefronts: below 40 additions.
ROW = 40


def norm(x, weight, bias, eps, dtype):
    """[(out, bound), (mean, bound), (rstd, bound)]"""
    d = x.shape[1]
    h = half_step(dtype)
    m = x.mean(1, keepdim=True)
    em = ROW * U * x.abs().mean(1, keepdim=True)
    c = x - m
    ec = em + U * c.abs()
    v = (c * c).mean(1, keepdim=True)
    # the mean's own error moves v by its square alone (the differences sum to zero)
    ev = (ROW + 4) * U * v + em * em + 2 * U * (c.abs() * (x.abs() + m.abs())).sum(1, keepdim=True) / d
    r = (v + eps) ** -0.5
    er = r * (0.5 * ev / (v + eps) + 4 * U)
    w = torch.ones_like(x[0]) if weight is None else weight
    b = torch.zeros_like(x[0]) if bias is None else bias
    y = c * r * w + b
    ey = (ec * r + c.abs() * er + 2 * U * (c * r).abs()) * w.abs() + U * (y.abs() + b.abs())
    return [(y, ey + h * (y.abs() + ey)), (m[:, 0], em[:, 0] + U * m[:, 0].abs()), (r[:, 0], er[:, 0])]


def norm_gradients(x, weight, mean, rstd, dout, residual, dtype, param_dtype):
    """[(dx, bound), (dweight, bound), (dbias, bound)] with the given mean and rstd."""
    h, hp = half_step(dtype), half_step(param_dtype)
    d, n = x.shape[1], x.shape[0]
    w = torch.ones_like(x[0]) if weight is None else weight
    hat = (x - mean[:, None]) * rstd[:, None]
    eh = 2 * U * hat.abs()
    g = dout * w
    sg, sgh = g.mean(1, keepdim=True), (g * hat).mean(1, keepdim=True)
    esg = ROW * U * g.abs().mean(1, keepdim=True)
    esgh = (ROW + 4) * U * (g * hat).abs().mean(1, keepdim=True)
    dx = (g - sg - hat * sgh) * rstd[:, None]
    inner = esg + esgh * hat.abs() + eh * sgh.abs() + 4 * U * (g.abs() + sg.abs() + (hat * sgh).abs())
    edx = inner * rstd[:, None] + U * dx.abs()
    if residual is not None:
        dx = dx + residual
        edx = edx + U * dx.abs()
    dw, db = (dout * hat).sum(0), dout.sum(0)
    edw = (n + 8) * U * (dout * hat).abs().sum(0) + 2 * U * (dout * hat).abs().sum(0)
    edb = (n + 8) * U * dout.abs().sum(0)
    return [(dx, edx + h * (dx.abs() + edx)), (dw, edw + hp * (dw.abs() + edw)),
            (db, edb + hp * (db.abs() + edb))]


def close(got, want_and_bound, what=""):
    want, bound = want_and_bound
    off = (got.double().to(want.device) - want).abs()
    # the smallest normal number: below it a result may be flushed
    bad = ~(off <= bound + 2.0 ** -126)
    assert not bool(bad.any()), (what, int(bad.sum()), float((off / (bound + 2.0 ** -126)).max()),
                                 torch.nonzero(bad)[:4].tolist())


def strided(t, pad, offset=0):
    """t as a view whose rows lie `pad` elements further apart and start `offset` elements in."""
    n, d = t.shape
    flat = torch.full(((n + 1) * (d + pad) + offset,), float("nan"), dtype=t.dtype, device=t.device)
    v = flat[offset:offset + n * (d + pad)].view(n, d + pad)[:, :d]
    v.copy_(t)
    return v
