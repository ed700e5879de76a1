"""The dense layer and the gated pair, forward and backward, against the formulas in 64 bits
(tests/layers.py has the bounds)."""
import pytest
import torch

from . import layers as ref

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")

F, B = torch.float32, torch.bfloat16
# (n, d_in, d_out): one row to many; every tile shape, whole tiles and cut ones, widths below a piece, sums that
# are split, lengths of less than a step of the summed index, and rows on both sides of 512
SHAPES = [(1, 1, 1), (1, 64, 128), (1, 2048, 1024), (2, 3, 5), (5, 7, 3), (8, 72, 136), (31, 130, 264), (33, 64, 8),
          (64, 1000, 200), (65, 128, 128), (128, 31, 257), (200, 520, 72), (129, 1030, 131), (257, 96, 515),
          (511, 64, 256), (512, 65, 256), (600, 256, 512), (777, 136, 1000), (2500, 40, 24)]
LARGE = [(4096, 768, 1024), (4100, 1032, 1032), (9000, 256, 2048)]


def normal(*shape, dtype, gen, scale=1.0):
    return (scale * torch.randn(*shape, generator=gen, device="cuda")).to(dtype)


def d64(t):
    return None if t is None else t.double()


def space(call, n, i, o, dtype, backward=False):
    return torch.empty(call(n, i, o, dtype, backward=backward), dtype=torch.uint8, device="cuda")


def linear_case(n, i, o, dtype, name, gen, place=lambda t: t, bias=True, residual=True):
    """Forward and backward of a linear layer against the formulas."""
    x, w = place(normal(n, i, dtype=dtype, gen=gen)), place(normal(i, o, dtype=dtype, gen=gen, scale=i ** -0.5))
    b = normal(o, dtype=dtype, gen=gen) if bias else None
    r = place(normal(n, o, dtype=dtype, gen=gen)) if residual else None
    out, pre = (place(torch.zeros(n, o, device="cuda", dtype=dtype)) for _ in range(2))
    gm.gnn_linear(x, w, out, space(gm.gnn_linear_workspace_size, n, i, o, dtype), bias=b, activation=name,
                  residual=r, pre=pre)
    y, ey, z, ez = ref.linear(d64(x), d64(w), d64(b), name, d64(r), dtype)
    ref.close(out, (y, ey), "out")
    ref.close(pre, (z, ez), "pre")
    dout = place(normal(n, o, dtype=dtype, gen=gen))
    dx, dw = place(torch.zeros(n, i, device="cuda", dtype=dtype)), place(torch.zeros(i, o, device="cuda", dtype=dtype))
    db = torch.empty(o, device="cuda", dtype=dtype)
    gm.gnn_linear_backward(x, w, dout, space(gm.gnn_linear_workspace_size, n, i, o, dtype, True), activation=name,
                           pre=pre, dx=dx, dw=dw, dbias=db)
    want = ref.linear_gradients(d64(x), d64(w), d64(dout), name, d64(pre), dtype)
    for got, exact, what in zip((dx, dw, db), want, ("dx", "dw", "dbias")):
        ref.close(got, exact, what)
    return out, pre, dx, dw


def gated_case(n, i, o, dtype, name, gen, place=lambda t: t, bias=True):
    x = place(normal(n, i, dtype=dtype, gen=gen))
    wg, wu = (place(normal(i, o, dtype=dtype, gen=gen, scale=i ** -0.5)) for _ in range(2))
    bg, bu = (normal(o, dtype=dtype, gen=gen) if bias else None for _ in range(2))
    out, gate, up = (place(torch.zeros(n, o, device="cuda", dtype=dtype)) for _ in range(3))
    gm.gnn_gated_linear(x, wg, wu, out, space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype), bias_gate=bg,
                        bias_up=bu, activation=name, gate=gate, up=up)
    want = ref.gated(d64(x), d64(wg), d64(wu), d64(bg), d64(bu), name, dtype)
    for got, exact, what in zip((out, gate, up), want, ("out", "gate", "up")):
        ref.close(got, exact, what)
    dout = place(normal(n, o, dtype=dtype, gen=gen))
    dx = place(torch.zeros(n, i, device="cuda", dtype=dtype))
    dwg, dwu = (place(torch.zeros(i, o, device="cuda", dtype=dtype)) for _ in range(2))
    dbg, dbu = torch.empty(2, o, device="cuda", dtype=dtype)
    gm.gnn_gated_linear_backward(x, wg, wu, gate, up, dout,
                                 space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype, True), activation=name,
                                 dx=dx, dw_gate=dwg, dw_up=dwu, dbias_gate=dbg, dbias_up=dbu)
    want = ref.gated_gradients(d64(x), d64(wg), d64(wu), d64(dout), name, d64(gate), d64(up), dtype)
    for got, exact, what in zip((dx, dwg, dbg, dwu, dbu), want, ("dx", "dw_gate", "dbias_gate", "dw_up", "dbias_up")):
        ref.close(got, exact, what)
    return out, gate, up, dx, dwg, dwu


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape", SHAPES)
def test_linear(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    linear_case(*shape, dtype, ref.ACTS[sum(shape) % 6], g)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape", SHAPES)
def test_gated(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(sum(shape) + 1)
    gated_case(*shape, dtype, ref.ACTS[(sum(shape) + 1) % 6], g)


@pytest.mark.parametrize("name", ref.ACTS)
@pytest.mark.parametrize("dtype", [F, B])
def test_activations(name, dtype):
    g = torch.Generator(device="cuda").manual_seed(3)
    linear_case(150, 64, 96, dtype, name, g, bias=False, residual=False)
    gated_case(150, 64, 96, dtype, name, g, bias=False)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape", LARGE)
def test_large(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(4)
    linear_case(*shape, dtype, "silu", g)
    gated_case(*shape, dtype, "gelu", g)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("pad, offset", [(8, 0), (5, 0), (8, 3), (1, 1)])
@pytest.mark.parametrize("shape", [(3, 40, 24), (70, 136, 72), (300, 264, 520)])
def test_strided_rows(shape, pad, offset, dtype):
    """Rows apart: at multiples of 16 bytes (pad 8, or 4 in fp32), at others, and off any alignment.  What lies
    between the rows is neither read nor written."""
    g = torch.Generator(device="cuda").manual_seed(5)

    def place(t):
        return ref.strided(t, pad, offset)

    for results in (linear_case(*shape, dtype, "gelu_tanh", g, place), gated_case(*shape, dtype, "sigmoid", g, place)):
        for t in results:
            n, d = t.shape
            between = t._base[offset:offset + n * (d + pad)].view(n, d + pad)[:, d:]
            assert torch.isnan(between).all()


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("n, count", [(40, 7), (40, 0), (300, 300), (300, 100), (700, 513), (700, 300), (700, 9999), (300, -1)])
def test_the_rows_that_count(n, count, dtype):
    """Rows past the device count are neither written nor added, whatever they hold."""
    g = torch.Generator(device="cuda").manual_seed(6)
    i, o, m = 200, 328, max(0, min(n, count))
    nan = float("nan")
    d_n = torch.tensor([count], device="cuda")
    x, wg, wu = normal(n, i, dtype=dtype, gen=g), *normal(2, i, o, dtype=dtype, gen=g, scale=0.1)
    x[m:] = nan
    dout = normal(n, o, dtype=dtype, gen=g)
    dout[m:] = nan
    out, gate, up = torch.full((3, n, o), 7.0, device="cuda", dtype=dtype)
    dx = torch.full((n, i), 7.0, device="cuda", dtype=dtype)
    gm.gnn_gated_linear(x, wg, wu, out, space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype), gate=gate, up=up,
                        d_n=d_n)
    want = ref.gated(d64(x[:m]), d64(wg), d64(wu), None, None, "silu", dtype)
    for t, exact in zip((out, gate, up), want):
        assert (t[m:] == 7).all()
        ref.close(t[:m], exact)
    gate[m:], up[m:] = nan, nan
    dwg, dwu, dbs = torch.empty_like(wg), torch.empty_like(wu), torch.empty(2, o, device="cuda", dtype=dtype)
    gm.gnn_gated_linear_backward(x, wg, wu, gate, up, dout,
                                 space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype, True), dx=dx, dw_gate=dwg,
                                 dw_up=dwu, dbias_gate=dbs[0], dbias_up=dbs[1], d_n=d_n)
    assert (dx[m:] == 7).all()
    want = ref.gated_gradients(d64(x[:m]), d64(wg), d64(wu), d64(dout[:m]), "silu", d64(gate[:m]), d64(up[:m]), dtype)
    for got, exact in zip((dx[:m], dwg, dbs[0], dwu, dbs[1]), want):
        ref.close(got, exact)
    out.fill_(7.0)
    gm.gnn_linear(x, wg, out, space(gm.gnn_linear_workspace_size, n, i, o, dtype), residual=out, d_n=d_n)
    y, ey, _, _ = ref.linear(d64(x[:m]), d64(wg), None, "none", torch.full((m, o), 7.0, device="cuda").double(), dtype)
    assert (out[m:] == 7).all()
    ref.close(out[:m], (y, ey))


@pytest.mark.parametrize("dtype", [F, B])
def test_no_rows(dtype):
    i, o = 48, 40
    w = normal(i, o, dtype=dtype, gen=torch.Generator(device="cuda"))
    x, y = torch.empty(0, i, device="cuda", dtype=dtype), torch.empty(0, o, device="cuda", dtype=dtype)
    gm.gnn_linear(x, w, y, space(gm.gnn_linear_workspace_size, 0, i, o, dtype), activation="gelu", pre=y)
    dw, db = torch.full_like(w, 3.0), torch.full((o,), 3.0, device="cuda", dtype=dtype)
    gm.gnn_linear_backward(x, w, y, space(gm.gnn_linear_workspace_size, 0, i, o, dtype, True), activation="gelu",
                           pre=y, dx=x, dw=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()
    dw2 = torch.full_like(w, 3.0)
    gm.gnn_gated_linear(x, w, w, y, space(gm.gnn_gated_linear_workspace_size, 0, i, o, dtype))
    gm.gnn_gated_linear_backward(x, w, w, y, y, y, space(gm.gnn_gated_linear_workspace_size, 0, i, o, dtype, True),
                                 dx=x, dw_gate=dw.fill_(3.0), dw_up=dw2)
    assert (dw == 0).all() and (dw2 == 0).all()


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("n", [20, 600])
def test_halves_of_merged_matrices_and_parts_of_the_gradients(n, dtype):
    """w_gate and w_up as halves of one matrix, their sums and gradients too; each gradient by itself is what it is
    among all; the same call gives the same bits."""
    g = torch.Generator(device="cuda").manual_seed(7)
    i, o = 128, 192
    x, w, dout = normal(n, i, dtype=dtype, gen=g), normal(i, 2 * o, dtype=dtype, gen=g, scale=0.1), \
        normal(n, o, dtype=dtype, gen=g)
    out, kept, dw = torch.empty_like(dout), torch.empty(n, 2 * o, device="cuda", dtype=dtype), torch.empty_like(w)
    gm.gnn_gated_linear(x, w[:, :o], w[:, o:], out, space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype),
                        gate=kept[:, :o], up=kept[:, o:])
    want = ref.gated(d64(x), d64(w[:, :o]), d64(w[:, o:]), None, None, "silu", dtype)
    for t, exact in zip((out, kept[:, :o], kept[:, o:]), want):
        ref.close(t, exact)
    out2 = torch.empty_like(out)
    gm.gnn_gated_linear(x, w[:, :o], w[:, o:], out2, space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype))
    assert torch.equal(out2, out)
    ws = space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype, True)
    args = (x, w[:, :o], w[:, o:], kept[:, :o], kept[:, o:], dout, ws)
    dx, dbs = torch.empty_like(x), torch.empty(2, o, device="cuda", dtype=dtype)
    gm.gnn_gated_linear_backward(*args, dx=dx, dw_gate=dw[:, :o], dw_up=dw[:, o:], dbias_gate=dbs[0], dbias_up=dbs[1])
    want = ref.gated_gradients(d64(x), d64(w[:, :o]), d64(w[:, o:]), d64(dout), "silu", d64(kept[:, :o]),
                               d64(kept[:, o:]), dtype)
    for t, exact in zip((dx, dw[:, :o], dbs[0], dw[:, o:], dbs[1]), want):
        ref.close(t, exact)
    one = [torch.empty_like(dx), torch.empty_like(w[:, :o].contiguous()), torch.empty_like(w[:, :o].contiguous()),
           torch.empty_like(dbs[0]), torch.empty_like(dbs[1])]
    for name, t in zip(("dx", "dw_gate", "dw_up", "dbias_gate", "dbias_up"), one):
        gm.gnn_gated_linear_backward(*args, **{name: t})
    ref.close(one[1], want[1])
    ref.close(one[2], want[3])
    assert torch.equal(one[0], dx) and torch.equal(one[3], dbs[0]) and torch.equal(one[4], dbs[1])


@pytest.mark.parametrize("n", [4, 300])
def test_what_is_not_finite_stays_in_its_row(n):
    """An infinity or NaN of x reaches its own row of out alone, although tiles are filled up beside it."""
    g = torch.Generator(device="cuda").manual_seed(8)
    i, o = 70, 50
    for dtype in (F, B):
        x, w = normal(n, i, dtype=dtype, gen=g), normal(i, o, dtype=dtype, gen=g)
        ws = space(gm.gnn_linear_workspace_size, n, i, o, dtype)
        clean, out = torch.empty(2, n, o, device="cuda", dtype=dtype)
        gm.gnn_linear(x, w, clean, ws)
        x[1, 69], x[3, 0] = float("inf"), float("nan")
        gm.gnn_linear(x, w, out, ws)
        live = [r for r in range(n) if r not in (1, 3)]
        assert torch.equal(out[live], clean[live])
        assert torch.isinf(out[1]).all() and torch.isnan(out[3]).all()


def test_relu_keeps_nan_and_stops_infinity():
    x = torch.tensor([[float("nan")], [float("inf")], [-float("inf")], [-2.0], [0.0]], device="cuda")
    w, out = torch.ones(1, 1, device="cuda"), torch.empty(5, 1, device="cuda")
    gm.gnn_linear(x, w, out, space(gm.gnn_linear_workspace_size, 5, 1, 1, F), activation="relu")
    assert torch.isnan(out[0]).all() and out[1:, 0].tolist() == [float("inf"), 0.0, 0.0, 0.0]


@pytest.mark.parametrize("dtype", [F, B])
def test_far_arguments_of_the_activations(dtype):
    """act and act' at far arguments: the limits, no NaN where the limit is a number."""
    z = torch.tensor([[-1e4], [-200.0], [-50.0], [50.0], [200.0], [1e4]], device="cuda", dtype=dtype)
    one = torch.ones(1, 1, device="cuda", dtype=dtype)
    for name in ref.ACTS[2:]:
        out, dx = torch.empty_like(z), torch.empty_like(z)
        gm.gnn_linear(z, one, out, space(gm.gnn_linear_workspace_size, 6, 1, 1, dtype), activation=name)
        gm.gnn_linear_backward(z, one, torch.ones_like(z), space(gm.gnn_linear_workspace_size, 6, 1, 1, dtype, True),
                               activation=name, pre=z, dx=dx)
        y, s = ref.act(name, z.double())
        assert torch.allclose(out.double(), y, rtol=1e-2, atol=1e-18), name
        assert torch.allclose(dx.double(), s, rtol=1e-2, atol=1e-18), name


def test_captured_and_replayed_on_another_stream():
    """A small (split) and a large product, in a graph on a stream of its own, against eager calls."""
    g = torch.Generator(device="cuda").manual_seed(9)
    for n, i, o in ((3, 512, 256), (700, 256, 512)):
        x, w, dout = normal(n, i, dtype=B, gen=g), normal(i, o, dtype=B, gen=g, scale=0.1), normal(n, o, dtype=B, gen=g)
        out, pre, dx, dw = torch.empty_like(dout), torch.empty_like(dout), torch.empty_like(x), torch.empty_like(w)
        db = torch.empty(o, device="cuda", dtype=B)
        ws = space(gm.gnn_linear_workspace_size, n, i, o, B)
        wsb = space(gm.gnn_linear_workspace_size, n, i, o, B, True)

        def step():
            gm.gnn_linear(x, w, out, ws, activation="gelu", pre=pre)
            gm.gnn_linear_backward(x, w, dout, wsb, activation="gelu", pre=pre, dx=dx, dw=dw, dbias=db)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        results = (out, pre, dx, dw, db)
        for turn in range(3):
            x.copy_(normal(n, i, dtype=B, gen=g))
            for t in results:
                t.fill_(-1.0)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            replayed = [t.clone() for t in results]
            step()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(replayed, results)), turn


@pytest.mark.parametrize("name", ["gelu", "gelu_tanh", "silu", "sigmoid", "none"])
def test_gradients_against_differences(name):
    """L = sum(dout * out) along directions in x and the weights, by central differences of the kernels' outputs in
    fp32 at +-e.  The third derivatives are of order 1, so e^2 / 6 of the terms' sizes is below 2e-5 of them
    (e = 1e-2); the outputs and the moved inputs are rounded: 2^-24 / e of the terms, 6e-6, times some ten."""
    g = torch.Generator(device="cuda").manual_seed(12)
    n, i, o, e = 40, 64, 72, 1e-2
    x, wg, wu = normal(n, i, dtype=F, gen=g), *normal(2, i, o, dtype=F, gen=g, scale=i ** -0.5)
    dout = normal(n, o, dtype=F, gen=g)
    gate, up, dx = torch.empty_like(dout), torch.empty_like(dout), torch.empty_like(x)
    dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
    ws = space(gm.gnn_gated_linear_workspace_size, n, i, o, F)

    def loss(x, wg, wu, sizes=False):
        y = torch.empty_like(dout)
        gm.gnn_gated_linear(x, wg, wu, y, ws, activation=name, gate=gate, up=up)
        t = dout.double() * y.double()
        return float(t.abs().sum()) if sizes else float(t.sum())

    size = loss(x, wg, wu, True)
    gm.gnn_gated_linear_backward(x, wg, wu, gate, up, dout,
                                 space(gm.gnn_gated_linear_workspace_size, n, i, o, F, True), activation=name, dx=dx,
                                 dw_gate=dwg, dw_up=dwu)
    base = (x, wg, wu)
    for which, got in enumerate((dx, dwg, dwu)):
        v = normal(*got.shape, dtype=F, gen=g, scale=1.0 if which == 0 else i ** -0.5)
        hi, lo = ([t + s * e * v if j == which else t for j, t in enumerate(base)] for s in (1, -1))
        slope = float((got.double() * v.double()).sum())
        terms = float((got.double() * v.double()).abs().sum())
        assert abs((loss(*hi) - loss(*lo)) / (2 * e) - slope) <= 1e-3 * (terms + size) / n ** 0.5, which
