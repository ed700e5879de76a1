"""The norm and the dense layers at the ends of their ranges: operands past 4 GiB, rows of whole words, many
products' tiles, sums on both sides of their splits, the same bits every time, two streams at once."""
import pytest
import torch

from . import layers as ref
from .test_gpu_dense import B, F, d64, gated_case, linear_case, normal, space

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")


@pytest.mark.parametrize("shape", [(3, 130, 70), (40, 1034, 518), (90, 62, 1030), (700, 134, 516), (1500, 516, 1030),
                                   (4100, 258, 2050)])
@pytest.mark.parametrize("pad, offset", [(0, 0), (2, 2), (6, 4)])
def test_bf16_rows_of_whole_words(shape, pad, offset):
    """Rows at multiples of 4 bytes but not of 16."""
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    place = (lambda t: ref.strided(t, pad, offset)) if pad else (lambda t: t)
    linear_case(*shape, B, "gelu", g, place)
    gated_case(*shape, B, "silu", g, place)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape", [(1, 16, 20000), (2, 9000, 16), (6000, 16, 16), (17, 8200, 40), (300, 20, 8200),
                                   (2000, 1500, 8), (100000, 24, 40), (513, 2048, 300)])
def test_long_in_one_direction(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(7)
    linear_case(*shape, dtype, "relu", g)
    gated_case(*shape, dtype, "sigmoid", g)


@pytest.mark.parametrize("dtype", [F, B])
def test_layers_past_4_gib(dtype):
    """x of over 2^32 bytes, whose rows are zero but for the last: their results, and the weights' gradients."""
    i, o, last = 2048, 40, 70
    n = (1 << 32) // (i * (2 if dtype == B else 4)) + 1000
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(n, i, device="cuda", dtype=dtype)
    x[-last:] = normal(last, i, dtype=dtype, gen=g)
    w = normal(i, o, dtype=dtype, gen=g, scale=i ** -0.5)
    b = normal(o, dtype=dtype, gen=g)
    out = torch.full((n, o), 9.0, device="cuda", dtype=dtype)
    gm.gnn_linear(x, w, out, space(gm.gnn_linear_workspace_size, n, i, o, dtype), bias=b)
    y, ey, _, _ = ref.linear(d64(x[-last:]), d64(w), d64(b), "none", None, dtype)
    ref.close(out[-last:], (y, ey))
    assert torch.equal(out[:n - last], b.expand(n - last, o))
    dout = normal(n, o, dtype=dtype, gen=g)
    dx, dw = torch.full_like(x, 9.0), torch.empty_like(w)
    gm.gnn_linear_backward(x, w, dout, space(gm.gnn_linear_workspace_size, n, i, o, dtype, True), dx=dx, dw=dw)
    want = ref.linear_gradients(d64(x[-last:]), d64(w), d64(dout[-last:]), "none", None, dtype)
    ref.close(dx[-last:], want[0])
    ref.close(dw, want[1])
    first = ref.linear_gradients(d64(x[:last]), d64(w), d64(dout[:last]), "none", None, dtype)
    ref.close(dx[:last], first[0])


def test_wide_outputs_past_4_gib():
    n, i, o, last = 70_000, 32, 32_768, 40
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = normal(n, i, dtype=B, gen=g), normal(i, o, dtype=B, gen=g)
    out = torch.full((n, o), 9.0, device="cuda", dtype=B)
    gm.gnn_linear(x, w, out, space(gm.gnn_linear_workspace_size, n, i, o, B), activation="relu")
    for rows in (slice(0, last), slice(n - last, n)):
        y, ey, _, _ = ref.linear(d64(x[rows]), d64(w), None, "relu", None, B)
        ref.close(out[rows], (y, ey))
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    dout = torch.zeros_like(out)
    dout[-last:] = normal(last, o, dtype=B, gen=g)
    gm.gnn_linear_backward(x, w, dout, space(gm.gnn_linear_workspace_size, n, i, o, B, True), activation="relu",
                           pre=out, dx=dx, dw=dw)
    # (relu's output is its pre as far as the slope goes)
    want = ref.linear_gradients(d64(x[-last:]), d64(w), d64(dout[-last:]), "relu", d64(out[-last:]), B)
    ref.close(dx[-last:], want[0])
    assert (dx[:n - last] == 0).all()
    dw_want, dw_bound = want[1]
    # n = 70000 rows: one plane of dz; a slope of 0 or 1 rounds nothing
    ref.close(dw, (dw_want, dw_bound))


def test_norm_past_4_gib():
    n, d, last = 530_000, 4096, 50
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.zeros(n, d, device="cuda", dtype=B)
    x[-last:] = normal(last, d, dtype=B, gen=g)
    w, b = normal(d, dtype=B, gen=g), normal(d, dtype=B, gen=g)
    out, mean, rstd = torch.empty_like(x), *torch.empty(2, n, device="cuda")
    gm.gnn_layer_norm(x, w, b, 1e-5, out, mean=mean, rstd=rstd)
    ref.close(out[-last:], ref.norm(d64(x[-last:]), d64(w), d64(b), 1e-5, B)[0])
    assert torch.equal(out[:1000], b.expand(1000, d)) and (mean[:n - last] == 0).all()
    dout, dx = torch.zeros_like(x), torch.full_like(x, 9.0)
    dout[-last:] = normal(last, d, dtype=B, gen=g)
    dw, db = torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(gm.gnn_layer_norm_workspace_size(n, d), dtype=torch.uint8, device="cuda")
    gm.gnn_layer_norm_backward(x, w, mean, rstd, dout, dx, ws, dweight=dw, dbias=db)
    want = ref.norm_gradients(d64(x[-last:]), d64(w), mean[-last:].double(), rstd[-last:].double(),
                              d64(dout[-last:]), None, B, B)
    for got, exact in zip((dx[-last:], dw, db), want):
        ref.close(got, exact)
    assert (dx[:n - last] == 0).all()


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape", [(2, 1000, 300), (700, 300, 520), (3000, 1024, 1032)])
def test_the_same_bits_every_time_and_two_streams_at_once(shape, dtype):
    n, i, o = shape
    g = torch.Generator(device="cuda").manual_seed(4)
    x, wg, wu = normal(n, i, dtype=dtype, gen=g), *normal(2, i, o, dtype=dtype, gen=g, scale=0.1)
    dout = normal(n, o, dtype=dtype, gen=g)
    w, b = normal(i, dtype=F, gen=g), normal(i, dtype=F, gen=g)

    def run(stream):
        with torch.cuda.stream(stream):
            y, (mean, rstd) = torch.empty_like(x), torch.empty(2, n, device="cuda")
            out, gate, up = torch.empty(3, n, o, device="cuda", dtype=dtype)
            dx, dwg, dwu, dy = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu), torch.empty_like(x)
            db, dn = torch.empty(2, o, device="cuda", dtype=dtype), torch.empty(2, i, device="cuda")
            ws = space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype)
            wsb = space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype, True)
            wsn = torch.empty(gm.gnn_layer_norm_workspace_size(n, i), dtype=torch.uint8, device="cuda")
            for _ in range(3):
                gm.gnn_layer_norm(x, w, b, 1e-5, y, mean=mean, rstd=rstd)
                gm.gnn_gated_linear(y, wg, wu, out, ws, gate=gate, up=up)
                gm.gnn_gated_linear_backward(y, wg, wu, gate, up, dout, wsb, dx=dy, dw_gate=dwg, dw_up=dwu,
                                             dbias_gate=db[0], dbias_up=db[1])
                gm.gnn_layer_norm_backward(x, w, mean, rstd, dy, dx, wsn, dweight=dn[0], dbias=dn[1])
            return out, gate, up, dx, dwg, dwu, db, dn

    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    first, second = (run(s) for s in streams)
    torch.cuda.synchronize()
    third = run(torch.cuda.current_stream())
    torch.cuda.synchronize()
    for a, b, c in zip(first, second, third):
        assert torch.equal(a, b) and torch.equal(a, c)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape", [(1, 515, 1371), (3, 1, 520), (5, 130, 8), (7, 99, 843), (8, 1000, 9), (8, 65, 1032)])
def test_a_few_rows(shape, dtype):
    """Gradients of weights that a few rows give: whole and cut lines and columns, rows off any alignment."""
    g = torch.Generator(device="cuda").manual_seed(8)
    for place in (lambda t: t, lambda t: ref.strided(t, 3, 1)):
        results = linear_case(*shape, dtype, "gelu", g, place) + gated_case(*shape, dtype, "silu", g, place)
        for t in results:
            if t._base is not None and t._base.dim() == 1:
                n, d = t.shape
                assert torch.isnan(t._base[1:1 + n * (d + 3)].view(n, d + 3)[:, d:]).all()


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("count", [0, 1, 5, 8, 9])
def test_a_few_rows_that_count(count, dtype):
    g = torch.Generator(device="cuda").manual_seed(9)
    n, i, o, m = 8, 300, 328, min(count, 8)
    x, wg, wu = normal(n, i, dtype=dtype, gen=g), *normal(2, i, o, dtype=dtype, gen=g, scale=0.1)
    dout, gate, up = normal(n, o, dtype=dtype, gen=g), *normal(2, n, o, dtype=dtype, gen=g)
    for t in (x, dout, gate, up):
        t[m:] = float("nan")
    dx, dwg, dwu = torch.full_like(x, 7.0), torch.empty_like(wg), torch.empty_like(wu)
    gm.gnn_gated_linear_backward(x, wg, wu, gate, up, dout,
                                 space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype, True), dx=dx, dw_gate=dwg,
                                 dw_up=dwu, d_n=torch.tensor([count], device="cuda"))
    want = ref.gated_gradients(d64(x[:m]), d64(wg), d64(wu), d64(dout[:m]), "silu", d64(gate[:m]), d64(up[:m]), dtype)
    assert (dx[m:] == 7).all()
    for got, exact in zip((dx[:m], dwg, dwu), (want[0], want[1], want[3])):
        ref.close(got, exact)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape", [(4, 40, 24), (20, 70, 50), (300, 64, 640), (600, 136, 72)])
def test_infinite_gradients_stay_infinite(shape, dtype):
    """One infinity of dout: its row of dx and its column of dw and dbias are infinite with the sign of the other
    factor, and all others are what they are without it.  (Sums of one and of two planes of dz.)"""
    n, i, o = shape
    g = torch.Generator(device="cuda").manual_seed(10)
    x, w, dout = normal(n, i, dtype=dtype, gen=g), normal(i, o, dtype=dtype, gen=g), normal(n, o, dtype=dtype, gen=g)
    x[1] = torch.where(x[1] < 0, x[1] - 0.1, x[1] + 0.1)      # no zeros meet the infinity
    w[:, 2] = torch.where(w[:, 2] < 0, w[:, 2] - 0.1, w[:, 2] + 0.1)
    pre = torch.ones_like(dout)      # a slope above 0
    ws = space(gm.gnn_linear_workspace_size, n, i, o, dtype, True)

    def gradients():
        dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty(o, device="cuda", dtype=dtype)
        gm.gnn_linear_backward(x, w, dout, ws, activation="gelu", pre=pre, dx=dx, dw=dw, dbias=db)
        return dx, dw, db

    clean = gradients()
    dout[1, 2] = float("inf")
    dx, dw, db = gradients()
    assert torch.equal(dx[1], w[:, 2].sign() * float("inf"))
    assert torch.equal(dw[:, 2], x[1].sign() * float("inf"))
    assert float(db[2]) == float("inf")
    rows, cols = torch.arange(n, device="cuda") != 1, torch.arange(o, device="cuda") != 2
    assert torch.equal(dx[rows], clean[0][rows]) and torch.equal(dw[:, cols], clean[1][:, cols])
    assert torch.equal(db[cols], clean[2][cols])


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("n, d", [(9, 7), (33, 101), (20, 521), (11, 1031), (5, 4099), (5, 8195), (3, 16383)])
def test_norms_in_place_at_odd_widths(n, d, dtype):
    """out over x and dx over residual_grad where a row's last pieces overlap."""
    g = torch.Generator(device="cuda").manual_seed(11)
    x, w, dout, dres = normal(n, d, dtype=dtype, gen=g), normal(d, dtype=dtype, gen=g), \
        normal(n, d, dtype=dtype, gen=g), normal(n, d, dtype=dtype, gen=g)
    out, y, mean, rstd = torch.empty_like(x), x.clone(), *torch.empty(2, n, device="cuda")
    gm.gnn_layer_norm(x, w, None, 1e-5, out, mean=mean, rstd=rstd)
    gm.gnn_layer_norm(y, w, None, 1e-5, y)
    ws = torch.empty(gm.gnn_layer_norm_workspace_size(n, d), dtype=torch.uint8, device="cuda")
    dx, over = torch.empty_like(x), dres.clone()
    gm.gnn_layer_norm_backward(x, w, mean, rstd, dout, dx, ws, residual_grad=dres)
    gm.gnn_layer_norm_backward(x, w, mean, rstd, dout, over, ws, residual_grad=over)
    assert torch.equal(y, out) and torch.equal(over, dx)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape", [(1, 512, 256), (3, 1030, 257), (77, 515, 137), (700, 300, 520), (2500, 64, 1032)])
def test_out_over_the_residual(shape, dtype):
    n, i, o = shape
    g = torch.Generator(device="cuda").manual_seed(12)
    x, w, r = normal(n, i, dtype=dtype, gen=g), normal(i, o, dtype=dtype, gen=g), normal(n, o, dtype=dtype, gen=g)
    ws = space(gm.gnn_linear_workspace_size, n, i, o, dtype)
    for place in (lambda t: t.clone(), lambda t: ref.strided(t, 3, 1)):
        over = place(r)
        apart = place(torch.zeros_like(r))
        gm.gnn_linear(x, w, apart, ws, activation="silu", residual=place(r))
        gm.gnn_linear(x, w, over, ws, activation="silu", residual=over)
        assert torch.equal(over, apart)


@pytest.mark.parametrize("dtype", [F, B])
def test_a_few_rows_captured(dtype):
    g = torch.Generator(device="cuda").manual_seed(13)
    n, i, o = 5, 515, 328
    x, wg, wu = normal(n, i, dtype=dtype, gen=g), *normal(2, i, o, dtype=dtype, gen=g, scale=0.1)
    dout, gate, up = normal(n, o, dtype=dtype, gen=g), *normal(2, n, o, dtype=dtype, gen=g)
    dx, dwg, dwu, db = torch.empty_like(x), torch.empty_like(wg), torch.empty_like(wu), \
        torch.empty(2, o, device="cuda", dtype=dtype)
    ws, count = space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype, True), torch.tensor([5], device="cuda")

    def step():
        gm.gnn_gated_linear_backward(x, wg, wu, gate, up, dout, ws, dx=dx, dw_gate=dwg, dw_up=dwu, dbias_gate=db[0],
                                     dbias_up=db[1], d_n=count)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    results = (dx, dwg, dwu, db)
    for m in (5, 2, 0):      # the count is read at the replay
        count.fill_(m)
        x.copy_(normal(n, i, dtype=dtype, gen=g))
        for t in results:
            t.fill_(-1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in results]
        for t in results:
            t.fill_(-1.0)
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, results)), m
