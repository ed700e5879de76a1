"""Layer norm and its backward pass against the formulas in 64 bits (tests/layers.py has the bounds)."""
import pytest
import torch

from . import layers as ref

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")

F, B = torch.float32, torch.bfloat16
# a lane group of each width, its ends, a workgroup's, and widths that are no whole pieces
SHAPES = [(1, 1), (3, 7), (1, 4096), (37, 64), (33, 65), (130, 100), (19, 129), (65, 256), (9, 300), (21, 512),
          (11, 1000), (7, 1025), (5, 2048), (6, 2049), (3, 4095), (3, 4097), (2, 8191), (3, 16384)]
TYPES = [(F, F, F), (B, B, B), (F, B, F), (B, F, B), (F, F, B)]


def rows(n, d, dtype, gen, scale=1.0, shift=0.0):
    return (scale * torch.randn(n, d, generator=gen, device="cuda") + shift).to(dtype)


def d64(t):
    return None if t is None else t.double()


def space(n, d):
    return torch.empty(gm.gnn_layer_norm_workspace_size(n, d), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("x_type, out_type, param", TYPES)
@pytest.mark.parametrize("n, d", SHAPES)
def test_against_the_formulas(n, d, x_type, out_type, param):
    g = torch.Generator(device="cuda").manual_seed(n * 7919 + d)
    x = rows(n, d, x_type, g, 2.0, 0.5)
    w, b = rows(1, d, param, g, 0.3, 1.0)[0], rows(1, d, param, g)[0]
    out, mean, rstd = torch.empty(n, d, device="cuda", dtype=out_type), *torch.empty(2, n, device="cuda")
    gm.gnn_layer_norm(x, w, b, 1e-5, out, mean=mean, rstd=rstd)
    want = ref.norm(d64(x), d64(w), d64(b), 1e-5, out_type)
    for got, exact, name in zip((out, mean, rstd), want, ("out", "mean", "rstd")):
        ref.close(got, exact, name)
    dout, dres = rows(n, d, out_type, g), rows(n, d, x_type, g) if n % 2 else None
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    gm.gnn_layer_norm_backward(x, w, mean, rstd, dout, dx, space(n, d), dweight=dw, dbias=db,
                               residual_grad=dres)
    want = ref.norm_gradients(d64(x), d64(w), mean.double(), rstd.double(), d64(dout), d64(dres), x_type, param)
    for got, exact, name in zip((dx, dw, db), want, ("dx", "dweight", "dbias")):
        ref.close(got, exact, name)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("offset", [0, 1])
def test_strided_rows_and_no_parameters(dtype, offset):
    """Rows apart and off any alignment, no weight, no bias; more rows than a workgroup's turn."""
    g = torch.Generator(device="cuda").manual_seed(5)
    n, d = 3001, 75
    x = ref.strided(rows(n, d, dtype, g), 6, offset)
    dout = ref.strided(rows(n, d, dtype, g), 3, offset)
    out, dx = (ref.strided(torch.zeros(n, d, device="cuda", dtype=dtype), 9, offset) for _ in range(2))
    mean, rstd = torch.empty(2, n, device="cuda")
    gm.gnn_layer_norm(x, None, None, 1e-5, out, mean=mean, rstd=rstd)
    ref.close(out, ref.norm(d64(x), None, None, 1e-5, dtype)[0])
    assert torch.isnan(out._base.view(-1)[offset + d:offset + d + 9]).all()      # between the rows
    dw = torch.empty(d, device="cuda", dtype=dtype)
    gm.gnn_layer_norm_backward(x, None, mean, rstd, dout, dx, space(n, d), dweight=dw)
    want = ref.norm_gradients(d64(x), None, mean.double(), rstd.double(), d64(dout), None, dtype, dtype)
    ref.close(dx, want[0])
    ref.close(dw, want[1])
    assert torch.isnan(dx._base.view(-1)[offset + d:offset + d + 9]).all()


def test_a_large_offset_keeps_its_digits():
    """Rows of 1000 + noise in fp32: the variance is of the differences from the mean."""
    g = torch.Generator(device="cuda").manual_seed(6)
    x = rows(64, 768, F, g, 0.01, 1000.0)
    out = torch.empty_like(x)
    gm.gnn_layer_norm(x, None, None, 0.0, out)
    ref.close(out, ref.norm(d64(x), None, None, 0.0, F)[0])


def test_constant_rows():
    x = torch.full((5, 100), 3.25, device="cuda")
    w, b = torch.randn(100, device="cuda"), torch.randn(100, device="cuda")
    out, mean, rstd = torch.empty_like(x), *torch.empty(2, 5, device="cuda")
    gm.gnn_layer_norm(x, w, b, 1e-5, out, mean=mean, rstd=rstd)
    assert torch.equal(out, b.expand_as(out)) and torch.equal(mean, torch.full_like(mean, 3.25))


@pytest.mark.parametrize("d", [100, 3000])
def test_a_row_that_is_not_finite_stays_alone(d):
    g = torch.Generator(device="cuda").manual_seed(7)
    x = rows(9, d, F, g)
    clean = torch.empty_like(x)
    gm.gnn_layer_norm(x, None, None, 1e-5, clean)
    x[2, 3], x[7, 0] = float("inf"), float("nan")
    out = torch.empty_like(x)
    gm.gnn_layer_norm(x, None, None, 1e-5, out)
    live = torch.ones(9, dtype=torch.bool, device="cuda")
    live[[2, 7]] = False
    assert torch.equal(out[live], clean[live]) and torch.isnan(out[~live]).all()


@pytest.mark.parametrize("count", [0, 1, 41, 100, 1000, -3])
@pytest.mark.parametrize("d", [72, 2500])
def test_the_rows_that_count(count, d):
    """Rows past the device count are neither written nor added; a count beyond n is n."""
    g = torch.Generator(device="cuda").manual_seed(8)
    n = 100
    m = max(0, min(n, count))
    x, dout = rows(n, d, F, g), rows(n, d, F, g)
    x[m:], dout[m:] = float("nan"), float("nan")
    w = rows(1, d, F, g)[0]
    d_n = torch.tensor([count], device="cuda")
    out, dx = torch.full_like(x, 7.0), torch.full_like(x, 7.0)
    mean, rstd = torch.full((2, n), 7.0, device="cuda")
    gm.gnn_layer_norm(x, w, w, 1e-5, out, mean=mean, rstd=rstd, d_n=d_n)
    assert (out[m:] == 7).all() and (mean[m:] == 7).all() and (rstd[m:] == 7).all()
    ref.close(out[:m], ref.norm(d64(x[:m]), d64(w), d64(w), 1e-5, F)[0])
    dw, db = torch.empty_like(w), torch.empty_like(w)
    gm.gnn_layer_norm_backward(x, w, mean, rstd, dout, dx, space(n, d), dweight=dw, dbias=db, d_n=d_n)
    want = ref.norm_gradients(d64(x[:m]), d64(w), mean[:m].double(), rstd[:m].double(), d64(dout[:m]), None, F, F)
    assert (dx[m:] == 7).all()
    for got, exact in zip((dx[:m], dw, db), want):
        ref.close(got, exact)


def test_no_rows():
    e, w = torch.empty(0, 40, device="cuda"), torch.ones(40, device="cuda")
    none = torch.empty(0, device="cuda")
    gm.gnn_layer_norm(e, w, w, 1e-5, e)
    dw, db = torch.full((2, 40), 5.0, device="cuda")
    gm.gnn_layer_norm_backward(e, w, none, none, e, e, space(0, 40), dweight=dw, dbias=db)
    assert (dw == 0).all() and (db == 0).all()


def test_in_place_and_parts_of_the_gradients():
    g = torch.Generator(device="cuda").manual_seed(9)
    n, d = 257, 512
    x, w, dout, dres = rows(n, d, B, g), rows(1, d, B, g)[0], rows(n, d, B, g), rows(n, d, B, g)
    mean, rstd = torch.empty(2, n, device="cuda")
    out, y = torch.empty_like(x), x.clone()
    gm.gnn_layer_norm(x, w, None, 1e-5, out, mean=mean, rstd=rstd)
    gm.gnn_layer_norm(y, w, None, 1e-5, y)
    assert torch.equal(y, out)
    ws = space(n, d)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(w)
    gm.gnn_layer_norm_backward(x, w, mean, rstd, dout, dx, ws, dweight=dw, dbias=db, residual_grad=dres)
    over, dw2, db2 = dres.clone(), torch.empty_like(w), torch.empty_like(w)
    gm.gnn_layer_norm_backward(x, w, mean, rstd, dout, over, ws, residual_grad=over)
    gm.gnn_layer_norm_backward(x, w, mean, rstd, dout, None, ws, dweight=dw2)
    gm.gnn_layer_norm_backward(x, w, mean, rstd, dout, None, ws, dbias=db2)
    assert torch.equal(over, dx) and torch.equal(dw2, dw) and torch.equal(db2, db)


def test_captured_and_replayed_on_another_stream():
    g = torch.Generator(device="cuda").manual_seed(10)
    n, d = 3000, 384
    x, dout, w = rows(n, d, F, g), rows(n, d, F, g), rows(1, d, F, g)[0]
    out, dx, mean, rstd = torch.empty_like(x), torch.empty_like(x), *torch.empty(2, n, device="cuda")
    dw, db, ws = torch.empty_like(w), torch.empty_like(w), space(n, d)

    def step():
        gm.gnn_layer_norm(x, w, w, 1e-5, out, mean=mean, rstd=rstd)
        gm.gnn_layer_norm_backward(x, w, mean, rstd, dout, dx, ws, dweight=dw, dbias=db)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    results = [t for t in (out, mean, rstd, dx, dw, db)]
    for turn in range(3):
        x.copy_(rows(n, d, F, g, 1.0 + turn))
        for t in results:
            t.fill_(-1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        replayed = [t.clone() for t in results]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, results)), turn


def test_gradients_against_differences():
    """L = sum(dout * norm(x)) along a direction v, by central differences of the kernel's outputs at +-e.
    L's third derivative along v, times e^2 / 6, is below 1e-4 of |dL| here (e = 1e-2, rstd near 1), and the
    outputs' roundings give 2 u sum |dout out| / (2 e) at most, 3e-6 sum |dout out|."""
    g = torch.Generator(device="cuda").manual_seed(11)
    n, d, e = 20, 200, 1e-2
    x, dout, w, b = rows(n, d, F, g), rows(n, d, F, g), rows(1, d, F, g)[0], rows(1, d, F, g)[0]
    out, mean, rstd = torch.empty_like(x), *torch.empty(2, n, device="cuda")
    gm.gnn_layer_norm(x, w, b, 1e-5, out, mean=mean, rstd=rstd)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(b)
    gm.gnn_layer_norm_backward(x, w, mean, rstd, dout, dx, space(n, d), dweight=dw, dbias=db)
    noise = 3e-6 * float((dout * out).abs().sum())

    def loss(x, w, b):
        y = torch.empty_like(x)
        gm.gnn_layer_norm(x, w, b, 1e-5, y)
        return float((dout.double() * y.double()).sum())

    v = rows(n, d, F, g)
    slope = float((dx.double() * v.double()).sum())
    size = float((dx.double() * v.double()).abs().sum())
    assert abs((loss(x + e * v, w, b) - loss(x - e * v, w, b)) / (2 * e) - slope) <= 1e-3 * size + noise
    v = rows(1, d, F, g)[0]
    for first, got in ((True, dw), (False, db)):
        hi = loss(x, w + e * v, b) if first else loss(x, w, b + e * v)
        lo = loss(x, w - e * v, b) if first else loss(x, w, b - e * v)
        slope = float((got.double() * v.double()).sum())
        # linear in w and b; w +- e v is rounded: u / e of each term
        assert abs((hi - lo) / (2 * e) - slope) <= 1e-4 * float((got * v).abs().sum()) + 10 * noise
