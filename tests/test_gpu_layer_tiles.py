"""The dense layers' largest tiles, 128 x 128 and 256 x 256, by every way of their operands into LDS, forward and both
gradients: whole and cut, with rows that do not count, with sums that are split, and with two planes of dz."""
import pytest
import torch

from . import layers as ref
from .test_gpu_dense import B, F, d64, gated_case, linear_case, normal, space

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")

# (n, d_in, d_out): rows at multiples of 16 bytes, of 4, and (bf16) of 2
TILES = [(2048, 2048, 2048), (4096, 2048, 2048), (2047, 2049, 2047), (2050, 2046, 2054), (4096, 1031, 4097),
         (1030, 4104, 1032), (2100, 1000, 2056), (2100, 1001, 2055), (2100, 1002, 2054)]
# few terms in dx's sums: two planes of dz for it
NARROW = [(8192, 2048, 248), (8192, 2046, 250), (5000, 2047, 503), (16384, 4096, 250)]


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape", TILES + NARROW)
def test_large_tiles(shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    linear_case(*shape, dtype, "gelu", g)
    gated_case(*shape, dtype, "silu", g)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("count", [0, 300, 1900])
@pytest.mark.parametrize("shape", [TILES[0], TILES[2], TILES[3], TILES[6], NARROW[0], NARROW[2]])
def test_large_tiles_under_a_device_count(shape, count, dtype):
    """The count ends inside a tile of rows (and below 512 rows, where dw takes two planes of dz)."""
    n, i, o = shape
    g = torch.Generator(device="cuda").manual_seed(count + i)
    nan = float("nan")
    d_n = torch.tensor([count], device="cuda")
    x, dout = normal(n, i, dtype=dtype, gen=g), normal(n, o, dtype=dtype, gen=g)
    wg, wu = (normal(i, o, dtype=dtype, gen=g, scale=i ** -0.5) for _ in range(2))
    x[count:], dout[count:] = nan, nan
    out, gate, up, pre, y = torch.full((5, n, o), 7.0, device="cuda", dtype=dtype)
    gm.gnn_gated_linear(x, wg, wu, out, space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype), activation="gelu",
                        gate=gate, up=up, d_n=d_n)
    want = ref.gated(d64(x[:count]), d64(wg), d64(wu), None, None, "gelu", dtype)
    for t, exact in zip((out, gate, up), want):
        assert (t[count:] == 7).all()
        ref.close(t[:count], exact)
    gm.gnn_linear(x, wg, y, space(gm.gnn_linear_workspace_size, n, i, o, dtype), activation="silu", pre=pre, d_n=d_n)
    want = ref.linear(d64(x[:count]), d64(wg), None, "silu", None, dtype)
    for t, exact in ((y, want[:2]), (pre, want[2:])):
        assert (t[count:] == 7).all()
        ref.close(t[:count], exact)
    gate[count:], up[count:], pre[count:] = nan, nan, nan
    dx, dwg, dwu, dbs = torch.full_like(x, 7.0), torch.empty_like(wg), torch.empty_like(wu), \
        torch.empty(2, o, device="cuda", dtype=dtype)
    gm.gnn_gated_linear_backward(x, wg, wu, gate, up, dout,
                                 space(gm.gnn_gated_linear_workspace_size, n, i, o, dtype, True), activation="gelu",
                                 dx=dx, dw_gate=dwg, dw_up=dwu, dbias_gate=dbs[0], dbias_up=dbs[1], d_n=d_n)
    want = ref.gated_gradients(d64(x[:count]), d64(wg), d64(wu), d64(dout[:count]), "gelu", d64(gate[:count]),
                               d64(up[:count]), dtype)
    assert (dx[count:] == 7).all()
    for t, exact in zip((dx[:count], dwg, dbs[0], dwu, dbs[1]), want):
        ref.close(t, exact)
    dx.fill_(7.0)
    gm.gnn_linear_backward(x, wg, dout, space(gm.gnn_linear_workspace_size, n, i, o, dtype, True), activation="silu",
                           pre=pre, dx=dx, dw=dwg, dbias=dbs[0], d_n=d_n)
    want = ref.linear_gradients(d64(x[:count]), d64(wg), d64(dout[:count]), "silu", d64(pre[:count]), dtype)
    assert (dx[count:] == 7).all()
    for t, exact in zip((dx[:count], dwg, dbs[0]), want):
        ref.close(t, exact)


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape, count", [(TILES[0], 300), (TILES[2], 511), (TILES[3], 200), (TILES[6], 511),
                                          (TILES[7], 300), (NARROW[0], 8000), (NARROW[1], 400), (NARROW[2], 5000)])
def test_infinities_in_large_tiles(shape, count, dtype):
    """As in smaller tiles: one infinity of x, one of w, and nothing else is touched."""
    n, i, o = shape
    g = torch.Generator(device="cuda").manual_seed(count)
    x, w, dout = normal(n, i, dtype=dtype, gen=g), normal(i, o, dtype=dtype, gen=g), normal(n, o, dtype=dtype, gen=g)
    pre = normal(n, o, dtype=dtype, gen=g).abs()
    ws, d_n = space(gm.gnn_linear_workspace_size, n, i, o, dtype, True), torch.tensor([count], device="cuda")

    def gradients():
        dx, dw = torch.zeros_like(x), torch.empty_like(w)
        gm.gnn_linear_backward(x, w, dout, ws, activation="gelu", pre=pre, dx=dx, dw=dw, d_n=d_n)
        return dx[:count], dw

    clean = gradients()
    row, col, line, at = count // 2, i // 3, i - 1, o - 2
    x[row, col], w[line, at] = float("inf"), float("inf")
    dx, dw = gradients()
    assert torch.equal(dw[col].float(), dout[row].float().sign() * float("inf"))
    assert torch.equal(dx[:, line].float(), dout[:count, at].float().sign() * float("inf"))
    lines = torch.arange(i, device="cuda")
    assert torch.equal(dw[lines != col], clean[1][lines != col])
    assert torch.equal(dx[:, lines != line], clean[0][:, lines != line])


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("n, i, o, count", [(4096, 768, 1024, 4096), (9000, 256, 2048, 9000), (9000, 256, 2048, 7001),
                                            (2048, 2048, 2048, 1939), (4099, 1030, 1026, 4099), (4097, 1031, 4097, 4001)])
@pytest.mark.parametrize("name", ["none", "gelu"])
def test_out_over_the_residual_in_large_tiles(n, i, o, count, name, dtype):
    """out is the residual itself where rows of it are loaded ahead of the rows that are stored, and where the last
    rows end inside a wavefront's 32; rows that do not count keep what they hold."""
    g = torch.Generator(device="cuda").manual_seed(n + count)
    x, w, r = normal(n, i, dtype=dtype, gen=g), normal(i, o, dtype=dtype, gen=g, scale=i ** -0.5), \
        normal(n, o, dtype=dtype, gen=g)
    b = normal(o, dtype=dtype, gen=g)
    ws, d_n = space(gm.gnn_linear_workspace_size, n, i, o, dtype), torch.tensor([count], device="cuda")
    over, apart = r.clone(), r.clone()
    gm.gnn_linear(x, w, over, ws, bias=b, activation=name, residual=over, d_n=d_n)
    gm.gnn_linear(x, w, apart, ws, bias=b, activation=name, residual=r, d_n=d_n)
    assert torch.equal(over, apart) and torch.equal(over[count:], r[count:])
    y, ey, _, _ = ref.linear(d64(x[:count]), d64(w), d64(b), name, d64(r[:count]), dtype)
    ref.close(over[:count], (y, ey))


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("shape", [(4, 4098, 4098), (1, 2050, 1030), (4, 4097, 4099), (1, 2048, 1032), (17, 4098, 4102)])
def test_wide_layers_of_a_few_rows(shape, dtype):
    """Tiles of 32 rows by each way, their sums split."""
    g = torch.Generator(device="cuda").manual_seed(sum(shape))
    linear_case(*shape, dtype, "gelu_tanh", g)
    gated_case(*shape, dtype, "silu", g)
