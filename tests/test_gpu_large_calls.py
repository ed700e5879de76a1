"""Sizes within the documented limits whose kernels take 2^32 threads and more, which one launch cannot
have (its grid has fewer in a dimension): they are enqueued in pieces."""
import math

import pytest
import torch

from tests.test_gpu_attention import BF16, formulas

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")


def room(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib << 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def test_attention_over_two_to_the_29_query_rows_and_heads():
    """Rows of two states; those next to the pieces' borders and some heads' sums against the formulas."""
    room(60)
    nq, heads, d, nk = 2 ** 19 + 3, 1024, 8, 2
    g = torch.Generator(device="cuda").manual_seed(0)

    def rows(n):
        return torch.randn(n, heads, d, generator=g, device="cuda", dtype=BF16)

    q, dout, k, v = rows(nq), rows(nq), rows(nk), rows(nk)
    out, dq = torch.empty_like(q), torch.empty_like(q)
    dk, dv = torch.empty_like(k), torch.empty_like(v)
    lse = torch.empty(nq, heads, device="cuda")
    qp, kp = (torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in (nq, nk))
    ws = torch.empty(gm.gnn_cross_attention_workspace_size(1, nq, nk, nq, nk, heads, heads, d, BF16, True),
                     dtype=torch.uint8, device="cuda")
    scale = 0.375
    gm.gnn_cross_attention(q, k, v, qp, kp, nq, nk, scale, out, ws, lse=lse)
    gm.gnn_cross_attention_backward(q, k, v, qp, kp, nq, nk, scale, out, lse, dout, dq, dk, dv, ws)
    torch.cuda.synchronize()
    # lines (row, head) go in pieces of 2^28
    some = torch.tensor([0, 1, 2 ** 18 - 1, 2 ** 18, 2 ** 18 + 1, 2 ** 19 - 1, 2 ** 19, nq - 1], device="cuda")
    host = lambda t: t.double().cpu()
    for h in (0, 1, 511, 1023):
        ref = formulas(host(q[some, h]), host(k[:, h]), host(v[:, h]), host(dout[some, h]), scale, 2.0 ** -8)
        for name, x in (("out", out), ("dq", dq)):
            want, bound = ref[name]
            assert torch.all((host(x[some, h]) - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound)), (h, name)
    for h in (0, 700, 1023):
        ref = formulas(host(q[:, h]), host(k[:, h]), host(v[:, h]), host(dout[:, h]), scale, 2.0 ** -8)
        for name, x in (("dk", dk), ("dv", dv)):
            want, bound = ref[name]
            assert torch.all((host(x[:, h]) - want).abs() <= bound + 2.0 ** -8 * (want.abs() + bound)), (h, name)


def test_lookup_of_two_to_the_34_vectors():
    """137 GB of rows."""
    n, d, rows = 2 ** 34 // 9 + 1000, 36, 1001
    room(150)
    table = torch.randn(rows, d, device="cuda")
    ids = torch.randint(rows, (n,), dtype=torch.int32, device="cuda")
    out = torch.empty(n, d, dtype=BF16, device="cuda")
    gm.gnn_embedding_lookup(table, ids, 1.5, out, pad_id=7)
    # a piece has 2^23 workgroups of 1024 vectors, nine a row
    edge = 2 ** 33 // 9
    for lo, hi in ((0, 3000), (edge - 3000, edge + 3000), (n - 3000, n)):
        want = 1.5 * table[ids[lo:hi].long()]
        want[ids[lo:hi] == 7] = 0
        assert torch.equal(out[lo:hi], want.to(BF16))
