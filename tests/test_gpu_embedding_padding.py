"""A padding id that lies outside the table: one past its end, as a table without a padding row has it, or
further.  It is no error."""
import pytest
import torch

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")


@pytest.mark.parametrize("pad", [100, 101, 2 ** 31 - 1])
@pytest.mark.parametrize("n", [50, 3000, 9000, 20_000])
def test_padding_id_outside_the_table(n, pad):
    rows, d = 100, 12
    g = torch.Generator().manual_seed(n)
    ids = torch.randint(rows, (n,), generator=g, dtype=torch.int32)
    ids[::7] = pad
    table, dout = torch.randn(rows, d, generator=g), torch.randint(-4, 5, (n, d), generator=g).float()
    inside = ids != pad
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.full((n, d), 9.0, device="cuda")
    gm.gnn_embedding_lookup(table.cuda(), ids.cuda(), 2.0, out, pad_id=pad, d_status=status)
    want = torch.zeros(n, d)
    want[inside] = 2 * table[ids[inside].long()]
    assert torch.equal(out.cpu(), want) and status.item() == gm.GNN_OK
    # sums of small whole numbers are exact
    ws = torch.empty(gm.gnn_embedding_grad_workspace_size(n, rows, d), dtype=torch.uint8, device="cuda")
    want = torch.zeros(rows, d).index_add_(0, ids[inside].long(), dout[inside])
    grad = torch.full((rows, d), 9.0, device="cuda")
    gm.gnn_embedding_grad(ids.cuda(), dout.cuda(), 1.0, grad, ws, pad_id=pad, d_status=status)
    assert torch.equal(grad.cpu(), want) and status.item() == gm.GNN_OK
    uniq = torch.empty(rows, dtype=torch.int32, device="cuda")
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    gm.gnn_embedding_grad_rows(ids.cuda(), dout.cuda(), 1.0, rows, uniq, count, grad, ws, pad_id=pad,
                               d_status=status)
    named = torch.unique(ids[inside])
    assert status.item() == gm.GNN_OK and torch.equal(uniq[:count.item()].cpu(), named)
    assert torch.equal(grad[:len(named)].cpu(), want[named.long()])
    # any other id outside it is still one
    ids[3] = 102
    gm.gnn_embedding_lookup(table.cuda(), ids.cuda(), 2.0, out, pad_id=pad, d_status=status)
    assert status.item() == gm.GNN_ERR_OUT_OF_RANGE
    status.zero_()
    gm.gnn_embedding_grad(ids.cuda(), dout.cuda(), 1.0, grad, ws, pad_id=pad, d_status=status)
    assert status.item() == gm.GNN_ERR_OUT_OF_RANGE


def test_no_padding_id_is_no_id():
    """pad_id = -1: an id of -1 is out of range."""
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ids = torch.tensor([-1, 2], dtype=torch.int32, device="cuda")
    out = torch.empty(2, 4, device="cuda")
    gm.gnn_embedding_lookup(torch.ones(3, 4, device="cuda"), ids, 1.0, out, d_status=status)
    assert status.item() == gm.GNN_ERR_OUT_OF_RANGE
