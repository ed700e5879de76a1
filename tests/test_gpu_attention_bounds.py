"""Bounds and sizes of zero: what does not fit them is reported by the forward and the backward call alike,
and nothing is written."""
import pytest
import torch

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")

CAP, RANGE = gm.GNN_ERR_CAPACITY, gm.GNN_ERR_OUT_OF_RANGE


def call(q_indptr, k_indptr, n_q, n_k, max_q, max_k, backward, dtype=torch.float32):
    q, k = torch.ones(n_q, 4, 16, device="cuda", dtype=dtype), torch.ones(n_k, 2, 16, device="cuda", dtype=dtype)
    outs = {x: torch.full_like(t, 7.0) for x, t in (("out", q), ("dq", q), ("dk", k), ("dv", k))}
    lse = torch.full((n_q, 4), 7.0, device="cuda")
    qp, kp = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (q_indptr, k_indptr))
    ws = torch.empty(gm.gnn_cross_attention_workspace_size(len(qp) - 1, n_q, n_k, max_q, max_k, 4, 2, 16, dtype,
                                                           True), dtype=torch.uint8, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if backward:
        gm.gnn_cross_attention_backward(q, k, k, qp, kp, max_q, max_k, 1.0, outs["out"], lse, q, outs["dq"],
                                        outs["dk"], outs["dv"], ws, d_status=status)
    else:
        gm.gnn_cross_attention(q, k, k, qp, kp, max_q, max_k, 1.0, outs["out"], ws, lse=lse, d_status=status)
    return status.item(), dict(outs, lse=lse)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("backward", [False, True])
def test_sequences_beyond_a_bound_of_zero(backward, dtype):
    for max_q, max_k in ((0, 0), (0, 9)):
        status, outs = call([0, 5, 8], [0, 9, 9], 8, 9, max_q, max_k, backward, dtype)
        assert status == CAP
        for x in ("out", "lse", "dq"):
            assert torch.all(outs[x] == 7.0), x
    status, outs = call([0, 5, 8], [0, 9, 9], 8, 9, 8, 0, backward, dtype)
    assert status == CAP
    assert torch.all(outs["dk"] == 7.0) and torch.all(outs["dv"] == 7.0)


@pytest.mark.parametrize("backward", [False, True])
def test_rows_that_are_not_there(backward):
    """indptrs over tensors without rows."""
    assert call([0, 3], [0, 4], 0, 4, 3, 4, backward)[0] == RANGE
    assert call([0, 3], [0, 4], 3, 0, 3, 4, backward)[0] == RANGE
    assert call([0, 3], [0, 4], 0, 0, 3, 4, backward)[0] == RANGE


@pytest.mark.parametrize("backward", [False, True])
def test_nothing_is_no_error(backward):
    for n_q, n_k in ((0, 0), (0, 4), (3, 0)):
        status, outs = call([0, n_q], [0, n_k], n_q, n_k, n_q, n_k, backward)
        assert status == gm.GNN_OK
        if backward:
            assert torch.all(outs["dq"] == 0) and torch.all(outs["dk"] == 0) and torch.all(outs["dv"] == 0)
        elif n_q:
            assert torch.all(outs["out"] == 0) and torch.all(torch.isneginf(outs["lse"]))
    assert call([0, 0, 0], [0, 0, 0], 0, 0, 0, 0, backward)[0] == gm.GNN_OK
