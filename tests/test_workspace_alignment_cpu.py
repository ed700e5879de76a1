"""The learned operators refuse a workspace that does not start at a multiple of 16 bytes, where counters
that are added to atomically would lie across words.  No pointer is read."""
import ctypes

import pytest

import graph_mini_pipeline_amd as gm
from graph_mini_pipeline_amd import _abi

P = 4096


def grad(ws):
    return gm.lib().gnn_embedding_grad(P, None, 4, P, 0, 8, 1.0, -1, 10, 8, P, 1, 8, 0, None, ws, 1, None)


def grad_rows(ws):
    return gm.lib().gnn_embedding_grad_rows(P, None, 4, P, 0, 8, 1.0, -1, 10, 8, P, 4, P, P, 1, 8, None, ws, 1, None)


def attention():
    return ctypes.byref(_abi.gnn_attention(0, 8, 2, 64, 3, 30, 100, 20, 60, 0.125, P, P, None, P, P, P, 512, 128,
                                           128, P, 512, P, None))


def attend(ws):
    return gm.lib().gnn_cross_attention(attention(), ws, 1, None)


def attend_backward(ws):
    g = _abi.gnn_attention_grad(P, 512, P, P, P, 512, 128, 128)
    return gm.lib().gnn_cross_attention_backward(attention(), ctypes.byref(g), ws, 1, None)


def orthogonalize(ws):
    return gm.lib().gnn_orthogonalize(P, 0, 2, 20, 30, 30, 600, 5, None, 1e-7, 1.0, P, 30, 600, ws, 1, None)


@pytest.mark.parametrize("call", [grad, grad_rows, attend, attend_backward, orthogonalize])
def test_workspaces_start_at_multiples_of_16(call):
    for off in (1, 2, 4, 8, 15):
        assert call(P + off) == gm.GNN_ERR_INVALID_ARG, off
    for off in (0, 16, 256):
        assert call(P + off) == gm.GNN_ERR_CAPACITY, off     # (of one byte)
