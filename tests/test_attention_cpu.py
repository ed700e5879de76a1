"""Refusals of gnn_cross_attention and its backward pass on the host, before any device work: each
call differs from a well-formed one (whose pointers are never read) in one field."""
import ctypes

import pytest
import torch

import graph_mini_pipeline_amd as gm
from graph_mini_pipeline_amd import _abi

BAD, CAP, UNS = gm.GNN_ERR_INVALID_ARG, gm.GNN_ERR_CAPACITY, gm.GNN_ERR_UNSUPPORTED
P = 4096


def good(**changes):
    x = _abi.gnn_attention(0, 8, 2, 64, 3, 30, 100, 20, 60, 0.125, P, P, None, P, P, P, 512, 128, 128,
                           P, 512, P, None)
    for k, v in changes.items():
        setattr(x, k, v)
    return ctypes.byref(x)


def grads(**changes):
    g = _abi.gnn_attention_grad(P, 512, P, P, P, 512, 128, 128)
    for k, v in changes.items():
        setattr(g, k, v)
    return ctypes.byref(g)


SIZES = [("heads", 0, BAD), ("kv_heads", 0, BAD), ("kv_heads", 3, BAD), ("head_dim", 0, BAD),
         ("head_dim", 60, UNS), ("head_dim", 136, UNS), ("type", 2, UNS), ("n_seq", -1, BAD),
         ("n_seq", 65536, UNS), ("n_q", -1, BAD), ("n_q", 2 ** 31, UNS), ("n_q", 2 ** 28, UNS),
         ("n_k", -1, BAD), ("n_k", 2 ** 30, UNS), ("max_q", -1, BAD), ("max_k", -1, BAD),
         ("heads", 2048, UNS)]
POINTERS = [("q_indptr", None, BAD), ("k_indptr", None, BAD), ("q", None, BAD), ("k", None, BAD),
            ("v", None, BAD), ("out", None, BAD), ("ld_q", 511, BAD), ("ld_k", 127, BAD),
            ("ld_v", 127, BAD), ("ld_out", 511, BAD), ("ld_q", 2 ** 21 + 1, UNS),
            ("ld_k", 2 ** 21 + 1, UNS), ("ld_v", 2 ** 21 + 1, UNS), ("scale", float("nan"), BAD)]


@pytest.mark.parametrize("field,value,want", SIZES + POINTERS)
def test_refusals(field, value, want):
    L = gm.lib()
    x = good(**{field: value})
    assert L.gnn_cross_attention(x, P, 1 << 40, None) == want
    assert L.gnn_cross_attention_backward(x, grads(), P, 1 << 40, None) == want
    n = ctypes.c_size_t()
    if (field, value, want) in SIZES:
        assert L.gnn_cross_attention_workspace_size(x, 1, ctypes.byref(n)) == want


@pytest.mark.parametrize("field,value", [("dout", None), ("dq", None), ("dk", None), ("dv", None),
                                         ("ld_dout", 511), ("ld_dq", 511), ("ld_dk", 127),
                                         ("ld_dv", 127)])
def test_backward_refusals(field, value):
    assert gm.lib().gnn_cross_attention_backward(good(), grads(**{field: value}), P, 1 << 40,
                                                 None) == BAD


def test_missing_arguments_and_small_workspaces():
    L = gm.lib()
    n = ctypes.c_size_t()
    assert L.gnn_cross_attention(None, P, 1 << 40, None) == BAD
    assert L.gnn_cross_attention(good(), None, 1 << 40, None) == BAD
    assert L.gnn_cross_attention_backward(good(), None, P, 1 << 40, None) == BAD
    assert L.gnn_cross_attention_backward(good(lse=None), grads(), P, 1 << 40, None) == BAD
    assert L.gnn_cross_attention_workspace_size(good(), 0, None) == BAD
    assert L.gnn_cross_attention_workspace_size(good(), 1, ctypes.byref(n)) == gm.GNN_OK
    assert n.value >= 30 * 8 * 8
    assert L.gnn_cross_attention_backward(good(), grads(), P, n.value - 1, None) == CAP
    assert L.gnn_cross_attention(good(), P, 0, None) == CAP


def test_nothing_to_do():
    """No sequences: nothing is enqueued, so no device is needed."""
    assert gm.lib().gnn_cross_attention(good(n_seq=0), P, 1 << 30, None) == gm.GNN_OK


def test_binding_checks_tensors():
    q, k = torch.zeros(4, 2, 8), torch.zeros(6, 2, 8)
    ptr = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        gm.gnn_cross_attention(q, k, k, ptr, ptr, 4, 6, 1.0, q, q)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        gm.gnn_cross_attention(q.half(), k, k, ptr, ptr, 4, 6, 1.0, q, q)
    with pytest.raises(ValueError, match="q: "):
        gm.gnn_cross_attention(q[0], k, k, ptr, ptr, 4, 6, 1.0, q, q)
