"""Refusals of the embedding calls, on the host and before any device work: each call differs from a
well-formed one (whose pointers are never read) in one argument."""
import ctypes

import pytest
import torch

import graph_mini_pipeline_amd as gm

BAD, CAP, UNS = gm.GNN_ERR_INVALID_ARG, gm.GNN_ERR_CAPACITY, gm.GNN_ERR_UNSUPPORTED
P = 4096      # a pointer that no refused call reads

#         table type rows d ld ids d_n n scale pad out type ld_out status stream
LOOKUP = [P, 0, 10, 8, 8, P, None, 4, 1.0, -1, P, 1, 8, None, None]
#       ids d_n n dout type ld scale pad rows d grad type ld acc status ws bytes stream
GRAD = [P, None, 4, P, 0, 8, 1.0, -1, 10, 8, P, 1, 8, 0, None, P, 1 << 20, None]
#       ids d_n n dout type ld scale pad rows d uniq cap n_uniq grad type ld status ws bytes stream
ROWS = [P, None, 4, P, 0, 8, 1.0, -1, 10, 8, P, 4, P, P, 1, 8, None, P, 1 << 20, None]


def refused(call, args, changes):
    for i, v, want in changes:
        bad = list(args)
        bad[i] = v
        assert call(*bad) == want, (i, v)


def test_lookup_refusals():
    refused(gm.lib().gnn_embedding_lookup, LOOKUP, [
        (0, None, BAD), (1, 2, UNS), (1, -1, UNS), (2, 0, BAD), (2, 2 ** 31, UNS), (3, 0, BAD),
        (3, 2 ** 24 + 1, UNS), (4, 7, BAD), (5, None, BAD), (7, -1, BAD), (7, 2 ** 31, UNS),
        (9, -2, BAD), (10, None, BAD), (11, 5, UNS), (12, 7, BAD)])


def test_lookup_too_many_elements():
    bad = list(LOOKUP)
    bad[3] = bad[4] = bad[12] = 2 ** 20
    bad[7] = 2 ** 20 + 1
    assert gm.lib().gnn_embedding_lookup(*bad) == UNS


def test_grad_refusals():
    refused(gm.lib().gnn_embedding_grad, GRAD, [
        (0, None, BAD), (2, -1, BAD), (2, 2 ** 31, UNS), (3, None, BAD), (4, 3, UNS), (5, 7, BAD),
        (7, -2, BAD), (8, 0, BAD), (9, 0, BAD), (10, None, BAD), (11, 9, UNS), (12, 7, BAD),
        (15, None, BAD), (16, 16, CAP)])


def test_grad_rows_refusals():
    refused(gm.lib().gnn_embedding_grad_rows, ROWS, [
        (0, None, BAD), (3, None, BAD), (10, None, BAD), (11, -1, BAD), (12, None, BAD),
        (13, None, BAD), (15, 7, BAD), (17, None, BAD), (18, 16, CAP)])


def test_workspace_size():
    n = ctypes.c_size_t()
    size = gm.lib().gnn_embedding_grad_workspace_size
    assert size(100, 10, 8, None) == BAD
    assert size(-1, 10, 8, ctypes.byref(n)) == BAD
    assert size(100, 0, 8, ctypes.byref(n)) == BAD
    assert size(2 ** 31, 10, 8, ctypes.byref(n)) == UNS
    a = gm.gnn_embedding_grad_workspace_size(1000, 50, 16)
    b = gm.gnn_embedding_grad_workspace_size(100_000, 50, 16)
    assert 0 < a < b and b >= 100_000 * 16      # two (key, position) lists at least
    assert gm.gnn_embedding_grad_workspace_size(0, 1, 1) > 0


def test_binding_checks_tensors():
    f, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        gm.gnn_embedding_lookup(f, ids, 1.0, f)
    with pytest.raises(TypeError, match="ids"):
        gm.gnn_embedding_lookup(f, ids.long(), 1.0, f)
    with pytest.raises(ValueError, match="device"):
        gm.gnn_embedding_grad(ids, f, 1.0, f, f)
    meta = torch.zeros(4, 8, dtype=torch.float16)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        gm._need_rows(meta, "x")
