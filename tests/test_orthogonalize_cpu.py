"""Refusals of gnn_orthogonalize on the host, before any device work (the pointers are never read),
and the bound on the values that the coefficients can reach."""
import ctypes

import pytest
import torch

import graph_mini_pipeline_amd as gm

BAD, CAP, UNS = gm.GNN_ERR_INVALID_ARG, gm.GNN_ERR_CAPACITY, gm.GNN_ERR_UNSUPPORTED
P = 4096


def coefs(*c):
    return (ctypes.c_float * 3)(*c)


#       g type batch rows cols ld stride steps coefs eps scale out ld stride ws bytes stream
ARGS = [P, 0, 2, 20, 30, 30, 600, 5, None, 1e-7, 1.0, P, 30, 600, P, 1 << 30, None]


@pytest.mark.parametrize("i,v,want", [
    (0, None, BAD), (1, 2, UNS), (2, -1, BAD), (2, 65536, UNS), (3, 0, BAD), (3, 32769, UNS),
    (4, 0, BAD), (4, 32769, UNS), (5, 29, BAD), (6, 599, BAD), (7, 0, BAD), (7, 17, UNS),
    (9, -1.0, BAD), (9, float("nan"), BAD), (11, None, BAD), (12, 29, BAD), (13, 599, BAD),
    (14, None, BAD), (15, 100, CAP)])
def test_refusals(i, v, want):
    bad = list(ARGS)
    bad[i] = v
    assert gm.lib().gnn_orthogonalize(*bad) == want


@pytest.mark.parametrize("c,steps,fits", [
    ((1.5, -0.5, 0.0), 16, True),          # stays in [0, 1]
    ((2.0, -1.5, 0.5), 16, True),
    ((3.4445, -4.7750, 2.0315), 16, True),
    ((1.0, 0.0, 0.0), 16, True),
    ((3.5, 0.0, 0.0), 1, False),           # 1 goes to 3.5
    ((2.0, 0.0, 0.0), 1, True),
    ((2.0, 0.0, 0.0), 2, False),           # and 2 to 4
    ((16.0, -16.0, 0.0), 1, False),        # the polynomial's factor itself reaches 16
    ((float("nan"), 0.0, 0.0), 1, False),
    ((1.0, float("inf"), 0.0), 1, False)])
def test_coefficients_must_keep_values_in_range(c, steps, fits):
    a = list(ARGS)
    a[7], a[8], a[15] = steps, coefs(*c), 100
    # the workspace is checked after the coefficients
    assert gm.lib().gnn_orthogonalize(*a) == (CAP if fits else UNS)


def test_workspace_size():
    n = ctypes.c_size_t()
    size = gm.lib().gnn_orthogonalize_workspace_size
    assert size(1, 10, 10, 0, None) == BAD
    assert size(1, 0, 10, 0, ctypes.byref(n)) == BAD
    assert size(1, 10, 10, 7, ctypes.byref(n)) == UNS
    one = gm.gnn_orthogonalize_workspace_size(1, 500, 300, torch.bfloat16)
    assert one >= 3 * 500 * 300 * 2
    assert gm.gnn_orthogonalize_workspace_size(1, 300, 500, torch.bfloat16) == one
    assert gm.gnn_orthogonalize_workspace_size(1, 500, 300, torch.float32) > 1.9 * one


def test_binding_checks_tensors():
    x = torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device"):
        gm.gnn_orthogonalize(x, x, x)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        gm.gnn_orthogonalize(x.half(), x, x)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        gm.gnn_orthogonalize_workspace_size(1, 4, 4, torch.int32)
