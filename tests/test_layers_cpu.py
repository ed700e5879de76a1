"""Refusals of the layer norm and of the dense layers, on the host and before any device work: each call
differs from a well-formed one (whose pointers are never read) in one field.  And the structs' layouts."""
import ctypes
import os
import subprocess

import pytest
import torch

import graph_mini_pipeline_amd as gm
from graph_mini_pipeline_amd import _abi

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, BAD, CAP, UNS = gm.GNN_OK, gm.GNN_ERR_INVALID_ARG, gm.GNN_ERR_CAPACITY, gm.GNN_ERR_UNSUPPORTED
P = 4096      # a pointer that no refused call reads
NAN = float("nan")

NORM = dict(x_type=0, out_type=1, param_type=0, eps=1e-5, n=4, d=24, x=P, ld_x=24, weight=P, bias=P, out=P,
            ld_out=24, mean=P, rstd=P)
NORM_GRAD = dict(dout=P, ld_dout=24, residual_grad=P, ld_residual_grad=24, dx=P, ld_dx=24, dweight=P, dbias=P)
DENSE = dict(type=1, activation=2, n=4, d_in=16, d_out=24, x=P, ld_x=16, w=P, ld_w=24, bias=P, residual=P,
             ld_residual=24, out=P, ld_out=24, pre=P, ld_pre=24)
DENSE_GRAD = dict(dout=P, ld_dout=24, dx=P, ld_dx=16, dw=P, ld_dw=24, dbias=P)
GATED = dict(type=1, activation=4, n=4, d_in=16, d_out=24, x=P, ld_x=16, w_gate=P, w_up=P, ld_w=24, bias_gate=P,
             bias_up=P, out=P, ld_out=24, gate=P, up=P, ld_pre=24)
GATED_GRAD = dict(dout=P, ld_dout=24, dx=P, ld_dx=16, dw_gate=P, dw_up=P, ld_dw=24, dbias_gate=P, dbias_up=P)


def build(struct, base, **changes):
    s = struct()
    for k, v in dict(base, **changes).items():
        setattr(s, k, v)
    return s


def norm(ws=P, size=1 << 30, **c):
    return gm.lib().gnn_layer_norm(ctypes.byref(build(_abi.gnn_norm, NORM, **c)), None)


def norm_backward(ws=P, size=1, grad=(), **c):
    x, g = build(_abi.gnn_norm, NORM, **c), build(_abi.gnn_norm_grad, NORM_GRAD, **dict(grad))
    return gm.lib().gnn_layer_norm_backward(ctypes.byref(x), ctypes.byref(g), ws, size, None)


def linear(ws=P, size=1, **c):
    return gm.lib().gnn_linear(ctypes.byref(build(_abi.gnn_dense, DENSE, **c)), ws, size, None)


def linear_backward(ws=P, size=1, grad=(), **c):
    x, g = build(_abi.gnn_dense, DENSE, **c), build(_abi.gnn_dense_grad, DENSE_GRAD, **dict(grad))
    return gm.lib().gnn_linear_backward(ctypes.byref(x), ctypes.byref(g), ws, size, None)


def gated(ws=P, size=1, **c):
    return gm.lib().gnn_gated_linear(ctypes.byref(build(_abi.gnn_gated, GATED, **c)), ws, size, None)


def gated_backward(ws=P, size=1, grad=(), **c):
    x, g = build(_abi.gnn_gated, GATED, **c), build(_abi.gnn_gated_grad, GATED_GRAD, **dict(grad))
    return gm.lib().gnn_gated_linear_backward(ctypes.byref(x), ctypes.byref(g), ws, size, None)


SIZES = [dict(n=-1), dict(x=None)]


@pytest.mark.parametrize("change, want", [(c, BAD) for c in SIZES + [
    dict(d=0), dict(ld_x=23), dict(ld_out=23), dict(out=None), dict(eps=-1.0), dict(eps=NAN)]] + [
    (dict(n=2 ** 31), UNS), (dict(d=16385), UNS), (dict(x_type=2), UNS), (dict(out_type=-1), UNS),
    (dict(param_type=7), UNS)])
def test_norm_refusals(change, want):
    assert norm(**change) == want


@pytest.mark.parametrize("change, want", [(c, BAD) for c in SIZES + [
    dict(d=0), dict(ld_x=23), dict(mean=None), dict(rstd=None), dict(grad=dict(dout=None)),
    dict(grad=dict(ld_dout=23)), dict(grad=dict(ld_dx=23)), dict(grad=dict(ld_residual_grad=23)),
    dict(ws=None), dict(ws=P + 8)]] + [
    (dict(n=2 ** 31), UNS), (dict(d=16385), UNS), (dict(x_type=2), UNS), (dict(), CAP)])
def test_norm_backward_refusals(change, want):
    assert norm_backward(**change) == want


LAYER = [(c, BAD) for c in SIZES + [dict(d_in=0), dict(d_out=0), dict(ld_x=15), dict(ld_w=23), dict(ws=None),
                                    dict(ws=P + 8)]] + [
    (dict(type=2), UNS), (dict(activation=6), UNS), (dict(activation=-1), UNS), (dict(n=2 ** 30 + 1), UNS),
    (dict(d_in=2 ** 20 + 1, ld_x=2 ** 21), UNS), (dict(d_out=2 ** 20 + 1), UNS), (dict(ld_x=2 ** 21 + 1), UNS),
    (dict(ld_w=2 ** 21 + 1), UNS)]
FORWARD = [(dict(out=None), BAD), (dict(ld_out=23), BAD), (dict(ld_pre=23), BAD), (dict(ld_out=2 ** 21 + 1), UNS)]
BACKWARD = [(dict(grad=dict(dout=None)), BAD), (dict(grad=dict(ld_dout=23)), BAD), (dict(grad=dict(ld_dx=15)), BAD),
            (dict(grad=dict(ld_dw=23)), BAD), (dict(ld_pre=23), BAD), (dict(), CAP)]


@pytest.mark.parametrize("change, want", LAYER + FORWARD + [(dict(w=None), BAD), (dict(ld_residual=23), BAD)])
def test_linear_refusals(change, want):
    assert linear(**change) == want


@pytest.mark.parametrize("change, want", LAYER + BACKWARD + [(dict(w=None), BAD), (dict(pre=None), BAD)])
def test_linear_backward_refusals(change, want):
    assert linear_backward(**change) == want


@pytest.mark.parametrize("change, want", LAYER + FORWARD + [(dict(w_gate=None), BAD), (dict(w_up=None), BAD)])
def test_gated_refusals(change, want):
    assert gated(**change) == want


@pytest.mark.parametrize("change, want", LAYER + BACKWARD + [
    (dict(w_gate=None), BAD), (dict(w_up=None), BAD), (dict(gate=None), BAD), (dict(up=None), BAD)])
def test_gated_backward_refusals(change, want):
    assert gated_backward(**change) == want


def test_too_small_a_forward_workspace():
    for call, size in ((linear, gm.gnn_linear_workspace_size), (gated, gm.gnn_gated_linear_workspace_size)):
        need = size(4, 16, 24, torch.bfloat16)
        assert need > 0 and call(size=need - 1) == CAP


def test_null_structs():
    L, n = gm.lib(), ctypes.c_size_t()
    assert L.gnn_layer_norm(None, None) == BAD
    assert L.gnn_linear(None, P, 1, None) == BAD and L.gnn_gated_linear(None, P, 1, None) == BAD
    assert L.gnn_linear_workspace_size(None, 0, ctypes.byref(n)) == BAD
    assert L.gnn_gated_linear_workspace_size(ctypes.byref(build(_abi.gnn_gated, GATED)), 0, None) == BAD
    assert L.gnn_layer_norm_workspace_size(4, 8, None) == BAD
    assert L.gnn_linear_backward(ctypes.byref(build(_abi.gnn_dense, DENSE)), None, P, 1, None) == BAD


def test_workspace_sizes():
    for size in (gm.gnn_linear_workspace_size, gm.gnn_gated_linear_workspace_size):
        assert size(0, 1, 1, torch.float32) > 0
        # the gradient of the sums has a line of whole 128 bytes for each row
        assert size(1000, 64, 100, torch.bfloat16, backward=True) >= 1000 * 128 * 2
        for bad in ((-1, 8, 8), (8, 0, 8), (8, 8, 0)):
            with pytest.raises(gm.GnnError) as e:
                size(*bad, torch.float32)
            assert e.value.status == BAD
    assert gm.gnn_layer_norm_workspace_size(10, 64) >= 2 * 64 * 4
    with pytest.raises(gm.GnnError):
        gm.gnn_layer_norm_workspace_size(10, 20000)
    # the sizes never need a device, nor more than a card has for a large layer
    assert gm.gnn_linear_workspace_size(1 << 20, 4096, 16384, torch.bfloat16) < 1 << 33


def test_binding_checks_tensors():
    x, w, out = torch.zeros(4, 16), torch.zeros(16, 24), torch.zeros(4, 24)
    with pytest.raises(ValueError, match="device"):
        gm.gnn_linear(x, w, out, x)
    with pytest.raises(ValueError, match="activation"):
        gm.gnn_linear(x, w, out, x, activation="tanh")
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        gm.gnn_linear(x.half(), w, out, x)
    with pytest.raises(ValueError, match="matrix"):
        gm.gnn_layer_norm(x[0], None, None, 1e-5, x[0])
    with pytest.raises(ValueError, match="device"):
        gm.gnn_layer_norm(x, None, None, 1e-5, x)
    with pytest.raises(ValueError, match="one row stride"):
        gm._same_stride((1, 24), (2, 48), "w_gate, w_up")
    assert gm._same_stride((None, 0), (2, 48), "gate, up") == (None, 2, 48)


def test_tensors_on_another_device_are_refused(monkeypatch):
    """A call runs on the stream's device, the current one's without a stream; every tensor has to be there."""
    class Tensor:
        is_cuda = True

        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    assert gm._device_of(Tensor(1), None) == 1 and gm._device_of(Tensor(1), 12345) == 1
    with pytest.raises(ValueError, match="x: is on device 0, the call on device 1"):
        gm._device_of(Tensor(0), None)
    with pytest.raises(ValueError, match="ws: is on device 0, the call on device 1"):
        gm._space(Tensor(0), 1)
    host = torch.zeros(4)
    with pytest.raises(ValueError, match="w: must be a device tensor"):
        gm._vector(host, host.dtype, 4, "w", 1)


def test_layouts_match_the_header(tmp_path):
    structs = [_abi.gnn_norm, _abi.gnn_norm_grad, _abi.gnn_dense, _abi.gnn_dense_grad, _abi.gnn_gated,
               _abi.gnn_gated_grad]
    want = {}
    lines = []
    for s in structs:
        want[s.__name__] = ctypes.sizeof(s)
        lines.append(f"S({s.__name__})")
        for name, _ in s._fields_:
            want[f"{s.__name__}.{name}"] = getattr(s, name).offset
            lines.append(f"O({s.__name__}, {name})")
    src = tmp_path / "layout.c"
    src.write_text('#include <stddef.h>\n#include <stdio.h>\n#include "gnnmb.h"\n'
                   '#define S(T) printf(#T " %zu\\n", sizeof(T));\n'
                   '#define O(T, f) printf(#T "." #f " %zu\\n", offsetof(T, f));\n'
                   "int main(void) { " + " ".join(lines) + " return 0; }\n")
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)])
    out = subprocess.check_output([str(exe)]).decode().split("\n")
    got = {k: int(v) for k, v in (line.rsplit(" ", 1) for line in out if line)}
    assert got == want
