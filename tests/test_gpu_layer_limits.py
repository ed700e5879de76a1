"""The norm and the dense layers where values are extreme: far arguments, infinities, rows far from zero."""
import pytest
import torch

from . import layers as ref
from .test_gpu_dense import B, F, space

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")


@pytest.mark.parametrize("dtype", [F, B])
@pytest.mark.parametrize("name", ref.ACTS)
def test_activations_of_the_farthest_arguments(name, dtype):
    """act and act' up to the type's largest number: z, 1 or 0, the functions' limits there."""
    top = torch.finfo(dtype).max
    z = torch.tensor([[s * v] for v in (1e5, 1e10, 1e19, 1e20, 1e30, top) for s in (1, -1)], device="cuda", dtype=dtype)
    one = torch.ones(1, 1, device="cuda", dtype=dtype)
    out, dx = torch.empty_like(z), torch.empty_like(z)
    n = z.shape[0]
    gm.gnn_linear(z, one, out, space(gm.gnn_linear_workspace_size, n, 1, 1, dtype), activation=name)
    gm.gnn_linear_backward(z, one, torch.ones_like(z), space(gm.gnn_linear_workspace_size, n, 1, 1, dtype, True),
                           activation=name, pre=z, dx=dx)
    up = z > 0
    if name == "none":
        want, slope = z, torch.ones_like(z)
    elif name == "sigmoid":
        want, slope = up.to(dtype), torch.zeros_like(z)
    else:
        want, slope = torch.where(up, z, 0.0), up.to(dtype)
    assert torch.equal(out, want) and torch.equal(dx, slope)
