"""A workspace of the dense layers that is sized for a batch serves every smaller one."""
import random

import pytest
import torch

import graph_mini_pipeline_amd as gm

LAYERS = [(1, 1), (16, 24), (64, 16), (256, 128), (515, 1371), (1024, 4096), (4096, 4096), (4096, 10240), (16384, 4096)]


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [gm.gnn_linear_workspace_size, gm.gnn_gated_linear_workspace_size])
@pytest.mark.parametrize("d_in, d_out", LAYERS)
def test_sizes_grow_with_the_rows(d_in, d_out, size, dtype, backward):
    rng = random.Random(d_in + d_out)
    rows = sorted(set(list(range(0, 140)) + [255, 256, 257, 511, 512, 513] + [int(2 ** rng.uniform(7, 24)) for _ in range(300)]))
    sizes = [size(n, d_in, d_out, dtype, backward=backward) for n in rows]
    assert sizes == sorted(sizes)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_forward_pass_takes_no_more_than_a_part_of_the_last_cache(dtype):
    """Whatever the rows, and beside what the gradients keep of each row."""
    for size in (gm.gnn_linear_workspace_size, gm.gnn_gated_linear_workspace_size):
        for d_in, d_out in LAYERS + [(4096, 128256), (1 << 20, 1 << 20)]:
            for n in (1, 64, 1000, 1 << 20, 1 << 30):
                assert size(n, d_in, d_out, dtype) <= (128 << 20) + 256
