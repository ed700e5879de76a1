"""Norm, gated pair and linear layer run together, as a feed-forward block beside the lookup and attention
(examples/text_on_graph.py with a hidden width): the gradients of one step against automatic differentiation of
the same model in 64 bits on the host, and a few steps in each type."""
import importlib.util
import math
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

gm = pytest.importorskip("graph_mini_pipeline_amd")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    spec = importlib.util.spec_from_file_location("text_on_graph",
                                                  os.path.join(ROOT, "examples", "text_on_graph.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def graph(nodes=300):
    g = torch.Generator().manual_seed(3)
    degree = torch.randint(0, 9, (nodes,), generator=g)
    indptr = torch.cat([torch.zeros(1, dtype=torch.int64), degree.cumsum(0)])
    indices = torch.randint(nodes, (int(indptr[-1]),), generator=g).to(torch.int32)
    return gm.DeviceGraph(nodes, indptr.cuda(), indices.cuda())


def test_gradients_against_autograd():
    """fp32.  Every gradient is a sum of at most some thousand terms through seven products of widths up to 64 and a
    norm: relative errors of 2^-24 per operation, some thousand of them at worst in a row, 1e-4 of a gradient's
    largest entry."""
    ex = example()
    model = ex.TextOnGraph(graph(), vocab=101, d=32, heads=4, kv_heads=2, classes=5, seeds=40, fanout=6, tokens=7,
                           dtype=torch.float32, seed=1, hidden=56)
    model.norm["weight"].normal_(1.0, 0.2)
    model.norm["bias"].normal_(0.0, 0.2)
    ids, texts, labels = next(ex.synthetic_batches(300, 101, 5, 40, 7, 2))
    loss, grads, token_grad, (nodes, count, rows) = model.gradients(ids, texts, labels, 77)
    edges = int(model.blocks.counts[0])
    ptr = model.blocks.indptr[0].tolist()
    near = model.blocks.gid[0][:edges].long().cpu()

    leaf = lambda t: t.detach().double().cpu().requires_grad_()
    tokens, table = leaf(model.token_table), leaf(model.node_table)
    w = {k: leaf(v) for k, v in model.weights.items()}
    norm = {k: leaf(v) for k, v in model.norm.items()}
    flat = texts.reshape(-1).long().cpu()
    x = tokens[flat] * float(torch.tensor(math.sqrt(32), dtype=torch.float32))
    x = torch.where((flat == ex.PAD)[:, None], torch.zeros_like(x), x)
    q = (x @ w["q"]).view(40, 7, 4, 8)
    states = (table[near] @ w["kv"]).view(edges, 4, 8)
    attended = []
    for s in range(40):
        k, v = states[ptr[s]:ptr[s + 1], :2], states[ptr[s]:ptr[s + 1], 2:]
        if k.shape[0] == 0:
            attended.append(torch.zeros(7, 32, dtype=torch.float64))
            continue
        heads = [torch.softmax(8 ** -0.5 * q[s, :, h] @ k[:, h // 2].T, 1) @ v[:, h // 2] for h in range(4)]
        attended.append(torch.cat(heads, 1))
    r = x + torch.cat(attended)
    y = torch.nn.functional.layer_norm(r, (32,), norm["weight"], norm["bias"], ex.EPS)
    r = r + (torch.nn.functional.silu(y @ w["gate"]) * (y @ w["up"])) @ w["down"]
    want = torch.nn.functional.cross_entropy(r.view(40, 7, 32).mean(1) @ w["o"], labels.cpu())
    want.backward()
    assert abs(float(loss) - float(want.detach())) < 1e-5

    def near_enough(got, exact):
        assert float((got.double().cpu() - exact).abs().max()) <= 1e-4 * float(exact.abs().max())

    for k in w:
        near_enough(grads[k], w[k].grad)
    for k in norm:
        near_enough(model.norm_grads[k], norm[k].grad)
    near_enough(token_grad, tokens.grad)
    n = int(count)
    dense = torch.zeros_like(table)
    dense[nodes[:n].long().cpu()] = rows[:n].double().cpu()
    near_enough(dense, table.grad)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_a_few_steps_run(dtype):
    losses = example().train(steps=4, dtype=dtype, hidden=96)
    assert len(losses) == 4 and all(math.isfinite(x) for x in losses)
