"""Trains a small model of texts on a graph with the library's learned operators, on one GPU.

Every seed node carries a text of a few tokens.  One step on a mini-batch:
  1. gnn_sample_khop draws each seed's neighbours;
  2. gnn_embedding_lookup reads the texts' token vectors (scaled by sqrt(d)) and the sampled
     neighbours' node vectors, both from fp32 tables that are trained;
  3. gnn_cross_attention lets a seed's tokens attend to its own sampled neighbours: the block's indptr
     is the states' indptr, so seeds have different numbers of them, or none;
  4. with --hidden, a feed-forward block follows: gnn_layer_norm, gnn_gated_linear and gnn_linear, which
     adds its input (the residual) in its epilogue;
  5. the tokens are averaged and classified;
  6. backward: gnn_linear_backward, gnn_gated_linear_backward and gnn_layer_norm_backward (which adds the
     residual's gradient), gnn_cross_attention_backward, then gnn_embedding_grad for the token table
     and gnn_embedding_grad_rows for the touched rows of the node table;
  7. the weight matrices move along their momentum, orthogonalised by gnn_orthogonalize; the tables
     by plain gradient steps.
The projections are ordinary torch products.

    python examples/text_on_graph.py [--steps 60] [--hidden 128]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import graph_mini_pipeline_amd as gm  # noqa: E402
import synth  # noqa: E402

PAD = 0      # the padding token
EPS = 1e-5   # of the norm


class TextOnGraph:
    def __init__(self, graph: gm.DeviceGraph, vocab: int, d: int = 64, heads: int = 4, kv_heads: int = 2,
                 classes: int = 8, seeds: int = 256, fanout: int = 10, tokens: int = 12,
                 dtype=torch.bfloat16, seed: int = 0, hidden: int = 0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return scale * torch.randn(*shape, generator=g, device="cuda")

        self.graph, self.dtype = graph, dtype
        self.d, self.heads, self.kv, self.hd = d, heads, kv_heads, d // heads
        self.seeds, self.fanout, self.tokens = seeds, fanout, tokens
        self.token_table = normal(vocab, d, scale=d ** -0.5)
        self.node_table = normal(graph.num_nodes, d, scale=1.0)
        width = kv_heads * self.hd
        self.weights = {"q": normal(d, d, scale=d ** -0.5), "kv": normal(d, 2 * width, scale=d ** -0.5),
                        "o": normal(d, classes, scale=d ** -0.5)}
        self.hidden = hidden
        if hidden:
            self.weights.update(gate=normal(d, hidden, scale=d ** -0.5), up=normal(d, hidden, scale=d ** -0.5),
                                down=normal(hidden, d, scale=hidden ** -0.5))
            self.norm = {"weight": torch.ones(d, device="cuda"), "bias": torch.zeros(d, device="cuda")}
        self.momentum = {k: torch.zeros_like(w) for k, w in self.weights.items()}

        # what a program keeps from step to step: blocks, workspaces, outputs
        self.caps = gm.gnn_capacity(seeds, [fanout], graph.num_nodes)
        self.blocks = gm.Blocks(self.caps)
        edges, rows = self.caps.edges[0], seeds * tokens

        def space(n):
            return torch.empty(n, dtype=torch.uint8, device="cuda")

        self.ws_sample = space(gm.gnn_workspace_size(self.caps, graph.num_nodes))
        self.ws_attend = space(gm.gnn_cross_attention_workspace_size(
            seeds, rows, edges, tokens, fanout, heads, kv_heads, self.hd, dtype, backward=True))
        self.ws_tokens = space(gm.gnn_embedding_grad_workspace_size(rows, vocab, d))
        self.ws_nodes = space(gm.gnn_embedding_grad_workspace_size(edges, graph.num_nodes, d))
        self.ws_ortho = {k: space(gm.gnn_orthogonalize_workspace_size(1, *w.shape, w.dtype))
                         for k, w in self.weights.items()}
        if hidden:
            self.ws_ff = space(max(
                gm.gnn_layer_norm_workspace_size(rows, d),
                *(gm.gnn_gated_linear_workspace_size(rows, d, hidden, dtype, backward=b) for b in (False, True)),
                *(gm.gnn_linear_workspace_size(rows, hidden, d, dtype, backward=b) for b in (False, True))))
        self.q_indptr = torch.arange(seeds + 1, device="cuda", dtype=torch.int32) * tokens
        self.token_grad = torch.empty_like(self.token_table)
        self.nodes = torch.empty(edges, dtype=torch.int32, device="cuda")
        self.n_nodes = torch.empty(1, dtype=torch.int64, device="cuda")
        self.node_grad = torch.empty(edges, d, device="cuda")

    def feed_forward(self, r: torch.Tensor):
        """r + down(silu(gate y) * up y) with y the norm of r, and what its backward pass needs."""
        w = {k: self.weights[k].to(self.dtype) for k in ("gate", "up", "down")}
        rows = r.shape[0]
        y, (mean, rstd) = torch.empty_like(r), torch.empty(2, rows, device="cuda")
        gm.gnn_layer_norm(r, self.norm["weight"], self.norm["bias"], EPS, y, mean=mean, rstd=rstd)
        h, gate, up = torch.empty(3, rows, self.hidden, device="cuda", dtype=self.dtype)
        gm.gnn_gated_linear(y, w["gate"], w["up"], h, self.ws_ff, gate=gate, up=up)
        out = torch.empty_like(r)
        gm.gnn_linear(h, w["down"], out, self.ws_ff, residual=r)
        return out, (w, r, mean, rstd, y, gate, up, h)

    def feed_forward_gradients(self, kept, dout: torch.Tensor, grads: dict):
        """The gradient of feed_forward's input; those of its weights go into grads."""
        w, r, mean, rstd, y, gate, up, h = kept
        dw = {k: torch.empty_like(v) for k, v in w.items()}
        dh, dy, dr = torch.empty_like(h), torch.empty_like(y), torch.empty_like(r)
        gm.gnn_linear_backward(h, w["down"], dout, self.ws_ff, dx=dh, dw=dw["down"])
        gm.gnn_gated_linear_backward(y, w["gate"], w["up"], gate, up, dh, self.ws_ff, dx=dy,
                                     dw_gate=dw["gate"], dw_up=dw["up"])
        dn = {k: torch.empty_like(v) for k, v in self.norm.items()}
        gm.gnn_layer_norm_backward(r, self.norm["weight"], mean, rstd, dy, dr, self.ws_ff,
                                   dweight=dn["weight"], dbias=dn["bias"], residual_grad=dout)
        grads.update({k: v.float() for k, v in dw.items()})
        self.norm_grads = dn
        return dr

    def gradients(self, ids: torch.Tensor, texts: torch.Tensor, labels: torch.Tensor, draw: int):
        """The loss of one mini-batch and its gradients: of the weights (a dict), the token table, and
        (nodes, their number, rows) of the node table."""
        d, dt, rows = self.d, self.dtype, self.seeds * self.tokens
        gm.gnn_sample_khop(self.graph, ids, [self.fanout], draw, self.blocks, self.ws_sample)
        edges = int(self.blocks.counts[0])
        near, k_indptr = self.blocks.gid[0][:edges], self.blocks.indptr[0]

        x = torch.empty(rows, d, device="cuda", dtype=dt)
        gm.gnn_embedding_lookup(self.token_table, texts.reshape(-1), math.sqrt(d), x, pad_id=PAD)
        y = torch.empty(edges, d, device="cuda", dtype=dt)
        gm.gnn_embedding_lookup(self.node_table, near, 1.0, y)

        w = {k: v.to(dt) for k, v in self.weights.items()}
        q = (x @ w["q"]).view(rows, self.heads, self.hd)
        states = (y @ w["kv"]).view(edges, 2 * self.kv, self.hd)
        k, v = states[:, :self.kv], states[:, self.kv:]      # halves of one projection's rows
        out, lse = torch.empty_like(q), torch.empty(rows, self.heads, device="cuda")
        scale = self.hd ** -0.5
        gm.gnn_cross_attention(q, k, v, self.q_indptr, k_indptr, self.tokens, self.fanout, scale, out,
                               self.ws_attend, lse=lse)
        # the tokens' own vectors pass beside what they attended to
        h = x.float() + out.view(rows, d).float()
        if self.hidden:
            y2, kept = self.feed_forward(h.to(dt))
            h = y2.float()
        h = h.view(self.seeds, self.tokens, d).mean(1)
        logits = h @ self.weights["o"]
        p = torch.softmax(logits, 1)
        loss = -torch.log(p[torch.arange(self.seeds, device="cuda"), labels]).mean()

        dlogits = (p - torch.nn.functional.one_hot(labels, p.shape[1])) / self.seeds
        grads = {"o": h.T @ dlogits}
        dh = (dlogits @ self.weights["o"].T / self.tokens).to(dt)
        dout = dh[:, None, :].expand(-1, self.tokens, -1).contiguous().view(rows, d)
        if self.hidden:
            dout = self.feed_forward_gradients(kept, dout, grads)
        dout = dout.view(rows, self.heads, self.hd)
        dq, dstates = torch.empty_like(q), torch.empty_like(states)
        gm.gnn_cross_attention_backward(q, k, v, self.q_indptr, k_indptr, self.tokens, self.fanout, scale,
                                        out, lse, dout, dq, dstates[:, :self.kv],
                                        dstates[:, self.kv:], self.ws_attend)
        dq, dstates = dq.view(rows, d), dstates.view(edges, -1)
        grads["q"], grads["kv"] = (x.T @ dq).float(), (y.T @ dstates).float()
        dx = dout.view(rows, d) + dq @ w["q"].T
        gm.gnn_embedding_grad(texts.reshape(-1), dx, math.sqrt(d), self.token_grad, self.ws_tokens,
                              pad_id=PAD)
        dy = dstates @ w["kv"].T
        gm.gnn_embedding_grad_rows(near, dy, 1.0, self.graph.num_nodes, self.nodes, self.n_nodes,
                                   self.node_grad, self.ws_nodes)
        return loss, grads, self.token_grad, (self.nodes, self.n_nodes, self.node_grad)

    def step(self, ids, texts, labels, draw, lr=0.05, table_lr=20.0, beta=0.9) -> torch.Tensor:
        loss, grads, token_grad, (nodes, count, rows) = self.gradients(ids, texts, labels, draw)
        for k, w in self.weights.items():
            m = self.momentum[k].mul_(beta).add_(grads[k])
            update = torch.empty_like(w)
            gm.gnn_orthogonalize(grads[k] + beta * m, update, self.ws_ortho[k])
            w.sub_(lr * update)
        if self.hidden:
            for k, v in self.norm.items():
                v.sub_(lr * self.norm_grads[k])
        self.token_table.sub_(table_lr * token_grad)
        n = int(count)
        self.node_table[nodes[:n].long()] -= table_lr * rows[:n]
        return loss


def synthetic_batches(num_nodes: int, vocab: int, classes: int, seeds: int, tokens: int, seed: int):
    """Seeds, their texts and labels: a label's texts draw most tokens from its own part of the
    vocabulary, and end in padding."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    while True:
        ids = torch.randperm(num_nodes, generator=g, device="cuda")[:seeds].to(torch.int32)
        labels = torch.randint(classes, (seeds,), generator=g, device="cuda")
        part = (vocab - 1) // classes
        own = 1 + labels[:, None] * part + torch.randint(part, (seeds, tokens), generator=g, device="cuda")
        other = torch.randint(1, vocab, (seeds, tokens), generator=g, device="cuda")
        texts = torch.where(torch.rand(seeds, tokens, generator=g, device="cuda") < 0.6, own, other)
        length = torch.randint(1, tokens + 1, (seeds, 1), generator=g, device="cuda")
        texts = texts.masked_fill(torch.arange(tokens, device="cuda") >= length, PAD)
        yield ids, texts.to(torch.int32), labels


def train(steps: int = 60, seed: int = 0, vocab: int = 1001, classes: int = 8, **model_args):
    """Losses of `steps` steps on the tiny synthetic graph."""
    cfg = synth.CONFIGS["tiny"]
    g = synth.build_graph(cfg)
    graph = gm.DeviceGraph(cfg.num_nodes, g.indptr.cuda(), g.indices.cuda())
    model = TextOnGraph(graph, vocab, classes=classes, seed=seed, **model_args)
    batches = synthetic_batches(cfg.num_nodes, vocab, classes, model.seeds, model.tokens, seed)
    losses = [model.step(*next(batches), gm.gnn_batch_seed(cfg.rng_seed, i)) for i in range(steps)]
    return [float(x) for x in losses]


if __name__ == "__main__":
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("--steps", type=int, default=60)
    parser.add_argument("--hidden", type=int, default=0, help="width of a feed-forward block (0: none)")
    args = parser.parse_args()
    for i, loss in enumerate(train(args.steps, hidden=args.hidden)):
        if i % 10 == 0 or i + 1 == args.steps:
            print(f"step {i:4d}  loss {loss:.4f}", flush=True)
