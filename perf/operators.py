"""The measured cases of the training-side operators: embedding lookup with scaling, its gradient by
sorted ids, and the orthogonalisation of a weight matrix's update by Newton-Schulz products.

`run` computes them with the library's calls where `own` is true and in plain torch operations
where it is not; `exact` gives the same results in 64 bits.
"""
import math

import torch

own = False

#: The quintic p(s) = a s + b s^3 + c s^5 that every step applies to the singular values, the number
#: of steps, and what is added to the norm.
QUINTIC = (3.4445, -4.7750, 2.0315)
STEPS = 5
EPS = 1e-7

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
PAD = 0   # the padding id of the cases with padding: its rows are zero and get no gradient


def listed():
    return [
        # the seeds of one mini-batch read their learned node vectors: one short launch
        dict(name="lookup seeds", op="lookup", n=1024, rows=233_000, d=602, table="f32", out="f32",
             ids="frontier", pad=False),
        # text tokens of a batch of sequences with padding at their ends, scaled by sqrt(d)
        dict(name="lookup tokens", op="lookup", n=16_384, rows=50_257, d=768, table="bf16",
             out="bf16", ids="zipf", pad=True),
        # the whole last frontier of a three-hop mini-batch, single-precision table, bf16 activations
        dict(name="lookup frontier", op="lookup", n=1_081_344, rows=2_450_000, d=100, table="f32",
             out="bf16", ids="frontier", pad=False),
        # a small graph's node vectors: latency counts
        dict(name="grad small", op="grad", n=1024, rows=10_000, d=64, dout="f32", out="f32",
             form="dense", ids="uniform", pad=False),
        # the gradient of a token table from a batch of sequences: few words hold most positions
        dict(name="grad tokens", op="grad", n=131_072, rows=50_257, d=1024, dout="bf16", out="f32",
             form="dense", ids="zipf", pad=True),
        # one gradient row for each sampled edge of a mini-batch, over the nodes that it reaches; hubs
        # repeat; only the touched rows of a large table come back
        dict(name="grad edges", op="grad", n=901_120, rows=2_450_000, d=100, dout="f32", out="f32",
             form="rows", ids="edges", nodes=400_000, pad=False),
        # odd width, so that rows are not aligned, and a ragged number of tokens
        dict(name="grad odd", op="grad", n=33_333, rows=100_003, d=515, dout="bf16", out="bf16",
             form="dense", ids="zipf", pad=True),
        # the weights [2 d, d_out] of one mean-aggregating layer
        dict(name="ortho layer", op="ortho", batch=1, m=256, n=256, dtype="f32"),
        # many equal small matrices at once (the projections of the heads of a model)
        dict(name="ortho heads", op="ortho", batch=24, m=128, n=768, dtype="bf16"),
        # one wide projection of a mid-sized model
        dict(name="ortho wide", op="ortho", batch=1, m=1024, n=4096, dtype="bf16"),
        # tall, odd in both directions, single precision
        dict(name="ortho tall odd", op="ortho", batch=2, m=2571, n=1030, dtype="f32"),
        # the largest square weights
        dict(name="ortho large", op="ortho", batch=1, m=4096, n=4096, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lookup", "grad", "ortho"])
    if op == "ortho":
        dtype = rng.choice(["f32", "bf16"])
        m, n = _spread(rng, 64, 4096), _spread(rng, 64, 4096)
        top = 68e9 if dtype == "bf16" else 10e9     # of m n min(m, n), over the batch
        while m * n * min(m, n) > top:
            m, n = _spread(rng, 64, 4096), _spread(rng, 64, 4096)
        most = int(min(32, top / (m * n * min(m, n))))
        return dict(op=op, batch=_spread(rng, 1, max(1, most)), m=m, n=n, dtype=dtype)
    rows = _spread(rng, 1000, 2_450_000)
    d = _spread(rng, 32, 1024)
    if rng.random() < 0.6:
        d = -(-d // 8) * 8
    while rows * d > 300_000_000:
        rows = _spread(rng, 1000, 2_450_000)
    n = _spread(rng, 256, max(512, min(1_081_344, 130_000_000 // d)))
    if op == "lookup":
        ids = rng.choice(["frontier", "zipf", "uniform"])
        return dict(op=op, n=min(n, rows) if ids == "frontier" else n, rows=rows, d=d,
                    table=rng.choice(["f32", "bf16"]), out=rng.choice(["f32", "bf16"]), ids=ids,
                    pad=rng.random() < 0.5)
    case = dict(op=op, n=n, rows=rows, d=d, dout=rng.choice(["f32", "bf16"]),
                out=rng.choice(["f32", "bf16"]), pad=rng.random() < 0.5)
    if rng.random() < 0.5:
        return dict(case, form="rows", ids="edges", nodes=_spread(rng, 64, min(n, rows - 1)))
    while case["rows"] * d > 60_000_000:
        case["rows"] = _spread(rng, 1000, 2_450_000)
    return dict(case, form="dense", ids=rng.choice(["zipf", "uniform"]))


def _by_frequency(n, count, gen):
    """n ranks below count, rank r in proportion to 1 / (r + 1): word and hub frequencies."""
    cdf = torch.cumsum(1.0 / torch.arange(1, count + 1, device="cuda", dtype=torch.float64), 0)
    u = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64) * cdf[-1]
    return torch.searchsorted(cdf, u).clamp_(max=count - 1)


def _ids(case, gen):
    n, rows = case["n"], case["rows"]
    if case["ids"] == "edges":          # each node of the batch once, then by frequency, mixed
        k = case["nodes"]
        nodes = 1 + torch.randperm(rows - 1, generator=gen, device="cuda")[:k]
        more = nodes[_by_frequency(n - k, k, gen)]
        if case["pad"]:
            more = more.masked_fill(torch.rand(n - k, generator=gen, device="cuda") < 1 / 16, PAD)
        mixed = torch.randperm(n, generator=gen, device="cuda")
        return torch.cat([nodes, more])[mixed].to(torch.int32)
    if case["ids"] == "frontier":       # a mini-batch's node list: distinct, ascending
        ids = torch.randperm(rows, generator=gen, device="cuda")[:n].sort()[0]
    elif case["ids"] == "zipf":
        ids = torch.randperm(rows, generator=gen, device="cuda")[_by_frequency(n, rows, gen)]
    else:
        ids = torch.randint(rows, (n,), generator=gen, device="cuda")
    if case["pad"]:                     # about one position in sixteen is padding
        ids = ids.masked_fill(torch.rand(n, generator=gen, device="cuda") < 1 / 16, PAD)
    return ids.to(torch.int32)


def _scale(case):
    """sqrt(d), rounded to 32 bits."""
    return float(torch.tensor(math.sqrt(case["d"]), dtype=torch.float32))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "ortho":
        b, m, n = case["batch"], case["m"], case["n"]
        k = max(1, min(m, n) // 8)
        # a momentum: a few strong directions over a floor of noise
        strong = torch.randn(b, m, k, generator=gen, device="cuda") @ torch.randn(
            b, k, n, generator=gen, device="cuda")
        g = 1e-3 * (strong / math.sqrt(k) + torch.randn(b, m, n, generator=gen, device="cuda"))
        s["g"] = g.to(DTYPES[case["dtype"]])
        s["out"] = torch.empty_like(s["g"])
        if own:
            import graph_mini_pipeline_amd as gm
            s["ws"] = torch.empty(gm.gnn_orthogonalize_workspace_size(b, m, n, s["g"].dtype),
                                  dtype=torch.uint8, device="cuda")
        return s
    n, rows, d = case["n"], case["rows"], case["d"]
    s["ids"] = _ids(case, gen)
    s["pad"] = PAD if case["pad"] else -1
    s["scale"] = _scale(case)
    out = DTYPES[case["out"]]
    if case["op"] == "lookup":
        s["table"] = torch.randn(rows, d, generator=gen, device="cuda", dtype=DTYPES[case["table"]])
        s["out"] = torch.empty(n, d, device="cuda", dtype=out)
        return s
    s["dout"] = torch.randn(n, d, generator=gen, device="cuda", dtype=DTYPES[case["dout"]])
    if case["form"] == "dense":
        s["grad"] = torch.empty(rows, d, device="cuda", dtype=out)
    else:
        # the length of the batch's node list is known before its backward pass
        s["nodes"] = torch.empty(case["nodes"], dtype=torch.int32, device="cuda")
        s["count"] = torch.empty(1, dtype=torch.int64, device="cuda")
        s["grad"] = torch.empty(case["nodes"], d, device="cuda", dtype=out)
    if own:
        import graph_mini_pipeline_amd as gm
        s["ws"] = torch.empty(gm.gnn_embedding_grad_workspace_size(n, rows, d), dtype=torch.uint8,
                              device="cuda")
    return s


def run(s):
    return {"lookup": _lookup, "grad": _grad, "ortho": _ortho}[s["case"]["op"]](s)


def _lookup(s):
    if own:
        import graph_mini_pipeline_amd as gm
        gm.gnn_embedding_lookup(s["table"], s["ids"], s["scale"], s["out"], pad_id=s["pad"])
        return s["out"]
    x = s["table"][s["ids"]].float() * s["scale"]
    if s["case"]["pad"]:
        x = torch.where((s["ids"] == s["pad"])[:, None], 0.0, x)
    return x.to(s["out"].dtype)


def _grad(s):
    case = s["case"]
    if own:
        import graph_mini_pipeline_amd as gm
        if case["form"] == "dense":
            gm.gnn_embedding_grad(s["ids"], s["dout"], s["scale"], s["grad"], s["ws"],
                                  pad_id=s["pad"])
            return s["grad"]
        gm.gnn_embedding_grad_rows(s["ids"], s["dout"], s["scale"], case["rows"], s["nodes"],
                                   s["count"], s["grad"], s["ws"], pad_id=s["pad"])
        return s["nodes"], s["count"], s["grad"]
    g = s["dout"].float()
    if case["pad"]:
        g = torch.where((s["ids"] == s["pad"])[:, None], 0.0, g)
    if case["form"] == "dense":
        acc = torch.zeros(case["rows"], case["d"], device="cuda")
        acc.index_add_(0, s["ids"], g)
        return (acc * s["scale"]).to(s["grad"].dtype)
    nodes, place = torch.unique(s["ids"], sorted=True, return_inverse=True)
    acc = torch.zeros(nodes.numel(), case["d"], device="cuda")
    acc.index_add_(0, place, g)
    if case["pad"]:
        kept = nodes != s["pad"]
        nodes, acc = nodes[kept], acc[kept]
    count = torch.full((1,), nodes.numel(), device="cuda")
    return nodes, count, (acc * s["scale"]).to(s["grad"].dtype)


def _ortho(s):
    if own:
        import graph_mini_pipeline_amd as gm
        gm.gnn_orthogonalize(s["g"], s["out"], s["ws"], steps=STEPS, coefs=QUINTIC, eps=EPS)
        return s["out"]
    a, b, c = QUINTIC
    x = s["g"].float()
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    x = x / (x.square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2).contiguous()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if tall:
        x = x.transpose(1, 2).contiguous()
    return x.to(s["g"].dtype)


def _distinct(case):
    """The expected number of distinct ids, without the padding."""
    n, rows = case["n"] * (15 / 16 if case["pad"] else 1.0), case["rows"]
    if case["ids"] == "edges":
        return case["nodes"]
    if case["ids"] == "frontier":
        return n
    if case["ids"] == "uniform":
        return rows * -math.expm1(n * math.log1p(-1 / rows))
    p = 1.0 / torch.arange(1, rows + 1, dtype=torch.float64)
    p = (p / p.sum()).clamp_(max=1 - 1e-12)
    return float(-torch.expm1(n * torch.log1p(-p)).sum())


def work(case):
    size = {"f32": 4, "bf16": 2}
    if case["op"] == "ortho":
        s, l = sorted((case["m"], case["n"]))
        # of the two symmetric products one triangle is needed, with its diagonal
        flops = STEPS * (s * (s + 1) * l + s * (s + 1) * s + 2 * s * s * l)
        return dict(bytes=2 * case["batch"] * s * l * size[case["dtype"]],
                    flops=case["batch"] * flops)
    n, d = case["n"], case["d"]
    kept = n - (n - case.get("nodes", 0)) * (1 / 16 if case["pad"] else 0.0)
    if case["op"] == "lookup":
        return dict(bytes=4 * n + _distinct(case) * d * size[case["table"]] +
                    n * d * size[case["out"]], flops=n * d)
    if case["form"] == "dense":
        written = case["rows"] * d * size[case["out"]]
    else:
        written = _distinct(case) * (4 + d * size[case["out"]])
    return dict(bytes=4 * n + kept * d * size[case["dout"]] + written, flops=kept * d)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "ortho":
        return _exact_ortho(s["g"].double())
    ids, scale = s["ids"].long(), torch.tensor(s["scale"], dtype=torch.float64, device="cuda")
    if case["op"] == "lookup":
        out = torch.zeros(case["n"], case["d"], dtype=torch.float64, device="cuda")
        live = torch.nonzero(ids != s["pad"]).squeeze(1)
        out[live] = torch.index_select(s["table"], 0, ids[live]).double() * scale
        return out
    # the positions in the order of their ids, running sums over them, and their differences at
    # the ends of every id's run
    live = torch.nonzero(ids != s["pad"]).squeeze(1)
    order = live[torch.argsort(ids[live], stable=True)]
    nodes, counts = torch.unique_consecutive(ids[order], return_counts=True)
    last = torch.cumsum(counts, 0) - 1
    sums = torch.empty(nodes.numel(), case["d"], dtype=torch.float64, device="cuda")
    for j in range(0, case["d"], 128):
        part = torch.cumsum(s["dout"][:, j:j + 128][order].double(), 0)[last]
        sums[:, j:j + 128] = torch.diff(part, dim=0, prepend=torch.zeros_like(part[:1])) * scale
    if case["form"] == "rows":
        return nodes.to(torch.int32), torch.tensor([nodes.numel()], device="cuda"), sums
    out = torch.zeros(case["rows"], case["d"], dtype=torch.float64, device="cuda")
    out[nodes] = sums
    return out


def _exact_ortho(g):
    """Every step multiplies X from the left by Q = a I + b A + c A^2 with A = X X^T, and takes A to
    Q A Q; all of them are polynomials of the first A, so their product is gathered first and X is
    multiplied once."""
    a, b, c = QUINTIC
    outs = []
    for x in g:
        wide = x if x.shape[0] <= x.shape[1] else x.T.contiguous()
        wide = wide / (torch.linalg.matrix_norm(wide) + EPS)
        gram = wide @ wide.T
        eye = torch.eye(gram.shape[0], dtype=torch.float64, device=gram.device)
        total = eye
        for _ in range(STEPS):
            q = a * eye + gram @ (b * eye + c * gram)
            total = q @ total
            gram = q @ gram @ q
        wide = total @ wide
        outs.append(wide if x.shape[0] <= x.shape[1] else wide.T)
    return torch.stack(outs)
