"""The measured cases of the learned side of the path: embedding lookup with scaling, its gradient by
sorted ids, cross attention of queries to a mini-batch's states and its backward pass, and the
orthogonalisation of a weight matrix's update by Newton-Schulz products.

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
        # one token of each of the group's sequences attends to its mini-batch's first-hop states
        dict(name="attend one token", op="attend", batch=16, lq=1, lk=16_384, heads=16, kv=4, d=128,
             dtype="bf16", train=False, empty=False),
        # prompts of a few tokens over short neighbourhoods, one of them without a neighbour
        dict(name="attend short odd", op="attend", batch=12, lq=19, lk=333, heads=8, kv=2, d=80,
             dtype="f32", train=False, empty=True),
        # a training step over ragged states, grouped heads
        dict(name="attend train", op="attend", batch=4, lq=1024, lk=2600, heads=16, kv=4, d=128,
             dtype="bf16", train=True, empty=False),
        # the same in single precision, one sequence without states
        dict(name="attend train f32", op="attend", batch=3, lq=201, lk=1025, heads=8, kv=8, d=64,
             dtype="f32", train=True, empty=True),
        # the weights [2 d, d_out] of one mean-aggregating layer
        dict(name="ortho layer", op="ortho", batch=1, m=256, n=256, dtype="f32"),
        # tall, odd in both directions, single precision
        dict(name="ortho tall odd", op="ortho", batch=2, m=2571, n=1030, dtype="f32"),
        # the largest square weights
        dict(name="ortho large", op="ortho", batch=1, m=4096, n=4096, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lookup", "grad", "attend", "ortho"])
    if op == "attend":
        train = rng.random() < 0.5
        while True:
            heads = rng.choice([4, 8, 16])
            case = dict(op=op, batch=_spread(rng, 1, 16), lq=_spread(rng, 1, 1024),
                        lk=_spread(rng, 1, 16_384), heads=heads,
                        kv=heads // rng.choice([1, 2, 4]), d=rng.choice([32, 40, 64, 80, 128]),
                        dtype=rng.choice(["f32", "bf16"]), train=train, empty=rng.random() < 0.3)
            case["empty"] = case["empty"] and case["batch"] > 1
            if case["batch"] * heads * case["lq"] * case["lk"] <= (50e6 if train else 150e6):
                return case
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


def _lengths(case):
    """Queries and states of each sequence, from the case alone: between a quarter and all of lk."""
    lq, lk = [], []
    for b in range(case["batch"]):
        part = (0.618034 * (b + 1)) % 1.0 if b else 1.0
        lk.append(max(1, round(case["lk"] * (0.25 + 0.75 * part))))
        lq.append(max(1, round(case["lq"] * (0.5 + 0.5 * (0.7548777 * b % 1.0)))) if b else case["lq"])
    if case["empty"]:
        lk[case["batch"] // 2] = 0
    return lq, lk


def _indptr(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "attend":
        lq, lk = _lengths(case)
        h, kv, d, dtype = case["heads"], case["kv"], case["d"], DTYPES[case["dtype"]]

        def rows(n, heads):
            return torch.randn(n, heads, d, generator=gen, device="cuda", dtype=dtype)

        s["q"], s["k"], s["v"] = rows(sum(lq), h), rows(sum(lk), kv), rows(sum(lk), kv)
        s["q_indptr"], s["k_indptr"] = _indptr(lq), _indptr(lk)
        s["max_q"], s["max_k"], s["scale"] = max(lq), max(lk), d ** -0.5
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(sum(lq), h, device="cuda")
        if case["train"]:
            s["dout"] = rows(sum(lq), h)
            s["dq"], s["dk"], s["dv"] = (torch.empty_like(s[x]) for x in "qkv")
        if own:
            import graph_mini_pipeline_amd as gm
            s["ws"] = torch.empty(gm.gnn_cross_attention_workspace_size(
                case["batch"], sum(lq), sum(lk), s["max_q"], s["max_k"], h, kv, d, dtype,
                backward=case["train"]), dtype=torch.uint8, device="cuda")
        return s
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
    return {"lookup": _lookup, "grad": _grad, "attend": _attend, "ortho": _ortho}[s["case"]["op"]](s)


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


def _padded(indptr, most, x, heads):
    """Rows of a packed x as [batch, heads, most, d] in 32 bits, and which of them there are."""
    at = indptr[:-1, None].long() + torch.arange(most, device="cuda")
    there = at < indptr[1:, None]
    if x.shape[0] == 0:
        return x.new_zeros(at.shape[0], heads, most, x.shape[2], dtype=torch.float32), there
    y = torch.where(there[:, :, None, None], x[at.clamp(max=x.shape[0] - 1)].float(), 0.0)
    return y.transpose(1, 2).contiguous(), there


def _attend(s):
    case = s["case"]
    if own:
        import graph_mini_pipeline_amd as gm
        gm.gnn_cross_attention(s["q"], s["k"], s["v"], s["q_indptr"], s["k_indptr"], s["max_q"],
                               s["max_k"], s["scale"], s["out"], s["ws"], lse=s["lse"])
        if not case["train"]:
            return s["out"], s["lse"]
        gm.gnn_cross_attention_backward(s["q"], s["k"], s["v"], s["q_indptr"], s["k_indptr"],
                                        s["max_q"], s["max_k"], s["scale"], s["out"], s["lse"],
                                        s["dout"], s["dq"], s["dk"], s["dv"], s["ws"])
        return s["out"], s["lse"], s["dq"], s["dk"], s["dv"]
    b, h, kv, d = case["batch"], case["heads"], case["kv"], case["d"]
    lq, lk, dtype = s["max_q"], s["max_k"], s["q"].dtype

    def shared(x):      # [b, h, lq, d] with the heads that share states in one matrix
        return x.reshape(b * kv, h // kv * lq, d)

    def times(x, y):    # batched x @ y^T
        return x @ y.transpose(1, 2).contiguous()

    q, there_q = _padded(s["q_indptr"], lq, s["q"], h)
    k, there_k = _padded(s["k_indptr"], lk, s["k"], kv)
    v, _ = _padded(s["k_indptr"], lk, s["v"], kv)
    q, k, v = shared(q), k.reshape(b * kv, lk, d), v.reshape(b * kv, lk, d)
    live = there_k[:, None, None, :].expand(b, kv, 1, lk).reshape(b * kv, 1, lk)
    score = torch.where(live, times(q, k) * s["scale"], -math.inf)
    top = score.amax(2, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(2, keepdim=True)
    lse = torch.where(top == -math.inf, -math.inf, top + torch.log(total))
    p = p / torch.where(total == 0, 1.0, total)
    out = p @ v

    def packed(x, there, heads, most):
        return x.reshape(b, heads, most, -1).transpose(1, 2)[there]

    answer = (packed(out, there_q, h, lq).to(dtype), packed(lse, there_q, h, lq)[:, :, 0])
    if not case["train"]:
        return answer
    g = shared(_padded(s["q_indptr"], lq, s["dout"], h)[0])
    dv = p.transpose(1, 2).contiguous() @ g
    ds = p * (times(g, v) - (g * out).sum(2, keepdim=True)) * s["scale"]
    dq, dk = ds @ k, ds.transpose(1, 2).contiguous() @ q
    return answer + (packed(dq, there_q, h, lq).to(dtype), packed(dk, there_k, kv, lk).to(dtype),
                     packed(dv, there_k, kv, lk).to(dtype))


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
    if case["op"] == "attend":
        lq, lk = _lengths(case)
        h, d, z = case["heads"], case["d"], size[case["dtype"]]
        pairs = sum(x * y for x, y in zip(lq, lk)) * h * d
        rows_q, rows_k = sum(lq) * h * d * z, sum(lk) * case["kv"] * d * z
        if case["train"]:       # seven products of every query with every state
            return dict(bytes=4 * rows_q + 4 * rows_k + sum(lq) * h * 4, flops=14 * pairs)
        return dict(bytes=2 * rows_q + 2 * rows_k + sum(lq) * h * 4, flops=4 * pairs)
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
    if case["op"] == "attend":
        return _exact_attend(s)
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


def _exact_attend(s):
    """Sequence by sequence and head by head."""
    case = s["case"]
    group, scale = case["heads"] // case["kv"], s["scale"]
    names = ("out", "lse", "dq", "dk", "dv") if case["train"] else ("out", "lse")
    r = {x: torch.zeros(s[x].shape, dtype=torch.float64, device="cuda") for x in names}
    q_at, k_at = s["q_indptr"].tolist(), s["k_indptr"].tolist()
    for b in range(case["batch"]):
        i, j = slice(q_at[b], q_at[b + 1]), slice(k_at[b], k_at[b + 1])
        for h in range(case["heads"]):
            q, k, v = s["q"][i, h].double(), s["k"][j, h // group].double(), s["v"][j, h // group].double()
            if k.shape[0] == 0:
                r["lse"][i, h] = -math.inf
                continue
            score = scale * torch.mm(q, k.t())
            lse = torch.logsumexp(score, 1)
            p = torch.exp(score - lse[:, None])
            r["out"][i, h], r["lse"][i, h] = torch.mm(p, v), lse
            if not case["train"]:
                continue
            g = s["dout"][i, h].double()
            r["dv"][j, h // group] += torch.mm(p.t(), g)
            dp = torch.mm(g, v.t())
            ds = scale * p * (dp - (p * dp).sum(1, keepdim=True))
            r["dq"][i, h] = torch.mm(ds, k)
            r["dk"][j, h // group] += torch.mm(ds.t(), q)
    return tuple(r[x] for x in names)


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
