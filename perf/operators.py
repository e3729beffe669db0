"""The feed-forward operators on compressed weights, as they are measured.

Three operators, each in a plain form (elementary torch operations in 32 bits, rounded once) and
as a user of the library calls it:

* ``linear``: y = act(x . W^T + bias) * mul + residual, W stored as codebook indices
  (``VQLinear.forward_fused``);
* ``experts``: the same product grouped by expert, y[r] = act(x[rows[r]] . W_e^T + bias_e) for the
  rows r of expert e, with an optional gated pair of weight halves (``VQExperts.forward``);
* ``route`` / ``combine``: the k best experts of every token with their weights and the order of
  the rows by expert, and the weighted sum of a token's rows (``VQRouter``).

W is N x K in groups of 8 consecutive inputs, G = K / 8 groups per row; group g of row n decodes to
scale * (cb1[i1] + cb2[i2]), or scale * cb1[i1] where the format has one stage.  The index planes
are stored slice by slice (16 groups, 128 inputs), the rows of a slice one after another.
"""

import math

import torch

own = False

RVQ12, RVQ12_4, VQ16 = 1, 2, 3
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------------------------ the cases


def listed():
    lin = dict(op="linear", sg=64, bias=False, mul=False, res=False)
    exp = dict(op="experts", sg=64, bias=False, gather=True, shared=False, skew=0.5)
    return [
        # one token through a small model's gate: latency
        dict(lin, name="gate 1 token", N=1536, K=576, M=1, fmt=RVQ12_4, dt="fp16", act="silu", mul=True),
        # the down projection of a serving batch, added to the residual stream
        dict(lin, name="down 16 tokens", N=4096, K=14336, M=16, fmt=RVQ12_4, dt="bf16", act="none", res=True),
        # an odd output width (a classifier, a cut vocabulary) on a ragged prompt, one index stage, a scale per row
        dict(lin, name="odd width 77 tokens", N=1003, K=960, M=77, fmt=RVQ12, dt="fp16", act="gelu", bias=True, sg=0),
        # a whole prompt through a large projection
        dict(lin, name="prompt 1024 tokens", N=8192, K=8192, M=1024, fmt=RVQ12_4, dt="bf16", act="gelu_tanh", bias=True,
             res=True),
        # one token, 8 of 64 experts: gate and up of each, gated
        dict(exp, name="experts 1 token", E=64, N=2048, K=2048, tokens=1, k=8, fmt=RVQ12_4, dt="bf16", glu=True,
             act="silu"),
        # a serving batch through the down projections, rows already in order
        dict(exp, name="experts 32 tokens down", E=64, N=2048, K=1024, tokens=32, k=8, fmt=RVQ12_4, dt="bf16",
             glu=False, act="none", gather=False),
        # a short prompt over a few wide experts with 16-bit indices and one table for all of them
        dict(exp, name="experts 16-bit 100 tokens", E=16, N=1536, K=576, tokens=100, k=2, fmt=VQ16, dt="fp16",
             glu=False, act="relu", bias=True, shared=True, sg=0),
        # a long prompt: gate and up of every expert
        dict(exp, name="experts 4096 tokens", E=32, N=4096, K=2048, tokens=4096, k=4, fmt=RVQ12_4, dt="bf16", glu=True,
             act="silu"),
        # routing of one decoded token, and of a prompt
        dict(op="route", name="route 1 token", tokens=1, E=64, k=8, dt="bf16", renorm=True),
        dict(op="route", name="route 8192 tokens", tokens=8192, E=128, k=8, dt="fp32", renorm=False),
        # the experts' rows of a serving batch and of a prompt, back to their tokens
        dict(op="combine", name="combine 32 tokens", tokens=32, E=64, k=8, N=2048, dt="bf16", res=True),
        dict(op="combine", name="combine 8192 tokens", tokens=8192, E=32, k=4, N=4096, dt="bf16", res=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("linear", "linear", "experts", "experts", "route", "combine"))
    if op == "linear":
        K = 64 * _log(rng, 4, 224)
        N = _log(rng, 64, min(14336, (1 << 26) // K))
        N = N if rng.random() < 0.4 else max(8, N // 8 * 8)
        M = _log(rng, 1, min(2048, (1 << 36) // (N * K)))
        return dict(op=op, N=N, K=K, M=M, fmt=rng.choice((RVQ12, RVQ12_4, RVQ12_4, VQ16)), dt=rng.choice(("fp16", "bf16")),
                    sg=rng.choice((0, 64)), act=rng.choice(ACTS), bias=rng.random() < 0.5, mul=rng.random() < 0.4,
                    res=rng.random() < 0.5)
    if op == "experts":
        E = _log(rng, 4, 64)
        k = rng.choice([v for v in (1, 2, 4, 8) if v <= E])
        K = 64 * _log(rng, 4, 64)
        N = 16 * _log(rng, 8, min(256, (1 << 28) // (E * K * 16)))
        tokens = _log(rng, 1, min(4096, (1 << 37) // (k * N * K)))
        return dict(op=op, E=E, N=N, K=K, tokens=tokens, k=k, fmt=rng.choice((RVQ12, RVQ12_4, RVQ12_4, VQ16)),
                    dt=rng.choice(("fp16", "bf16")), sg=rng.choice((0, 64)), act=rng.choice(ACTS),
                    glu=rng.random() < 0.5, bias=rng.random() < 0.5, gather=rng.random() < 0.5,
                    shared=rng.random() < 0.5, skew=rng.choice((0.0, 0.5, 1.5)))
    E = _log(rng, 4, 256)
    k = rng.choice([v for v in (1, 2, 3, 4, 6, 8) if v <= E])
    tokens = _log(rng, 1, 8192)
    if op == "route":
        return dict(op=op, tokens=tokens, E=E, k=k, dt=rng.choice(("fp16", "bf16", "fp32")), renorm=rng.random() < 0.5)
    return dict(op=op, tokens=tokens, E=E, k=k, N=8 * _log(rng, 8, min(1024, (1 << 24) // tokens)),
                dt=rng.choice(("fp16", "bf16")), res=rng.random() < 0.5)


def _index_bytes(c):
    """Index bytes of one weight matrix, its scales, and its codebooks."""
    groups = c["N"] * c["K"] // 8
    planes = groups * {RVQ12: 1.5, RVQ12_4: 2, VQ16: 2}[c["fmt"]]
    scales = 2 * c["N"] * (c["K"] // 64 if c["sg"] else 1)
    books = 16 * {RVQ12: 4096, RVQ12_4: 4112, VQ16: 65536}[c["fmt"]]
    return planes + scales, books


def work(c):
    if c["op"] == "linear":
        planes, books = _index_bytes(c)
        io = 2 * c["M"] * (c["K"] + c["N"] * (1 + c["mul"] + c["res"])) + 2 * c["N"] * c["bias"]
        return {"bytes": planes + books + io, "flops": 2.0 * c["M"] * c["N"] * c["K"]}
    if c["op"] == "experts":
        planes, books = _index_bytes(c)
        rows = c["tokens"] * c["k"]
        used = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["tokens"])  # experts that get a row, on average
        n_out = c["N"] // 2 if c["glu"] else c["N"]
        x = 2 * c["K"] * (c["tokens"] if c["gather"] else rows)
        by = used * (planes + 2 * c["N"] * c["bias"]) + books * (1 if c["shared"] else used)
        return {"bytes": by + x + 2 * rows * n_out + 4 * (c["E"] + 1 + rows * c["gather"]), "flops": 2.0 * rows * c["N"] * c["K"]}
    rows = c["tokens"] * c["k"]
    if c["op"] == "route":
        size = 4 if c["dt"] == "fp32" else 2
        return {"bytes": c["tokens"] * c["E"] * size + 16 * rows + 4 * (c["E"] + 1), "flops": 4.0 * c["tokens"] * c["E"]}
    return {"bytes": 2 * c["N"] * (rows + c["tokens"] * (1 + c["res"])) + 8 * rows, "flops": 2.0 * rows * c["N"]}


# ------------------------------------------------------------------------------------ the inputs


def _weights(gen, c, E):
    """Index planes, codebooks and scales of E matrices (leading dimension E; codebooks 1 where shared)."""
    N, K, fmt = c["N"], c["K"], c["fmt"]
    n = N * K // 8
    books = 1 if c.get("shared") else E
    dev = "cuda"

    def ints(hi, *shape):
        return torch.randint(0, hi, shape, generator=gen, device=dev, dtype=torch.int32)

    def book(entries):
        return torch.randn((books, entries, 8), generator=gen, device=dev).half()

    w = {}
    if fmt == VQ16:
        w["idx16"] = ints(65536, E, n).to(torch.int16)  # the low 16 bits
        w["cb1"] = book(65536)
    else:
        w["lo"] = ints(256, E, n).to(torch.uint8)
        w["hi4"] = ints(256, E, n // 2).to(torch.uint8)
        w["cb1"] = book(4096)
        if fmt == RVQ12_4:
            w["s2"] = ints(256, E, n // 2).to(torch.uint8)
            w["cb2"] = book(16)
    per_row = K // 64 if c["sg"] else 1
    w["scales"] = torch.exp(torch.randn((E, N * per_row), generator=gen, device=dev) * 0.5 - 4.0).half()
    return w


def _routing(gen, tokens, E, k, skew):
    """ids [tokens, k] of a router whose experts differ in how often they are taken; a token's experts are distinct."""
    pop = skew * torch.randn((1, E), generator=gen, device="cuda")
    logits = 2.0 * torch.randn((tokens, E), generator=gen, device="cuda") + pop
    return logits.topk(k, dim=1).indices


def _sorted(ids, E):
    """The rows in the order of their experts (token order within one): offsets, row -> token, (token, j) -> row."""
    flat = ids.reshape(-1)
    order = torch.sort(flat, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=ids.device)
    offsets[1:] = torch.cumsum(torch.bincount(flat, minlength=E), 0)
    slots = torch.empty_like(flat)
    slots[order] = torch.arange(flat.numel(), device=ids.device)
    return offsets, (order // ids.shape[1]).to(torch.int32), slots.view_as(ids).to(torch.int32)


def _numpy(w):
    """The planes of one matrix on the host, as a layer's file gives them."""
    out = {k: v[0].cpu() for k, v in w.items()}
    return {k: (v.view(torch.int16).numpy().view("uint16") if v.dtype in (torch.int16, torch.float16) else v.numpy())
            for k, v in out.items()}


def prepare(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DT[c["dt"]]

    def randn(*shape):
        return torch.randn(shape, generator=gen, device="cuda").to(dt)

    s = {"c": c}
    if c["op"] == "linear":
        s["w"] = _weights(gen, c, 1)
        s["x"] = randn(c["M"], c["K"])
        s["bias"] = randn(c["N"]) if c["bias"] else None
        s["mul"] = randn(c["M"], c["N"]) if c["mul"] else None
        s["res"] = randn(c["M"], c["N"]) if c["res"] else None
        if own:
            import compressed_index_matmul_b200 as vq

            s["layer"] = vq.VQLinear(c["N"], c["K"], c["fmt"], 64 if c["sg"] else c["K"],
                                     vq.VQ_BF16 if c["dt"] == "bf16" else vq.VQ_F16, c["M"], _numpy(s["w"]))
            s["act"] = getattr(vq, "VQ_ACT_" + c["act"].upper())
    elif c["op"] == "experts":
        rows = c["tokens"] * c["k"]
        s["w"] = _weights(gen, c, c["E"])
        s["bias"] = randn(c["E"], c["N"]) if c["bias"] else None
        s["offsets"], order, _ = _sorted(_routing(gen, c["tokens"], c["E"], c["k"], c["skew"]), c["E"])
        s["rows"] = order if c["gather"] else None
        s["x"] = randn(c["tokens"] if c["gather"] else rows, c["K"])
        if own:
            import compressed_index_matmul_b200 as vq

            s["layer"] = vq.VQExperts(c["E"], c["N"], c["K"], c["fmt"], 64 if c["sg"] else c["K"],
                                      vq.VQ_BF16 if c["dt"] == "bf16" else vq.VQ_F16, rows, s["w"],
                                      act=getattr(vq, "VQ_ACT_" + c["act"].upper()), glu=c["glu"], bias=s["bias"],
                                      shared_codebooks=c["shared"])
    elif c["op"] == "route":
        s["logits"] = (2.0 * torch.randn((c["tokens"], c["E"]), generator=gen, device="cuda")).to(dt)
        if own:
            import compressed_index_matmul_b200 as vq

            s["router"] = vq.VQRouter(c["E"], c["k"], c["tokens"], renorm=c["renorm"])
    else:
        ids = _routing(gen, c["tokens"], c["E"], c["k"], 0.5)
        _, _, s["slots"] = _sorted(ids, c["E"])
        s["weights"] = torch.softmax(torch.randn((c["tokens"], c["k"]), generator=gen, device="cuda"), 1)
        s["y"] = randn(c["tokens"] * c["k"], c["N"])
        s["res"] = randn(c["tokens"], c["N"]) if c["res"] else None
    return s


# ------------------------------------------------------------------------------------ the plain form


def _rows_first(flat, N, per_slice, total):
    """[A, N * total] stored slice by slice (per_slice entries a row, the last slice what is left) -> [A, N, total]."""
    A, full = flat.shape[0], total // per_slice
    head = flat[:, : full * per_slice * N].reshape(A, full, N, per_slice).permute(0, 2, 1, 3).reshape(A, N, full * per_slice)
    return torch.cat([head, flat[:, full * per_slice * N:].reshape(A, N, total - full * per_slice)], 2)


def _nibbles(packed):
    return torch.stack([packed & 15, packed >> 4], 2).reshape(packed.shape[0], -1)


def _decode(c, w):
    """The weights [A, N, K] in 32 bits of the A matrices in w."""
    N, K = c["N"], c["K"]
    G, A = K // 8, w["scales"].shape[0]

    def look_up(book, flat):
        at = _rows_first(flat, N, 16, G).long()
        which = torch.arange(A if book.shape[0] > 1 else 1, device=at.device).view(-1, 1, 1)
        return book.float()[which, at]  # [A, N, G, 8]

    if c["fmt"] == VQ16:
        v = look_up(w["cb1"], w["idx16"].int() & 65535)
    else:
        v = look_up(w["cb1"], w["lo"].int() | (_nibbles(w["hi4"]).int() << 8))
        if c["fmt"] == RVQ12_4:
            v = v + look_up(w["cb2"], _nibbles(w["s2"]))
    if c["sg"]:
        scales = _rows_first(w["scales"], N, 2, K // 64).float()
        return (v.view(A, N, K // 64, 64) * scales.unsqueeze(3)).view(A, N, K)
    return v.view(A, N, K) * w["scales"].float().unsqueeze(2)


def _act(name, v):
    if name == "relu":
        return torch.clamp(v, min=0.0)
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _linear(s):
    c = s["c"]
    v = s["x"].float() @ _decode(c, s["w"])[0].t()
    if s["bias"] is not None:
        v = v + s["bias"].float()
    v = _act(c["act"], v)
    if s["mul"] is not None:
        v = v * s["mul"].float()
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(s["x"].dtype)


def _experts(s):
    c = s["c"]
    x = (s["x"] if s["rows"] is None else s["x"][s["rows"].long()]).float()
    counts = (s["offsets"][1:] - s["offsets"][:-1]).long()
    used = counts.nonzero().view(-1)
    w = {k: v if v.shape[0] == 1 else v[used] for k, v in s["w"].items()}
    # the rows of each expert side by side, padded with zero rows to the longest
    n = counts[used]
    place = torch.arange(used.numel(), device=x.device).repeat_interleave(n)
    rank = torch.arange(x.shape[0], device=x.device) - s["offsets"][:-1].long()[used].repeat_interleave(n)
    padded = torch.zeros((used.numel(), int(n.max()), c["K"]), device=x.device)
    padded[place, rank] = x
    v = torch.bmm(padded, _decode(c, w).transpose(1, 2))[place, rank]
    if s["bias"] is not None:
        v = v + s["bias"].float()[used][place]
    if c["glu"]:
        return (_act(c["act"], v[:, : c["N"] // 2]) * v[:, c["N"] // 2:]).to(s["x"].dtype)
    return _act(c["act"], v).to(s["x"].dtype)


def _route(s):
    c = s["c"]
    v = s["logits"].float()
    # ties go to the lowest expert: a stable sort from the largest down
    order = torch.sort(v, dim=1, descending=True, stable=True).indices[:, : c["k"]]
    e = torch.exp(v - v.max(1, keepdim=True).values)
    taken = e.gather(1, order)
    weights = taken / (taken if c["renorm"] else e).sum(1, keepdim=True)
    offsets, rows, slots = _sorted(order, c["E"])
    return {"ids": order.to(torch.int32), "weights": weights, "offsets": offsets, "rows": rows, "slots": slots}


def _combine(s):
    v = (s["y"].float()[s["slots"].long()] * s["weights"].unsqueeze(2)).sum(1)
    if s["res"] is not None:
        v = v + s["res"].float()
    return v.to(s["y"].dtype)


def run(s):
    op = s["c"]["op"]
    if not own:
        return {"linear": _linear, "experts": _experts, "route": _route, "combine": _combine}[op](s)
    if op == "linear":
        return s["layer"].forward_fused(s["x"], act=s["act"], bias=s["bias"], mul=s["mul"], residual=s["res"])
    if op == "experts":
        return s["layer"].forward(s["x"], s["offsets"], rows=s["rows"])
    if op == "route":
        r = s["router"].forward(s["logits"])
        return {"ids": r.ids, "weights": r.weights, "offsets": r.offsets, "rows": r.rows, "slots": r.slots}
    import compressed_index_matmul_b200 as vq

    return vq.combine(s["y"], s["weights"], s["slots"], residual=s["res"])


# ------------------------------------------------------------------------------------ 64 bits


def _exact_weights(c, w, e):
    """Matrix e in 64 bits, every entry found from its place in the planes."""
    N, K = c["N"], c["K"]
    G = K // 8
    dev = w["scales"].device
    n = torch.arange(N, device=dev).view(N, 1)
    g = torch.arange(G, device=dev).view(1, G)
    width = torch.clamp(G - 16 * (g // 16), max=16)
    at = 16 * (g // 16) * N + n * width + g % 16
    b = e if w["cb1"].shape[0] > 1 else 0

    def half(plane):
        return (plane[e].long()[at // 2] >> (4 * (at % 2))) & 15

    if c["fmt"] == VQ16:
        v = w["cb1"][b].double()[w["idx16"][e].long()[at] % 65536]
    else:
        v = w["cb1"][b].double()[w["lo"][e].long()[at] + 256 * half(w["hi4"])]
        if c["fmt"] == RVQ12_4:
            v = v + w["cb2"][b].double()[half(w["s2"])]
    sc = w["scales"][e].double()
    if c["sg"]:
        v = v * sc[2 * (g // 16) * N + n * (width // 8) + (g % 16) // 8].unsqueeze(2)
    else:
        v = v * sc.view(N, 1, 1)
    return v.reshape(N, K)


def _exact_act(name, v):
    if name == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v))
    if name == "silu":
        return v * torch.sigmoid(v)
    if name == "gelu":
        return v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
    if name == "gelu_tanh":
        return v * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3))
    return v


def exact(c, seed):
    global own
    before, own = own, False
    s = prepare(c, seed)
    own = before
    if c["op"] == "linear":
        v = torch.einsum("mk,nk->mn", s["x"].double(), _exact_weights(c, s["w"], 0))
        v = _exact_act(c["act"], v if s["bias"] is None else v + s["bias"].double())
        v = v if s["mul"] is None else v * s["mul"].double()
        return v if s["res"] is None else v + s["res"].double()
    if c["op"] == "experts":
        at = s["offsets"].tolist()
        x = s["x"].double() if s["rows"] is None else s["x"].double()[s["rows"].long()]
        parts = []
        for e in range(c["E"]):
            if at[e] == at[e + 1]:
                continue
            v = x[at[e]:at[e + 1]] @ _exact_weights(c, s["w"], e).t()
            v = v if s["bias"] is None else v + s["bias"][e].double()
            if c["glu"]:
                gate, up = v.chunk(2, 1)
                parts.append(_exact_act(c["act"], gate) * up)
            else:
                parts.append(_exact_act(c["act"], v))
        return torch.cat(parts)
    if c["op"] == "route":
        p = torch.softmax(s["logits"].double(), 1)
        left = s["logits"].double().clone()
        ids = []
        for _ in range(c["k"]):  # the largest that is left, the lowest of equals
            best = (left == left.max(1, keepdim=True).values).to(torch.uint8).argmax(1)
            ids.append(best)
            left.scatter_(1, best.view(-1, 1), -math.inf)
        ids = torch.stack(ids, 1)
        taken = p.gather(1, ids)
        weights = taken / taken.sum(1, keepdim=True) if c["renorm"] else taken
        flat = ids.reshape(-1)
        key = flat * flat.numel() + torch.arange(flat.numel(), device=flat.device)
        order = torch.argsort(key)
        counts = (flat.view(1, -1) == torch.arange(c["E"], device=flat.device).view(-1, 1)).sum(1)
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
        return {"ids": ids.int(), "weights": weights, "offsets": offsets.int(), "rows": (order // c["k"]).int(),
                "slots": torch.argsort(order).view_as(ids).int()}
    v = torch.einsum("tk,tkn->tn", s["weights"].double(), s["y"].double()[s["slots"].long()])
    return v if s["res"] is None else v + s["res"].double()
