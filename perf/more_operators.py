"""Measured cases of attention over spans of keys and of the per-head norm with rotation.

Four operators of a decoder layer on packed documents: the RMSNorm of every query and key
head with the rotation at given positions (``rdt_qk_norm_rope``) and its backward pass
(``rdt_qk_norm_rope_backward``), attention in which each query sees one span of keys, with
scores that may be capped by a tanh (``rdt_attention``), and its backward pass
(``rdt_attention_backward``).

With ``own`` false ``run`` computes them from elementary torch operations in fp32 (angles in
64 bits), with ``own`` true through ``resident_decoder_trainer_gb300.rdt``.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6

# query heads, key heads, head dim of the package's workloads
HEADS = {"tiny": (4, 2, 16), "small": (16, 8, 64), "q4b": (32, 8, 128)}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token of the q4b decoder: latency counts
        _norm(name="norm_rope 1 token bf16", shape="q4b", tokens=1, dtype="bf16", out="bf16",
              axes=1, far=32768, theta=1e6),
        # the fp32 projections of a packed batch, restarted positions, to bf16 operands
        _norm(name="norm_rope 4096 tokens f32", shape="q4b", tokens=4096, dtype="f32", out="bf16",
              axes=1, far=1024, theta=1e6),
        # text with images: positions in time, height and width, far into a long context
        _norm(name="norm_rope 32768 tokens 3 axes", shape="q4b", tokens=32768, dtype="bf16",
              out="bf16", axes=3, far=1 << 20, theta=1e6),
        # a ragged batch of the small decoder
        _norm(name="norm_rope grad 509 tokens f32", op="norm_grad", shape="small", tokens=509,
              dtype="f32", out="f32", axes=1, far=1024, theta=1e4),
        # a training batch of four 4096-token rows of packed documents
        _norm(name="norm_rope grad 16384 tokens", op="norm_grad", shape="q4b", tokens=16384,
              dtype="bf16", out="bf16", axes=1, far=4096, theta=1e6),
        # the next token of one sequence, its scores against a long context
        _cont(name="attention 1 token of 32768", shape="q4b", seqs=1, new=1, cache=32768),
        # four 1024-token rows of packed documents, the end of the last row unused
        _docs(name="attention 4096 tokens packed", shape="q4b", tokens=4096, longest=1024, pad=131,
              layout=1),
        # capped scores in a sliding window, odd length
        _docs(name="attention 8191 capped window", shape="small", tokens=8191, longest=8191, pad=0,
              layout=2, window=1024, softcap=50.0),
        # one long sequence whose first quarter (the prompt) is seen whole
        _docs(name="attention 8192 prefix", shape="q4b", tokens=8192, longest=8192, pad=0,
              layout=3, prefix=0.25),
        # the tiny decoder's batch: launch-bound
        _docs(name="attention grad tiny", op="attn_grad", shape="tiny", tokens=32, longest=20,
              pad=0, layout=4),
        # the packed training batch
        _docs(name="attention grad 4096 packed", op="attn_grad", shape="q4b", tokens=4096,
              longest=1024, pad=131, layout=1),
        # one long sequence with its prompt seen whole
        _docs(name="attention grad 8192 prefix", op="attn_grad", shape="q4b", tokens=8192,
              longest=8192, pad=0, layout=3, prefix=0.25),
    ]


def _heads(kw):
    if "shape" in kw:
        kw["heads"], kw["kv_heads"], kw["dim"] = HEADS[kw.pop("shape")]
    return kw


def _norm(op="norm", **kw):
    return dict(op=op, **_heads(kw))


def _docs(op="attn", window=0, prefix=0.0, softcap=0.0, **kw):
    return dict(op=op, kind="docs", window=window, prefix=prefix, softcap=softcap, **_heads(kw))


def _cont(op="attn", window=0, softcap=0.0, layout=0, **kw):
    return dict(op=op, kind="cont", window=window, softcap=softcap, layout=layout, **_heads(kw))


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "attn", "attn", "attn_grad", "attn_grad"])
    heads = dict(zip(("heads", "kv_heads", "dim"), rng.choice(
        [HEADS["tiny"], HEADS["small"], HEADS["q4b"], HEADS["q4b"], (8, 8, 64), (16, 1, 128),
         (20, 4, 128), (6, 2, 96), (9, 3, 32), (12, 12, 80)])))
    if op in ("norm", "norm_grad"):
        most = 32768 if op == "norm" else 16384
        dtype = rng.choice(["f32", "bf16", "bf16", "f16"])
        return _norm(op=op, tokens=_log_uniform(rng, 1, most), dtype=dtype,
                     out=rng.choice([dtype, "bf16"]), axes=rng.choice([1, 1, 2, 3]),
                     far=_log_uniform(rng, 16, 1 << 20), theta=rng.choice([1e4, 1e6]), **heads)
    # a query of one key has gradients 0 for query and key, and what any arithmetic leaves there
    # is its rounding: gradients are drawn with more keys
    least = 1 if op == "attn" else 16
    window = rng.choice([0, 0, _log_uniform(rng, least, 4096)])
    softcap = rng.choice([0.0, 0.0, 30.0, 50.0])
    layout = rng.randint(10, 1 << 20)
    if op == "attn" and rng.random() < 0.4:
        cache = _log_uniform(rng, 16, 32768)
        new = rng.choice([1, 1, _log_uniform(rng, 1, min(64, cache // 2))])
        return _cont(seqs=_log_uniform(rng, 1, min(64, 131072 // cache)), new=new, cache=cache,
                     window=window, softcap=softcap, layout=layout, **heads)
    tokens = _log_uniform(rng, least, 8192)
    return _docs(op=op, tokens=tokens, longest=_log_uniform(rng, least, tokens),
                 pad=rng.choice([0, 0, rng.randint(0, tokens // 8)]), layout=layout, window=window,
                 prefix=rng.choice([0.0, 0.0, round(rng.uniform(0.1, 1.0), 2)]), softcap=softcap,
                 **heads)


def _spans(case):
    """First and last + 1 key of each query (int64, on the host), and the number of keys."""
    gen = torch.Generator().manual_seed(case["layout"])
    lo, hi, start = [], [], 0
    if case["kind"] == "cont":
        for _ in range(case["seqs"]):
            most = case["cache"]
            length = most if case["seqs"] == 1 else int(
                torch.randint(max(case["new"], most // 2), most + 1, (1,), generator=gen))
            t = torch.arange(length - case["new"], length)
            first = (t + 1 - case["window"]).clamp(min=0) if case["window"] else t * 0
            lo.append(start + first)
            hi.append(start + t + 1)
            start += length
        return torch.cat(lo), torch.cat(hi), start
    total = case["tokens"] - case["pad"]
    while start < total:
        # document lengths spread over their logarithm
        u = float(torch.rand(1, generator=gen, dtype=torch.float64))
        length = total if case["longest"] >= total else max(1, int(case["longest"] ** u))
        length = min(length, total - start)
        t = torch.arange(length)
        first = (t + 1 - case["window"]).clamp(min=0) if case["window"] else t * 0
        lo.append(start + first)
        hi.append(start + (t + 1).clamp(min=int(case["prefix"] * length)))
        start += length
    nothing = torch.zeros(case["pad"], dtype=torch.int64)
    return torch.cat(lo + [nothing]), torch.cat(hi + [nothing]), case["tokens"]


def work(case):
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] in ("norm", "norm_grad"):
        n = case["tokens"] * (h + g) * d
        more = 2 * d * 4 + 4 * case["axes"] * case["tokens"]
        if case["op"] == "norm":
            return {"bytes": n * (BYTES[case["dtype"]] + BYTES[case["out"]]) + more, "flops": 8 * n}
        return {"bytes": n * (2 + BYTES[case["dtype"]] + BYTES[case["out"]]) + 2 * more,
                "flops": 16 * n}
    lo, hi, keys = _spans(case)
    queries, pairs = len(lo), int((hi - lo).clamp(min=0).sum())
    if case["op"] == "attn":
        return {"bytes": 4 * d * (queries * h + keys * g) + 4 * queries * (h + 2),
                "flops": 4 * d * h * pairs}
    return {"bytes": 8 * d * (queries * h + keys * g) + 4 * queries * (h + 2),
            "flops": 10 * d * h * pairs}


# ----------------------------------------------------------------- inputs
def _sections(case):
    """Pairs of each axis: all, or the first quarter in time and the rest in the plane."""
    half = case["dim"] // 2
    if case["axes"] == 1:
        return [half]
    first = max(1, half // 4)
    if case["axes"] == 2:
        return [first, half - first]
    return [first, (half - first) // 2, half - first - (half - first) // 2]


def _prepare_norm(case, gen):
    t, h, g, d = case["tokens"], case["heads"], case["kv_heads"], case["dim"]

    def normal(*size):
        return torch.randn(*size, generator=gen, device="cuda")

    # the projections of one token lie together: queries, keys, values
    qkv = (normal(t, h + 2 * g, d) * 1.3).to(DTYPES[case["dtype"]])
    st = {"q": qkv[:, :h], "k": qkv[:, h:h + g], "theta": case["theta"],
          "sections": _sections(case), "gain_q": 1 + 0.1 * normal(d), "gain_k": 1 + 0.1 * normal(d),
          "positions": torch.randint(0, case["far"], (case["axes"], t), generator=gen,
                                     device="cuda", dtype=torch.int32)}
    out = DTYPES[case["out"]]
    if case["op"] == "norm":
        st["out"] = {"q": torch.zeros(t, h, d, dtype=out, device="cuda"),
                     "k": torch.zeros(t, g, d, dtype=out, device="cuda")}
        return st
    st["d_q"] = (0.01 * normal(t, h, d)).to(torch.bfloat16)
    st["d_k"] = (0.01 * normal(t, g, d)).to(torch.bfloat16)
    dx = torch.zeros(t, h + 2 * g, d, dtype=out, device="cuda")
    st["out"] = {"q": dx[:, :h], "k": dx[:, h:h + g],
                 "gain_q": torch.zeros(d, device="cuda"), "gain_k": torch.zeros(d, device="cuda")}
    if own:
        from resident_decoder_trainer_gb300 import rdt
        st["ws"] = torch.empty(rdt.qk_norm_rope_backward_workspace_bytes(t, h, g, d),
                               dtype=torch.uint8, device="cuda")
    return st


def _prepare_attention(case, gen):
    h, g, d = case["heads"], case["kv_heads"], case["dim"]
    lo, hi, keys = _spans(case)
    queries = len(lo)

    def normal(*size):
        return torch.randn(*size, generator=gen, device="cuda")

    st = {"lo": lo.int().cuda(), "hi": hi.int().cuda(), "softcap": case["softcap"],
          "scale": 1 / math.sqrt(d), "q": (1.5 * normal(queries, h, d)).to(torch.bfloat16),
          "k": normal(keys, g, d).to(torch.bfloat16), "v": normal(keys, g, d).to(torch.bfloat16)}
    backward = case["op"] == "attn_grad"
    if backward:
        st["d_o"] = (0.01 * normal(queries, h, d)).to(torch.bfloat16)
        kept = _plain_attention(st)  # what the forward pass kept
        st["o"], st["lse"] = kept["o"], kept["lse"]
        st["out"] = {n: torch.zeros_like(st[n]) for n in ("q", "k", "v")}
    else:
        st["out"] = {"o": torch.zeros_like(st["q"]), "lse": torch.zeros(queries, h, device="cuda")}
    if own:
        from resident_decoder_trainer_gb300 import rdt
        st["ws"] = torch.empty(rdt.attention_workspace_bytes(queries, keys, h, g, d,
                                                             backward=backward),
                               dtype=torch.uint8, device="cuda")
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    norm = case["op"] in ("norm", "norm_grad")
    st = (_prepare_norm if norm else _prepare_attention)(case, gen)
    st["op"] = case["op"]
    return st


# ------------------------------------------------------------- plain form
def _turn(st, half):
    """Cosine and sine of every token's angles, [tokens, 1, half]."""
    axis = torch.repeat_interleave(torch.arange(len(st["sections"])),
                                   torch.tensor(st["sections"])).cuda()
    rate = st["theta"] ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = (st["positions"][axis].T.double() * rate)[:, None]
    return angle.cos().float(), angle.sin().float()


def _plain_norm(st):
    out = {}
    for name in ("q", "k"):
        x = st[name].float()
        half = x.shape[2] // 2
        cos, sin = _turn(st, half)
        n = x * torch.rsqrt(x.square().mean(2, keepdim=True) + EPS) * st["gain_" + name]
        a, b = n[..., :half], n[..., half:]
        out[name] = torch.cat([a * cos - b * sin, b * cos + a * sin], 2).to(st["out"][name].dtype)
    return out


def _plain_norm_grad(st):
    out = {}
    for name in ("q", "k"):
        x, dy, gain = st[name].float(), st["d_" + name].float(), st["gain_" + name]
        half = x.shape[2] // 2
        cos, sin = _turn(st, half)
        r = torch.rsqrt(x.square().mean(2, keepdim=True) + EPS)
        unit = x * r
        a, b = dy[..., :half], dy[..., half:]
        dn = torch.cat([a * cos + b * sin, b * cos - a * sin], 2)
        out["gain_" + name] = (dn * unit).sum((0, 1))
        dn = dn * gain
        dx = r * (dn - unit * (dn * unit).mean(2, keepdim=True))
        out[name] = dx.to(st["out"][name].dtype)
    return out


def _grouped(x, groups):
    """[tokens, heads, d] as fp32 [groups, heads of a group x tokens, d]."""
    t, h, d = x.shape
    return x.float().view(t, groups, h // groups, d).permute(1, 2, 0, 3).reshape(groups, -1, d)


def _ungrouped(x, tokens):
    groups, n, d = x.shape
    x = x.view(groups, n // tokens, tokens, d).permute(2, 0, 1, 3)
    return x.reshape(tokens, -1, d)


def _plain_scores(st):
    """Scores with -inf where a query does not see a key, [groups, heads of a group, queries,
    keys], and the cap's tanh."""
    q, k = st["q"], st["k"]
    groups = k.shape[1]
    s = _grouped(q, groups) @ k.float().permute(1, 2, 0)
    s = s.view(groups, -1, q.shape[0], k.shape[0]) * st["scale"]
    cap = st["softcap"]
    tanh = torch.tanh(s / cap) if cap else None
    s = tanh * cap if cap else s
    j = torch.arange(k.shape[0], device=q.device)
    unseen = (j < st["lo"][:, None]) | (j >= st["hi"][:, None])
    return s.masked_fill(unseen, -math.inf), tanh


def _plain_attention(st):
    s, _ = _plain_scores(st)
    groups, _, queries, keys = s.shape
    top = s.amax(3, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    p = torch.exp(s - top)
    del s
    total = p.sum(3, keepdim=True)
    o = p.view(groups, -1, keys) @ st["v"].float().transpose(0, 1)
    o = o / total.masked_fill(total == 0, 1.0).view(groups, -1, 1)
    lse = (top + total.log()).view(-1, queries).T.contiguous()
    return {"o": _ungrouped(o, queries).to(st["q"].dtype), "lse": lse}


def _plain_attention_grad(st):
    queries, h, _ = st["q"].shape
    groups, keys = st["k"].shape[1], st["k"].shape[0]
    s, tanh = _plain_scores(st)
    lse = st["lse"].T.reshape(groups, -1, queries, 1)
    p = torch.exp(s - lse.masked_fill(lse == -math.inf, 0.0)).view(groups, -1, keys)
    del s
    d_o = _grouped(st["d_o"], groups)
    rows = (d_o * _grouped(st["o"], groups)).sum(2, keepdim=True)
    ds = p * (d_o @ st["v"].float().permute(1, 2, 0) - rows)
    if tanh is not None:
        ds = ds * (1 - tanh.square()).view(groups, -1, keys)
    dq = _ungrouped(ds @ st["k"].float().transpose(0, 1), queries) * st["scale"]
    dk = (ds.transpose(1, 2) @ _grouped(st["q"], groups)).transpose(0, 1) * st["scale"]
    dv = (p.transpose(1, 2) @ d_o).transpose(0, 1)
    return {n: x.to(torch.bfloat16) for n, x in (("q", dq), ("k", dk), ("v", dv))}


# -------------------------------------------------------------------- run
def run(state):
    st = state
    if not own:
        return {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "attn": _plain_attention,
                "attn_grad": _plain_attention_grad}[st["op"]](st)
    from resident_decoder_trainer_gb300 import rdt
    out = st["out"]
    if st["op"] == "norm":
        rdt.qk_norm_rope(st["q"], st["k"], out["q"], out["k"], gain_q=st["gain_q"],
                         gain_k=st["gain_k"], eps=EPS, positions=st["positions"],
                         sections=st["sections"], theta=st["theta"])
    elif st["op"] == "norm_grad":
        rdt.qk_norm_rope_backward(st["q"], st["k"], st["d_q"], st["d_k"], out["q"], out["k"],
                                  st["ws"], gain_q=st["gain_q"], gain_k=st["gain_k"],
                                  d_gain_q=out["gain_q"], d_gain_k=out["gain_k"], eps=EPS,
                                  positions=st["positions"], sections=st["sections"],
                                  theta=st["theta"])
    elif st["op"] == "attn":
        rdt.attention(st["q"], st["k"], st["v"], out["o"], st["ws"], lse=out["lse"], lo=st["lo"],
                      hi=st["hi"], scale=st["scale"], softcap=st["softcap"])
    else:
        rdt.attention_backward(st["q"], st["k"], st["v"], st["o"], st["lse"], st["d_o"], out["q"],
                               out["k"], out["v"], st["ws"], lo=st["lo"], hi=st["hi"],
                               scale=st["scale"], softcap=st["softcap"])
    return out


# ------------------------------------------------------------------ exact
def _exact_norm(x, gain, st):
    """Norm and rotation by their definition, the pairs as complex numbers."""
    half = x.shape[2] // 2
    n = x / torch.sqrt((x * x).sum(2, keepdim=True) / x.shape[2] + EPS) * gain
    angle = torch.empty(x.shape[0], half, dtype=torch.float64, device=x.device)
    at = 0
    for axis, pairs in enumerate(st["sections"]):
        for i in range(at, at + pairs):
            angle[:, i] = st["positions"][axis].double() / st["theta"] ** (2 * i / x.shape[2])
        at += pairs
    z = torch.complex(n[..., :half].contiguous(), n[..., half:].contiguous())
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None]
    return torch.cat([z.real, z.imag], 2)


def _exact_head(q, k, v, seen, st):
    """One head's output and log-sum-exp."""
    s = q @ k.T * st["scale"]
    if st["softcap"]:
        s = st["softcap"] * torch.tanh(s / st["softcap"])
    s = torch.where(seen, s, -math.inf)
    return torch.where(seen, torch.softmax(s, 1), 0.0) @ v, torch.logsumexp(s, 1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm":
        return {n: _exact_norm(st[n].double(), st["gain_" + n].double(), st) for n in ("q", "k")}
    out = {}
    if case["op"] == "norm_grad":
        for n in ("q", "k"):
            x = st[n].double().requires_grad_()
            gain = st["gain_" + n].double().requires_grad_()
            loss = (_exact_norm(x, gain, st) * st["d_" + n].double()).sum()
            out[n], out["gain_" + n] = torch.autograd.grad(loss, [x, gain])
        return out
    j = torch.arange(st["k"].shape[0], device="cuda")
    seen = (j >= st["lo"][:, None]) & (j < st["hi"][:, None])
    each = case["heads"] // case["kv_heads"]
    if case["op"] == "attn":
        out["o"] = torch.zeros_like(st["q"], dtype=torch.float64)
        out["lse"] = torch.zeros_like(st["out"]["lse"], dtype=torch.float64)
    else:
        out = {n: torch.zeros_like(st[n], dtype=torch.float64) for n in ("q", "k", "v")}
    for head in range(case["heads"]):
        g = head // each
        part = [st["q"][:, head].double(), st["k"][:, g].double(), st["v"][:, g].double()]
        if case["op"] == "attn":
            out["o"][:, head], out["lse"][:, head] = _exact_head(*part, seen, st)
            continue
        part = [x.requires_grad_() for x in part]
        o, _ = _exact_head(*part, seen, st)
        grads = torch.autograd.grad((o * st["d_o"][:, head].double()).sum(), part)
        out["q"][:, head] += grads[0]
        out["k"][:, g] += grads[1]
        out["v"][:, g] += grads[2]
    return out
