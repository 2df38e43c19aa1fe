"""Measured cases of the token log-probability and many-tensor optimizer operators.

Four operators of one training step: the log probabilities of given tokens with
entropy and top alternatives (``rdt_token_logprobs``), their gradient with
respect to the logits (``rdt_token_logprobs_backward``), the squared sum of
many tensors' gradients (``rdt_tensors_sq_sum``) and one AdamW update of many
tensors with 32-bit or 8-bit states (``rdt_tensors_adamw``).

With ``own`` false ``run`` computes them from elementary torch operations, with
``own`` true through ``resident_decoder_trainer_gb300.rdt``. The arithmetic of
AdamW is defined in fp32, operation by operation (include/rdt.h), because its
8-bit states are rounded from those values; the plain form follows that order.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
QBLOCK = 256  # elements that share one scale of an 8-bit state
E4M3_MAX = 448.0
E4M3_TINY = 2.0 ** -9
ABSMAX_TINY = 2.0 ** -100  # a block whose largest value is below this is stored as zeros
BETA1, BETA2, EPS = 0.9, 0.95, 1e-8

# the decoder shapes of the package's workloads: hidden, heads, kv heads, head_dim, FFN width
SHAPES = {"tiny": (64, 4, 2, 16, 176), "small": (1024, 16, 8, 64, 2816),
          "q4b": (2560, 32, 8, 128, 9728)}
VOCAB = {"tiny": 256, "small": 32000, "q4b": 151936}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one generated token: the vocabulary's logits of one position, the drawn token's log
        # probability and 20 alternatives; latency counts
        dict(name="logprobs 1 row bf16 top 20", op="logprobs", rows=1, vocab=151936, pad=0,
             dtype="bf16", scale=1.0, top=20, skip=0.0, mask=0.0),
        # prompts with unscored positions and a constrained vocabulary, at a sampling temperature
        # of 0.7, rows of odd length in a wider buffer
        dict(name="logprobs ragged f16 top 8", op="logprobs", rows=509, vocab=32001, pad=6,
             dtype="f16", scale=1.0 / 0.7, top=8, skip=0.4, mask=0.3),
        # the LM head's fp32 logits of one 1024-token sequence, with alternatives
        dict(name="logprobs 1024 rows f32 top 20", op="logprobs", rows=1024, vocab=151936, pad=0,
             dtype="f32", scale=1.0, top=20, skip=0.0, mask=0.0),
        # a training batch of four 1024-token sequences: log probabilities and entropies only
        dict(name="logprobs 4096 rows bf16", op="logprobs", rows=4096, vocab=151936, pad=0,
             dtype="bf16", scale=1.0, top=0, skip=0.0, mask=0.0),
        # the tiny workload's batch, every gradient at once: launch-bound
        dict(name="grad 32 rows f32", op="grad", rows=32, vocab=256, pad=0, dtype="f32",
             out="f32", scale=1.0, skip=0.25, mask=0.0, entropy=True, lse=True),
        # the training batch's gradient as the bf16 operand of the head's weight gradient
        dict(name="grad 4096 rows bf16", op="grad", rows=4096, vocab=151936, pad=0, dtype="bf16",
             out="bf16", scale=1.0, skip=0.0, mask=0.0, entropy=True, lse=False),
        # LM head, final norm and one block: what a memory-bound update costs
        dict(name="sq_sum head and block f32", op="sq_sum", kind="model", shape="q4b", layers=1,
             head=True, g="f32"),
        # adapters of 36 blocks with bf16 gradients: hundreds of tensors of very unlike size
        dict(name="sq_sum adapters bf16", op="sq_sum", kind="adapters", shape="q4b", layers=36,
             rank=16, g="bf16"),
        # every tensor of the tiny decoder, fp32 states: launch-bound
        dict(name="adamw32 tiny decoder", op="adamw", bits=32, kind="model", shape="tiny",
             layers=2, head=True, g="f32", shadow=True, step=3),
        # one block's eleven tensors, fp32 states and the bf16 operand copy
        dict(name="adamw32 block", op="adamw", bits=32, kind="model", shape="q4b", layers=1,
             head=False, g="f32", shadow=True, step=100),
        # the adapters, 8-bit states rounded to nearest, bf16 gradients
        dict(name="adamw8 adapters bf16", op="adamw", bits=8, kind="adapters", shape="q4b",
             layers=36, rank=16, g="bf16", shadow=False, step=10, stochastic=False),
        # LM head, final norm and one block, 8-bit states rounded up or down at random
        dict(name="adamw8 head and block", op="adamw", bits=8, kind="model", shape="q4b",
             layers=1, head=True, g="f32", shadow=True, step=1000, stochastic=True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["logprobs", "logprobs", "grad", "sq_sum", "adamw", "adamw"])
    if op in ("logprobs", "grad"):
        vocab = rng.choice([_log_uniform(rng, 100, 151936), _log_uniform(rng, 1000, 151936), 32000,
                            151936])
        top = rng.choice([0, 0, 1, 5, 8, 20, 32]) if op == "logprobs" else 0
        most = 1024 * 151936 if top else 4096 * 151936 // 2
        rows = _log_uniform(rng, 1, max(1, min(8192, most // vocab)))
        case = dict(op=op, rows=rows, vocab=vocab, pad=rng.choice([0, 0, rng.randint(1, 64)]),
                    dtype=rng.choice(["f32", "bf16", "bf16", "f16"]),
                    scale=rng.choice([1.0, 1.0, round(rng.uniform(0.5, 2.0), 3)]),
                    skip=rng.choice([0.0, 0.0, 0.3, 0.7]), mask=rng.choice([0.0, 0.0, 0.5, 0.9]))
        if op == "logprobs":
            case["top"] = top
        else:
            case.update(out=rng.choice([case["dtype"], "bf16", "f32"]),
                        entropy=rng.random() < 0.7, lse=rng.random() < 0.3)
        return case
    kind = rng.choice(["ragged", "ragged", "model", "adapters"])
    if kind == "ragged":
        case = dict(op=op, kind=kind, count=_log_uniform(rng, 1, 1500),
                    largest=_log_uniform(rng, 256, 150000), layout=rng.randint(0, 1 << 20))
    elif kind == "model":
        shape = rng.choice(["tiny", "small", "small"])
        case = dict(op=op, kind=kind, shape=shape, layers=rng.randint(1, 9),
                    head=rng.random() < 0.5)
    else:
        case = dict(op=op, kind=kind, shape=rng.choice(["small", "q4b"]),
                    layers=rng.randint(1, 36), rank=rng.choice([8, 16]))
    case["g"] = rng.choice(["f32", "bf16"])
    if op == "adamw":
        case.update(bits=rng.choice([8, 8, 32]), shadow=rng.random() < 0.5,
                    step=_log_uniform(rng, 1, 20000))
        if case["bits"] == 8:
            case["stochastic"] = rng.random() < 0.6
    return case


def _sizes(case):
    """Element counts of the case's tensors, in order."""
    if case["kind"] == "ragged":
        g = torch.Generator().manual_seed(case["layout"])
        u = torch.rand(case["count"], generator=g, dtype=torch.float64)
        return [max(1, int(math.exp(x * math.log(case["largest"])))) for x in u.tolist()]
    H, nh, nkv, d, ffn = SHAPES[case["shape"]]
    proj = [(nh * d, H), (nkv * d, H), (nkv * d, H), (H, nh * d), (ffn, H), (ffn, H), (H, ffn)]
    if case["kind"] == "adapters":
        r = case["rank"]
        return ([r * i for _, i in proj] + [o * r for o, _ in proj]) * case["layers"]
    one = [o * i for o, i in proj] + [H, H, d, d]
    return one * case["layers"] + ([H, VOCAB[case["shape"]] * H] if case["head"] else [])


def _scored(case):
    return case["rows"] - int(case["rows"] * case["skip"])


def work(case):
    if case["op"] == "logprobs":
        n = _scored(case) * case["vocab"]
        return {"bytes": n * BYTES[case["dtype"]] + case["rows"] * (4 + 20 + 8 * case["top"]),
                "flops": 6 * n}
    if case["op"] == "grad":
        n = _scored(case) * case["vocab"]
        return {"bytes": n * BYTES[case["dtype"]] + case["rows"] * (28 + case["vocab"] *
                                                                   BYTES[case["out"]]),
                "flops": 8 * n}
    n = sum(_sizes(case))
    if case["op"] == "sq_sum":
        return {"bytes": n * BYTES[case["g"]] + 8, "flops": 2 * n}
    state = 16 if case["bits"] == 32 else 4 + 16 / QBLOCK
    return {"bytes": n * (8 + BYTES[case["g"]] + state + (2 if case["shadow"] else 0)),
            "flops": 16 * n}


# ----------------------------------------------------------------- inputs
def _logits(case, gen):
    """Rows as a language model gives them: a broad bulk, a few likely tokens in each row."""
    rows, vocab = case["rows"], case["vocab"]
    z = torch.randn(rows, vocab, generator=gen, device="cuda").mul_(2.0)
    hot = torch.randint(0, vocab, (rows, 8), generator=gen, device="cuda")
    z.scatter_add_(1, hot, 4 + 10 * torch.rand(rows, 8, generator=gen, device="cuda"))
    targets = torch.where(torch.rand(rows, generator=gen, device="cuda") < 0.7, hot[:, 0],
                          torch.randint(0, vocab, (rows,), generator=gen, device="cuda"))
    if case["mask"]:
        gone = torch.rand(rows, vocab, generator=gen, device="cuda") < case["mask"]
        z.masked_fill_(gone, -math.inf)
        if rows > 8:
            z[3] = -math.inf  # nothing of this row is allowed
    order = torch.randperm(rows, generator=gen, device="cuda")
    targets[order[:rows - _scored(case)]] = -1
    store = torch.full((rows, vocab + case["pad"]), 7.0, device="cuda",
                       dtype=DTYPES[case["dtype"]])
    store[:, :vocab] = z
    return store[:, :vocab], targets.to(torch.int32)


def _prepare_rows(case, gen):
    logits, targets = _logits(case, gen)
    rows, vocab = logits.shape
    st = {"logits": logits, "targets": targets, "scale": case["scale"]}

    def f32(*size):
        return torch.zeros(*size, dtype=torch.float32, device="cuda")

    if case["op"] == "logprobs":
        k = case["top"]
        st["out"] = {"logp": f32(rows), "entropy": f32(rows), "lse": f32(rows),
                     "stats": f32(rows, 2)}
        if k:
            st["out"].update(top_ids=torch.zeros(rows, k, dtype=torch.int32, device="cuda"),
                             top_logp=f32(rows, k))
        return st
    # what the forward kept for the gradient
    z = logits.double()
    top = z.amax(1, keepdim=True)
    d = ((z - top) * case["scale"]).masked_fill_(z == -math.inf, -math.inf)
    del z
    log_sum = d.exp().sum(1, keepdim=True).log()
    lp = d - log_sum
    del d
    ent = -(lp.exp() * lp.masked_fill(lp == -math.inf, 0.0)).sum(1)
    del lp
    empty = top == -math.inf
    log_sum.masked_fill_(empty, 0.0)
    ent.masked_fill_(empty[:, 0], 0.0)
    st["stats"] = torch.cat([top, log_sum], 1).float()
    st["entropy"] = ent.float()
    st["d_logp"] = torch.randn(rows, generator=gen, device="cuda")
    st["d_entropy"] = (0.1 * torch.randn(rows, generator=gen, device="cuda")
                       if case["entropy"] else None)
    st["d_lse"] = 0.01 * torch.randn(rows, generator=gen, device="cuda") if case["lse"] else None
    st["d_logits"] = torch.zeros(rows, vocab, dtype=DTYPES[case["out"]], device="cuda")
    return st


def _prepare_tensors(case, gen):
    sizes = _sizes(case)
    n = torch.tensor(sizes, dtype=torch.int64)
    blocks = (n + QBLOCK - 1) // QBLOCK
    start = (blocks.cumsum(0) - blocks) * QBLOCK
    total = int(blocks.sum()) * QBLOCK
    owner = torch.repeat_interleave(torch.arange(len(sizes)), blocks).cuda()
    place = torch.arange(total // QBLOCK, device="cuda")[:, None] * QBLOCK + \
        torch.arange(QBLOCK, device="cuda")
    held = place < (start + n).cuda()[owner][:, None]  # the rest is padding between tensors
    del place
    # gradients of unlike magnitude from tensor to tensor
    size = torch.exp(torch.randn(len(sizes), 1, generator=gen, device="cuda") - 7.0)[owner]

    def normal(std):
        return torch.randn(total // QBLOCK, QBLOCK, generator=gen, device="cuda").mul_(std) * held

    st = {"n": n, "start": start, "owner": owner, "g": normal(size).to(DTYPES[case["g"]])}
    if case["op"] == "sq_sum":
        st["sumsq"] = torch.zeros(1, dtype=torch.float64, device="cuda")
    else:
        matrix = n > 4096  # no decay on gains and other small tensors
        st["lr"] = torch.where(matrix, 3e-4, 1e-4).float()
        st["wd"] = torch.where(matrix, 0.1, 0.0).float()
        st["w"] = normal(0.02)
        m = normal(0.3 * size)
        v = (normal(size).square_() * (0.5 + torch.rand(total // QBLOCK, 1, generator=gen,
                                                         device="cuda")))
        st["scale"] = torch.full((1,), 0.37, device="cuda")
        st["skip"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        st["step"], st["bits"] = case["step"], case["bits"]
        st["seed"] = 2024 + case["step"] if case.get("stochastic") else None
        st["wb"] = st["w"].to(torch.bfloat16) if case["shadow"] else None
        if case["bits"] == 32:
            st["m"], st["v"], st["ms"], st["vs"] = m, v, None, None
        else:
            st["m"], st["ms"] = _to_8_bits(m, None, False)
            st["v"], st["vs"] = _to_8_bits(v.sqrt_(), None, True)
    if own:
        from resident_decoder_trainer_gb300 import rdt
        spans = list(zip(start.tolist(), n.tolist()))

        def cut(buf):
            return None if buf is None else [buf.view(-1)[a:a + k] for a, k in spans]

        def cut_scales(buf):
            return None if buf is None else [buf.view(-1)[a // QBLOCK:-(-(a + k) // QBLOCK)]
                                             for a, k in spans]

        if case["op"] == "sq_sum":
            st["list"] = rdt.OptTensors(g=cut(st["g"]))
            st["ws"] = torch.empty(rdt.tensors_sq_sum_workspace_bytes(st["list"]),
                                   dtype=torch.uint8, device="cuda")
        else:
            st["list"] = rdt.OptTensors(
                g=cut(st["g"]), w=cut(st["w"]), m=cut(st["m"]), v=cut(st["v"]),
                m_scale=cut_scales(st["ms"]), v_scale=cut_scales(st["vs"]), w_bf16=cut(st["wb"]),
                lr=st["lr"].tolist(), weight_decay=st["wd"].tolist())
    return st


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = (_prepare_rows if case["op"] in ("logprobs", "grad") else _prepare_tensors)(case, gen)
    st["op"] = case["op"]
    return st


# ------------------------------------------------------------- plain form
def _plain_logprobs(st):
    z, k = st["logits"].float(), st["out"].get("top_ids")
    t, s = st["targets"].long(), st["scale"]
    skipped, top = t < 0, z.amax(1)
    empty = top == -math.inf
    d = (z - top.masked_fill(empty, 0.0)[:, None]) * s
    e = torch.exp(d)
    total = e.sum(1)
    log_sum = torch.log(total).masked_fill_(empty, 0.0)
    # p log p is 0 where p is 0
    entropy = log_sum - (e * d.masked_fill(e == 0, 0.0)).sum(1) / total
    logp = d.gather(1, t.clamp(min=0)[:, None])[:, 0] - log_sum
    out = {"logp": logp, "entropy": entropy.masked_fill(empty, 0.0), "lse": top * s + log_sum,
           "stats": torch.stack([top, log_sum], 1)}
    if k is not None:
        k = k.shape[1]
        bits = (z + 0.0).view(torch.int32).long()  # + 0.0: both zeros are one value
        bits = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
        # value, then lowest index: one whole number, no two of a row alike
        key = bits * 2 ** 32 + (2 ** 31 - torch.arange(z.shape[1], device=z.device))
        best = torch.topk(key, min(k, z.shape[1]), dim=1).indices
        lp = d.gather(1, best) - log_sum[:, None]
        best = best.masked_fill(lp == -math.inf, -1)
        more = k - best.shape[1]
        out["top_ids"] = torch.nn.functional.pad(best, (0, more), value=-1).int()
        out["top_logp"] = torch.nn.functional.pad(lp, (0, more), value=-math.inf)
    for name, x in out.items():
        x.masked_fill_(skipped.view(-1, *[1] * (x.dim() - 1)), -1 if name == "top_ids" else 0)
    return out


def _plain_grad(st):
    z, s, t = st["logits"].float(), st["scale"], st["targets"].long()
    top, log_sum = st["stats"][:, :1], st["stats"][:, 1:]
    void = (t < 0) | (top[:, 0] == -math.inf)
    lp = (z - top.masked_fill(void[:, None], 0.0)) * s - log_sum
    p = torch.exp(lp)
    g = st["d_logp"]
    a = -g if st["d_lse"] is None else st["d_lse"] - g
    if st["d_entropy"] is None:
        out = p * a[:, None]
    else:
        h = st["d_entropy"]
        out = p * ((a - h * st["entropy"])[:, None] - h[:, None] * lp.masked_fill(p == 0, 0.0))
    out.scatter_add_(1, t.clamp(min=0)[:, None], g[:, None])
    return (out * s).masked_fill_(void[:, None], 0.0).to(st["d_logits"].dtype)


def _f32(x):
    return torch.tensor(x, dtype=torch.float32).item()


def _mix(x):
    """A whole number below 2^32 from another: two rounds of multiplying and folding."""
    x = x ^ (x >> 16)
    x = (x * 0x3C6EF373) & 0xFFFFFFFF
    x = x ^ (x >> 14)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def _random_halves(st):
    """Two 16-bit whole numbers for every element, by seed, step, tensor and place."""
    tensor = torch.arange(len(st["n"]), device="cuda")
    key = _mix((_mix(_mix(st["step"]) + st["seed"] & 0xFFFFFFFF) + tensor) & 0xFFFFFFFF)
    first = st["start"].cuda()[st["owner"]]
    at = torch.arange(len(st["owner"]), device="cuda") * QBLOCK - first
    x = _mix((at[:, None] + torch.arange(QBLOCK, device="cuda")) ^ key[st["owner"]][:, None])
    return x & 0xFFFF, x >> 16


def _to_8_bits(x, half, floor):
    """Codes (e4m3) and one scale for each row of 256 values, rounded to nearest, or with 16
    random bits up or down in proportion; floor: no value > 0 becomes 0."""
    big = x.abs().amax(1, keepdim=True)
    there = big >= ABSMAX_TINY
    q = (x * torch.where(there, E4M3_MAX / big, 0.0)).clamp_(-E4M3_MAX, E4M3_MAX)
    if half is not None:
        # three mantissa bits stay: the other twenty get the random ones added and are cut off;
        # below 2^-6 the steps are those of [2^-6, 2^-5)
        low = torch.where(q.abs() < 2.0 ** -6, 2.0 ** -6, 0.0)
        bits = (q.abs() + low).view(torch.int32) + (half * 16 + 8).int()
        q = torch.copysign((bits & -0x100000).view(torch.float32) - low, q)
        q = q.clamp_(-E4M3_MAX, E4M3_MAX)
    if floor:
        q = torch.where((x > 0) & there & (q < E4M3_TINY), E4M3_TINY, q)
    most = torch.full_like(big, E4M3_MAX)  # a tensor: division by it rounds once
    return q.to(torch.float8_e4m3fn), torch.where(there, big / most, 0.0)


def _plain_adamw(st):
    b1, b2, eps = _f32(BETA1), _f32(BETA2), _f32(EPS)
    by1, by2 = _f32(1.0 / (1.0 - b1 ** st["step"])), _f32(1.0 / math.sqrt(1.0 - b2 ** st["step"]))
    lr, wd = st["lr"].cuda(), st["wd"].cuda()
    rate, keep = (lr * by1)[st["owner"]][:, None], (1.0 - lr * wd)[st["owner"]][:, None]
    m, v = st["m"].float(), st["v"].float()
    if st["bits"] == 8:
        m, v = m * st["ms"], v * st["vs"]
        v = v * v
    g = st["g"].float() * st["scale"]
    m = m * b1 + g * _f32(1.0 - b1)
    v = v * b2 + (g * _f32(1.0 - b2)) * g
    root = torch.sqrt(v)
    w = st["w"] * keep - (m / (root * by2 + eps)) * rate
    skip = st["skip"] != 0  # a step of a non-finite norm changes nothing
    st["w"].copy_(torch.where(skip, st["w"], w))
    if st["wb"] is not None:
        st["wb"].copy_(torch.where(skip, st["wb"], w.to(torch.bfloat16)))
    if st["bits"] == 8:
        up = (None, None) if st["seed"] is None else _random_halves(st)
        (m, ms), (v, vs) = _to_8_bits(m, up[0], False), _to_8_bits(root, up[1], True)
        st["ms"].copy_(torch.where(skip, st["ms"], ms))
        st["vs"].copy_(torch.where(skip, st["vs"], vs))
        m, v = m.view(torch.uint8), v.view(torch.uint8)
        st["m"].view(torch.uint8).copy_(torch.where(skip, st["m"].view(torch.uint8), m))
        st["v"].view(torch.uint8).copy_(torch.where(skip, st["v"].view(torch.uint8), v))
    else:
        st["m"].copy_(torch.where(skip, st["m"], m))
        st["v"].copy_(torch.where(skip, st["v"], v))
    return _updated(st)


def _updated(st):
    """The step's results. 8-bit states are e4m3 values in units of their block's scale."""
    return {k: st[k] for k in ("w", "wb", "m", "v", "ms", "vs") if st[k] is not None}


# -------------------------------------------------------------------- run
def run(state):
    st = state
    if own:
        from resident_decoder_trainer_gb300 import rdt
        if st["op"] == "logprobs":
            rdt.token_logprobs(st["logits"], targets=st["targets"], logit_scale=st["scale"],
                               **st["out"])
            return st["out"]
        if st["op"] == "grad":
            rdt.token_logprobs_backward(
                st["logits"], st["targets"], st["stats"], st["d_logits"], d_logp=st["d_logp"],
                entropy=st["entropy"], d_entropy=st["d_entropy"], d_lse=st["d_lse"],
                logit_scale=st["scale"])
            return st["d_logits"]
        if st["op"] == "sq_sum":
            rdt.tensors_sq_sum(st["list"], st["sumsq"], st["ws"])
            return st["sumsq"]
        rdt.tensors_adamw(st["list"], st["step"], BETA1, BETA2, EPS, scale=st["scale"],
                          skip=st["skip"], seed=st["seed"])
        return _updated(st)
    if st["op"] == "logprobs":
        return _plain_logprobs(st)
    if st["op"] == "grad":
        return _plain_grad(st)
    if st["op"] == "sq_sum":
        return st["g"].double().square().sum().view(1)
    return _plain_adamw(st)


# ------------------------------------------------------------------ exact
def _exact_logprobs(case, st):
    rows, vocab, k = case["rows"], case["vocab"], case["top"]
    keys = ["logp", "entropy", "lse", "stats"] + (["top_ids", "top_logp"] if k else [])
    parts = {name: [] for name in keys}
    for a in range(0, rows, 512):
        z = st["logits"][a:a + 512].double() * case["scale"]
        t = st["targets"][a:a + 512].long()
        lse = torch.logsumexp(z, 1)
        none = lse == -math.inf
        lp = z - torch.where(none, 0.0, lse)[:, None]
        got = {"logp": lp.gather(1, t.clamp(min=0)[:, None])[:, 0],
               "entropy": -torch.special.xlogy(lp.exp(), lp.exp()).sum(1), "lse": lse}
        top = st["logits"][a:a + 512].double().amax(1)
        got["stats"] = torch.stack([top, torch.where(none, 0.0, lse - top * case["scale"])], 1)
        if k:
            order = torch.sort(st["logits"][a:a + 512].float(), dim=1, descending=True,
                               stable=True).indices[:, :k]
            values = lp.gather(1, order)
            got["top_ids"] = torch.full((len(t), k), -1, device=z.device, dtype=torch.int32)
            got["top_logp"] = torch.full((len(t), k), -math.inf, device=z.device).double()
            got["top_ids"][:, :vocab] = torch.where(values == -math.inf, -1, order).int()
            got["top_logp"][:, :vocab] = values
        for name in keys:
            got[name][t < 0] = -1 if name == "top_ids" else 0
            parts[name].append(got[name])
    return {name: torch.cat(parts[name]) for name in keys}


def _exact_grad(case, st):
    out = torch.zeros(case["rows"], case["vocab"], dtype=torch.float64, device="cuda")
    for r in range(0, case["rows"], 512):
        at = slice(r, r + 512)
        z, t = st["logits"][at].double() * case["scale"], st["targets"][at].long()
        alive = (t >= 0) & (z.amax(1) > -math.inf)
        lp = torch.log_softmax(z, 1)
        p = lp.exp()
        g = st["d_logp"][at].double()[:, None]
        grad = torch.nn.functional.one_hot(t.clamp(min=0), case["vocab"]) * g - p * g
        if case["entropy"]:
            plp = torch.special.xlogy(p, p)
            h = st["d_entropy"][at].double()[:, None]
            grad += h * (p * plp.sum(1, keepdim=True) - plp)
        if case["lse"]:
            grad += st["d_lse"][at].double()[:, None] * p
        out[at] = torch.where(alive[:, None], case["scale"] * grad, 0.0)
    return out


def _exact_adamw(case, st):
    b1, b2, eps = _f32(BETA1), _f32(BETA2), _f32(EPS)
    lr, wd = (st[k].double().cuda()[st["owner"]][:, None] for k in ("lr", "wd"))
    m, r = st["m"].double(), st["v"].double()
    if case["bits"] == 8:
        m, r = m * st["ms"].double(), r * st["vs"].double()
        r = r ** 2
    g = st["g"].double() * float(st["scale"])
    m = b1 * m + (1 - b1) * g
    v = b2 * r + (1 - b2) * g ** 2
    del r, g
    hat = (m / (1 - b1 ** case["step"])) / ((v / (1 - b2 ** case["step"])).sqrt() + eps)
    w = st["w"].double() - lr * (hat + wd * st["w"].double())
    out = {"w": w}
    if case["shadow"]:
        out["wb"] = w
    if case["bits"] == 32:
        out.update(m=m, v=v)
        return out
    for name, scale, x, low in (("m", "ms", m, 0.0), ("v", "vs", v.sqrt(), E4M3_TINY)):
        unit = x.abs().amax(1, keepdim=True) / E4M3_MAX
        unit = torch.where(unit * E4M3_MAX < ABSMAX_TINY, 0.0, unit)
        out[scale] = unit
        if case["stochastic"]:
            out[name] = None  # the codes follow the fp32 values' low bits
            continue
        q = torch.where(unit > 0, x / unit, 0.0)
        # three bits below the leading one, steps of 2^-9 at the smallest; ties to even
        step = torch.exp2(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -6))) - 3)
        code = torch.round(q / step) * step
        out[name] = torch.where((q > 0) & (code < low), low, code)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logprobs":
        return _exact_logprobs(case, st)
    if case["op"] == "grad":
        return _exact_grad(case, st)
    if case["op"] == "sq_sum":
        total = torch.zeros(1, dtype=torch.float64, device="cuda")
        for part in st["g"].view(-1).split(1 << 26):
            total += torch.dot(part.double(), part.double())
        return total
    return _exact_adamw(case, st)
