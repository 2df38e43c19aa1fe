"""Token log probabilities, entropy, log-sum-exp, alternatives and their
gradient (rdt_token_logprobs, rdt_token_logprobs_backward, rdt_head_logprobs)
against the definition in 64 bits."""
import math

import pytest
import torch

from resident_decoder_trainer_gb300 import rdt, synth

from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu

INF = math.inf
TYPES = [torch.float32, torch.bfloat16, torch.float16]
U = 2.0 ** -24  # half a step of fp32


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()
    yield
    assert rdt.device_error() == 0


def rows_in(values, pad=0, shift=0):
    """The values as rows of a wider buffer that starts `shift` elements into its storage."""
    rows, vocab = values.shape
    store = torch.full((shift + rows * (vocab + pad),), 9.0, dtype=values.dtype, device="cuda")
    view = store[shift:].view(rows, vocab + pad)[:, :vocab]
    view.copy_(values)
    return view


def random_logits(rows, vocab, dtype, seed, spread=2.0, mask=0.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    z = spread * torch.randn(rows, vocab, generator=gen, device="cuda")
    z[:, vocab // 2] += 9
    if mask:
        z[torch.rand(rows, vocab, generator=gen, device="cuda") < mask] = -INF
    t = torch.randint(0, vocab, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    t[::3] = vocab // 2
    return z.to(dtype), t


def outputs(rows, top):
    """Outputs full of values that no call leaves."""
    out = {k: torch.full((rows,), 77.0, device="cuda") for k in ("logp", "entropy", "lse")}
    out["stats"] = torch.full((rows, 2), 77.0, device="cuda")
    if top:
        out["top_ids"] = torch.full((rows, top), 777777777, dtype=torch.int32, device="cuda")
        out["top_logp"] = torch.full((rows, top), 77.0, device="cuda")
    return out


def definition(z, targets, top, scale):
    """Values in 64 bits, and how far fp32 arithmetic may be from them (see check)."""
    x = z.double()
    rows, vocab = x.shape
    m = x.amax(1)
    none = m == -INF
    d = (x - m.masked_fill(none, 0.0)[:, None]) * scale
    e = d.exp()
    s = e.sum(1)
    ls = s.log().masked_fill(none, 0.0)
    p = e / s[:, None]
    p[none] = 0
    pd = (p * d.masked_fill(p == 0, 0.0))
    want = {"entropy": ls - pd.sum(1), "lse": scale * m + ls, "stats": torch.stack([m, ls], 1)}
    want["entropy"][none] = 0
    # each d has two roundings and one of the exponent's factor; the exponential is right to
    # 2^-21; a sum's terms pass through at most vocab / 256 + 40 additions
    add = (vocab / 256 + 40) * U
    far = pd.abs().sum(1)
    e_sum = 2.0 ** -21 + 4 * U * far + add
    e_ls = e_sum + 2 * U * ls.abs()
    e_ent = (e_ls + far * (2.0 ** -21 + add + e_sum) +
             6 * U * (p * d.masked_fill(p == 0, 0.0) ** 2).sum(1) + U * want["entropy"].abs())
    tol = {"entropy": e_ent, "stats": torch.stack([0 * ls, e_ls], 1),
           "lse": e_ls + U * (scale * m).abs() + U * want["lse"].abs()}
    if targets is not None:
        at = targets.long().clamp(0, vocab - 1)[:, None]
        dt = d.gather(1, at)[:, 0]
        want["logp"] = dt - ls
        want["logp"][targets >= vocab] = math.nan
        tol["logp"] = e_ls + 3 * U * dt.abs() + U * (dt - ls).abs()
    if top:
        # larger first, equal ones by index; masked tokens are no alternatives
        k = min(top, vocab)
        order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
        dt = d.gather(1, order)
        want["top_ids"] = torch.full((rows, top), -1, dtype=torch.int32, device="cuda")
        want["top_ids"][:, :k] = torch.where(dt == -INF, -1, order).int()
        want["top_logp"] = torch.full((rows, top), -INF, dtype=torch.float64, device="cuda")
        want["top_logp"][:, :k] = dt - ls[:, None]
        tol["top_logp"] = torch.zeros_like(want["top_logp"])
        tol["top_logp"][:, :k] = e_ls[:, None] + 3 * U * dt.abs() + U * (dt - ls[:, None]).abs()
    bad = x.isnan().any(1) | (x == INF).any(1)
    skipped = targets < 0 if targets is not None else torch.zeros(rows, dtype=torch.bool,
                                                                   device="cuda")
    for k, v in want.items():
        v[bad] = -1 if k == "top_ids" else math.nan
        v[skipped] = -1 if k == "top_ids" else 0
    for v in tol.values():
        v[bad | skipped] = 0  # these are exact
    return want, tol


def check(z, targets, top=0, scale=1.0, out=None):
    rows = z.shape[0]
    if out is None:
        out = outputs(rows, top)
        if targets is None:
            del out["logp"]
        rdt.token_logprobs(z, targets=targets, logit_scale=scale, **out)
    scale = torch.tensor(scale, dtype=torch.float32).item()
    want, tol = definition(z, targets, top, scale)
    for k, got in out.items():
        if k == "top_ids":
            assert torch.equal(got, want[k]), k
            continue
        w, g = want[k], got.double()
        beyond = w.abs() > torch.finfo(torch.float32).max  # what fp32 rounds to infinity
        w = torch.where(beyond, torch.copysign(torch.full_like(w, INF), w), w)
        fine = w.isfinite()
        assert torch.equal(g.isnan(), w.isnan()), k
        assert torch.equal(g[~fine & ~w.isnan()], w[~fine & ~w.isnan()]), k
        off = (g - w)[fine].abs() - tol[k][fine]
        assert off.numel() == 0 or off.max() <= 0, (k, float(off.max()))
    return out


SHAPES = [(1, 1), (3, 2), (5, 31), (2, 33), (7, 255), (4, 1023), (3, 4099), (33, 777), (2, 32001),
          (1, 151936), (3, 151936), (160, 32000), (700, 1008), (5000, 97)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", SHAPES)
def test_values_and_alternatives(rows, vocab, dtype):
    for top, pad, shift, scale, mask in ((0, 0, 0, 1.0, 0.0), (1, 1, 1, 0.7, 0.3),
                                         (5, 3, 5, 1.0, 0.9), (20, 0, 3, 1.3, 0.0),
                                         (32, 7, 0, 1.0, 0.5)):
        z, t = random_logits(rows, vocab, dtype, seed=rows + vocab + top, mask=mask)
        z = rows_in(z, pad, shift)
        check(z, t, top, scale)
        t[1::4] = -1
        check(z, t, top, scale)
        check(z, None, top, scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [5, 1000, 32001, 151936])
def test_rows_that_masks_leave_empty_or_nearly(vocab, dtype):
    low = torch.finfo(dtype).min
    z, _ = random_logits(9, vocab, dtype, seed=vocab)
    z[0] = -INF                            # nothing left
    z[1] = -INF
    z[1, vocab - 1] = 3.0                  # one token left
    z[2] = low                             # the type's lowest value everywhere: uniform
    z[3] = low
    z[3, 1] = 0.5                          # ... or everywhere else
    z[4, ::2] = low
    z[5, ::2] = -INF
    z[6] = -INF
    z[6, 2] = low                          # only a lowest value left
    z[7] = -INF
    z[7, :2] = torch.finfo(dtype).max      # as large as they come
    z[8, 3] = torch.finfo(dtype).max
    t = torch.tensor([0, vocab - 1, 1, 1, 0, 0, 2, 1, 3], dtype=torch.int32, device="cuda")
    out = check(z, t, top=8)
    assert out["lse"][0] == -INF and out["logp"][0] == -INF and out["entropy"][0] == 0
    assert out["logp"][1] == 0 and out["top_ids"][1].tolist() == [vocab - 1] + [-1] * 7
    assert abs(float(out["entropy"][2]) - math.log(vocab)) < 1e-5


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [40, 4097, 151936])
def test_ties_go_to_the_lowest_id(vocab, dtype):
    z = torch.zeros(6, vocab, dtype=dtype, device="cuda")  # every value the same
    z[1, 1::2] = -0.0                                       # both zeros are one value
    z[2] = torch.arange(vocab, device="cuda").float().div(vocab / 100).to(dtype)  # rising
    z[3] = z[2].flip(0)                                     # falling
    z[4] = (torch.arange(vocab, device="cuda") % 7).to(dtype)
    z[5, vocab // 2:] = 1
    check(z.repeat(200, 1)[:700], None, top=32)  # more rows than SMs: whole rows to a CTA
    out = check(z, None, top=32)
    first = torch.arange(32, dtype=torch.int32, device="cuda")
    assert torch.equal(out["top_ids"][0], first) and torch.equal(out["top_ids"][1], first)
    assert torch.equal(out["top_ids"][5], first[:min(32, vocab - vocab // 2)] + vocab // 2) or \
        vocab == 40


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [3, 600, 40001])
def test_nan_and_infinite_logits(vocab, dtype):
    """A NaN or +inf anywhere in a row makes the row NaN, wherever it lies and whatever is
    beside it; the rows around it are not touched."""
    places = [0, vocab - 1, vocab // 2]
    rows = []
    for bad in (math.nan, INF):
        for at in places:
            for rest in (0.0, -INF):
                row = torch.full((vocab,), rest, device="cuda")
                row[at] = bad
                rows += [row, torch.linspace(-1, 1, vocab, device="cuda")]
    z = torch.stack(rows).to(dtype)
    t = torch.zeros(len(rows), dtype=torch.int32, device="cuda")
    out = check(z, t, top=4)
    assert out["logp"][::2].isnan().all() and not out["logp"][1::2].isnan().any()
    # every logit NaN, with both signs and payloads
    z = torch.full((2, vocab), math.nan, device="cuda").to(dtype)
    z[1] = -z[1]
    check(z, t[:2], top=3)


def test_targets_outside_the_vocabulary():
    z, t = random_logits(6, 500, torch.float32, 1)
    t[:4] = torch.tensor([-1, -2 ** 31, 500, 2 ** 31 - 1], dtype=torch.int32)
    z[0] = math.nan  # not scored: not looked at
    out = check(z, t, top=3)
    assert out["logp"][0] == 0 and out["top_ids"][0].tolist() == [-1, -1, -1]
    assert out["logp"][2:4].isnan().all() and out["entropy"][2:4].isfinite().all()


def test_large_logits_keep_their_digits():
    """fp32 logits around 1e6: lse has 1/16 of a unit left, stats keeps log p exact."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    z = torch.round(8 * torch.randn(4, 5000, generator=gen, device="cuda")) / 8 + 1e6
    out = check(z, torch.zeros(4, dtype=torch.int32, device="cuda"), top=5)
    again = check(z - 1e6, torch.zeros(4, dtype=torch.int32, device="cuda"), top=5)
    for k in ("logp", "entropy", "top_ids", "top_logp"):
        assert torch.equal(out[k], again[k]), k


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("scale", [1e-6, 1e-3, 30.0, 1e6])
@pytest.mark.parametrize("vocab", [600, 40001])
def test_temperatures(vocab, scale, dtype):
    """From nearly uniform to one token only, with masked tokens (for fp16 at low scales the
    floor is not clear of the maximum, and a masked token still has probability 0)."""
    z, t = random_logits(5, vocab, dtype, 31, mask=0.4)
    z[1] = -INF
    z[2, ::3] = torch.finfo(dtype).min
    z[3] = torch.finfo(dtype).min
    z[3, 5:9] = torch.finfo(dtype).min * 0.999
    check(z, t, top=6, scale=scale)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [5, 40, 100])
def test_rows_shared_by_a_cluster(rows, dtype):
    """Few long rows: parts of a row that hold nothing, everything, the NaN, or equal values."""
    vocab = 151936
    z, t = random_logits(rows, vocab, dtype, 32)
    part = vocab // 8
    z[0, :-part] = -INF                   # only the last part holds anything
    z[1, part:] = -INF                    # only the first
    z[2] = -INF
    z[2, torch.arange(5) * part + 17] = torch.arange(5, device="cuda").to(dtype)
    z[3, 3 * part + 5] = math.nan         # one part's NaN is the row's
    z[4] = -INF
    z[4, 7 * part + 3] = torch.finfo(dtype).min
    if rows > 5:
        z[5] = 1.5                        # ties across the parts
        z[6, -20:] = 50                   # the best all in the last part
        z[7] = -INF
        t[8] = -1
    check(z, t, top=20)
    check(z, t, top=0)


@pytest.mark.parametrize("keep", ["logp", "entropy", "lse", "stats", "top"])
def test_each_output_alone(keep):
    z, t = random_logits(19, 3001, torch.bfloat16, 4)
    full = outputs(19, 6)
    rdt.token_logprobs(z, targets=t, **full)
    one = {k: v for k, v in outputs(19, 6).items() if k.startswith(keep)}
    rdt.token_logprobs(z, targets=t, **one)
    for k, v in one.items():
        assert torch.equal(v, full[k]), k


def test_more_rows_than_a_grid_dimension():
    z, t = random_logits(70001, 40, torch.float16, 5)
    check(z, t, top=2)
    check(z[:0], t[:0], out=outputs(0, 0))
    rdt.token_logprobs(z[:0], targets=t[:0], **outputs(0, 3))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_beyond_32_bit_offsets(dtype):
    """21 rows 110 M elements apart: the last begin behind 2^31 elements."""
    ld, vocab, rows = 110_000_003, 2000, 21
    store = torch.empty(rows * ld, dtype=dtype, device="cuda")
    z = store.view(rows, ld)[:, :vocab]
    values, t = random_logits(rows, vocab, dtype, 6)
    z.copy_(values)
    out = check(z, t, top=4)
    grad = torch.empty(rows, vocab, dtype=dtype, device="cuda")
    up = torch.ones(rows, device="cuda")
    rdt.token_logprobs_backward(z, t, out["stats"], z, d_logp=up)
    rdt.token_logprobs_backward(values, t, out["stats"], grad, d_logp=up)
    assert torch.equal(z, grad)


def test_the_same_call_gives_the_same_bits():
    z, t = random_logits(300, 32001, torch.bfloat16, 7)
    a, b = outputs(300, 32), outputs(300, 32)
    rdt.token_logprobs(z, targets=t, **a)
    rdt.token_logprobs(z, targets=t, **b)
    for k in a:
        assert torch.equal(a[k], b[k]), k


def test_other_streams_and_two_calls_at_once():
    z, t = random_logits(64, 50001, torch.bfloat16, 8)
    y, r = random_logits(3, 151936, torch.float32, 9)
    a, b = outputs(64, 20), outputs(3, 20)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        rdt.token_logprobs(z, targets=t, **a, stream=s1)
        rdt.token_logprobs(y, targets=r, **b, stream=s2)
    torch.cuda.synchronize()
    check(z, t, 20, out=a)
    check(y, r, 20, out=b)


def test_captured_and_replayed():
    z, t = random_logits(40, 32000, torch.bfloat16, 10)
    z0, t0 = z.clone(), t.clone()
    out = outputs(40, 8)
    d = torch.zeros_like(z)
    up = torch.randn(40, device="cuda")
    call = lambda: (rdt.token_logprobs(z0, targets=t0, **out),  # noqa: E731
                    rdt.token_logprobs_backward(z0, t0, out["stats"], d, d_logp=up,
                                                entropy=out["entropy"], d_entropy=up))
    g, h = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    call()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    with torch.cuda.graph(h):
        call()
    for seed, graph in ((11, g), (12, h), (13, g)):
        y, r = random_logits(40, 32000, torch.bfloat16, seed)
        z0.copy_(y)
        t0.copy_(r)
        graph.replay()
        torch.cuda.synchronize()
        check(z0, t0, 8, out=out)
        eager = torch.zeros_like(d)
        rdt.token_logprobs_backward(z0, t0, out["stats"], eager, d_logp=up,
                                    entropy=out["entropy"], d_entropy=up)
        assert torch.equal(d, eager)


@pytest.mark.parametrize("rows,vocab", [(1, 151936), (64, 32000), (4000, 4096), (600, 40000)])
def test_overlapping_launches_keep_the_order_of_the_stream(rows, vocab):
    """Copies, other kernels and calls in turn, nothing waited for in between: every call sees
    what was written before it and none of what is written after it."""
    values = [random_logits(rows, vocab, torch.bfloat16, 40 + i)[0] for i in range(4)]
    t = random_logits(rows, vocab, torch.bfloat16, 40)[1]
    up = torch.ones(rows, device="cuda")
    alone = []
    for z in values:
        out, d = outputs(rows, 4), torch.empty_like(z)
        rdt.token_logprobs(z, targets=t, **out)
        rdt.token_logprobs_backward(z, t, out["stats"], d, d_logp=up)
        torch.cuda.synchronize()
        alone.append({**out, "d": d})
    z, d, out = torch.empty_like(values[0]), torch.empty_like(values[0]), outputs(rows, 4)
    got = []
    for i in range(12):
        source = values[i % 4]
        if i % 3 == 0:
            z.copy_(source)                # a copy without a kernel
        elif i % 3 == 1:
            torch.add(source, 0.0, out=z)  # a kernel
        else:
            z.zero_()
            z.copy_(source.clone())
        rdt.token_logprobs(z, targets=t, **out)
        rdt.token_logprobs_backward(z, t, out["stats"], d, d_logp=up)
        got.append({k: v.clone() for k, v in out.items()})
        got[-1]["d"] = d.clone()
        z.fill_(float("nan"))
        for v in out.values():
            v.fill_(-5)
        d.fill_(-5)
    torch.cuda.synchronize()
    for i, one in enumerate(got):
        for k, v in one.items():
            assert torch.equal(v, alone[i % 4][k]), (i, k)


def test_refusals_of_the_binding():
    z, t = random_logits(4, 64, torch.float32, 1)
    e = torch.empty(4, device="cuda")
    with pytest.raises(ValueError, match="type"):
        rdt.token_logprobs(z.double(), entropy=e)
    with pytest.raises(ValueError, match="contiguous rows"):
        rdt.token_logprobs(z.t(), entropy=torch.empty(64, device="cuda"))
    with pytest.raises(ValueError, match="shape"):
        rdt.token_logprobs(z, entropy=e[:3])
    with pytest.raises(ValueError, match="type"):
        rdt.token_logprobs(z, targets=t.long(), logp=e)
    with pytest.raises(ValueError, match="CUDA"):
        rdt.token_logprobs(z, targets=t.cpu(), logp=e)
    with pytest.raises(rdt.RdtError, match="top"):
        rdt.token_logprobs(z, top_ids=torch.empty(4, 33, dtype=torch.int32, device="cuda"),
                           top_logp=torch.empty(4, 33, device="cuda"))
    with pytest.raises(rdt.RdtError, match="top_ids"):
        rdt.token_logprobs(z, top_ids=torch.empty(4, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(rdt.RdtError, match="overlaps"):
        wide = torch.zeros(8, 64, device="cuda")
        rdt.token_logprobs_backward(wide[:4], t, torch.zeros(4, 2, device="cuda"), wide[2:6],
                                    d_logp=e)
    with pytest.raises(ValueError, match="shape of logits"):
        rdt.token_logprobs_backward(z, t, torch.zeros(4, 2, device="cuda"), z[:, :32], d_logp=e)


# ------------------------------------------------------------------ gradient
def objective(z, targets, ups, scale):
    """sum of upstream x value, in 64 bits, differentiable; rows not scored give nothing."""
    lp = torch.log_softmax(z * scale, 1)
    p = lp.exp()
    total = z.new_zeros(())
    alive = torch.ones(len(z), dtype=torch.bool, device=z.device)
    if targets is not None:
        alive = targets >= 0
        chosen = lp.gather(1, targets.long().clamp(min=0)[:, None])[:, 0]
        if ups[0] is not None:
            total = total + (ups[0].double() * chosen)[alive].sum()
    if ups[1] is not None:
        ent = -(p * torch.where(p > 0, lp, 0.0)).sum(1)
        total = total + (ups[1].double() * ent)[alive].sum()
    if ups[2] is not None:
        total = total + (ups[2].double() * torch.logsumexp(z * scale, 1))[alive].sum()
    return total


def kept(z, scale, targets=None):
    """stats and entropy as the forward leaves them."""
    rows = z.shape[0]
    out = {"stats": torch.empty(rows, 2, device="cuda"), "entropy": torch.empty(rows, device="cuda")}
    rdt.token_logprobs(z, targets=targets, logit_scale=scale, **out)
    return out["stats"], out["entropy"]


def check_grad(z, targets, ups, scale, d, out=None):
    """d holds the gradient of rows without masks, NaN or stray targets."""
    scale = torch.tensor(scale, dtype=torch.float32).item()
    x = z.double()
    lp = torch.log_softmax(x * scale, 1)
    p = lp.exp()
    zero = torch.zeros(len(z), device="cuda")
    g, h, gl = ((zero if u is None else u).double()[:, None] for u in ups)
    ent = -(p * lp).sum(1, keepdim=True)
    hit = torch.zeros_like(p)
    if targets is not None:
        hit.scatter_(1, targets.long().clamp(min=0)[:, None], 1.0)
    coef = gl - g - h * (lp + ent)
    want = scale * (hit * g + p * coef)
    size = scale * (hit * g.abs() + p * (gl.abs() + g.abs() + h.abs() * (lp.abs() + ent)))
    # p's relative error: d (3 roundings), the kept log-sum (its error in the forward's check,
    # with the largest rows here), the exponential (2^-21); then five operations
    ls = (lp.amax(1, keepdim=True)).abs()
    e_p = 2.0 ** -21 + U * (4 * (lp.abs() + ls) + 2 * ls) + 2.0 ** -20 + (z.shape[1] / 256 + 40) * U
    tol = size * (2 * e_p + 8 * U) + torch.finfo(d.dtype).eps / 2 * want.abs() * 1.01 + \
        torch.finfo(d.dtype).smallest_normal * torch.finfo(d.dtype).eps
    if targets is not None:
        want[targets < 0] = 0
    off = (d.double() - want).abs() - tol
    assert off.max() <= 0, float(off.max())


UPS = [(True, False, False), (True, True, False), (False, True, False), (True, True, True),
       (False, False, True)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("d_dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(1, 1), (3, 2), (5, 33), (4, 1023), (33, 776), (2, 32001),
                                        (1, 151936), (700, 1008)])
def test_gradient(rows, vocab, dtype, d_dtype):
    for i, (pad, shift, pad_d, shift_d) in enumerate(((0, 0, 0, 0), (1, 1, 1, 1), (3, 5, 0, 0),
                                                      (0, 0, 5, 3), (8, 8, 16, 8))):
        scale = 1.0 if i % 2 == 0 else 0.8
        z, t = random_logits(rows, vocab, dtype, seed=rows + vocab + i)
        z = rows_in(z, pad, shift)
        if i > 1:
            t[1::4] = -1
        gen = torch.Generator(device="cuda").manual_seed(i)
        ups = [torch.randn(rows, generator=gen, device="cuda") if on else None for on in UPS[i]]
        stats, ent = kept(z, scale)
        back = torch.full((shift_d + rows * (vocab + pad_d) + 64,), 55.0, dtype=d_dtype,
                          device="cuda")
        wide = back[shift_d:shift_d + rows * (vocab + pad_d)].view(rows, vocab + pad_d)
        d = wide[:, :vocab]
        rdt.token_logprobs_backward(z, t, stats, d, d_logp=ups[0], entropy=ent, d_entropy=ups[1],
                                    d_lse=ups[2], logit_scale=scale)
        check_grad(z, t, ups, scale, d)
        assert (wide[:, vocab:] == 55).all() and (back[:shift_d] == 55).all()
        assert (back[shift_d + rows * (vocab + pad_d):] == 55).all()
        if ups[0] is None:
            again = torch.empty(rows, vocab, dtype=d_dtype, device="cuda")
            rdt.token_logprobs_backward(z, None, stats, again, entropy=ent, d_entropy=ups[1],
                                        d_lse=ups[2], logit_scale=scale)
            check_grad(z, None, ups, scale, again)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(0, 0), (3, 1)])
def test_gradient_in_place(dtype, pad, shift):
    z, t = random_logits(50, 4099, dtype, 21)
    z = rows_in(z, pad, shift)
    t[::7] = -1
    up = torch.randn(50, device="cuda")
    stats, ent = kept(z, 0.9)
    d = torch.empty(50, 4099, dtype=dtype, device="cuda")
    args = dict(d_logp=up, entropy=ent, d_entropy=up, logit_scale=0.9)
    rdt.token_logprobs_backward(z, t, stats, d, **args)
    rdt.token_logprobs_backward(z, t, stats, z, **args)
    assert torch.equal(z, d)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradient_in_place_is_read_at_once(dtype):
    """Rows that share cache lines, their gradient written over them, and its squared sum, its
    own log probabilities and one more gradient taken without a wait: as with waits."""
    rows, vocab = 301, 4099
    z0, t = random_logits(rows, vocab, dtype, 61)
    up = torch.full((rows,), 0.5, device="cuda")
    ways = []
    for wait in (True, False):
        z = torch.empty_like(z0)
        lst = rdt.OptTensors(g=[z])
        ws = torch.empty(rdt.tensors_sq_sum_workspace_bytes(lst), dtype=torch.uint8, device="cuda")
        sums = torch.zeros(8, dtype=torch.float64, device="cuda")
        out, again = outputs(rows, 3), outputs(rows, 3)
        kept_out = []
        for i in range(8):
            z.copy_(z0 * (1 + i / 4))
            for call in (lambda: rdt.token_logprobs(z, targets=t, **out),
                         lambda: rdt.token_logprobs_backward(z, t, out["stats"], z, d_logp=up),
                         lambda: rdt.tensors_sq_sum(lst, sums[i:i + 1], ws),
                         lambda: rdt.token_logprobs(z, targets=t, **again),
                         lambda: rdt.token_logprobs_backward(z, t, again["stats"], z, d_logp=up)):
                call()
                if wait:
                    torch.cuda.synchronize()
            kept_out.append([z.clone()] + [x.clone() for x in again.values()])
        torch.cuda.synchronize()
        ways.append((sums.clone(), kept_out))
    assert torch.equal(ways[0][0], ways[1][0]) and (ways[0][0] > 0).all()
    for a, b in zip(ways[0][1], ways[1][1]):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype", TYPES)
def test_gradient_of_masked_empty_and_broken_rows(dtype):
    vocab = 1201
    z, t = random_logits(8, vocab, dtype, 22, mask=0.5)
    low = torch.finfo(dtype).min
    z[0] = -INF
    z[1, 5] = math.nan
    z[2, 6] = INF
    z[3] = -INF
    z[3, 7] = low
    z[4] = low
    t[:8] = torch.tensor([3, 3, 3, 7, 8, 9, vocab, -1], dtype=torch.int32)
    z[5, 9] = -INF  # its own target is masked: log p is -inf, its gradient the formula's
    z[7] = math.nan
    ups = torch.randn(3, 8, device="cuda")
    stats, ent = kept(z, 1.0, t)
    d = torch.full((8, vocab), 5.0, device="cuda")
    rdt.token_logprobs_backward(z, t, stats, d, d_logp=ups[0], entropy=ent, d_entropy=ups[1],
                                d_lse=ups[2])
    assert (d[0] == 0).all() and (d[7] == 0).all()
    assert d[1].isnan().all() and d[2].isnan().all() and d[6].isnan().all()
    good = d[3:6]
    assert good.isfinite().all()
    masked = z[3:6] == -INF
    masked[2, 9] = False
    assert (good[masked] == 0).all()
    assert abs(float(d[5, 9] - ups[0, 5])) <= 4 * U * abs(float(ups[0, 5]))
    # rows 3 and 4: p is 1 at one place, 1 / vocab everywhere; d entropy is 0 for both
    assert abs(float(d[3, 7] - ups[2, 3])) <= 1e-5 * float(ups[:, 3].abs().max())
    p = 1.0 / vocab
    want = torch.full((vocab,), float(ups[2, 4] - ups[0, 4]) * p, device="cuda")
    want[8] += float(ups[0, 4])
    assert (d[4] - want).abs().max() <= 1e-5 * float(ups[:, 4].abs().max())


def test_gradient_against_the_formula_and_differences():
    """The kernel's gradient against automatic differentiation of the definition, and that
    against central differences, both in 64 bits."""
    z, t = random_logits(6, 23, torch.float32, 23, spread=1.0)
    t[2] = -1
    scale = 0.75
    gen = torch.Generator(device="cuda").manual_seed(1)
    ups = [torch.randn(6, generator=gen, device="cuda") for _ in range(3)]
    x = z.double().requires_grad_()
    objective(x, t, ups, scale).backward()
    h = 1e-5
    for r, c in ((0, 0), (0, 11), (1, int(t[1])), (2, 3), (4, 7), (5, 22)):
        step = torch.zeros_like(x)
        step[r, c] = h
        diff = (objective(x.detach() + step, t, ups, scale) -
                objective(x.detach() - step, t, ups, scale)) / (2 * h)
        assert abs(float(diff - x.grad[r, c])) < 1e-8
    stats, ent = kept(z, scale)
    d = torch.empty_like(z)
    rdt.token_logprobs_backward(z, t, stats, d, d_logp=ups[0], entropy=ent, d_entropy=ups[1],
                                d_lse=ups[2], logit_scale=scale)
    # values of order 1, some twenty fp32 operations and the exponential
    assert (d.double() - x.grad).abs().max() < 40 * U * 8


# ---------------------------------------------------------- head and trainer
def head_reference(cfg, h, gamma, w):
    """The head's logits in 64 bits of the operands the GPU multiplies: hn rounded to bf16."""
    x = h.double()
    hn = x / (x.square().mean(1, keepdim=True) + cfg.rms_eps).sqrt() * gamma.double()
    return hn.to(torch.bfloat16).double() @ w.double().t()


@pytest.mark.parametrize("tokens", [1, 77, 300])
def test_head_logprobs(tokens):
    shape = synth.WORKLOADS["small"].replace(hidden=256, vocab=32000)
    cfg = rdt.Config.from_shape(shape)
    gen = torch.Generator(device="cuda").manual_seed(tokens)
    h = torch.randn(tokens, 256, generator=gen, device="cuda")
    gamma = 1 + 0.1 * torch.randn(256, generator=gen, device="cuda")
    w = (0.1 * torch.randn(32000, 256, generator=gen, device="cuda")).bfloat16()
    t = torch.randint(0, 32000, (tokens,), generator=gen, device="cuda", dtype=torch.int32)
    t[3::5] = -1
    ws = torch.full((rdt.head_logprobs_workspace_bytes(cfg, tokens),), 255, dtype=torch.uint8,
                    device="cuda")
    out = outputs(tokens, 10)
    del out["stats"]
    rdt.head_logprobs(cfg, h, gamma, w, ws, targets=t, logit_scale=0.9, **out)
    z = head_reference(cfg, h, gamma, w)
    want, _ = definition(z, t, 10, 0.9)
    # hn may round to the other neighbour where fp32 puts it across a border: one in ~2^13
    # elements, each 2^-8 of |hn w| ~ 0.1 to 0.4; and fp32 sums of 256 products
    for k in ("logp", "entropy", "lse", "top_logp"):
        assert (out[k].double() - want[k]).abs().max() < 5e-3, k
    # the alternatives are those of values that close to the definition's
    mine = z.gather(1, out["top_ids"].long().clamp(min=0))
    best = torch.sort(z, dim=1, descending=True).values[:, :10]
    alive = t >= 0
    assert (mine - best)[alive].abs().max() < 5e-3
    assert (out["top_ids"][~alive] == -1).all()


def test_head_logprobs_in_several_chunks():
    """A vocabulary that leaves 128 rows a chunk: three chunks, the last ragged."""
    shape = synth.WORKLOADS["tiny"].replace(vocab=2_000_000)
    cfg = rdt.Config.from_shape(shape)
    gen = torch.Generator(device="cuda").manual_seed(1)
    h = torch.randn(300, 64, generator=gen, device="cuda")
    gamma = torch.ones(64, device="cuda")
    w = (0.2 * torch.randn(2_000_000, 64, generator=gen, device="cuda")).bfloat16()
    t = torch.randint(0, 2_000_000, (300,), generator=gen, device="cuda", dtype=torch.int32)
    size = rdt.head_logprobs_workspace_bytes(cfg, 300)
    assert size < (1 << 30) + (1 << 20)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    lp, lse = torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
    rdt.head_logprobs(cfg, h, gamma, w, ws, targets=t, logp=lp, lse=lse)
    for a in (0, 127, 128, 255, 256, 299):
        z = head_reference(cfg, h[a:a + 1], gamma, w)
        want = torch.logsumexp(z, 1)
        assert abs(float(lse[a] - want)) < 5e-3
        assert abs(float(lp[a] - (z[0, int(t[a])] - want))) < 5e-3
