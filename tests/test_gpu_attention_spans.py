"""Attention over spans of keys and its gradient on the GPU, against the formulas in 64 bits and
against differences.

Tolerances, from the roundings alone. A score is an fp32 sum of head_dim products of bf16 values:
it is off by at most head_dim 2^-24 (2^-17) of scale sum |q||k|, at most A over a row; the
exponential, the cap and the running sums add a few 2^-21 of a score's size. So an unrounded p is
off by a share of at most
    delta = 2^-15 A + cap 2^-19 + 2^-17
(four times the bound, for the share p / sum p and the order of sums). p is rounded to bf16 (half
a step is 2^-8 of the value) before its product with v, and so is ds before its products:
    |o - o'|   <= (2^-8 + delta) p |v| + 2^-8 |o|
    |lse - ..| <= delta + 2^-20 |lse|
    |ds - ..|  <= (2^-8 + delta) |ds| + slope p ((delta + 2^-17) |d_o||v| + 2^-17 |d_o||o|) =: e
    |dq - ..|  <= scale e |k| + 2^-8 |dq|, dk alike, |dv - ..| <= (2^-8 + delta) p^T |d_o| + 2^-8 |dv|
with o, and so D, as the forward call wrote it. 2^-100 is added for values next to 0."""
import math

import pytest
import torch

from gpu_helpers import ensure_built
from resident_decoder_trainer_gb300 import rdt

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
HALF = torch.finfo(BF16).eps / 2
TINY = 2.0 ** -100


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


# ------------------------------------------------------------------ spans
def causal(n, first=0):
    t = torch.arange(n)
    return torch.full((n,), first), first + t + 1


def documents(lengths, window=0, prefix=0.0):
    lo, hi, at = [], [], 0
    for n in lengths:
        t = torch.arange(n)
        lo.append(at + ((t + 1 - window).clamp(min=0) if window else 0 * t))
        hi.append(at + (t + 1).clamp(min=int(prefix * n)))
        at += n
    return torch.cat(lo), torch.cat(hi)


def with_nothing(spans, n):
    z = torch.zeros(n, dtype=torch.int64)
    return torch.cat([spans[0], z]), torch.cat([spans[1], z])


def scattered(queries, keys, seed):
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(-3, keys + 3, (queries,), generator=g)
    b = torch.randint(-3, keys + 3, (queries,), generator=g)
    return a, b  # a > b: sees nothing


MASKS = {
    "causal 1": (1, lambda: causal(1)),
    "causal 130": (130, lambda: causal(130)),
    "causal 257": (257, lambda: causal(257)),
    "documents": (500, lambda: documents([1, 2, 130, 17, 255, 95])),
    "documents of ones": (70, lambda: documents([1] * 70)),
    "window": (420, lambda: documents([300, 120], window=33)),
    "prefix": (400, lambda: documents([270, 130], prefix=0.4)),
    "all": (200, lambda: documents([200], prefix=1.0)),
    "padded": (300, lambda: with_nothing(documents([100, 57]), 143)),
    "nothing": (90, lambda: with_nothing(documents([0]), 90)),
    "cache 1": (777, lambda: (torch.tensor([0]), torch.tensor([777]))),
    "cache 5": (650, lambda: causal(5, 645) and (torch.zeros(5, dtype=torch.int64),
                                                 torch.arange(646, 651))),
    "scattered": (333, lambda: scattered(210, 333, 3)),
    "scattered short": (40, lambda: scattered(300, 40, 4)),
    "one key": (1, lambda: scattered(140, 1, 5)),
}
HEADS = [(4, 2, 16), (8, 2, 64), (4, 1, 128), (3, 3, 128), (10, 2, 80), (6, 2, 96), (16, 1, 48),
         (9, 3, 32)]


def problem(mask, heads, seed=0, layout="plain", size=1.0):
    keys, spans = MASKS[mask]
    nh, nkv, d = heads
    lo, hi = spans()
    queries = len(lo)
    g = torch.Generator(device="cuda").manual_seed(seed + 17 * nh + d)

    def normal(t, h):
        x = torch.randn(t, h, d, generator=g, device="cuda")
        if layout == "head_major":
            return (size * x).to(BF16).transpose(0, 1).contiguous().transpose(0, 1)
        return (size * x).to(BF16)

    st = dict(q=normal(queries, nh), k=normal(keys, nkv), v=normal(keys, nkv),
              d_o=normal(queries, nh), lo=lo.int().cuda(), hi=hi.int().cuda(),
              d_lse=torch.randn(queries, nh, generator=g, device="cuda"), scale=1 / math.sqrt(d),
              cap=0.0)
    if layout == "fused" and queries == keys:
        both = torch.cat([st["q"], st["k"], st["v"]], 1)
        st["q"], st["k"], st["v"] = both[:, :nh], both[:, nh:nh + nkv], both[:, nh + nkv:]
    return st


def scores(q, k, lo, hi, scale, cap):
    """Capped scores [heads, queries, keys], what each query sees, and the cap's slope."""
    rep = q.shape[1] // k.shape[1]
    kk = k.repeat_interleave(rep, 1)
    s = scale * torch.einsum("thd,jhd->htj", q, kk)
    slope = torch.ones_like(s)
    if cap:
        th = torch.tanh(s / cap)
        s, slope = cap * th, 1 - th * th
    j = torch.arange(k.shape[0], device=q.device)
    sees = (j >= lo[:, None].long()) & (j < hi[:, None].long())
    return s, sees, slope


def forward_exact(st):
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    s, sees, _ = scores(q, k, st["lo"], st["hi"], st["scale"], st["cap"])
    s = s.masked_fill(~sees, -math.inf)
    lse = torch.logsumexp(s, 2)
    p = torch.exp(s - lse.masked_fill(lse == -math.inf, 0.0)[..., None]).masked_fill(~sees, 0.0)
    rep = q.shape[1] // k.shape[1]
    o = torch.einsum("htj,jhd->thd", p, v.repeat_interleave(rep, 1))
    return o, lse.T, p


def delta(st):
    """A row's share by which p may be off, [heads, queries, 1]."""
    s, sees, _ = scores(st["q"].double().abs(), st["k"].double().abs(), st["lo"], st["hi"],
                        st["scale"], 0.0)
    top = s.masked_fill(~sees, 0.0).amax(2, keepdim=True) if s.shape[2] else s.sum(2, True)
    return 2.0 ** -15 * top + st["cap"] * 2.0 ** -19 + 2.0 ** -17


def run_forward(st, with_lse=True):
    t, nh, d = st["q"].shape
    keys, nkv = st["k"].shape[:2]
    o = torch.full((t, nh, d), 7.0, device="cuda", dtype=BF16)
    lse = torch.full((t, nh), 7.0, device="cuda") if with_lse else None
    ws = torch.full((rdt.attention_workspace_bytes(t, keys, nh, nkv, d),), 255, dtype=torch.uint8,
                    device="cuda")
    rdt.attention(st["q"], st["k"], st["v"], o, ws, lse=lse, lo=st["lo"], hi=st["hi"],
                  scale=st["scale"], softcap=st["cap"])
    return o, lse


def run_backward(st, o, lse, d_lse=True):
    t, nh, d = st["q"].shape
    keys, nkv = st["k"].shape[:2]
    out = {n: torch.full((m, h, d), 7.0, device="cuda", dtype=BF16)
           for n, m, h in (("q", t, nh), ("k", keys, nkv), ("v", keys, nkv))}
    ws = torch.full((rdt.attention_workspace_bytes(t, keys, nh, nkv, d, backward=True),), 255,
                    dtype=torch.uint8, device="cuda")
    rdt.attention_backward(st["q"], st["k"], st["v"], o, lse, st["d_o"], out["q"], out["k"],
                           out["v"], ws, d_lse=st["d_lse"] if d_lse else None, lo=st["lo"],
                           hi=st["hi"], scale=st["scale"], softcap=st["cap"])
    return out


def within(got, want, bound, what):
    bad = (got.double() - want).abs() / (bound + TINY)
    assert not bad.isnan().any(), what
    assert bad.numel() == 0 or bad.max() <= 1, f"{what}: {float(bad.max())} of its bound"


def check_forward(st, o, lse):
    want, want_lse, p = forward_exact(st)
    dl = delta(st)
    rep = st["q"].shape[1] // st["k"].shape[1]
    av = st["v"].double().abs().repeat_interleave(rep, 1)
    bound = torch.einsum("htj,jhd->thd", (HALF + dl) * p, av) + HALF * want.abs()
    within(o, want, bound, "o")
    nothing = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, nothing)
    z = want_lse.masked_fill(nothing, 0.0)
    within(lse.masked_fill(nothing, 0.0), z, dl[..., 0].T + 2.0 ** -20 * z.abs(), "lse")


def backward_exact(st, o, lse, d_lse=True):
    """The formulas and their bounds, for the o and lse that the forward call wrote."""
    q, k, v, g, oo = (x.double() for x in (st["q"], st["k"], st["v"], st["d_o"], o))
    rep = q.shape[1] // k.shape[1]
    kk, vv = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    s, sees, slope = scores(q, k, st["lo"], st["hi"], st["scale"], st["cap"])
    ll = lse.double().T
    p = torch.exp(s - ll.masked_fill(ll == -math.inf, 0.0)[..., None]).masked_fill(~sees, 0.0)
    own = (g * oo).sum(2)
    if d_lse:
        own = own - st["d_lse"].double()
    dp = torch.einsum("thd,jhd->htj", g, vv)
    ds = p * (dp - own.T[..., None]) * slope
    dl = delta(st)
    sizes = torch.einsum("thd,jhd->htj", g.abs(), vv.abs())
    own_size = (g * oo).abs().sum(2) + (st["d_lse"].double().abs() if d_lse else 0)
    # the cap's slope 1 - tanh^2 is off by 2 2^-19 where tanh is by 2^-19
    e = ((HALF + dl) * ds.abs() + slope * p * ((dl + 2.0 ** -17) * sizes
                                               + 2.0 ** -17 * own_size.T[..., None]))
    if st["cap"]:
        e = e + 2.0 ** -18 * p * (dp - own.T[..., None]).abs()
    sc = st["scale"]

    def shared(x):  # sum over the heads of a group
        return x.view(x.shape[0], -1, rep, x.shape[2]).sum(2)

    out = {"q": sc * torch.einsum("htj,jhd->thd", ds, kk),
           "k": shared(sc * torch.einsum("htj,thd->jhd", ds, q)),
           "v": shared(torch.einsum("htj,thd->jhd", p, g))}
    bound = {"q": sc * torch.einsum("htj,jhd->thd", e, kk.abs()),
             "k": shared(sc * torch.einsum("htj,thd->jhd", e, q.abs())),
             "v": shared(torch.einsum("htj,thd->jhd", (HALF + dl) * p, g.abs()))}
    return out, {n: bound[n] + HALF * out[n].abs() for n in out}


def check_backward(st, o, lse, got, d_lse=True):
    want, bound = backward_exact(st, o, lse, d_lse)
    for n in want:
        within(got[n], want[n], bound[n], "d" + n)


@pytest.mark.parametrize("heads", HEADS, ids=str)
@pytest.mark.parametrize("mask", MASKS)
def test_forward_and_gradient(mask, heads):
    st = problem(mask, heads)
    o, lse = run_forward(st)
    check_forward(st, o, lse)
    check_backward(st, o, lse, run_backward(st, o, lse))


@pytest.mark.parametrize("mask", ["documents", "window", "cache 1", "scattered", "padded"])
@pytest.mark.parametrize("cap,size", [(30.0, 1.0), (50.0, 4.0), (2.0, 3.0)])
def test_capped_scores(mask, cap, size):
    for heads in ((4, 2, 16), (4, 1, 128), (6, 2, 96), (8, 8, 64)):
        st = dict(problem(mask, heads, seed=5, size=size), cap=cap)
        o, lse = run_forward(st)
        check_forward(st, o, lse)
        check_backward(st, o, lse, run_backward(st, o, lse))


@pytest.mark.parametrize("layout", ["fused", "head_major"])
@pytest.mark.parametrize("heads", [(8, 2, 64), (4, 1, 128), (10, 2, 80)], ids=str)
def test_layouts(layout, heads):
    for mask in ("documents", "causal 257"):
        a, b = problem(mask, heads), problem(mask, heads, layout=layout)
        o, lse = run_forward(a)
        o2, lse2 = run_forward(b)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
        g, g2 = run_backward(a, o, lse), run_backward(b, o, lse)
        for n in g:
            assert torch.equal(g[n], g2[n])


@pytest.mark.parametrize("heads,queries,keys", [((32, 8, 128), 1, 5000), ((32, 8, 128), 3, 9001),
                                                ((16, 8, 64), 1, 4097), ((20, 4, 128), 40, 2500),
                                                ((4, 2, 16), 2, 3000)])
def test_few_queries_many_keys(heads, queries, keys):
    nh, nkv, d = heads
    g = torch.Generator(device="cuda").manual_seed(7)

    def normal(t, h):
        return torch.randn(t, h, d, generator=g, device="cuda").to(BF16)

    st = dict(q=normal(queries, nh), k=normal(keys, nkv), v=normal(keys, nkv),
              d_o=normal(queries, nh), d_lse=None, scale=d ** -0.5, cap=0.0,
              lo=torch.zeros(queries, dtype=torch.int32, device="cuda"),
              hi=torch.arange(keys - queries + 1, keys + 1, dtype=torch.int32, device="cuda"))
    o, lse = run_forward(st)
    check_forward(st, o, lse)
    check_backward(st, o, lse, run_backward(st, o, lse, d_lse=False), d_lse=False)


def test_long_packed_batch():
    """Several tiles of everything, documents that end inside tiles, an unused end."""
    lengths, g = [], torch.Generator().manual_seed(1)
    while sum(lengths) < 1800:
        lengths.append(int(torch.randint(1, 400, (1,), generator=g)))
    lo, hi = with_nothing(documents(lengths), 77)
    MASKS["long"] = (len(lo), lambda: (lo, hi))
    for heads in ((8, 2, 128), (4, 2, 64)):
        st = problem("long", heads)
        o, lse = run_forward(st)
        check_forward(st, o, lse)
        check_backward(st, o, lse, run_backward(st, o, lse))


def test_large_scores():
    """Scores of hundreds: exponentials far below and above the running maximum's."""
    for mask in ("causal 257", "documents"):
        st = problem(mask, (4, 2, 64), size=8.0)
        o, lse = run_forward(st)
        check_forward(st, o, lse)
        check_backward(st, o, lse, run_backward(st, o, lse))


def test_gradient_against_differences():
    """Along random directions, with the exact loss of the formulas. The kernel's D comes from
    the rounded o, off by 2^-8 of |d_o||o| and by what o is, and the sums along a direction
    are bounded by the elements' bounds."""
    for cap in (0.0, 5.0):
        st = dict(problem("documents", (4, 2, 32), seed=2), cap=cap)
        o, lse = run_forward(st)
        got = run_backward(st, o, lse)
        want, bound = backward_exact(st, o, lse)
        o_exact, _, p = forward_exact(st)
        d_own = (st["d_o"].double() * (o.double() - o_exact)).sum(2).abs()  # [queries, heads]
        for n in ("q", "k", "v"):
            g = torch.Generator(device="cuda").manual_seed(3)
            u = torch.randn(st[n].shape, generator=g, device="cuda", dtype=torch.float64)

            def loss(h):
                x = dict(st)
                x[n] = st[n].double() + h * u
                y, l, _ = forward_exact(x)
                return ((y * st["d_o"].double()).sum()
                        + (l * st["d_lse"].double()).masked_fill(l == -math.inf, 0.0).sum())

            diff = (loss(1e-4) - loss(-1e-4)) / 2e-4
            rep = st["q"].shape[1] // st["k"].shape[1]
            k, q = st["k"].double().repeat_interleave(rep, 1), st["q"].double()
            more = p * d_own.T[..., None] * st["scale"]
            extra = {"q": torch.einsum("htj,jhd->thd", more, k.abs()),
                     "k": torch.einsum("htj,thd->jhd", more, q.abs())
                     .view(k.shape[0], -1, rep, k.shape[2]).sum(2),
                     "v": torch.zeros((), device="cuda", dtype=torch.float64)}[n]
            room = ((bound[n] + extra) * u.abs()).sum() + 1e-5 * (want[n] * u).abs().sum()
            assert (diff - (got[n].double() * u).sum()).abs() <= room, (n, cap)


@pytest.mark.parametrize("heads", [(4, 2, 16), (8, 2, 64), (4, 1, 128)], ids=str)
@pytest.mark.parametrize("junk", [math.nan, math.inf, -math.inf])
def test_what_is_not_seen_does_not_count(heads, junk):
    """Infinities and NaN in keys that no query sees, in keys that some do not see, and in
    queries that see nothing: what does not see them stays within its bounds."""
    st = problem("padded", heads)
    o, lse = run_forward(st)
    want_o, want_lse, p = forward_exact(st)
    rep = heads[0] // heads[1]
    av = st["v"].double().abs().repeat_interleave(rep, 1)
    room = torch.einsum("htj,jhd->thd", (HALF + delta(st)) * p, av) + HALF * want_o.abs()
    want, bound = backward_exact(st, o, lse)

    def same_o(o2, part):
        within(o2[part], want_o[part], room[part], "o")

    def same(got, n, part):
        within(got[n][part], want[n][part], bound[n][part], "d" + n)

    everything = slice(None)
    dirty = {n: st[n].clone() for n in ("q", "k", "v", "d_o")}
    for n in dirty:
        dirty[n][157:] = junk
    bad = dict(st, **dirty)
    o2, lse2 = run_forward(bad)
    same_o(o2, everything)
    assert torch.equal(lse, lse2)
    got = run_backward(bad, o, lse)
    for n in got:
        same(got, n, everything)
    # key 120 (document 100 to 157): queries 0 to 119 do not see it, the later ones do
    for n in ("k", "v"):
        part = st[n].clone()
        part[120] = junk
        bad = dict(st, **{n: part})
        o2, lse2 = run_forward(bad)
        for part in (slice(0, 120), slice(157, None)):
            same_o(o2, part)
            assert torch.equal(lse[part], lse2[part])
        assert n == "k" or not o2[120:157].isfinite().any()
        got = run_backward(bad, o, lse)
        same(got, "q", slice(0, 120))
        for m in ("k", "v"):  # the document before shares no query with key 120
            same(got, m, slice(0, 100))
    # query 110's gradient: the keys after it, and those of the other document, do not see it
    part = st["d_o"].clone()
    part[110] = junk
    got = run_backward(dict(st, d_o=part), o, lse)
    for m in ("k", "v"):
        same(got, m, slice(0, 100))
        same(got, m, slice(111, None))
        assert not got[m][100:111].isfinite().any()
    same(got, "q", slice(0, 110))
    same(got, "q", slice(111, None))


@pytest.mark.parametrize("heads", [(4, 2, 16), (4, 1, 128)], ids=str)
def test_what_is_not_finite_stays_so(heads):
    """A query that is NaN, a key that all see, a batch that is NaN throughout."""
    st = problem("documents", heads)  # 1, 2, 130, 17, 255, 95 tokens
    o, lse = run_forward(st)
    q = st["q"].clone()
    q[200] = math.nan  # in the fifth document, tokens 150 to 404
    bad = dict(st, q=q)
    o2, lse2 = run_forward(bad)
    assert o2[200].isnan().all() and lse2[200].isnan().all()
    keep = torch.arange(len(q), device="cuda") != 200
    assert o2[keep].isfinite().all() and torch.equal(lse[keep], lse2[keep])
    got = run_backward(bad, o2, lse2)
    assert got["q"][200].isnan().all() and got["q"][keep].isfinite().all()
    seen = torch.zeros(len(q), dtype=torch.bool, device="cuda")
    seen[150:201] = True  # the keys that query 200 sees
    for n in ("k", "v"):
        assert not got[n][seen].isfinite().any() and got[n][~seen].isfinite().all()
    v = st["v"].clone()
    v[150] = math.inf  # seen by the whole document
    o2, _ = run_forward(dict(st, v=v))
    assert not o2[150:405].isfinite().any()
    assert o2[:150].isfinite().all() and o2[405:].isfinite().all()
    nan = dict(st, **{n: torch.full_like(st[n], math.nan) for n in ("q", "k", "v", "d_o")})
    o2, lse2 = run_forward(nan)
    assert o2.isnan().all() and lse2.isnan().all()
    assert all(x.isnan().all() for x in run_backward(nan, o2, lse2).values())


@pytest.mark.parametrize("heads", [(128, 1, 16), (71, 1, 32), (100, 2, 64), (33, 3, 112)], ids=str)
def test_many_query_heads_of_a_key_head(heads):
    for mask in ("causal 1", "documents of ones", "cache 5", "scattered short"):
        st = problem(mask, heads)
        o, lse = run_forward(st)
        check_forward(st, o, lse)
        check_backward(st, o, lse, run_backward(st, o, lse))


def test_offsets_beyond_32_bits():
    """A cache whose elements lie up to 2^31 and more apart: results as of its copy."""
    keys, nkv, d = 33000, 2, 64
    cache = torch.empty(keys, 1 << 16, device="cuda", dtype=BF16)  # 2.2e9 elements
    g = torch.Generator(device="cuda").manual_seed(0)
    k = cache[:, :nkv * d].view(keys, nkv, d)
    v = cache[:, 4096:4096 + nkv * d].view(keys, nkv, d)
    for x in (k, v):
        x.copy_(torch.randn(keys, nkv, d, generator=g, device="cuda"))
    q = torch.randn(70, 4, d, generator=g, device="cuda").to(BF16)
    hi = torch.arange(keys - 69, keys + 1, device="cuda", dtype=torch.int32)
    st = dict(q=q, k=k, v=v, d_o=q.flip(0).contiguous(), d_lse=None, lo=hi - 32900, hi=hi,
              scale=d ** -0.5, cap=0.0)
    st["lo"].clamp_(min=0)
    copy = dict(st, k=k.contiguous(), v=v.contiguous())
    o, lse = run_forward(st)
    o2, lse2 = run_forward(copy)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_forward(copy, o, lse)
    a, b = (run_backward(x, o, lse, d_lse=False) for x in (st, copy))
    assert all(torch.equal(a[n], b[n]) for n in a)


def test_far_past_the_cap():
    """Scores past the cap's polynomial in some tiles and rows only."""
    st = dict(problem("causal 257", (4, 2, 64), seed=9), cap=3.0)
    st["q"][130:140] *= 30
    st["k"][200] *= 40
    o, lse = run_forward(st)
    check_forward(st, o, lse)
    check_backward(st, o, lse, run_backward(st, o, lse))


@pytest.mark.parametrize("cap,scale", [(12400.0, 0.125), (1e-6, 1e-6), (1.1e-5, 1.0), (11.0, 1e6),
                                       (0.0, 1e-6), (0.09, 1e-6)])
def test_caps_and_scales_at_the_ends_of_their_range(cap, scale):
    """A cap far above every score caps nothing: held to the formula without one (a score of 20
    loses 20^3 / (3 12400^2) < 2^-15). Where scores pass the cap by more than 2^15, a score's own
    error (2^-21 of its size and more) moves score / cap by a good part of the slope's width, so
    that no figure of a gradient of q or k is left to hold it to: those only have to be
    finite."""
    st = dict(problem("documents", (4, 2, 64), seed=12), cap=cap, scale=scale)
    st["q"][7] = 0
    o, lse = run_forward(st)
    got = run_backward(st, o, lse)
    if cap > 1e4:
        st["cap"] = 0.0
    check_forward(st, o, lse)
    if cap and scale / cap > 2.0 ** 15:
        assert all(x.isfinite().all() for x in got.values())
        want, bound = backward_exact(st, o, lse)
        within(got["v"], want["v"], bound["v"], "dv")
    else:
        check_backward(st, o, lse, got)


@pytest.mark.parametrize("heads", [(3, 1, 48), (10, 2, 80), (31, 1, 96), (100, 1, 32), (4, 2, 128)],
                         ids=str)
@pytest.mark.parametrize("cap", [0.0, 3.0])
def test_results_do_not_hang_on_what_else_is_there(cap, heads):
    """Not on what a call before left on the chip, nor on large values in keys that nobody sees:
    scores on both sides of where the cap's polynomial ends."""
    st = dict(problem("padded", heads, seed=6), cap=cap)
    o, lse = run_forward(st)
    check_forward(st, o, lse)
    got = run_backward(st, o, lse)
    check_backward(st, o, lse, got)
    large = dict(problem("causal 257", heads, seed=7, size=50.0), cap=cap)
    for value in (0.0, 1e4, -1e4):
        run_backward(large, *run_forward(large))
        other = dict(st, **{n: st[n].clone() for n in ("k", "v")})
        for n in ("k", "v"):
            other[n][157:] = value
        o2, lse2 = run_forward(other)
        assert torch.equal(o, o2) and torch.equal(lse, lse2), value
        run_backward(large, *run_forward(large))
        again = run_backward(other, o, lse)
        assert all(torch.equal(got[n], again[n]) for n in got), value


@pytest.mark.parametrize("heads", [(8, 2, 64), (4, 1, 128)], ids=str)
def test_spans_at_the_ends_of_their_type(heads):
    """Between queries that see something: ends of -2^31 and 2^31 - 1 either way round."""
    st = problem("causal 257", heads, seed=3)
    low, high = -(1 << 31), (1 << 31) - 1
    for part, lo, hi in ((0, 0, low), (1, high, low), (2, low, high), (3, high, high),
                         (4, low, low)):
        st["lo"][3 + part::9] = lo
        st["hi"][3 + part::9] = hi
    o, lse = run_forward(st)
    check_forward(st, o, lse)
    check_backward(st, o, lse, run_backward(st, o, lse))


def test_two_calls_at_once():
    """On two streams, each with its own workspace."""
    sts = [problem("documents", (8, 2, 128), seed=s) for s in range(2)]
    want = [run_forward(st) for st in sts]
    grads = [run_backward(st, *w) for st, w in zip(sts, want)]
    streams = [torch.cuda.Stream() for _ in sts]
    for _ in range(5):
        got = []
        for st, s in zip(sts, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                o, lse = run_forward(st)
                got.append((o, lse, run_backward(st, o, lse)))
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        for (o, lse, g), w, wg in zip(got, want, grads):
            assert torch.equal(o, w[0]) and torch.equal(lse, w[1])
            assert all(torch.equal(g[n], wg[n]) for n in g)


def test_rows_around_are_left():
    st = problem("padded", (8, 2, 64))
    t, nh, d = st["q"].shape
    nkv = st["k"].shape[1]
    o, lse = run_forward(st)
    want = run_backward(st, o, lse)
    big = {n: torch.full((t + 2, h + 2, d), 5.0, device="cuda", dtype=BF16)
           for n, h in (("o", nh), ("q", nh), ("k", nkv), ("v", nkv))}
    view = {n: x[1:-1, 1:-1] for n, x in big.items()}
    ws = torch.empty(rdt.attention_workspace_bytes(t, t, nh, nkv, d, backward=True) + 256,
                     dtype=torch.uint8, device="cuda")
    common = dict(lo=st["lo"], hi=st["hi"], scale=st["scale"])
    rdt.attention(st["q"], st["k"], st["v"], view["o"], ws, **common)
    rdt.attention_backward(st["q"], st["k"], st["v"], view["o"], lse, st["d_o"], view["q"],
                           view["k"], view["v"], ws, d_lse=st["d_lse"], **common)
    assert torch.equal(view["o"], o)
    for n in want:
        assert torch.equal(view[n], want[n])
    for x in big.values():
        edge = x.clone()
        edge[1:-1, 1:-1] = 5.0
        assert (edge == 5.0).all()


def test_without_spans_every_query_sees_every_key():
    st = problem("all", (4, 2, 64))
    o, lse = run_forward(st)
    g = run_backward(st, o, lse)
    bare = dict(st, lo=None, hi=None)
    o2, lse2 = run_forward(bare)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g2 = run_backward(bare, o, lse)
    for n in g:
        assert torch.equal(g[n], g2[n])
    assert torch.equal(run_forward(st, with_lse=False)[0], o)


def test_no_queries_and_no_keys():
    st = problem("causal 130", (4, 2, 64))
    none = torch.empty(0, 4, 64, device="cuda", dtype=BF16)
    no_keys = torch.empty(0, 2, 64, device="cuda", dtype=BF16)
    spans = torch.empty(0, dtype=torch.int32, device="cuda")
    rdt.attention(none, st["k"], st["v"], none, lo=spans, hi=spans)
    dk, dv = torch.ones_like(st["k"]), torch.ones_like(st["k"])
    ws = torch.empty(rdt.attention_workspace_bytes(0, 130, 4, 2, 64, backward=True) + 256,
                     dtype=torch.uint8, device="cuda")
    rdt.attention_backward(none, st["k"], st["v"], none, torch.empty(0, 4, device="cuda"), none,
                           none, dk, dv, ws, lo=spans, hi=spans)
    assert (dk == 0).all() and (dv == 0).all()
    o, dq = torch.ones_like(st["q"]), torch.ones_like(st["q"])
    lse = torch.ones(130, 4, device="cuda")
    ws = torch.empty(rdt.attention_workspace_bytes(130, 0, 4, 2, 64, backward=True) + 256,
                     dtype=torch.uint8, device="cuda")
    rdt.attention(st["q"], no_keys, no_keys, o, ws, lse=lse)
    assert (o == 0).all() and (lse == -math.inf).all()
    rdt.attention_backward(st["q"], no_keys, no_keys, o, lse, st["d_o"], dq, no_keys, no_keys, ws)
    assert (dq == 0).all()


@pytest.mark.parametrize("mask,heads", [("documents", (8, 2, 128)), ("cache 1", (8, 2, 128)),
                                        ("padded", (4, 2, 16)), ("scattered", (6, 2, 96))])
def test_repeats_replays_and_other_stream(mask, heads):
    st = problem(mask, heads)
    o, lse = run_forward(st)
    g = run_backward(st, o, lse)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        o2, lse2 = run_forward(st)
        g2 = run_backward(st, o2, lse2)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(g[n], g2[n]) for n in g)
    t, nh, d = st["q"].shape
    keys, nkv = st["k"].shape[:2]
    ws = torch.empty(max(rdt.attention_workspace_bytes(t, keys, nh, nkv, d, backward=b)
                         for b in (False, True)) + 256, dtype=torch.uint8, device="cuda")
    out = {n: torch.zeros_like(x) for n, x in g.items()}
    o3, lse3 = torch.zeros_like(o), torch.zeros_like(lse)
    common = dict(lo=st["lo"], hi=st["hi"], scale=st["scale"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rdt.attention(st["q"], st["k"], st["v"], o3, ws, lse=lse3, **common)
        rdt.attention_backward(st["q"], st["k"], st["v"], o3, lse3, st["d_o"], out["q"], out["k"],
                               out["v"], ws, d_lse=st["d_lse"], **common)
    for _ in range(3):
        for x in (o3, lse3, *out.values()):
            x.fill_(3.0)
        ws.fill_(255)
        graph.replay()
        assert torch.equal(o, o3) and torch.equal(lse, lse3)
        assert all(torch.equal(g[n], out[n]) for n in g)
    assert rdt.device_error() == 0


def test_layer_of_packed_documents():
    """The operators as a decoder layer uses them: projections of a packed batch, norm and
    rotation, attention, and back, against torch's differentiation of the formulas in 64 bits
    of each document alone."""
    nh, nkv, d, lengths = 8, 2, 64, [40, 1, 87, 72]
    total = sum(lengths)
    g = torch.Generator(device="cuda").manual_seed(0)

    def normal(*size):
        return torch.randn(*size, generator=g, device="cuda")

    qkv = normal(total, nh + 2 * nkv, d)
    gq, gk = 1 + 0.1 * normal(d), 1 + 0.1 * normal(d)
    lo, hi = (x.int().cuda() for x in documents(lengths))
    positions = torch.cat([torch.arange(n) for n in lengths]).int().cuda()
    q, k = (torch.empty(total, h, d, device="cuda", dtype=BF16) for h in (nh, nkv))
    v = qkv[:, nh + nkv:].to(BF16)
    norm = dict(gain_q=gq, gain_k=gk, eps=1e-6, positions=positions, theta=1e4)
    rdt.qk_norm_rope(qkv[:, :nh], qkv[:, nh:nh + nkv], q, k, **norm)
    o, lse = torch.empty_like(q), torch.empty(total, nh, device="cuda")
    ws = torch.empty(max(rdt.attention_workspace_bytes(total, total, nh, nkv, d, True),
                         rdt.attention_workspace_bytes(total, total, nh, nkv, d),
                         rdt.qk_norm_rope_backward_workspace_bytes(total, nh, nkv, d)),
                     dtype=torch.uint8, device="cuda")
    rdt.attention(q, k, v, o, ws, lse=lse, lo=lo, hi=hi)
    d_o = normal(total, nh, d).to(BF16)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    rdt.attention_backward(q, k, v, o, lse, d_o, dq, dk, dv, ws, lo=lo, hi=hi)
    dqkv = torch.empty_like(qkv)
    dgq, dgk = torch.empty_like(gq), torch.empty_like(gk)
    rdt.qk_norm_rope_backward(qkv[:, :nh], qkv[:, nh:nh + nkv], dq, dk, dqkv[:, :nh],
                              dqkv[:, nh:nh + nkv], ws, d_gain_q=dgq, d_gain_k=dgk, **norm)

    x = qkv.double().requires_grad_()
    gains = [t.double().requires_grad_() for t in (gq, gk)]
    i = torch.arange(d // 2, device="cuda", dtype=torch.float64)
    outs, at = [], 0
    for n in lengths:
        angle = (torch.arange(n, device="cuda")[:, None] * 1e4 ** (-2 * i / d))[:, None]

        def rotated(y, gain):
            y = y / torch.sqrt(y.square().mean(2, keepdim=True) + 1e-6) * gain
            a, b = y[..., :d // 2], y[..., d // 2:]
            return torch.cat([a * angle.cos() - b * angle.sin(),
                              b * angle.cos() + a * angle.sin()], 2)

        part = x[at:at + n]
        qq, kk = rotated(part[:, :nh], gains[0]), rotated(part[:, nh:nh + nkv], gains[1])
        vv = part[:, nh + nkv:].repeat_interleave(nh // nkv, 1)
        s = torch.einsum("thd,jhd->htj", qq, kk.repeat_interleave(nh // nkv, 1)) * d ** -0.5
        s = s.masked_fill(~torch.ones(n, n, device="cuda", dtype=torch.bool).tril(), -math.inf)
        outs.append(torch.einsum("htj,jhd->thd", torch.softmax(s, 2), vv))
        at += n
    want = torch.cat(outs)
    grads = torch.autograd.grad((want * d_o.double()).sum(), [x, *gains])
    # q, k, v, p, o, ds, dq, dk: about eight roundings to bf16 (2^-9 in the mean square each),
    # so 1e-2 of the norm, as for the block's own gradients
    got = torch.cat([dqkv[:, :nh + nkv], dv.float()], 1)
    for a, b in ((o, want), (got, grads[0]), (dgq, grads[1]), (dgk, grads[2])):
        assert (a.double() - b).norm() <= 1e-2 * b.norm()
