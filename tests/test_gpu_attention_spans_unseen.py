"""Attention over spans and its gradient where something that is not finite lies beside what is
seen, and where warps of a CTA wait long for one another, against the formulas in 64 bits (bounds
as in test_gpu_attention_spans)."""
import math

import pytest
import torch

import test_gpu_attention_spans as spans
from gpu_helpers import ensure_built
from resident_decoder_trainer_gb300 import rdt
from test_gpu_attention_spans_items import caches, check_by_key_heads, problem

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def unsplit_queries():
    """Queries of one head whose pairs of row tiles leave no SM over for a second part of the
    keys."""
    return 128 * (torch.cuda.get_device_properties(0).multi_processor_count + 2)


def test_rows_computed_again_for_seconds():
    """A key that is NaN and that one query of a warp sees: the others' 31 rows are computed again,
    4 s over 2^19 keys, while the CTA's other warps wait for theirs."""
    t, keys = unsplit_queries(), 1 << 19
    lo = torch.zeros(t, dtype=torch.int64)
    hi = lo.clone()
    hi[0], hi[1:32] = keys, keys - 1
    st = problem(lo, hi, keys, (1, 1, 16), seed=1)
    bad = dict(st, v=st["v"].clone())
    bad["v"][-1] = math.nan
    o, lse = spans.run_forward(bad)
    assert rdt.device_error() == 0
    assert o[0].isnan().all()
    part = {n: st[n][1:32] for n in ("q", "lo", "hi")}
    spans.check_forward(dict(st, **part), o[1:32], lse[1:32])
    assert (o[32:] == 0).all() and (lse[32:] == -math.inf).all()


def test_keys_computed_again_for_seconds():
    """A query that is NaN and sees a key of its own, in a row tile with others that see 128 keys
    besides: these keys' gradients are computed again, 4 s over 2^19 queries."""
    t, keys = 1 << 19, 256
    lo = torch.zeros(t, dtype=torch.int64)
    hi = lo + 128
    lo[5], hi[5] = 200, 201
    st = problem(lo, hi, keys, (1, 1, 16), seed=2)
    st["q"][5] = math.nan
    o, lse = spans.run_forward(st)
    got = spans.run_backward(st, o, lse)
    assert rdt.device_error() == 0
    keep = torch.arange(t, device="cuda") != 5
    rest = dict(st, **{n: st[n][keep] for n in ("q", "d_o", "d_lse", "lo", "hi")})
    want, bound = spans.backward_exact(rest, o[keep], lse[keep])
    spans.within(got["q"][keep], want["q"], bound["q"], "dq")
    assert got["q"][5].isnan().all()
    for n in ("k", "v"):
        spans.within(got[n][:128], want[n][:128], bound[n][:128], "d" + n)
        assert got[n][200].isnan().all()
        got[n][200] = 0
        assert (got[n][128:] == 0).all()


def test_a_row_tile_that_sees_nothing_beside_one_that_sees_2_28_keys():
    """Its warps wait for their next item for as long as the other tile's walk takes, some
    seconds. One key has a score of 64, the others 0: p is 1 to 2^28 e^-64 < 2^-64."""
    t, keys = unsplit_queries(), 1 << 28
    q = torch.ones(t, 1, 16, device="cuda", dtype=torch.bfloat16)
    k = torch.zeros(keys, 1, 16, device="cuda", dtype=torch.bfloat16)
    k[keys - 3] = 4
    hi = torch.zeros(t, device="cuda", dtype=torch.int32)
    hi[0] = keys
    o, lse = torch.empty_like(q), torch.empty(t, 1, device="cuda")
    ws = torch.empty(rdt.attention_workspace_bytes(t, keys, 1, 1, 16), dtype=torch.uint8,
                     device="cuda")
    rdt.attention(q, k, k, o, ws, lse=lse, hi=hi, scale=1.0)
    assert rdt.device_error() == 0
    assert (o[0] == 4).all() and lse[0, 0] == 64
    assert (o[1:] == 0).all() and (lse[1:] == -math.inf).all()


def time_us(call):
    """The least of three, after a first."""
    call()
    least = math.inf
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        b.synchronize()
        least = min(least, 1e3 * a.elapsed_time(b))
    return least


def forward_call(st):
    t, nh, d = st["q"].shape
    keys, nkv = st["k"].shape[:2]
    o, lse = torch.empty_like(st["q"]), torch.empty(t, nh, device="cuda")
    ws = torch.empty(rdt.attention_workspace_bytes(t, keys, nh, nkv, d), dtype=torch.uint8,
                     device="cuda")
    return lambda: rdt.attention(st["q"], st["k"], st["v"], o, ws, lse=lse, lo=st["lo"],
                                 hi=st["hi"], scale=st["scale"], softcap=st["cap"])


def backward_call(st):
    """The gradient, of o and lse as the forward call writes them."""
    o, lse = spans.run_forward(st)
    t, nh, d = st["q"].shape
    keys, nkv = st["k"].shape[:2]
    dq, dk, dv = (torch.empty_like(st[n]) for n in ("q", "k", "v"))
    ws = torch.empty(rdt.attention_workspace_bytes(t, keys, nh, nkv, d, backward=True),
                     dtype=torch.uint8, device="cuda")
    return lambda: rdt.attention_backward(st["q"], st["k"], st["v"], o, lse, st["d_o"], dq, dk, dv,
                                          ws, lo=st["lo"], hi=st["hi"], scale=st["scale"],
                                          softcap=st["cap"])


@pytest.mark.parametrize("heads", [(32, 8, 128), (16, 16, 64)], ids=str)
def test_an_infinity_that_all_see_costs_little(heads):
    """Rows that are not finite by right are not computed again, which took 600 times as long."""
    lo, hi = spans.causal(4096)
    st = problem(lo, hi, 4096, heads)
    clean = time_us(forward_call(st))
    st["v"][5] = math.inf
    assert time_us(forward_call(st)) < 20 * clean


@pytest.mark.parametrize("heads", [(8, 2, 64), (4, 1, 128), (10, 2, 80), (4, 2, 16), (9, 3, 48)],
                         ids=str)
def test_columns_that_are_not_finite(heads):
    """Infinities and NaN in single columns of values: what sees them is not finite in those
    columns and is within its bounds in the others, whatever it does not see has in them."""
    lo, hi = spans.documents([100, 300], window=90)
    st = problem(lo, hi, 400, heads, seed=8)
    bad = dict(st, v=st["v"].clone())
    places = [(120, 3, math.inf), (150, 5, math.nan), (151, 3, -math.inf), (230, 5, math.inf),
              (95, heads[2] - 1, math.nan)]
    for key, column, value in places:
        bad["v"][key, :, column] = value
    o, lse = spans.run_forward(bad)
    want, _, p = spans.forward_exact(st)
    rep = heads[0] // heads[1]
    av = st["v"].double().abs().repeat_interleave(rep, 1)
    room = (torch.einsum("htj,jhd->thd", (spans.HALF + spans.delta(st)) * p, av)
            + spans.HALF * want.abs())
    sees = torch.zeros_like(o, dtype=torch.bool)
    for key, column, _ in places:
        rows = (st["lo"] <= key) & (key < st["hi"])
        sees[rows, :, column] = True
        # a weight that is 0 in fp32 makes NaN of an infinity, as 0 times it is
        assert not o[rows][:, :, column].isfinite().any()
    spans.within(o.masked_fill(sees, 0.0), want.masked_fill(sees, 0.0), room, "o")


def test_a_query_that_is_nan_costs_little_where_keys_are_split():
    """Nor does an infinity that it sees. Took 500 times as long."""
    st = problem(torch.tensor([0]), torch.tensor([32768]), 32768, (32, 8, 128))
    clean = time_us(forward_call(st))
    for n, at in (("q", 0), ("v", 5)):
        bad = dict(st, **{n: st[n].clone()})
        bad[n][at] = math.nan
        assert time_us(forward_call(bad)) < 20 * clean, n
        o, _ = spans.run_forward(bad)
        assert o.isnan().all()


@pytest.mark.parametrize("heads", [(8, 2, 64), (4, 1, 128), (10, 2, 80), (4, 2, 16)], ids=str)
def test_columns_that_are_not_finite_where_keys_are_split(heads):
    """Two queries, of which the first does not see the last key: NaN in a column of that, an
    infinity in a column of a key that both see."""
    st = problem(torch.tensor([0, 40]), torch.tensor([2999, 3000]), 3000, heads, seed=9)
    bad = dict(st, v=st["v"].clone())
    bad["v"][2999, :, 7] = math.nan
    bad["v"][1000, :, 2] = math.inf
    o, lse = spans.run_forward(bad)
    sees = torch.zeros_like(o, dtype=torch.bool)
    sees[1, :, 7] = True
    sees[:, :, 2] = True
    assert not o[sees].isfinite().any()
    want, _, p = spans.forward_exact(st)
    av = st["v"].double().abs().repeat_interleave(heads[0] // heads[1], 1)
    room = (torch.einsum("htj,jhd->thd", (spans.HALF + spans.delta(st)) * p, av)
            + spans.HALF * want.abs())
    spans.within(o.masked_fill(sees, 0.0), want.masked_fill(sees, 0.0), room, "o")


def minus_infinite_key(heads, tokens, key, column):
    """A causal batch whose key `key` is -infinity in one column in which every query is above 0:
    its weight is 0, and a gradient of a query that sees it is not finite in that column."""
    lo, hi = spans.causal(tokens)
    st = problem(lo, hi, tokens, heads, seed=4)
    st["q"][:, :, column] = st["q"][:, :, column].abs() + 0.5
    bad = dict(st, k=st["k"].clone())
    bad["k"][key, :, column] = -math.inf
    return st, bad


def test_the_gradient_of_a_key_with_an_infinity_costs_little():
    """Took 350 times as long."""
    st, bad = minus_infinite_key((32, 8, 128), 4096, 5, 3)
    clean = time_us(backward_call(st))
    assert time_us(backward_call(bad)) < 20 * clean


@pytest.mark.parametrize("heads", [(8, 2, 64), (4, 1, 128), (10, 2, 80)], ids=str)
def test_the_gradient_of_a_key_with_an_infinity(heads):
    """Finite, and within its bounds, in the other columns and for queries before the key."""
    st, bad = minus_infinite_key(heads, 300, 150, 3)
    o, lse = spans.run_forward(bad)
    assert o.isfinite().all() and lse.isfinite().all()
    # as if nobody saw the key: two spans for the queries after it, so by a mask of its own
    q, k, v, g = (st[n].double() for n in ("q", "k", "v", "d_o"))
    rep = heads[0] // heads[1]
    kk, vv = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    s, sees, _ = spans.scores(q, k, st["lo"], st["hi"], st["scale"], 0.0)
    sees[:, 150] = False
    p = torch.exp(s - lse.double().T[..., None]).masked_fill(~sees, 0.0)
    own = (g * o.double()).sum(2)
    dp = torch.einsum("thd,jhd->htj", g, vv)
    ds = p * (dp - own.T[..., None])
    dl = spans.delta(st)
    sizes = torch.einsum("thd,jhd->htj", g.abs(), vv.abs())
    own_size = (g * o.double()).abs().sum(2).T[..., None]
    e = (spans.HALF + dl) * ds.abs() + p * ((dl + 2.0 ** -17) * sizes + 2.0 ** -17 * own_size)
    want = st["scale"] * torch.einsum("htj,jhd->thd", ds, kk)
    room = (st["scale"] * torch.einsum("htj,jhd->thd", e, kk.abs()) + spans.HALF * want.abs())
    got = spans.run_backward(bad, o, lse, d_lse=False)["q"]
    after = torch.zeros_like(o, dtype=torch.bool)
    after[150:, :, 3] = True
    assert not got[after].isfinite().any()
    spans.within(got.masked_fill(after, 0.0), want.masked_fill(after, 0.0), room, "dq")


UNSEEN = {  # keys, spans; what no query sees is what lies between and behind
    "1 of a cache": (3000, lambda: (torch.tensor([0]), torch.tensor([2700]))),
    "1 of a short cache": (300, lambda: (torch.tensor([3]), torch.tensor([130]))),
    "5 of a cache": (900, lambda: (torch.zeros(5, dtype=torch.int64), torch.arange(641, 646))),
    "caches": (8 * 300, lambda: caches([300, 1, 17, 128, 129, 0, 255, 256], 1, 300)),
    "many caches": (70 * 64, lambda: caches([(7 * i) % 65 for i in range(70)], 1, 64)),
    "long caches": (3 * 2500, lambda: caches([2400, 77, 1300], 2, 2500)),
    "unused end": (500, lambda: spans.with_nothing(spans.documents([100, 57, 203]), 140)),
    "unused start": (500, lambda: tuple(x.roll(140) for x in spans.with_nothing(
        spans.documents([100, 57, 203]), 140))),
    "a window's past": (900, lambda: (torch.arange(400, 600), torch.arange(431, 631))),
    "descending": (1000, lambda: (torch.arange(900, 0, -3), torch.arange(902, 2, -3))),
    "none": (200, lambda: spans.with_nothing(spans.documents([0]), 60)),
}


def unseen_keys(st):
    seen = torch.zeros(st["k"].shape[0] + 1, dtype=torch.int64, device="cuda")
    lo = st["lo"].long().clamp(min=0)
    hi = st["hi"].long().clamp(max=st["k"].shape[0])
    some = lo < hi
    seen.index_add_(0, lo[some], torch.ones_like(lo[some]))
    seen.index_add_(0, hi[some], -torch.ones_like(lo[some]))
    return seen.cumsum(0)[:-1] == 0


@pytest.mark.parametrize("mask", UNSEEN)
@pytest.mark.parametrize("heads,cap", [((32, 8, 128), 0.0), ((8, 8, 64), 30.0), ((4, 1, 128), 20.0),
                                       ((9, 3, 48), 0.0), ((4, 2, 16), 0.0)], ids=str)
@pytest.mark.parametrize("junk", [math.nan, -math.inf])
def test_keys_that_nobody_sees(mask, heads, cap, junk):
    """Results are those with zeros there: within the same bounds, whether a row's item is taken
    once more with these keys cleared or a part's sum formed again key by key (without the rounding
    of p to bf16, so not to the bit)."""
    keys, of = UNSEEN[mask]
    lo, hi = of()
    st = problem(lo, hi, keys, heads, seed=11, cap=cap)
    empty = unseen_keys(st)
    assert empty.any()
    for n in ("k", "v"):
        st[n][empty] = 0
    o, lse = spans.run_forward(st)
    spans.check_forward(st, o, lse)
    bad = dict(st, **{n: st[n].clone() for n in ("k", "v")})
    for n in ("k", "v"):
        bad[n][empty] = junk
    o2, lse2 = spans.run_forward(bad)
    spans.check_forward(st, o2, lse2)
    assert torch.equal(lse, lse2)


def test_keys_that_nobody_sees_cost_little():
    """NaN past the end of a cache and between caches; took 480 and 24 times as long."""
    for lo, hi, keys in ((torch.tensor([0]), torch.tensor([32700]), 33000),
                         (*caches([1000 + 61 * i for i in range(16)], 1, 2048), 16 * 2048)):
        st = problem(lo, hi, keys, (32, 8, 128))
        clean = time_us(forward_call(st))
        for n in ("k", "v"):
            st[n][unseen_keys(st)] = math.nan
        assert time_us(forward_call(st)) < 10 * clean


@pytest.mark.parametrize("junk", [0.0, math.nan])
def test_more_items_than_a_round_has(junk):
    """80 items an SM, of heads that are all the same; where keys that nobody sees are NaN, the
    items that load some are taken twice."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    heads = 256
    total = -(-80 * sms // heads) * 256 - 57
    lengths, g = [], torch.Generator().manual_seed(5)
    while sum(lengths) < total - 300:
        lengths.append(int(torch.randint(1, 200, (1,), generator=g)))
    lengths[-1] -= sum(lengths) - (total - 300)
    lo, hi = spans.with_nothing(spans.documents(lengths), 300)
    one = problem(lo, hi, total, (1, 1, 16), seed=6)
    for n in ("k", "v"):
        one[n][total - 300:] = junk
    every = {n: one[n].expand(total, heads, 16).contiguous() for n in ("q", "k", "v")}
    o, lse = spans.run_forward(dict(one, **every))
    assert torch.equal(o, o[:, :1].expand_as(o)) and torch.equal(lse, lse[:, :1].expand_as(lse))
    for n in ("k", "v"):
        one[n][total - 300:] = 0
    spans.check_forward(one, o[:, :1], lse[:, :1])


def blind_queries(st):
    return st["lo"].clamp(min=0) >= st["hi"].clamp(max=st["k"].shape[0])


def packed(heads=(32, 8, 128)):
    g, lengths, unused = torch.Generator().manual_seed(1), [], 131
    while sum(lengths) < 4096 - unused:
        n = int(torch.randint(1, 1025, (1,), generator=g))
        lengths.append(min(n, 4096 - unused - sum(lengths)))
    lo, hi = spans.with_nothing(spans.documents(lengths), unused)
    return problem(lo, hi, 4096, heads)


@pytest.mark.parametrize("mask", UNSEEN)
@pytest.mark.parametrize("heads,cap", [((32, 8, 128), 0.0), ((8, 8, 64), 30.0), ((4, 1, 128), 20.0),
                                       ((9, 3, 48), 0.0), ((4, 2, 16), 0.0)], ids=str)
def test_the_gradient_of_queries_that_see_nothing(mask, heads, cap):
    """Whatever their rows hold."""
    keys, of = UNSEEN[mask]
    lo, hi = of()
    lo, hi = (torch.cat([x[:7], torch.tensor([3, 9, 2]), x[7:]]) for x in (lo, hi))
    hi[len(hi[:7]):len(hi[:7]) + 3] = 1  # some between the others
    st = problem(lo, hi, keys, heads, seed=13, cap=cap)
    blind = blind_queries(st)
    o, lse = spans.run_forward(st)
    bad = dict(st, **{n: st[n].clone() for n in ("q", "d_o", "d_lse")})
    for n, junk in (("q", math.nan), ("d_o", -math.inf), ("d_lse", math.nan)):
        bad[n][blind] = junk
    got = spans.run_backward(bad, o, lse)
    spans.check_backward(st, o, lse, got)


def test_the_gradient_of_queries_that_see_nothing_costs_little():
    """NaN in the unused end of a packed batch's q and d_o; took 100 times as long."""
    st = packed()
    clean = time_us(backward_call(st))
    for n in ("q", "d_o"):
        st[n][blind_queries(st)] = math.nan
    assert time_us(backward_call(st)) < 3 * clean


@pytest.mark.parametrize("mask", UNSEEN)
@pytest.mark.parametrize("heads,cap", [((32, 8, 128), 0.0), ((8, 8, 64), 30.0), ((4, 1, 128), 20.0),
                                       ((9, 3, 48), 0.0), ((4, 2, 16), 0.0)], ids=str)
@pytest.mark.parametrize("junk", [math.nan, math.inf])
def test_the_gradient_beside_keys_that_nobody_sees(mask, heads, cap, junk):
    keys, of = UNSEEN[mask]
    lo, hi = of()
    st = problem(lo, hi, keys, heads, seed=14, cap=cap)
    empty = unseen_keys(st)
    o, lse = spans.run_forward(st)
    bad = dict(st, **{n: st[n].clone() for n in ("k", "v")})
    for n in ("k", "v"):
        bad[n][empty] = junk
    got = spans.run_backward(bad, o, lse)
    for n in ("k", "v"):
        assert (got[n][empty] == 0).all()
    spans.check_backward(st, o, lse, got)


def test_the_gradient_beside_keys_that_nobody_sees_costs_little():
    """NaN in the unused end of a packed batch, in all that it reads; took 140 times as long."""
    st = packed()
    clean = time_us(backward_call(st))
    for n, which in (("k", unseen_keys(st)), ("v", unseen_keys(st)), ("q", blind_queries(st)),
                     ("d_o", blind_queries(st))):
        st[n][which] = math.nan
    assert time_us(backward_call(st)) < 4 * clean


@pytest.mark.parametrize("junk", [0.0, math.nan])
def test_the_gradient_of_more_items_than_a_round_has(junk):
    """As above, 80 items an SM of dQ."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    heads = 256
    total = -(-80 * sms // heads) * 128 - 57
    lengths, g = [], torch.Generator().manual_seed(5)
    while sum(lengths) < total - 300:
        lengths.append(int(torch.randint(1, 200, (1,), generator=g)))
    lengths[-1] -= sum(lengths) - (total - 300)
    lo, hi = spans.with_nothing(spans.documents(lengths), 300)
    one = problem(lo, hi, total, (1, 1, 16), seed=6)
    o, lse = spans.run_forward(one)
    for n in ("q", "k", "v", "d_o"):
        one[n][total - 300:] = junk
    every = {n: one[n].expand(total, heads, 16).contiguous() for n in ("q", "k", "v", "d_o")}
    every["d_lse"] = one["d_lse"].expand(total, heads).contiguous()
    got = spans.run_backward(dict(one, **every), o.expand(total, heads, 16).contiguous(),
                             lse.expand(total, heads).contiguous())
    for n in got:
        assert torch.equal(got[n], got[n][:, :1].expand_as(got[n])), n
    for n in ("q", "k", "v", "d_o"):
        one[n][total - 300:] = 0
    spans.check_backward(one, o, lse, {n: got[n][:, :1] for n in got})


def test_nan_beside_replays_and_other_streams():
    """A captured layer's attention whose unused memory turns to NaN and back between replays, and
    two such calls at once."""
    st = packed((8, 2, 128))
    sts = [st, problem(*caches([300, 1, 17, 128, 129, 0, 255, 256], 1, 300), 2400, (8, 2, 128))]
    calls = []
    for x in sts:
        t, nh, d = x["q"].shape
        keys, nkv = x["k"].shape[:2]
        out = {n: torch.zeros_like(x[n]) for n in ("q", "k", "v")}
        o, lse = torch.zeros_like(x["q"]), torch.zeros(t, nh, device="cuda")
        ws = torch.empty(max(rdt.attention_workspace_bytes(t, keys, nh, nkv, d, backward=b)
                             for b in (False, True)), dtype=torch.uint8, device="cuda")

        def call(x=x, o=o, lse=lse, ws=ws, out=out):
            common = dict(lo=x["lo"], hi=x["hi"], scale=x["scale"])
            rdt.attention(x["q"], x["k"], x["v"], o, ws, lse=lse, **common)
            rdt.attention_backward(x["q"], x["k"], x["v"], o, lse, x["d_o"], out["q"], out["k"],
                                   out["v"], ws, d_lse=x["d_lse"], **common)

        calls.append((call, o, lse, out, ws))
    streams = [torch.cuda.Stream() for _ in sts]
    graphs = []
    for call, *_ in calls:
        call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for junk in (0.0, math.nan, 0.0, math.inf, 0.0):
        for x in sts:
            for n in ("k", "v"):
                x[n][unseen_keys(x)] = junk
            for n in ("q", "d_o"):
                x[n][blind_queries(x)] = junk
        torch.cuda.synchronize()
        for graph, s, (_, o, lse, out, ws) in zip(graphs, streams, calls):
            with torch.cuda.stream(s):
                for y in (o, lse, *out.values()):
                    y.fill_(3.0)
                ws.fill_(255)
                for _ in range(3):
                    graph.replay()
        torch.cuda.synchronize()
        for x, (_, o, lse, out, _) in zip(sts, calls):
            clean = dict(x, **{n: x[n].clone() for n in ("q", "k", "v", "d_o")})
            for n in ("k", "v"):
                clean[n][unseen_keys(x)] = 0
            for n in ("q", "d_o"):
                clean[n][blind_queries(x)] = 0
            check_by_key_heads(clean, o, lse, out)
    assert rdt.device_error() == 0
