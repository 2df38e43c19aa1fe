"""Attention over spans and its gradient where a CTA takes several items one after the other, and
where many sequences have a cache each, against the formulas in 64 bits (bounds as in
test_gpu_attention_spans)."""
import pytest
import torch

import test_gpu_attention_spans as spans
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def check_by_key_heads(st, o, lse, got, d_lse=True):
    """The checks of one key head and its query heads at a time: all at once take much memory."""
    rep = st["q"].shape[1] // st["k"].shape[1]
    for g in range(st["k"].shape[1]):
        heads, one = slice(g * rep, (g + 1) * rep), slice(g, g + 1)
        part = dict(st, q=st["q"][:, heads], d_o=st["d_o"][:, heads], k=st["k"][:, one],
                    v=st["v"][:, one], d_lse=st["d_lse"][:, heads])
        spans.check_forward(part, o[:, heads], lse[:, heads])
        spans.check_backward(part, o[:, heads], lse[:, heads],
                             {"q": got["q"][:, heads], "k": got["k"][:, one],
                              "v": got["v"][:, one]}, d_lse=d_lse)


def problem(lo, hi, keys, heads, seed=0, cap=0.0):
    nh, nkv, d = heads
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(t, h):
        return torch.randn(t, h, d, generator=g, device="cuda").to(BF16)

    t = len(lo)
    return dict(q=normal(t, nh), k=normal(keys, nkv), v=normal(keys, nkv), d_o=normal(t, nh),
                d_lse=torch.randn(t, nh, generator=g, device="cuda"), lo=lo.int().cuda(),
                hi=hi.int().cuda(), scale=d ** -0.5, cap=cap)


@pytest.mark.parametrize("heads,cap", [((32, 8, 128), 0.0), ((32, 8, 128), 30.0),
                                       ((60, 60, 64), 0.0), ((60, 60, 64), 30.0),
                                       ((40, 20, 96), 0.0)], ids=str)
def test_a_cta_takes_many_items(heads, cap):
    """More than four items an SM of every kernel: what is handed on from item to item (stages,
    phases, the ring of items, accumulators) comes round. Ragged documents, an unused end."""
    nh, nkv, d = heads
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    per = 128 // (nh // nkv)  # queries of a row tile; an item of the forward pass is two
    pairs = -(-5 * sms // nkv)
    total = pairs * 2 * per - 57
    assert -(-total // (2 * per)) * nkv >= 5 * sms and -(-total // per) * nkv >= 5 * sms
    assert -(-total // 128) * nkv > 2 * sms  # key tiles of dK and dV, some of them halved
    g = torch.Generator().manual_seed(nh)
    lengths, unused = [], 77
    while sum(lengths) < total - unused:
        n = int(torch.randint(1, 900, (1,), generator=g))
        lengths.append(min(n, total - unused - sum(lengths)))
    lo, hi = spans.with_nothing(spans.documents(lengths), unused)
    st = problem(lo, hi, total, heads, seed=d, cap=cap)
    o, lse = spans.run_forward(st)
    got = spans.run_backward(st, o, lse)
    check_by_key_heads(st, o, lse, got)
    o2, lse2 = spans.run_forward(st)
    again = spans.run_backward(st, o, lse)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert all(torch.equal(got[n], again[n]) for n in got)


def caches(lengths, new, capacity):
    """Spans of `new` tokens of each sequence, whose keys lie at the start of `capacity` rows."""
    lo, hi = [], []
    for i, n in enumerate(lengths):
        end = torch.arange(n - new + 1, n + 1).clamp(min=0)
        lo.append(torch.full((new,), i * capacity))
        hi.append(i * capacity + end)
    return torch.cat(lo), torch.cat(hi)


@pytest.mark.parametrize("heads", [(32, 8, 128), (16, 8, 64), (4, 2, 16), (9, 3, 32), (8, 8, 128)],
                         ids=str)
@pytest.mark.parametrize("new,capacity,lengths", [
    (1, 300, [300, 1, 17, 128, 129, 0, 255, 256]),
    (1, 64, [int(x) for x in torch.randint(0, 65, (70,),
                                           generator=torch.Generator().manual_seed(0))]),
    (3, 700, [700, 3, 400, 131, 512]),
    (1, 2500, [2400, 77, 1300])], ids=["8 of 300", "70 of 64", "3 tokens", "long"])
def test_new_tokens_of_many_sequences(heads, new, capacity, lengths):
    lo, hi = caches(lengths, new, capacity)
    st = problem(lo, hi, capacity * len(lengths), heads, seed=3)
    o, lse = spans.run_forward(st)
    got = spans.run_backward(st, o, lse)
    check_by_key_heads(st, o, lse, got)
