"""Attention over spans and its gradient where something that is not finite lies beside what is
seen, and where warps of a CTA wait long for one another, against the formulas in 64 bits (bounds
as in test_gpu_attention_spans)."""
import math

import pytest
import torch

import test_gpu_attention_spans as spans
from gpu_helpers import ensure_built
from resident_decoder_trainer_gb300 import rdt
from test_gpu_attention_spans_items import problem

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
