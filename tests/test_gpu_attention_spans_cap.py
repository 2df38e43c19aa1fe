"""Gradient of capped scores far past their cap, where the slope 1 - tanh^2 is small but counts."""
import math

import pytest
import torch

import test_gpu_attention_spans as spans
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("beside", [False, True], ids=["", "beside NaN"])
@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("cap,sign", [(1.0, 1), (1.0, -1), (2.0, 1)])
def test_slope_of_a_saturated_score(d, cap, sign, beside):
    """Query t sees keys 2 t and 2 t + 1, with scores x_t cap and 0 that are exact products, x up to
    12. Key 2 t has the gradient ds = p (d_o . v - D) slope in its first column, the query
    x_t cap ds. Relative errors: 2^-8 for the rounding of ds to bf16 and 2^-8 for the result's;
    the slope's: 2 x log2 e in fp32 is off by 3 roundings of at most 35, 2^-18 of e^2x, and
    ex2 and the quotient by 2^-21; p's and those of (d_o . v - D), of which nothing cancels
    (d_o . v is 1 and 0, D between 0.26 and 0.89): 2^-17 each. Below 2^-7 + 2^-15 in all.
    Beside a query that is NaN and sees a key that is NaN, in the same tiles: rows and keys are
    computed one by one."""
    x = torch.arange(0.25, 12.01, 0.0625).to(BF16)
    n = len(x)
    more = 1 if beside else 0
    q = torch.zeros(n + more, 1, d, device="cuda", dtype=BF16)
    q[:n, :, 0] = 1
    k, v = (torch.zeros(2 * n + more, 1, d, device="cuda", dtype=BF16) for _ in range(2))
    k[:2 * n:2, 0, 0] = sign * x.cuda() * cap
    v[:2 * n:2, 0, 1] = 1
    d_o = torch.zeros_like(q)
    d_o[:n, :, 1] = 1
    lo = torch.arange(0, 2 * n + more, 2, device="cuda", dtype=torch.int32)
    hi = (lo + 2).clamp(max=2 * n + more)
    if beside:
        for y in (q, k, v):
            y[-1] = math.nan
        # a row tile in which the NaN lies between the others
        q, d_o, lo, hi = (y.roll(40, 0) for y in (q, d_o, lo, hi))
    st = dict(q=q, k=k, v=v, d_o=d_o, d_lse=None, lo=lo, hi=hi, scale=1.0, cap=cap)
    o, lse = spans.run_forward(st)
    got = spans.run_backward(st, o, lse, d_lse=False)
    keep = torch.arange(n + more, device="cuda") != (39 if beside else -1)
    part = dict(st, q=q[keep], d_o=d_o[keep], lo=lo[keep], hi=hi[keep], k=k[:2 * n], v=v[:2 * n])
    want, _ = spans.backward_exact(part, o[keep], lse[keep], d_lse=False)
    for a, b in ((got["k"][:2 * n:2, 0, 0], want["k"][::2, 0, 0]),
                 (got["q"][keep][:, 0, 0], want["q"][:, 0, 0])):
        assert (b.abs() > 0).all()
        worst = ((a.double() - b).abs() / b.abs()).max()
        assert worst <= 2.0 ** -7 + 2.0 ** -15, float(worst)
