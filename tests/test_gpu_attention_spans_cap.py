"""Gradient of capped scores far past their cap, where the slope 1 - tanh^2 is small but counts."""
import pytest
import torch

import test_gpu_attention_spans as spans
from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


@pytest.mark.parametrize("d", [16, 64, 128])
@pytest.mark.parametrize("cap,sign", [(1.0, 1), (1.0, -1), (2.0, 1)])
def test_slope_of_a_saturated_score(d, cap, sign):
    """Query t sees keys 2 t and 2 t + 1, with scores x_t cap and 0 that are exact products, x up to
    12. Key 2 t has the gradient ds = p (d_o . v - D) slope in its first column, the query
    x_t cap ds. Relative errors: 2^-8 for the rounding of ds to bf16 and 2^-8 for the result's;
    the slope's: 2 x log2 e in fp32 is off by 3 roundings of at most 35, 2^-18 of e^2x, and
    ex2 and the quotient by 2^-21; p's and those of (d_o . v - D), of which nothing cancels
    (d_o . v is 1 and 0, D between 0.26 and 0.89): 2^-17 each. Below 2^-7 + 2^-15 in all."""
    x = torch.arange(0.25, 12.01, 0.0625).to(BF16)
    n = len(x)
    q = torch.zeros(n, 1, d, device="cuda", dtype=BF16)
    q[:, :, 0] = 1
    k, v = (torch.zeros(2 * n, 1, d, device="cuda", dtype=BF16) for _ in range(2))
    k[::2, 0, 0] = sign * x.cuda() * cap
    v[::2, 0, 1] = 1
    d_o = torch.zeros_like(q)
    d_o[:, :, 1] = 1
    lo = torch.arange(0, 2 * n, 2, device="cuda", dtype=torch.int32)
    st = dict(q=q, k=k, v=v, d_o=d_o, d_lse=None, lo=lo, hi=lo + 2, scale=1.0, cap=cap)
    o, lse = spans.run_forward(st)
    got = spans.run_backward(st, o, lse, d_lse=False)
    want, _ = spans.backward_exact(st, o, lse, d_lse=False)
    for name, rows in (("k", slice(0, None, 2)), ("q", slice(None))):
        a, b = got[name][rows, 0, 0].double(), want[name][rows, 0, 0]
        assert (b.abs() > 0).all()
        worst = ((a - b).abs() / b.abs()).max()
        assert worst <= 2.0 ** -7 + 2.0 ** -15, (name, float(worst))
