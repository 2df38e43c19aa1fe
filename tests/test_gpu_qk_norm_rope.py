"""Per-head RMSNorm with rotation and its gradient on the GPU, against the formulas in 64 bits,
torch's differentiation of them, and differences.

Tolerances. All arithmetic is fp32: a value passes through about ten roundings (2^-24 each) and
a sum of head_dim squares, the angle is off by 2^-24 of a half turn (3 2^-24) at most, and the
result is rounded to its type once: half a step, eps / 2. With m = max |n| of the head (a pair
mixes two values), |out - exact| <= eps(out) / 2 |exact| + 2^-19 m."""
import itertools

import pytest
import torch

from gpu_helpers import ensure_built
from resident_decoder_trainer_gb300 import rdt

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
FP32_PART = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def built():
    ensure_built()


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def exact(x, gain, eps, positions, sections, theta):
    """The forward formulas in 64 bits (differentiable)."""
    d = x.shape[2]
    half = d // 2
    n = x
    if gain is not None:
        n = x / torch.sqrt(x.square().mean(2, keepdim=True) + eps) * gain
    if positions is None:
        return n
    axis = torch.cat([torch.full((c,), i) for i, c in enumerate(sections)]).to(x.device)
    i = torch.arange(half, device=x.device, dtype=torch.float64)
    angle = (positions[axis].T.double() * theta ** (-2 * i / d))[:, None]
    a, b = n[..., :half], n[..., half:]
    return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], 2)


def problem(tokens, nh, nkv, d, dtype=BF16, axes=1, far=1 << 20, layout="fused", seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed + 1000 * tokens + d)

    def normal(*size):
        return torch.randn(*size, generator=g, device="cuda")

    def heads(n):
        if layout == "head_major":  # [heads, tokens, d], seen as [tokens, heads, d]
            return normal(n, tokens, d).to(dtype).transpose(0, 1)
        return normal(tokens, n, d).to(dtype)

    if layout == "fused":
        qkv = normal(tokens, nh + 2 * nkv, d).to(dtype)
        q, k = qkv[:, :nh], qkv[:, nh:nh + nkv]
    else:
        q, k = heads(nh), heads(nkv)
    half = d // 2
    cut = sorted(int(x) for x in torch.randint(0, half + 1, (axes - 1,),
                                               generator=torch.Generator().manual_seed(seed)))
    sections = [b - a for a, b in zip([0] + cut, cut + [half])]
    return dict(q=q, k=k, gain_q=1 + 0.2 * normal(d), gain_k=1 - 0.2 * normal(d),
                positions=torch.randint(-far, far, (axes, tokens), generator=g, device="cuda",
                                        dtype=torch.int32), sections=sections,
                d_q=normal(tokens, nh, d), d_k=normal(tokens, nkv, d))


def close(got, want, m, dtype, what):
    bound = half_step(dtype) * want.abs() + FP32_PART * m
    worst = ((got.double() - want).abs() / bound.clamp(min=1e-30)).max() if want.numel() else 0
    assert worst <= 1, f"{what}: {float(worst)} of its bound"


SHAPES = [(1, 32, 8, 128), (7, 4, 2, 16), (33, 9, 3, 32), (130, 6, 2, 96), (5, 12, 12, 80),
          (64, 3, 1, 256), (257, 16, 8, 64), (1, 1, 1, 48), (2, 130, 1, 128)]


@pytest.mark.parametrize("tokens,nh,nkv,d", SHAPES)
@pytest.mark.parametrize("dtype,out", [(F32, F32), (F32, BF16), (BF16, BF16), (F16, F16),
                                       (F16, BF16), (BF16, F32)])
def test_forward(tokens, nh, nkv, d, dtype, out):
    for axes, layout in ((1, "fused"), (3, "head_major"), (4, "plain")):
        p = problem(tokens, nh, nkv, d, dtype, axes, layout=layout)
        got = {n: torch.full((tokens, h, d), 7.0, device="cuda", dtype=out)
               for n, h in (("q", nh), ("k", nkv))}
        rdt.qk_norm_rope(p["q"], p["k"], got["q"], got["k"], gain_q=p["gain_q"],
                         gain_k=p["gain_k"], eps=1e-6, positions=p["positions"],
                         sections=p["sections"], theta=1e4)
        for n in ("q", "k"):
            want = exact(p[n].double(), p["gain_" + n].double(), 1e-6, p["positions"],
                         p["sections"], 1e4)
            top = want.abs().amax(2, keepdim=True)
            close(got[n], want, top, out, n)


def gradient(p, accumulate=False, out=F32, d_dtype=F32, start=None, **kw):
    q, k = p["q"], p["k"]
    t, nh, d = q.shape
    nkv = k.shape[1]
    dq = torch.full((t, nh, d), 9.0, device="cuda", dtype=out)
    dk = torch.full((t, nkv, d), 9.0, device="cuda", dtype=out)
    gains = [torch.full((d,), 3.0 if start is None else start, device="cuda") for _ in range(2)]
    ws = torch.full((rdt.qk_norm_rope_backward_workspace_bytes(t, nh, nkv, d),), 255,
                    dtype=torch.uint8, device="cuda")
    args = dict(gain_q=p["gain_q"], gain_k=p["gain_k"], d_gain_q=gains[0], d_gain_k=gains[1],
                eps=1e-6, positions=p["positions"], sections=p["sections"], theta=1e4)
    args.update(kw)
    rdt.qk_norm_rope_backward(q, k, p["d_q"].to(d_dtype), p["d_k"].to(d_dtype), dq, dk, ws,
                              accumulate=accumulate, **args)
    return dict(q=dq, k=dk, gain_q=args["d_gain_q"], gain_k=args["d_gain_k"])


def exact_gradient(p, d_dtype=F32):
    """By the formulas: the upstream gradient turned back, then the norm's."""
    out = {}
    for n in ("q", "k"):
        x, gain = p[n].double(), p["gain_" + n].double()
        dy = p["d_" + n].to(d_dtype).double()
        dn = exact(dy, None, 0.0, -p["positions"], p["sections"], 1e4)
        r = 1 / torch.sqrt(x.square().mean(2, keepdim=True) + 1e-6)
        unit = x * r
        out["gain_" + n] = (dn * unit).sum((0, 1))
        out["gain_size_" + n] = (dn * unit).abs().sum((0, 1))
        dn = dn * gain
        out[n] = r * (dn - unit * (dn * unit).mean(2, keepdim=True))
        # what a rounding of an operand may change: the two terms apart
        out["size_" + n] = (r * (dn.abs() + unit.abs() * (dn * unit).abs().mean(2, keepdim=True))
                            ).amax(2, keepdim=True)
    return out


def check_gradient(got, want, out):
    for n in ("q", "k"):
        close(got[n], want[n], want["size_" + n], out, "d" + n)
        # fp32 terms (2^-19 each, as above) summed in any order: at most a few hundred additions
        # in a row a lane, their errors far below n 2^-24 of the sum of magnitudes
        bound = (2.0 ** -19 + 2.0 ** -24 * 512) * want["gain_size_" + n] + 1e-30
        err = (got["gain_" + n].double() - want["gain_" + n]).abs() / bound
        assert err.max() <= 1, (n, float(err.max()))


@pytest.mark.parametrize("tokens,nh,nkv,d", SHAPES)
@pytest.mark.parametrize("dtype,d_dtype,out", [(F32, F32, F32), (BF16, BF16, BF16),
                                               (F16, BF16, F16), (F32, F16, BF16),
                                               (BF16, F32, F32)])
def test_gradient(tokens, nh, nkv, d, dtype, d_dtype, out):
    for axes, layout in ((1, "fused"), (3, "head_major")):
        p = problem(tokens, nh, nkv, d, dtype, axes, layout=layout)
        check_gradient(gradient(p, out=out, d_dtype=d_dtype), exact_gradient(p, d_dtype), out)


def test_gradient_of_many_tokens():
    p = problem(3001, 32, 8, 128, axes=2)
    check_gradient(gradient(p, out=BF16), exact_gradient(p), BF16)


def test_gradient_against_differences():
    p = problem(5, 4, 2, 32, F32, axes=2)
    got = gradient(p)
    x = {n: p[n].double() for n in ("q", "k", "gain_q", "gain_k")}

    def loss(change, h):
        y = {n: x[n] + h * change.get(n, 0.0) for n in x}
        return sum((exact(y[n], y["gain_" + n], 1e-6, p["positions"], p["sections"], 1e4)
                    * p["d_" + n].double()).sum() for n in ("q", "k"))

    for seed, n in itertools.product(range(3), x):
        g = torch.Generator(device="cuda").manual_seed(seed)
        u = torch.randn(x[n].shape, generator=g, device="cuda", dtype=torch.float64)
        diff = (loss({n: u}, 1e-4) - loss({n: u}, -1e-4)) / 2e-4
        along = (got[n].double() * u).sum()
        # the difference's own error is h^2 times a third derivative: far below 1e-6 of the sum
        assert abs(diff - along) <= 2e-5 * (got[n].double() * u).abs().sum(), n


def test_accumulate_adds_and_repeats():
    p = problem(300, 8, 4, 64)
    a, b = gradient(p, start=0.0), gradient(p, accumulate=True, start=2.0)
    for n in ("gain_q", "gain_k"):
        assert torch.equal(a[n] + 2.0, b[n])
    c = gradient(p, start=5.0)
    for n in a:
        assert torch.equal(a[n], c[n])


def test_no_norm_no_rotation_and_one_tensor():
    p = problem(19, 4, 2, 64, F32)
    out = {n: torch.empty(p[n].shape, device="cuda") for n in ("q", "k")}
    rdt.qk_norm_rope(p["q"], p["k"], out["q"], out["k"])
    assert torch.equal(out["q"], p["q"]) and torch.equal(out["k"], p["k"])
    rdt.qk_norm_rope(p["q"], p["k"], out["q"], out["k"], positions=p["positions"][0], theta=1e4)
    want = exact(p["q"].double(), None, 0.0, p["positions"], p["sections"], 1e4)
    close(out["q"], want, want.abs().amax(2, keepdim=True), F32, "rotation alone")
    alone = torch.empty_like(out["k"])
    rdt.qk_norm_rope(None, p["k"], None, alone, positions=p["positions"][0], theta=1e4)
    assert torch.equal(alone, out["k"])
    # without a norm the gradient is the rotation back
    dq, dk = torch.empty_like(out["q"]), torch.empty_like(out["k"])
    rdt.qk_norm_rope_backward(p["q"], p["k"], p["d_q"], p["d_k"], dq, dk,
                              positions=p["positions"], theta=1e4)
    want = exact(p["d_q"].double(), None, 0.0, -p["positions"], p["sections"], 1e4)
    close(dq, want, want.abs().amax(2, keepdim=True), F32, "turned back")


def test_in_place():
    p = problem(70, 8, 2, 128, BF16)
    want = {n: torch.empty(p[n].shape, device="cuda", dtype=BF16) for n in ("q", "k")}
    args = dict(gain_q=p["gain_q"], gain_k=p["gain_k"], positions=p["positions"], theta=1e6)
    rdt.qk_norm_rope(p["q"], p["k"], want["q"], want["k"], **args)
    grads = [torch.empty(p[n].shape, device="cuda", dtype=BF16) for n in ("q", "k")]
    dq, dk = p["d_q"].to(BF16), p["d_k"].to(BF16)
    rdt.qk_norm_rope_backward(p["q"], p["k"], dq, dk, *grads, **args)
    rdt.qk_norm_rope_backward(p["q"], p["k"], dq, dk, dq, dk, **args)
    assert torch.equal(dq, grads[0]) and torch.equal(dk, grads[1])
    rdt.qk_norm_rope(p["q"], p["k"], p["q"], p["k"], **args)
    assert torch.equal(p["q"], want["q"]) and torch.equal(p["k"], want["k"])


def test_zero_rows_with_eps_zero_touch_no_other():
    """A head of zeros has no norm with eps 0; slots of a warp without a head count nowhere."""
    p = problem(3, 5, 1, 16, F32)  # 6 heads: slots of a warp stay empty
    got = gradient(p, eps=0.0)
    assert all(torch.isfinite(x).all() for x in got.values())


def test_rows_around_are_left():
    t, nh, nkv, d = 9, 4, 2, 64
    p = problem(t, nh, nkv, d)
    big = torch.full((t + 2, nh + nkv + 2, d), 5.0, device="cuda", dtype=BF16)
    q, k = big[1:-1, 1:1 + nh], big[1:-1, 1 + nh:-1]
    rdt.qk_norm_rope(p["q"], p["k"], q, k, gain_q=p["gain_q"], gain_k=p["gain_k"],
                     positions=p["positions"])
    assert (big[0] == 5).all() and (big[-1] == 5).all()
    assert (big[:, 0] == 5).all() and (big[:, -1] == 5).all()
    assert torch.isfinite(q).all() and not (q == 5).all()


def test_no_tokens():
    p = problem(0, 4, 2, 64)
    rdt.qk_norm_rope(p["q"], p["k"], p["q"], p["k"])
    dg = torch.ones(64, device="cuda")
    for accumulate, want in ((True, 1.0), (False, 0.0)):
        rdt.qk_norm_rope_backward(p["q"], p["k"], p["q"], p["k"], p["q"], p["k"],
                                  gain_q=p["gain_q"], d_gain_q=dg, accumulate=accumulate)
        assert (dg == want).all()


def test_replayed_graph_and_other_stream():
    p = problem(40, 8, 2, 128)
    want = gradient(p, out=BF16)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = gradient(p, out=BF16)
    torch.cuda.current_stream().wait_stream(s)
    for n in want:
        assert torch.equal(want[n], other[n])
    d = 128
    ws = torch.empty(rdt.qk_norm_rope_backward_workspace_bytes(40, 8, 2, d), dtype=torch.uint8,
                     device="cuda")
    out = {n: torch.zeros_like(want[n]) for n in want}
    dy = [p["d_q"].clone(), p["d_k"].clone()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rdt.qk_norm_rope_backward(p["q"], p["k"], *dy, out["q"], out["k"], ws,
                                  gain_q=p["gain_q"], gain_k=p["gain_k"],
                                  d_gain_q=out["gain_q"], d_gain_k=out["gain_k"], eps=1e-6,
                                  positions=p["positions"], sections=p["sections"], theta=1e4)
    for _ in range(2):
        for x in out.values():
            x.fill_(1.0)
        graph.replay()
        for n in want:
            assert torch.equal(want[n], out[n])
