"""Squared sum and AdamW over many tensors (rdt_tensors_sq_sum,
rdt_tensors_adamw) against their definitions: in 64 bits, and bit for bit
against the documented fp32 operations."""
import math

import pytest
import torch

from resident_decoder_trainer_gb300 import rdt

from gpu_helpers import ensure_built

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
RUN = rdt.STATE_RUN
B1, B2, EPS = 0.9, 0.95, 1e-8
SIZES = [1, 2, 3, 0, 7, 8, 255, 256, 257, 511, 512, 1000, 2047, 2048, 2049, 4096, 5001, 70000]


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()
    yield
    assert rdt.device_error() == 0


class Arena:
    """Tensors cut out of one buffer with a gap of 16 guard elements behind each."""

    def __init__(self, sizes, dtype, fill):
        starts, at = [], 0
        for n in sizes:
            starts.append(at)
            at += -(-n // 16) * 16 + 16
        raw = torch.uint8 if dtype == torch.float8_e4m3fn else dtype
        self.buf = torch.full((at,), fill, dtype=raw, device="cuda")
        self.parts = [self.buf[a:a + n] for a, n in zip(starts, sizes)]
        self.inside = torch.zeros(at, dtype=torch.bool, device="cuda")
        for a, n in zip(starts, sizes):
            self.inside[a:a + n] = True
        self.fill = fill

    def untouched(self):
        return bool((self.buf[~self.inside] == self.fill).all())


def codes_of(values, floor):
    """Codes and scales of one tensor, rounded to nearest (test set-up)."""
    n = values.numel()
    rows = torch.zeros(-(-n // RUN), RUN, device="cuda")
    rows.view(-1)[:n] = values
    big = rows.abs().amax(1, keepdim=True)
    q = torch.where(big > 0, rows * (448 / big), 0.0).clamp(-448, 448)
    if floor:
        q = torch.where((q > 0) & (q < 2.0 ** -9), 2.0 ** -9, q)
    return q.to(torch.float8_e4m3fn).view(-1)[:n].view(torch.uint8), big[:, 0] / 448


class Problem:
    def __init__(self, sizes, bits, g_dtype=torch.float32, shadow=True, seed=0, decades=2.0):
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def normal(n, std):
            return std * torch.randn(n, generator=gen, device="cuda")

        self.sizes, self.bits = sizes, bits
        self.g, self.w = Arena(sizes, g_dtype, 3.0), Arena(sizes, torch.float32, 5.0)
        state = torch.float32 if bits == 32 else torch.uint8
        self.m, self.v = Arena(sizes, state, 9), Arena(sizes, state, 11)
        runs = [-(-n // RUN) for n in sizes]
        self.ms, self.vs = Arena(runs, torch.float32, 13.0), Arena(runs, torch.float32, 15.0)
        self.wb = Arena(sizes, torch.bfloat16, 17.0) if shadow else None
        for i, n in enumerate(sizes):
            size = 10.0 ** float(decades * (torch.rand(1, generator=gen, device="cuda") - 2))
            spread = 10.0 ** normal(n, 0.7)
            self.g.parts[i].copy_(normal(n, size) * spread)
            self.w.parts[i].copy_(normal(n, 0.05))
            m, r = normal(n, size) * spread, (normal(n, size) * spread).abs()
            if n:
                m[0] = 0
                r[n // 2] = 0
            if bits == 32:
                self.m.parts[i].copy_(m)
                self.v.parts[i].copy_(r * r)
            else:
                for part, scales, x, low in ((self.m, self.ms, m, False), (self.v, self.vs, r, True)):
                    c, s = codes_of(x, low)
                    part.parts[i].copy_(c)
                    scales.parts[i].copy_(s)
        self.lr = [1e-3 * (1 + i % 3) for i in range(len(sizes))]
        self.wd = [0.1 * (i % 2) for i in range(len(sizes))]

    def list(self):
        states = {} if self.bits == 32 else {"m_scale": self.ms.parts, "v_scale": self.vs.parts}
        return rdt.OptTensors(g=self.g.parts, w=self.w.parts, m=self.m.parts, v=self.v.parts,
                              w_bf16=self.wb.parts if self.wb else None, lr=self.lr,
                              weight_decay=self.wd, **states)

    def arenas(self):
        return {k: x for k, x in vars(self).items() if isinstance(x, Arena)}

    def snapshot(self):
        return {k: [p.clone() for p in x.parts] for k, x in self.arenas().items()}


def f32(x):
    return torch.tensor(x, dtype=torch.float32).item()


def decode(codes, scales, n):
    x = codes.view(torch.float8_e4m3fn).float()
    return x * scales.repeat_interleave(RUN)[:n]


def mix(x):
    x = x ^ (x >> 16)
    x = (x * 0x3C6EF373) & 0xFFFFFFFF
    x = x ^ (x >> 14)
    x = (x * 0xBB67AE85) & 0xFFFFFFFF
    return x ^ (x >> 16)


def encode(x, half, floor):
    n = x.numel()
    rows = torch.zeros(-(-n // RUN), RUN, device=x.device)
    rows.view(-1)[:n] = x
    big = rows.abs().amax(1, keepdim=True)
    there = big >= 2.0 ** -100
    unit = torch.where(there, big.reciprocal() * 448.0, 0.0)
    scales = torch.where(there, big / torch.full_like(big, 448.0), 0.0)[:, 0]
    q = (rows * unit).view(-1)[:n].clamp(-448, 448)
    if half is not None:
        low = torch.where(q.abs() < 2.0 ** -6, 2.0 ** -6, 0.0)
        bits = (q.abs() + low).view(torch.int32) + (half * 16 + 8).int()
        q = torch.copysign((bits & -0x100000).view(torch.float32) - low, q).clamp(-448, 448)
    if floor:
        kept = there.expand(-1, RUN).reshape(-1)[:n]
        q = torch.where((x > 0) & kept & (q < 2.0 ** -9), 2.0 ** -9, q)
    return q.to(torch.float8_e4m3fn).view(torch.uint8), scales


def by_the_header(old, i, problem, step, scale, seed):
    """One tensor's state and bf16 copy after a step of the documented fp32 operations. Checks
    its w, whose quotient is right to 2^-22 and whose last difference is rounded again."""
    n = problem.sizes[i]
    b1, b2, eps = f32(B1), f32(B2), f32(EPS)
    lr, wd = (torch.tensor(x, dtype=torch.float32, device="cuda") for x in (problem.lr[i],
                                                                            problem.wd[i]))
    rate = lr * f32(1.0 / (1.0 - b1 ** step))
    keep = 1.0 - lr * wd
    m, v = old["m"][i], old["v"][i]
    if problem.bits == 8:
        m, r = decode(m, old["ms"][i], n), decode(v, old["vs"][i], n)
        v = r * r
    g = old["g"][i].float() * f32(scale)
    m = m * b1 + g * f32(1.0 - b1)
    v = v * b2 + (g * f32(1.0 - b2)) * g
    root = torch.sqrt(v)
    move = (m / (root * f32(1.0 / math.sqrt(1.0 - b2 ** step)) + eps)) * rate
    w = old["w"][i] * keep - move
    assert_near(problem.w.parts[i], w, 2.0 ** -22 * move.abs().double() + 2 * U * w.abs().double())
    out = {"wb": problem.w.parts[i].bfloat16()}
    if problem.bits == 32:
        return {**out, "m": m, "v": v}
    up = (None, None)
    if seed is not None:
        key = mix((mix((mix(step) + seed) & 0xFFFFFFFF) + i) & 0xFFFFFFFF)
        x = mix(torch.arange(n, device="cuda") ^ key)
        up = (x & 0xFFFF, x >> 16)
    (mc, ms), (vc, vs) = encode(m, up[0], False), encode(root, up[1], True)
    return {**out, "m": mc, "ms": ms, "v": vc, "vs": vs}


def assert_near(got, want, tol):
    off = (got.double() - want.double()).abs() - tol
    assert off.numel() == 0 or off.max() <= 0, float(off.max())


def in_64_bits(old, i, problem, step, scale):
    n = problem.sizes[i]
    b1, b2 = f32(B1), f32(B2)
    m, v = old["m"][i].double(), old["v"][i].double()
    if problem.bits == 8:
        m = decode(old["m"][i], old["ms"][i], n).double()
        v = decode(old["v"][i], old["vs"][i], n).double() ** 2
    g = old["g"][i].double() * f32(scale)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    w = old["w"][i].double()
    lr, wd = f32(problem.lr[i]), f32(problem.wd[i])
    hat = (m / (1 - b1 ** step)) / ((v / (1 - b2 ** step)).sqrt() + f32(EPS))
    return w - lr * (hat + wd * w), m, v, lr * hat.abs()


def check_step(p, step=3, scale=0.37, seed=None, **call):
    old = p.snapshot()
    lst = p.list()
    sc = torch.full((1,), scale, device="cuda")
    rdt.tensors_adamw(lst, call.pop("step_arg", step), B1, B2, EPS, scale=sc, seed=seed, **call)
    torch.cuda.synchronize()
    for name, arena in p.arenas().items():
        assert arena.untouched(), name
    for i, n in enumerate(p.sizes):
        want = by_the_header(old, i, p, step, scale, seed)
        for k, x in want.items():
            if k == "wb" and p.wb is None:
                continue
            assert torch.equal(getattr(p, k).parts[i], x), (k, i, n)
        assert torch.equal(p.g.parts[i], old["g"][i])
        # against 64 bits: the old state's squared root has two roundings, m and v two to
        # three more each, the quotient five, w two
        w, m, v, moved = in_64_bits(old, i, p, step, scale)
        tol = 2 * U * w.abs() + 4 * U * old["w"][i].abs() + 24 * U * moved + \
            f32(p.lr[i]) * 24 * U * (f32(B1) * decode(old["m"][i], old["ms"][i], n).double().abs()
                                     if p.bits == 8 else old["m"][i].double().abs()) / \
            ((v / (1 - f32(B2) ** step)).sqrt() + f32(EPS)) / (1 - f32(B1) ** step)
        off = (p.w.parts[i].double() - w).abs() - tol
        assert n == 0 or off.max() <= 0, (i, n, float(off.max()))
        if p.bits == 32:
            mag = old["m"][i].double().abs() + old["g"][i].double().abs()
            assert ((p.m.parts[i].double() - m).abs() <= 4 * U * mag).all()
            assert ((p.v.parts[i].double() - v).abs() <= 8 * U * v + 1e-44).all()
        elif n:
            # a code is off by half a step when rounded to nearest, by one when at random
            share = (2.0 ** -4 if seed is None else 2.0 ** -3) * 1.001
            least = (2.0 ** -10 if seed is None else 2.0 ** -9) * 1.001
            for part, scales, x in ((p.m, p.ms, m), (p.v, p.vs, v.sqrt())):
                got = decode(part.parts[i], scales.parts[i], n).double()
                unit = scales.parts[i].double().repeat_interleave(RUN)[:n]
                floor = (2.0 ** -9 if part is p.v else 0) * unit
                # a run whose largest magnitude is below 2^-100 is stored as zeros: scale 0, and
                # each element off by itself, so by less than 2^-100
                lost = torch.where(unit == 0, 2.0 ** -100, 1e-40)
                off = (got - x).abs() - torch.maximum(share * x.abs(), least * unit) - floor - lost
                assert off.max() <= 0, (i, n, float(off.max()))
    return p


@pytest.mark.parametrize("g_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shadow", [True, False])
@pytest.mark.parametrize("bits,seed", [(32, None), (8, None), (8, 0), (8, 2 ** 32 - 1)])
def test_one_step(bits, seed, g_dtype, shadow):
    check_step(Problem(SIZES, bits, g_dtype, shadow), seed=seed)
    check_step(Problem(SIZES, bits, g_dtype, shadow, seed=1), step=1, scale=1.0, seed=seed)
    check_step(Problem([5], bits, g_dtype, shadow, seed=2), step=100000, seed=seed)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("count", [31, 32, 33, 399, 400, 401, 1203])
def test_more_tensors_than_a_launch_takes(bits, count):
    """Launches hold a fixed number of entries; the rounding goes by the place in the list."""
    gen = torch.Generator().manual_seed(count)
    sizes = torch.randint(0, 700, (count,), generator=gen).tolist()
    check_step(Problem(sizes, bits), seed=5 if bits == 8 else None)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_large_tensor_beside_small_ones(bits):
    check_step(Problem([3, 20_000_001, 64, 1_000_000], bits, torch.bfloat16), seed=11)


@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_and_states(bits):
    p = Problem([1, 300, 4096], bits)
    for arena in (p.g, p.m, p.v, p.ms, p.vs):
        for part in arena.parts:
            part.zero_()
    old = p.snapshot()
    check_step(p, seed=3)
    for i, x in enumerate(old["w"]):  # decay only
        keep = 1 - f32(p.lr[i]) * f32(p.wd[i])
        assert (p.w.parts[i].double() - x.double() * keep).abs().max() <= 2 * U * x.abs().max()
        assert (p.m.parts[i] == 0).all() and (p.v.parts[i] == 0).all()


@pytest.mark.parametrize("seed", [None, 9])
def test_tiny_and_huge_runs_of_8_bit_states(seed):
    """Runs below 2^-100 are stored as zeros; a sqrt(v) > 0 elsewhere never becomes 0."""
    p = Problem([256, 256, 256, 600], 8)
    p.g.parts[0].fill_(1e-35)
    p.m.parts[0].zero_(), p.v.parts[0].zero_(), p.ms.parts[0].zero_(), p.vs.parts[0].zero_()
    p.g.parts[1].mul_(1e18 / p.g.parts[1].abs().max())
    p.g.parts[2].fill_(1e-12)
    p.v.parts[2].zero_(), p.m.parts[2].zero_()
    p.g.parts[2][7] = 1.0
    check_step(p, seed=seed)
    assert (p.m.parts[0] == 0).all() and (p.ms.parts[0] == 0).all()
    assert (p.v.parts[2] > 0).all()
    big = p.ms.parts[1]
    assert big.isfinite().all() and (p.v.parts[1] != 0x7F).all()


@pytest.mark.parametrize("bits", [32, 8])
def test_the_skip_flag_leaves_everything(bits):
    p = Problem(SIZES, bits)
    p.g.parts[-1][5] = math.nan
    old = p.snapshot()
    flag = torch.ones(1, dtype=torch.int32, device="cuda")
    rdt.tensors_adamw(p.list(), 1, B1, B2, EPS, skip=flag, seed=1)
    for k, parts in p.snapshot().items():
        for a, b in zip(parts, old[k]):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k
    flag.zero_()
    p.g.parts[-1][5] = 0.5
    check_step(p, seed=1, skip=flag)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_nan_gradient_stays_with_its_element(bits):
    p = Problem([1000], bits)
    q = Problem([1000], bits)
    p.g.parts[0][300] = math.nan
    for x in (p, q):
        rdt.tensors_adamw(x.list(), 2, B1, B2, EPS)
    rest = torch.arange(1000, device="cuda") != 300
    assert p.w.parts[0][300].isnan() and torch.equal(p.w.parts[0][rest], q.w.parts[0][rest])
    if bits == 8:
        assert int(p.m.parts[0][300]) & 0x7F == 0x7F and int(p.v.parts[0][300]) & 0x7F == 0x7F
        # the other runs are as they would be
        assert torch.equal(p.m.parts[0][:256], q.m.parts[0][:256])
        assert p.ms.parts[0].isfinite().all()


def test_no_scale_is_a_scale_of_one():
    p, q = Problem(SIZES, 8, seed=4), Problem(SIZES, 8, seed=4)
    rdt.tensors_adamw(p.list(), 7, B1, B2, EPS, scale=torch.ones(1, device="cuda"))
    rdt.tensors_adamw(q.list(), 7, B1, B2, EPS)
    for k, parts in p.snapshot().items():
        assert all(torch.equal(a, b) for a, b in zip(parts, q.snapshot()[k])), k


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("step", [1, 37, 20000])
def test_step_on_the_device(bits, step):
    p = Problem(SIZES, bits, seed=6)
    at = torch.full((1,), step, dtype=torch.int32, device="cuda")
    check_step(p, step=step, seed=8, step_arg=None, step_dev=at)


@pytest.mark.parametrize("bits,seed", [(32, None), (8, None), (8, 3)])
@pytest.mark.parametrize("b1,b2", [(B1, B2), (0.0, 0.999), (0.9999, 0.99999), (0.5, 0.0)])
def test_the_step_on_the_device_is_the_step_from_the_host(bits, seed, b1, b2):
    """The same bits: the bias corrections differ by a few 2^-53 of 1 before they are rounded to
    fp32, so a rounding falls otherwise once in some 2^25."""
    for step in (1, 2, 3, 10, 999, 65536, 2 ** 31 - 1):
        one, two = (Problem([300, 7, 5000], bits, seed=30) for _ in range(2))
        dev = torch.full((1,), step, dtype=torch.int32, device="cuda")
        rdt.tensors_adamw(one.list(), step, b1, b2, EPS, seed=seed)
        rdt.tensors_adamw(two.list(), None, b1, b2, EPS, seed=seed, step_dev=dev)
        for k, parts in one.snapshot().items():
            assert all(torch.equal(a, b) for a, b in zip(parts, two.snapshot()[k])), (k, step)


@pytest.mark.parametrize("bits", [32, 8])
def test_the_step_on_the_device_costs_little(bits):
    """134 M parameters: a quarter more than with a step from the host, at most (it took 1.7 to
    2.8 times as long while every thread formed the bias corrections)."""
    n = 1 << 27
    state = torch.float32 if bits == 32 else torch.uint8
    f = lambda k, dt=torch.float32: torch.zeros(k, dtype=dt, device="cuda")  # noqa: E731
    scales = {} if bits == 32 else {"m_scale": [f(n // RUN)], "v_scale": [f(n // RUN)]}
    lst = rdt.OptTensors(g=[torch.randn(n, device="cuda")], w=[f(n)], m=[f(n, state)],
                         v=[f(n, state)], lr=1e-3, **scales)
    dev = torch.full((1,), 7, dtype=torch.int32, device="cuda")

    def median(**kw):
        times = []
        for _ in range(15):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            for _ in range(3):
                rdt.tensors_adamw(lst, beta1=B1, beta2=B2, eps=EPS, **kw)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return sorted(times)[7]

    median(step=7)
    assert median(step=None, step_dev=dev) < 1.25 * median(step=7)


@pytest.mark.parametrize("sizes", [SIZES, [300, 5, 2048] * 280], ids=["one launch", "three"])
def test_captured_and_replayed(sizes):
    """A graph of squared sum, clip scale, step count and update; each replay is the next
    step, with rounding numbers of its own. Two graphs with one workspace, in turn."""
    p, q = Problem(sizes, 8, seed=7), Problem(sizes, 8, seed=7)
    sumsq = torch.zeros(1, dtype=torch.float64, device="cuda")
    scale = torch.ones(1, device="cuda")
    bad = torch.zeros(1, dtype=torch.int32, device="cuda")
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    lst = p.list()
    ws = torch.empty(rdt.tensors_sq_sum_workspace_bytes(lst), dtype=torch.uint8, device="cuda")

    def call(tensors):
        rdt.tensors_sq_sum(tensors, sumsq, ws)
        rdt.clip_scale(sumsq, 1.0, scale, bad)
        rdt.step_advance(step)
        rdt.tensors_adamw(tensors, None, B1, B2, EPS, scale=scale, skip=bad, step_dev=step, seed=4)

    eager = q.list()
    for _ in range(4):
        call(eager)
    torch.cuda.synchronize()
    step.zero_()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(lst)
        graphs.append(g)
    for g in graphs + graphs:
        g.replay()
    torch.cuda.synchronize()
    assert int(step) == 4
    for k, parts in p.snapshot().items():
        assert all(torch.equal(a, b) for a, b in zip(parts, q.snapshot()[k])), k


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes", [[300, 5, 2048] * 280, [3_000_000, 17]], ids=["three", "one"])
def test_overlapping_launches_keep_the_order_of_the_stream(sizes, bits):
    """Gradients written by a copy or a kernel, clip, step, gradients overwritten, step after
    step without a wait: the same as with one after every call."""
    ways = []
    for wait in (True, False):
        p = Problem(sizes, bits, seed=14)
        lst = p.list()
        ws = torch.empty(rdt.tensors_sq_sum_workspace_bytes(lst), dtype=torch.uint8, device="cuda")
        sumsq = torch.zeros(1, dtype=torch.float64, device="cuda")
        scale, bad = torch.ones(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        gen = torch.Generator(device="cuda").manual_seed(2)
        grads = [torch.randn(p.g.buf.numel(), generator=gen, device="cuda") for _ in range(3)]
        sums = []
        torch.cuda.synchronize()
        for step in range(1, 10):
            if step % 2:
                p.g.buf.copy_(grads[step % 3])
            else:
                torch.mul(grads[step % 3], 0.5, out=p.g.buf)
            for call in (lambda: rdt.tensors_sq_sum(lst, sumsq, ws),
                         lambda: rdt.clip_scale(sumsq, 1.0, scale, bad),
                         lambda: rdt.tensors_adamw(lst, step, B1, B2, EPS, scale=scale, skip=bad,
                                                   seed=1),
                         lambda: rdt.tensors_adamw(lst, step, B1, B2, EPS, seed=2)):
                call()
                if wait:
                    torch.cuda.synchronize()
            sums.append(sumsq.clone())
            p.g.buf.fill_(float("nan"))
        torch.cuda.synchronize()
        ways.append((p.snapshot(), torch.cat(sums)))
    assert torch.equal(ways[0][1], ways[1][1])
    for k, parts in ways[0][0].items():
        if k != "g":
            assert all(torch.equal(a, b) for a, b in zip(parts, ways[1][0][k])), k


def test_another_stream():
    p = Problem(SIZES, 8, seed=8)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    old = p.snapshot()
    torch.cuda.synchronize()
    rdt.tensors_adamw(p.list(), 5, B1, B2, EPS, stream=s, seed=2)
    torch.cuda.synchronize()
    for i in range(len(SIZES)):
        for k, x in by_the_header(old, i, p, 5, 1.0, 2).items():
            assert torch.equal(getattr(p, k).parts[i], x)


def test_random_rounding_is_exact_on_average():
    """256 seeds of the same step: the mean of the stored state is the value before rounding,
    within five standard errors of one element (a rounding's deviation is at most half a
    step) and, over all elements of a run, of the mean."""
    seeds = 256
    p = Problem([RUN] * seeds, 8, seed=9)
    for arena in (p.g, p.w, p.m, p.v, p.ms, p.vs):
        for part in arena.parts[1:]:
            part.copy_(arena.parts[0])
    old = p.snapshot()
    # the entry's place in the list is part of the random numbers, so one call has them all
    rdt.tensors_adamw(p.list(), 3, B1, B2, EPS, seed=77)
    _, m, v, _ = in_64_bits(old, 0, p, 3, 1.0)
    for part, scales, x in ((p.m, p.ms, m), (p.v, p.vs, v.sqrt())):
        got = torch.stack([decode(c, s, RUN) for c, s in zip(part.parts, scales.parts)]).double()
        unit = float(scales.parts[0])
        step = torch.exp2(torch.floor(torch.log2((x.abs() / unit).clamp(min=2.0 ** -6))) - 3) * unit
        free = (x.abs() / unit > 2.0 ** -9) | (part is p.m)  # below it sqrt(v) is raised
        off = ((got.mean(0) - x) / step)[free]
        assert off.abs().max() < 5 * 0.5 / seeds ** 0.5 + 2.0 ** -16
        assert abs(off.mean()) < 5 * 0.5 / (seeds * int(free.sum())) ** 0.5 + 2.0 ** -16


def test_slow_decay_of_the_second_moment():
    """No gradient but at the run's largest element, beta2 0.999, 300 steps: each step changes
    sqrt(v) by 0.05 %, far below a code's 6 to 12 %. Rounded at random the others decay as they
    should, on average over the run; rounded to nearest they stand still."""
    got = {}
    for seed in (5, None):
        n = 64 * RUN
        g = torch.zeros(n, device="cuda")
        g[::RUN] = 1.0
        m, ms = codes_of(torch.zeros(n, device="cuda"), False)
        r0 = torch.linspace(0.1, 0.9, n, device="cuda")
        r0[::RUN] = 1.0
        v, vs = codes_of(r0, True)
        start = decode(v, vs, n).double()
        w = torch.zeros(n, device="cuda")
        lst = rdt.OptTensors(g=[g], w=[w], m=[m.clone()], v=[v], m_scale=[ms], v_scale=[vs],
                             lr=1e-4)
        for step in range(1, 301):
            rdt.tensors_adamw(lst, step, 0.9, 0.999, EPS, seed=seed)
        end = decode(v, vs, n).double()
        rest = torch.arange(n, device="cuda") % RUN != 0
        got[seed] = float((end[rest].sum() / start[rest].sum()))
    want = 0.999 ** 150  # sqrt of 0.999^300
    # 16320 independent elements, each off by a random walk of at most sqrt(300 x 0.06) steps
    # of 12 % x 0.5
    assert abs(got[5] - want) < 5 * 0.06 * 300 ** 0.5 / 16320 ** 0.5
    assert got[None] > 0.99


def test_eight_bit_states_follow_thirty_two():
    """40 steps of the same gradients: the weights' way with 8-bit states stays near the way
    with 32-bit ones. A stored m is off by up to 1/16 (nearest) of itself and a stored sqrt(v)
    by the same, and both errors are carried, weighted by beta; a way is off by a third at
    most."""
    n = 50_000
    gen = torch.Generator(device="cuda").manual_seed(3)
    mean = 0.1 * torch.randn(n, generator=gen, device="cuda")
    ways = []
    for bits, seed in ((32, None), (8, None), (8, 6)):
        gen = torch.Generator(device="cuda").manual_seed(4)
        w, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
        if bits == 32:
            states = dict(m=[torch.zeros(n, device="cuda")], v=[torch.zeros(n, device="cuda")])
        else:
            runs = -(-n // RUN)
            states = dict(m=[torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda")],
                          v=[torch.zeros(n, dtype=torch.float8_e4m3fn, device="cuda")],
                          m_scale=[torch.zeros(runs, device="cuda")],
                          v_scale=[torch.zeros(runs, device="cuda")])
        lst = rdt.OptTensors(g=[g], w=[w], lr=1e-3, **states)
        for step in range(1, 41):
            g.copy_(mean + 0.1 * torch.randn(n, generator=gen, device="cuda"))
            rdt.tensors_adamw(lst, step, B1, B2, EPS, seed=seed)
        ways.append(w.double())
    for way in ways[1:]:
        assert way.isfinite().all()
        assert float((way - ways[0]).norm() / ways[0].norm()) < 1 / 3


def test_a_tensor_of_more_than_32_bits_of_elements():
    """2^32 + 1000 elements: addresses, scales and rounding numbers behind 2^32, against the
    same step of a short tensor (whose rounding goes by its own indexes: states to one code)."""
    n, tail = (1 << 32) + 1000, 5 * RUN + 1000
    a = n - tail
    gen = torch.Generator(device="cuda").manual_seed(15)
    big, short = {}, {}
    for k, dtype in (("g", torch.bfloat16), ("w", torch.float32), ("m", torch.uint8),
                     ("v", torch.uint8)):
        big[k] = torch.zeros(n, dtype=dtype, device="cuda")
        if k in "gw":
            big[k][a:] = torch.randn(tail, generator=gen, device="cuda").to(dtype)
        short[k] = big[k][a:].clone()
    for x, size in ((big, n), (short, tail)):
        for k in ("m_scale", "v_scale"):
            x[k] = torch.zeros(-(-size // RUN), device="cuda")
    for x in (big, short):
        lst = rdt.OptTensors(**{k: [t] for k, t in x.items()}, lr=1e-3)
        rdt.tensors_adamw(lst, 1, B1, B2, EPS, seed=3)
    assert torch.equal(big["w"][a:], short["w"]) and int(big["w"][:a].count_nonzero()) == 0
    for k in "mv":
        assert torch.equal(big[k + "_scale"][a // RUN:], short[k + "_scale"])
        x, y = (decode(c, s, tail).double() for c, s in (
            (big[k][a:], short[k + "_scale"]), (short[k], short[k + "_scale"])))
        unit = short[k + "_scale"].double().repeat_interleave(RUN)[:tail]
        assert ((x - y).abs() <= 2.0 ** -3 * 1.001 * torch.maximum(x.abs(), y.abs()) +
                2.0 ** -9 * unit).all()
    # the documented numbers there: the low 32 bits of the index, the key folded with the rest
    key = mix((mix((mix(1) + 3) & 0xFFFFFFFF) + 0) & 0xFFFFFFFF) ^ 0x9E3779B1
    at = torch.arange(1000, device="cuda")
    x = mix(at ^ key)
    g = big["g"][1 << 32:].float()
    m = g * f32(1.0 - f32(B1))
    root = torch.sqrt((g * f32(1.0 - f32(B2))) * g)
    for k, value, half, low in (("m", m, x & 0xFFFF, False), ("v", root, x >> 16, True)):
        codes, _ = encode(value, half, low)
        assert torch.equal(big[k][1 << 32:], codes), k
    want = float(big["g"][a:].double().square().sum())
    assert abs(sq_sum([big["g"]]) - want) <= 1e-12 * want


# --------------------------------------------------------------- squared sum
def sq_sum(parts):
    lst = rdt.OptTensors(g=parts)
    ws = torch.full((rdt.tensors_sq_sum_workspace_bytes(lst),), 255, dtype=torch.uint8,
                    device="cuda")
    out = torch.full((1,), math.nan, dtype=torch.float64, device="cuda")
    rdt.tensors_sq_sum(lst, out, ws)
    return float(out)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes", [[1], [0, 3], SIZES, [16] * 900, [30_000_000, 5, 2_000_003]])
def test_squared_sum(sizes, dtype):
    p = Problem(sizes, 32, dtype, shadow=False, seed=10, decades=6.0)
    want = sum(float(x.double().square().sum()) for x in p.g.parts)
    assert abs(sq_sum(p.g.parts) - want) <= 1e-12 * want
    assert sq_sum(p.g.parts) == sq_sum(p.g.parts)
    assert p.g.untouched()


def test_squared_sum_of_one_large_and_many_small_values():
    """2^26 values whose squares are each below half a step of the sum's first term in fp32."""
    g = torch.full((1 << 26,), 1e-6, device="cuda")
    g[0] = 1.0
    want = 1.0 + ((1 << 26) - 1) * f32(1e-6) ** 2
    assert abs(sq_sum([g]) - want) <= 1e-12 * want


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("first,rest", [(0.3, 0.3), (1e-3, 1e-3), (0.7, 0.7), (1.0, 1.7e-4),
                                        (1.0, 1.21e-4)])
def test_squared_sum_of_many_alike(first, rest, dtype):
    """Half a billion values whose additions round alike, so that nothing averages out; or a few
    thousand large values in front of ones whose squares are below half a step of the sum."""
    n, head = 500_000_000, 3_000_000
    g = torch.full((n,), rest, dtype=dtype, device="cuda")
    g[:head] = first
    a, b = float(g[0].double()) ** 2, float(g[-1].double()) ** 2
    want = head * a + (n - head) * b  # each square is exact in fp64
    assert abs(sq_sum([g]) - want) <= 1e-12 * want
    cut = list(g[: n // 8 * 8].view(8, -1)[:, :-16].unbind())  # rows of 62,499,984: ragged ends
    a8 = head * a + sum(c.numel() for c in cut) * b - head * b
    assert abs(sq_sum(cut) - a8) <= 1e-12 * a8


def test_squared_sum_of_a_list_with_more_tiles_than_32_bits_count():
    """2^31 - 1 tiles of 2048: one tensor of 2^34 elements named 256 times, once a tile shorter."""
    n = 1 << 34
    g = torch.full((n,), 0.5, dtype=torch.bfloat16, device="cuda")
    g[-2048:] = 2.0
    g[0] = 4.0
    one = 0.25 * (n - 2049) + 4.0 * 2048 + 16.0
    want = 256 * one - 4.0 * 2048
    assert abs(sq_sum([g] * 255 + [g[:-2048]]) - want) <= 1e-12 * want


def test_squared_sum_of_nothing_and_of_what_is_not_finite():
    assert sq_sum([]) == 0.0
    assert sq_sum([torch.zeros(100, device="cuda")]) == 0.0
    for bad in (math.nan, math.inf, -math.inf):
        g = torch.ones(5000, device="cuda")
        g[4321] = bad
        total = sq_sum([torch.ones(10, device="cuda"), g])
        scale, flag = torch.ones(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        rdt.clip_scale(torch.tensor([total], dtype=torch.float64, device="cuda"), 1.0, scale, flag)
        assert not math.isfinite(total) and int(flag) == 1


# ------------------------------------------------------------ the list itself
def test_refusals_of_the_list():
    def t(n, dtype=torch.float32):
        return torch.zeros(n, dtype=dtype, device="cuda")

    u8 = torch.uint8
    ok = dict(g=[t(300)], w=[t(300)], m=[t(300, u8)], v=[t(300, u8)], m_scale=[t(2)],
              v_scale=[t(2)])
    rdt.tensors_adamw(rdt.OptTensors(**ok), 1, B1, B2, EPS)
    for change, text in ((dict(w=[t(299)]), "w: want 300"), (dict(m=[t(300)]), "v: want 300"),
                         (dict(m_scale=[t(1)]), "m_scale: want 2"),
                         (dict(g=[t(300, torch.float16)]), "gradients"),
                         (dict(w=[t(600)[::2]]), "w: want 300 contiguous"),
                         (dict(w=[t(300), t(3)]), "2 tensors in w"),
                         (dict(m=[t(300, torch.int32)]), "moments"),
                         (dict(w=[torch.zeros(300)]), "CUDA")):
        with pytest.raises(ValueError, match=text):
            rdt.OptTensors(**{**ok, **change})
    with pytest.raises(ValueError, match="lr"):
        rdt.OptTensors(**ok, lr=[1.0, 2.0])
    with pytest.raises(ValueError, match="no moments"):
        rdt.tensors_adamw(rdt.OptTensors(g=[t(4)]), 1, B1, B2, EPS)
    with pytest.raises(rdt.RdtError, match="null"):
        rdt.tensors_adamw(rdt.OptTensors(**{k: ok[k] for k in ("g", "w", "m", "v")}), 1, B1, B2,
                          EPS)
    with pytest.raises(rdt.RdtError, match="overlap"):
        rdt.tensors_adamw(rdt.OptTensors(**{k: x * 2 for k, x in ok.items()}), 1, B1, B2, EPS)
    with pytest.raises(rdt.RdtError, match="aligned"):
        rdt.tensors_adamw(rdt.OptTensors(**{**ok, "w": [t(301)[1:]]}), 1, B1, B2, EPS)
    with pytest.raises(rdt.RdtError, match="step"):
        rdt.tensors_adamw(rdt.OptTensors(**ok), 0, B1, B2, EPS)


def test_refusals_of_workspaces_and_scalars():
    def t(n, dtype=torch.float32):
        return torch.zeros(n, dtype=dtype, device="cuda")

    lst = rdt.OptTensors(g=[t(300)], w=[t(300)], m=[t(300)], v=[t(300)])
    size = rdt.tensors_sq_sum_workspace_bytes(lst)
    sumsq = t(1, torch.float64)
    with pytest.raises(ValueError, match="contiguous"):
        rdt.tensors_sq_sum(lst, sumsq, t(1, torch.uint8).expand(size))
    with pytest.raises(ValueError, match="sumsq"):
        rdt.tensors_sq_sum(lst, sumsq[:0], t(size, torch.uint8))
    for kw in (dict(scale=t(0)), dict(skip=t(0, torch.int32)), dict(step_dev=t(0, torch.int32))):
        with pytest.raises(ValueError, match="no element"):
            rdt.tensors_adamw(lst, 1, B1, B2, EPS, **kw)


def test_rates_can_change_between_steps():
    p = Problem([500, 300], 32, seed=12)
    old = p.snapshot()
    lst = p.list()
    lst.set_lr([0.0, 2e-3])
    lst.set_weight_decay(0.0)
    p.lr, p.wd = [0.0, 2e-3], [0.0, 0.0]
    rdt.tensors_adamw(lst, 2, B1, B2, EPS)
    assert torch.equal(p.w.parts[0], old["w"][0]) and not torch.equal(p.w.parts[1], old["w"][1])
    for i in range(2):
        for k, x in by_the_header(old, i, p, 2, 1.0, None).items():
            assert torch.equal(getattr(p, k).parts[i], x)
