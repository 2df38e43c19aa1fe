"""Scoring and 8-bit optimizer states through the trainers, and the new calls
together as one policy step on a linear head."""
import numpy as np
import pytest
import torch

from oracle import model as om
from resident_decoder_trainer_gb300 import rdt, synth
from resident_decoder_trainer_gb300.nf4_step import Nf4LoraTrainer
from resident_decoder_trainer_gb300.step import DecoderTrainer

import test_gpu_tensors as tensors
from gpu_helpers import LOSS_REL, ensure_built, ragged_shape, rel_l2, to_np

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()
    yield
    assert rdt.device_error() == 0


def test_scores_are_the_training_losses():
    """The same forward pass as the fused cross-entropy's: log p is its loss with the sign
    turned, up to fp32 summation order; and the oracle's loss to the path's 1e-3."""
    shape = ragged_shape()
    blocks, head, x, tg = synth.make_model_inputs(shape, 5)
    tr = DecoderTrainer(shape)
    tr.load(blocks, head)
    xd, td = x.cuda(), tg.int().cuda()
    loss = tr.forward_backward(xd, td).clone()
    got = tr.score(xd, td, top=7)
    assert (got["logp"] + loss).abs().max() < 1e-5 * loss.abs().max()
    ref = om.train_step(blocks, head, x, tg.numpy(), shape, step=1, optim=synth.OPTIM)
    assert abs(-float(got["logp"].double().mean()) - ref["loss"]) < LOSS_REL * ref["loss"]
    # alternatives in order, their log p consistent with the entropy's distribution
    assert (got["top_logp"].diff(dim=1) <= 0).all()
    assert ((got["top_ids"] >= 0) & (got["top_ids"] < shape.vocab)).all()
    assert (got["entropy"] > 0).all() and (got["entropy"] < np.log(shape.vocab)).all()
    hot = tr.score(xd, td, logit_scale=0.5)
    assert (hot["entropy"] >= got["entropy"] - 1e-5).all()  # a higher temperature is flatter
    part = td.clone()
    part[::2] = -1
    some = tr.score(xd, part, top=7)
    assert (some["logp"][::2] == 0).all() and torch.equal(some["logp"][1::2], got["logp"][1::2])
    assert torch.equal(some["top_ids"][1::2], got["top_ids"][1::2])
    free = tr.score(xd)
    assert set(free) == {"entropy", "lse"} and torch.equal(free["lse"], got["lse"])


def test_scoring_leaves_training_alone():
    shape = ragged_shape()
    blocks, head, x, tg = synth.make_model_inputs(shape, 6)
    a, b = DecoderTrainer(shape), DecoderTrainer(shape)
    for tr in (a, b):
        tr.load(blocks, head)
    for step in range(2):
        a.train_step(x.cuda(), tg.cuda())
        b.score(x.cuda(), tg.cuda(), top=3)
        b.train_step(x.cuda(), tg.cuda())
    for name in ("w", "m", "v", "g"):
        assert torch.equal(getattr(a, name), getattr(b, name)), name


@pytest.mark.parametrize("kw", [dict(embedding=True), dict(embedding=True, accumulation_steps=2),
                                dict(), dict(checkpoint_segments=2)])
@pytest.mark.parametrize("graph", [False, True])
def test_scoring_leaves_the_staged_inputs_alone(kw, graph):
    """Steps without inputs train on the batch staged before, whatever was scored in between."""
    shape = ragged_shape()
    n, T = kw.get("accumulation_steps", 1), shape.tokens
    gen = torch.Generator(device="cuda").manual_seed(8)
    ids, other = (torch.randint(0, shape.vocab, (n * T,), dtype=torch.int32, device="cuda",
                                generator=gen) for _ in range(2))
    x, y = (torch.randn(n * T, shape.hidden, device="cuda", generator=gen) for _ in range(2))
    one = dict(ids=ids) if kw.get("embedding") else dict(x=x)
    two = dict(ids=other[:T]) if kw.get("embedding") else dict(x=y[:T])
    ways = []
    for scores in (False, True):
        tr = DecoderTrainer(shape, **kw)
        tr.init_random(4)
        tr.train_step(targets=ids.roll(-1), **one)
        if graph:
            tr.train_step_graph(targets=ids.roll(-1), **one)
        for _ in range(2):
            if scores:
                tr.score(targets=other[:T].roll(-1), top=3, **two)
            tr.train_step_graph() if graph else tr.train_step()
        torch.cuda.synchronize()
        ways.append(tr)
    for name in ("w", "m", "v") + (("emb", "emb_m") if kw.get("embedding") else ()):
        assert torch.equal(getattr(ways[0], name), getattr(ways[1], name)), name


def test_scoring_takes_ids_with_the_device_embedding_only():
    shape = ragged_shape()
    tr = DecoderTrainer(shape)
    with pytest.raises(ValueError, match="embedding"):
        tr.score(ids=torch.zeros(shape.tokens, dtype=torch.int32, device="cuda"))


def test_scoring_with_the_device_embedding():
    shape = ragged_shape()
    tr = DecoderTrainer(shape, embedding=True)
    tr.init_random(3)
    ids = torch.randint(0, shape.vocab, (shape.tokens,), dtype=torch.int32, device="cuda")
    tg = ids.roll(-1)
    loss = tr.forward_backward(targets=tg, ids=ids).clone()
    got = tr.score(targets=tg, ids=ids)
    assert (got["logp"] + loss).abs().max() < 1e-5 * loss.abs().max()


@pytest.mark.parametrize("kw", [dict(), dict(embedding=True), dict(accumulation_steps=2),
                                dict(state_seed=None), dict(checkpoint_segments=2)])
def test_first_step_with_8_bit_states_is_the_32_bit_one(kw):
    """States start at zero, so the first update reads no rounded state: the weights differ by
    the quotient's and the sums' roundings only (a few 2^-24 of lr and of w)."""
    shape = ragged_shape()
    n = kw.get("accumulation_steps", 1)
    blocks, head, _, _ = synth.make_model_inputs(shape, 7)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(n * shape.tokens, shape.hidden, generator=g).cuda()
    tg = torch.randint(0, shape.vocab, (n * shape.tokens,), generator=g, dtype=torch.int32).cuda()
    state_seed = kw.pop("state_seed", 0)
    ways = []
    for bits in (32, 8):
        tr = DecoderTrainer(shape, state_bits=bits, state_seed=state_seed, **kw)
        tr.load(blocks, head)
        if tr.embedding:
            gen = torch.Generator(device="cuda").manual_seed(2)
            tr.emb.normal_(0, 1, generator=gen)
            tr.train_step(targets=tg, ids=tg.roll(1))
        else:
            tr.train_step(x, tg)
        ways.append(tr)
    a, b = ways
    lr = a.optim["lr"]
    tol = 2.0 ** -20 * lr + 4 * 2.0 ** -24 * a.w.abs()
    assert ((a.w - b.w).abs() <= tol).all()
    assert torch.equal(b.wb[b.opt.tensors["w"][0].numel():][:16],
                       b.w[b.opt.tensors["w"][0].numel():][:16].bfloat16())
    if a.embedding:
        assert ((a.emb - b.emb).abs() <= 2.0 ** -20 * lr + 4 * 2.0 ** -24 * a.emb.abs()).all()
    # the states stand for the 32-bit ones: half a code (nearest) or one code off
    share = 2.0 ** -4 if state_seed is None else 2.0 ** -3
    for m8, s, g32 in zip(b.opt.tensors["m"], b.opt.tensors["m_scale"], a_slices(a, b)):
        x8 = m8.view(torch.float8_e4m3fn).float() * s.repeat_interleave(256)[:m8.numel()]
        unit = s.repeat_interleave(256)[:m8.numel()]
        assert ((x8 - g32).abs() <= share * 1.01 * g32.abs() + 2.0 ** -9 * unit).all()


def a_slices(a, b):
    """a's flat moments cut as b's list is."""
    base = b.m.data_ptr()
    for t in b.opt.tensors["m"]:
        at = t.data_ptr() - base
        yield a.m[at:at + t.numel()]


def test_8_bit_states_train_and_replay():
    """Ten steps on one batch: a replayed graph gives the eager steps' bits, another seed other
    bits, and the states take a quarter of the memory."""
    shape = ragged_shape()
    blocks, head, x, tg = synth.make_model_inputs(shape, 8)
    ways = []
    for mode, seed in (("eager", 3), ("graph", 3), ("eager", 4)):
        tr = DecoderTrainer(shape, state_bits=8, state_seed=seed)
        tr.load(blocks, head)
        first = tr.train_step(x.cuda(), tg.cuda()).clone()
        for _ in range(9):
            last = tr.train_step(x.cuda(), tg.cuda()) if mode == "eager" else \
                tr.train_step_graph(x.cuda(), tg.int().cuda())
        torch.cuda.synchronize()
        assert last.isfinite().all() and first.isfinite().all()
        ways.append(tr)
    for name in ("w", "m", "v", "wb"):
        assert torch.equal(getattr(ways[0], name), getattr(ways[1], name)), name
    assert not torch.equal(ways[0].m, ways[2].m)
    assert ways[0].m.element_size() == 1
    ways[0].reset_optimizer()
    assert int(ways[0].m.count_nonzero()) == 0
    assert all(int(s.count_nonzero()) == 0 for s in ways[0].opt.tensors["v_scale"])
    with pytest.raises(ValueError, match="state_bits"):
        DecoderTrainer(shape, state_bits=16)


def test_adapters_with_8_bit_states():
    shape = synth.WORKLOADS["q4b_nf4"].replace(hidden=256, n_heads=4, n_kv_heads=1, head_dim=64,
                                               intermediate=512, seq=128, vocab=256)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(shape.tokens, shape.hidden, generator=gen, device="cuda")
    dy = 1e-3 * torch.randn(shape.tokens, shape.hidden, generator=gen, device="cuda")
    ways = {}
    for key, bits, graph in (("a", 32, False), ("b", 8, False), ("c", 8, True)):
        tr = Nf4LoraTrainer(shape, rank=8, state_bits=bits)
        tr.init_random(5, b_std=0.02)
        tr.train_step(x, dy)
        if key == "a":
            ways["first"] = tr.lora.clone()
        if key == "b":
            tol = 2.0 ** -20 * tr.optim["lr"] + 4 * 2.0 ** -24 * tr.lora.abs()
            assert ((tr.lora - ways["first"]).abs() <= tol).all()
        for _ in range(5):
            tr.train_step_graph(x, dy) if graph else tr.train_step(x, dy)
        torch.cuda.synchronize()
        ways[key] = tr
    assert torch.equal(ways["b"].lora, ways["c"].lora) and torch.equal(ways["b"].v, ways["c"].v)
    assert ways["b"].lora.isfinite().all()
    with pytest.raises(ValueError, match="state_bits"):
        Nf4LoraTrainer(shape, rank=8, state_bits=4)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_policy_step_of_a_linear_head(bits):
    """Two steps of: logits, log probabilities and entropies, a policy-gradient loss with an
    entropy bonus and a log-sum-exp penalty, its gradient, the head's weight gradient, clip,
    AdamW; each step against 64 bits from the same weights and states."""
    T, V, H = 192, 2048, 128
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    w = 0.1 * torch.randn(V, H, generator=gen, device="cuda")
    bias = torch.zeros(V, device="cuda")  # a second, small tensor: a prior over tokens
    tg = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    tg[:T // 4] = -1  # prompt positions
    adv = torch.randn(T, generator=gen, device="cuda")
    wb = w.bfloat16()
    z, dz = torch.empty(T, V, device="cuda"), torch.empty(T, V, device="cuda",
                                                         dtype=torch.bfloat16)
    gw, gb = torch.empty(V, H, device="cuda"), torch.empty(V, device="cuda")
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    logp, ent, lse, stats = f(T), f(T), f(T), f(T, 2)
    dt = torch.float32 if bits == 32 else torch.uint8
    states = {k: [torch.zeros(n, dtype=dt, device="cuda") for n in (V * H, V)] for k in "mv"}
    scales = {} if bits == 32 else {k: [f(-(-n // 256)) for n in (V * H, V)]
                                    for k in ("m_scale", "v_scale")}
    lst = rdt.OptTensors(g=[gw, gb], w=[w, bias], w_bf16=[wb, bias.bfloat16()], lr=[1e-3, 1e-2],
                         weight_decay=[0.1, 0.0], **states, **scales)
    ws = torch.empty(rdt.tensors_sq_sum_workspace_bytes(lst), dtype=torch.uint8, device="cuda")
    sumsq = torch.zeros(1, dtype=torch.float64, device="cuda")
    scale, bad = torch.ones(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    n = T - T // 4
    up = [-adv / n, torch.full((T,), -0.01 / n, device="cuda"),
          torch.empty(T, device="cuda")]
    for step in (1, 2):
        before = wb.double().clone(), bias.double().clone(), w.double().clone()
        rdt.gemm(x, 0, wb, 0, T, V, H, z)
        z += bias
        rdt.token_logprobs(z, targets=tg, logp=logp, entropy=ent, lse=lse, stats=stats)
        torch.mul(lse, 2e-4 / n, out=up[2])  # of 1e-4 lse^2
        rdt.token_logprobs_backward(z, tg, stats, dz, d_logp=up[0], entropy=ent, d_entropy=up[1],
                                    d_lse=up[2])
        rdt.gemm(dz, 1, x, 1, V, H, T, gw)
        torch.sum(dz.float(), 0, out=gb)
        rdt.tensors_sq_sum(lst, sumsq, ws)
        rdt.clip_scale(sumsq, 0.05, scale, bad)
        rdt.tensors_adamw(lst, step, 0.9, 0.95, 1e-8, scale=scale, skip=bad, seed=9)
        # the same in 64 bits, differentiated automatically
        W, B = before[0].requires_grad_(), before[1].requires_grad_()
        lp = torch.log_softmax(x.double() @ W.t() + B, 1)
        alive = (tg >= 0).double()
        chosen = lp.gather(1, tg.long().clamp(min=0)[:, None])[:, 0]
        h = -(lp.exp() * lp).sum(1)
        big = torch.logsumexp(x.double() @ W.t() + B, 1)
        loss = ((-adv.double() * chosen - 0.01 * h + 1e-4 * big ** 2) * alive).sum() / n
        loss.backward()
        # dz is rounded to bf16 (2^-9 of each on average) before the product
        assert rel_l2(to_np(gw), W.grad.cpu().numpy()) < 2.0 ** -8
        assert rel_l2(to_np(gb), B.grad.cpu().numpy()) < 2.0 ** -8
        norm = float((gw.double().square().sum() + gb.double().square().sum()).sqrt())
        assert abs(float(sumsq) - norm ** 2) < 1e-12 * norm ** 2
        assert abs(float(scale) - min(1.0, 0.05 / norm)) < 1e-6 and int(bad) == 0
        if step == 1:  # states start at zero: the update is lr sign-like, decay aside
            g = gw.double() * float(scale)
            want = before[2] - 1e-3 * (g / (g.abs() + 1e-8) + 0.1 * before[2])
            assert (w.double() - want).abs().max() < 1e-3 * 2.0 ** -18 + 2.0 ** -22
        assert torch.equal(wb, w.bfloat16())


@pytest.mark.parametrize("captured", [False, True])
def test_calls_behind_events_of_another_stream(captured):
    """Each call follows one of its own kind in its stream and an event of a second stream, whose
    kernels, still running when the call is launched, write what it reads; eager and captured."""
    rows, vocab, sizes = 200, 5003, [300, 5, 2048] * 140
    gen = torch.Generator(device="cuda").manual_seed(20)
    z0 = torch.randn(rows, vocab, generator=gen, device="cuda")
    tg = torch.randint(0, vocab, (rows,), generator=gen, device="cuda", dtype=torch.int32)
    big = torch.randn(4096, 4096, generator=gen, device="cuda")
    p = tensors.Problem(sizes, 8, seed=21)
    g0 = p.g.buf.clone()
    lst, f = p.list(), lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    ws = torch.empty(rdt.tensors_sq_sum_workspace_bytes(lst), dtype=torch.uint8, device="cuda")
    sumsq, scale = torch.zeros(1, dtype=torch.float64, device="cuda"), f(1)
    z, d, slow = f(rows, vocab), f(rows, vocab), f(4096, 4096)
    out = dict(logp=f(rows), entropy=f(rows), lse=f(rows), stats=f(rows, 2))
    up, side = torch.ones(rows, device="cuda"), torch.cuda.Stream()

    def behind(write):
        """Runs `write` on the second stream behind a long kernel; this stream waits for it."""
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.mm(big, big, out=slow)
            write()
        torch.cuda.current_stream().wait_stream(side)

    def calls():
        rdt.token_logprobs(z, targets=tg, **out)
        behind(lambda: torch.mul(z0, 2.0, out=z))
        rdt.token_logprobs(z, targets=tg, **out)
        behind(lambda: torch.mul(out["logp"], -0.1, out=up))
        rdt.token_logprobs_backward(z, tg, out["stats"], d, d_logp=up)
        behind(lambda: torch.mul(g0, 0.5, out=p.g.buf))
        rdt.tensors_sq_sum(lst, sumsq, ws)
        behind(lambda: torch.rsqrt(sumsq, out=sumsq))
        scale.copy_(sumsq)
        rdt.tensors_adamw(lst, 2, 0.9, 0.95, 1e-8, scale=scale, seed=1)
        behind(lambda: scale.mul_(0.5))
        rdt.tensors_adamw(lst, 3, 0.9, 0.95, 1e-8, scale=scale, seed=1)

    old = p.snapshot()
    calls()
    torch.cuda.synchronize()
    # one by one, with nothing under way
    ref = {k: torch.zeros_like(x) for k, x in out.items()}
    d_ref = f(rows, vocab)
    rdt.token_logprobs(z0 * 2.0, targets=tg, **ref)
    torch.cuda.synchronize()
    rdt.token_logprobs_backward(z0 * 2.0, tg, ref["stats"], d_ref, d_logp=ref["logp"] * -0.1)
    q = tensors.Problem(sizes, 8, seed=21)
    q.g.buf.copy_(g0 * 0.5)
    total = torch.zeros(1, dtype=torch.float64, device="cuda")
    torch.cuda.synchronize()
    rdt.tensors_sq_sum(q.list(), total, ws)
    torch.cuda.synchronize()
    s1 = total.rsqrt().float()
    for step, s in ((2, s1), (3, s1 * 0.5)):
        rdt.tensors_adamw(q.list(), step, 0.9, 0.95, 1e-8, scale=s, seed=1)
        torch.cuda.synchronize()

    def check():
        assert all(torch.equal(out[k], ref[k]) for k in ref) and torch.equal(d, d_ref)
        for k in ("w", "m", "v", "ms", "vs", "wb"):
            assert torch.equal(getattr(p, k).buf, getattr(q, k).buf), k

    check()
    if not captured:
        return
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(2):
        for k, parts in old.items():
            for a, b in zip(getattr(p, k).parts, parts):
                a.copy_(b)
        for x in (z, d, p.g.buf, *out.values()):
            x.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check()


@pytest.mark.parametrize("bits,seed", [(32, None), (8, None), (8, 9)])
def test_the_updates_of_three_policy_steps(bits, seed):
    """The steps above, with every update checked: weight and bias, their moments (codes and
    scales), the bf16 copies, at the first step from zero states and at the next ones from the
    states the last one left; bit for bit by the documented operations and, with the tolerances
    of the many-tensor tests, in 64 bits. The bias has a rate and a decay of its own."""
    T, V, H = 192, 2048, 128
    gen = torch.Generator(device="cuda").manual_seed(16)
    x = torch.randn(T, H, generator=gen, device="cuda").bfloat16()
    tg = torch.randint(0, V, (T,), generator=gen, device="cuda", dtype=torch.int32)
    tg[:T // 4] = -1
    up = torch.randn(T, generator=gen, device="cuda") / T
    h_up = torch.full((T,), -0.01 / T, device="cuda")
    p = tensors.Problem([V * H, V], bits, seed=17)
    p.lr, p.wd = [1e-3, 2e-2], [0.1, 0.0]
    for arena in (p.m, p.v, p.ms, p.vs):
        for part in arena.parts:
            part.zero_()
    for w, wb in zip(p.w.parts, p.wb.parts):
        wb.copy_(w)
    z = torch.empty(T, V, device="cuda")
    dz = torch.empty(T, V, device="cuda", dtype=torch.bfloat16)
    f = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    logp, ent, stats = f(T), f(T), f(T, 2)
    lst = p.list()
    ws = torch.empty(rdt.tensors_sq_sum_workspace_bytes(lst), dtype=torch.uint8, device="cuda")
    sumsq = torch.zeros(1, dtype=torch.float64, device="cuda")
    scale, bad = torch.ones(1, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    for step in (1, 2, 3):
        rdt.gemm(x, 0, p.wb.parts[0].view(V, H), 0, T, V, H, z)
        z += p.w.parts[1]
        rdt.token_logprobs(z, targets=tg, logp=logp, entropy=ent, stats=stats)
        rdt.token_logprobs_backward(z, tg, stats, dz, d_logp=up, entropy=ent, d_entropy=h_up)
        rdt.gemm(dz, 1, x, 1, V, H, T, p.g.parts[0].view(V, H))
        torch.sum(dz.float(), 0, out=p.g.parts[1])
        rdt.tensors_sq_sum(lst, sumsq, ws)
        rdt.clip_scale(sumsq, 0.05, scale, bad)
        assert 0 < float(scale) <= 1 and int(bad) == 0
        assert all(int(part.count_nonzero()) > part.numel() // 2 for part in p.g.parts)
        before = [w.clone() for w in p.w.parts]
        tensors.check_step(p, step, scale=float(scale), seed=seed, skip=bad)
        assert all(not torch.equal(a, b) for a, b in zip(before, p.w.parts))
