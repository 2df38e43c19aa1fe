"""Refusals of the token log-probability and many-tensor calls: bad arguments
return RDT_EINVAL with a message before any device is touched (no GPU needed:
the pointers are never followed)."""
import ctypes

import pytest
import torch

from resident_decoder_trainer_gb300 import build, rdt, synth

P = ctypes.c_void_p
A = 4096  # an aligned address that no call may read


@pytest.fixture(scope="module")
def lib():
    build.build()
    return rdt.lib()


def einval(lib, status, text):
    assert status == rdt.RDT_EINVAL, (status, lib.rdt_last_error())
    assert text in lib.rdt_last_error(), lib.rdt_last_error()


FWD = dict(logits=P(A), dtype=0, ld=8, rows=2, vocab=8, scale=1.0, targets=P(A), logp=P(A),
           entropy=None, lse=None, stats=None, top=0, top_ids=None, top_logp=None, stream=None)


@pytest.mark.parametrize("change,text", [
    (dict(dtype=3), b"dtype"), (dict(dtype=-1), b"dtype"), (dict(rows=-1), b"rows"),
    (dict(vocab=0), b"vocab"), (dict(ld=7), b"ld"), (dict(scale=0.0), b"logit_scale"),
    (dict(scale=-1.0), b"logit_scale"), (dict(scale=float("inf")), b"logit_scale"),
    (dict(scale=float("nan")), b"logit_scale"), (dict(logits=None), b"null"),
    (dict(logits=P(A + 2)), b"aligned"), (dict(dtype=1, logits=P(A + 1)), b"aligned"),
    (dict(targets=None), b"targets"), (dict(logp=None), b"no output"),
    (dict(top=33, top_ids=P(A), top_logp=P(A)), b"top"), (dict(top=-1), b"top"),
    (dict(top=4), b"top_ids"), (dict(top=4, top_ids=P(A)), b"top_ids"),
    (dict(top_logp=P(A)), b"top_ids"), (dict(logp=P(A + 1)), b"aligned"),
    (dict(stats=P(A + 4)), b"aligned"), (dict(targets=P(A + 2)), b"aligned")])
def test_token_logprobs_refuses(lib, change, text):
    einval(lib, lib.rdt_token_logprobs(*{**FWD, **change}.values()), text)


def test_token_logprobs_of_no_rows_is_fine(lib):
    assert lib.rdt_token_logprobs(*{**FWD, "rows": 0, "logits": None}.values()) == rdt.RDT_OK


BWD = dict(logits=P(A), dtype=0, ld=8, rows=2, vocab=8, scale=1.0, targets=P(A), stats=P(A),
           entropy=P(A), d_logp=P(A), d_entropy=P(A), d_lse=None, d_logits=P(2 * A), d_dtype=1,
           ld_d=8, stream=None)


@pytest.mark.parametrize("change,text", [
    (dict(d_dtype=4), b"d_dtype"), (dict(ld_d=7), b"ld_d"), (dict(stats=None), b"null"),
    (dict(d_logits=None), b"null"), (dict(d_logp=None, d_entropy=None), b"upstream"),
    (dict(targets=None), b"targets"), (dict(entropy=None), b"entropy"),
    (dict(stats=P(A + 4)), b"aligned"), (dict(d_logits=P(2 * A + 1)), b"aligned"),
    (dict(logits=None), b"null"), (dict(vocab=0), b"vocab"), (dict(scale=0.0), b"logit_scale"),
    # over the logits, but not them: another type, another stride, another place
    (dict(d_logits=P(A)), b"overlaps"), (dict(d_logits=P(A), d_dtype=0, ld_d=9), b"overlaps"),
    (dict(d_logits=P(A + 8), d_dtype=0), b"overlaps")])
def test_token_logprobs_backward_refuses(lib, change, text):
    einval(lib, lib.rdt_token_logprobs_backward(*{**BWD, **change}.values()), text)


def test_token_logprobs_backward_of_no_rows_is_fine(lib):
    assert lib.rdt_token_logprobs_backward(*{**BWD, "rows": 0}.values()) == rdt.RDT_OK


def test_head_logprobs_refuses(lib):
    s = synth.WORKLOADS["tiny"]
    cfg = rdt.Config.from_shape(s)
    size = rdt.head_logprobs_workspace_bytes(cfg, 32)
    assert size >= 32 * s.vocab * 4 + 32 * s.hidden * 2 and size % 256 == 0
    assert rdt.head_logprobs_workspace_bytes(cfg, 0) == 0
    big = rdt.Config.from_shape(synth.WORKLOADS["q4b_full"])
    assert rdt.head_logprobs_workspace_bytes(big, 1 << 20) < (1 << 30) + (1 << 20) * (2560 * 2 + 8)
    base = dict(cfg=ctypes.byref(cfg), tokens=32, h=P(A), gamma=P(A), w=P(A), scale=1.0,
                targets=P(A), logp=P(A), entropy=None, lse=None, top=0, ids=None, top_logp=None,
                ws=P(A), ws_bytes=size, stream=None)
    for change, text in ((dict(tokens=0), b"tokens"), (dict(h=None), b"null"),
                         (dict(w=P(A + 8)), b"aligned"), (dict(ws=P(A + 16)), b"aligned"),
                         (dict(ws_bytes=size - 1), b"workspace"), (dict(targets=None), b"targets"),
                         (dict(logp=None), b"no output"), (dict(top=40, ids=P(A), top_logp=P(A)),
                                                           b"top"),
                         (dict(scale=0.0), b"logit_scale")):
        einval(lib, lib.rdt_head_logprobs(*{**base, **change}.values()), text)
    bad = rdt.Config.from_shape(s.replace(hidden=40))
    assert lib.rdt_head_logprobs(*{**base, "cfg": ctypes.byref(bad)}.values()) == rdt.RDT_EINVAL
    assert rdt.head_logprobs_workspace_bytes(bad, 32) == 0


def entries(*changes, **first):
    e = (rdt.OptTensor * max(1, len(changes)))()
    for i, change in enumerate(changes):
        base = dict(w=A * (i + 1), g=A, m=A, v=A, m_scale=A, v_scale=A, w_bf16=None, n=100, lr=1e-3,
                    weight_decay=0.0)
        for k, x in {**base, **change}.items():
            setattr(e[i], k, x)
    return e


def adamw(lib, e, count, **change):
    base = dict(g_dtype=0, bits=8, seed=-1, scale=None, skip=None, step=1, step_dev=None, b1=0.9,
                b2=0.95, eps=1e-8, stream=None)
    return lib.rdt_tensors_adamw(e, count, *{**base, **change}.values())


@pytest.mark.parametrize("change,text", [
    (dict(g_dtype=2), b"g_dtype"), (dict(bits=16), b"state_bits"), (dict(seed=1 << 32), b"seed"),
    (dict(step=0), b"step"), (dict(b1=1.0), b"beta"), (dict(b2=-0.1), b"beta"),
    (dict(b2=float("nan")), b"beta"), (dict(eps=-1.0), b"eps"), (dict(eps=0.0), b"eps"), (dict(scale=P(2)), b"aligned"),
    (dict(step_dev=P(6)), b"aligned")])
def test_tensors_adamw_refuses(lib, change, text):
    einval(lib, adamw(lib, entries({}), 1, **change), text)


@pytest.mark.parametrize("entry,text", [
    (dict(n=-1), b"n of a tensor"), (dict(n=1 << 41), b"n of a tensor"), (dict(g=None), b"null"),
    (dict(w=None), b"null"), (dict(m=None), b"null"), (dict(v=None), b"null"),
    (dict(m_scale=None), b"null"), (dict(v_scale=None), b"null"), (dict(g=A + 8), b"aligned"),
    (dict(w=A + 4), b"aligned"), (dict(v=A + 8), b"aligned"), (dict(w_bf16=A + 2), b"aligned"),
    (dict(m_scale=A + 2), b"aligned")])
def test_tensors_adamw_refuses_entries(lib, entry, text):
    einval(lib, adamw(lib, entries({}, entry), 2), text)


def test_tensors_adamw_refuses_overlapping_tensors(lib):
    einval(lib, adamw(lib, entries(dict(w=A), dict(w=A)), 2), b"overlap")
    einval(lib, adamw(lib, entries(dict(w=A + 16, n=4), dict(w=A, n=5)), 2), b"overlap")
    einval(lib, adamw(lib, entries(dict(w=A), dict(w=4 * A), dict(w=A + 384)), 3), b"overlap")


def test_empty_lists_and_tensors_launch_nothing(lib):
    assert adamw(lib, None, 0) == rdt.RDT_OK
    e = entries(dict(n=0, w=None, g=None, m=None, v=None))
    assert adamw(lib, e, 1) == rdt.RDT_OK
    einval(lib, adamw(lib, None, 1), b"null")
    einval(lib, adamw(lib, e, -1), b"count")


def test_tensors_sq_sum_refuses(lib):
    e = entries({}, {})
    size = lib.rdt_tensors_sq_sum_workspace_bytes(e, 2)
    assert size > 0
    assert lib.rdt_tensors_sq_sum_workspace_bytes(entries(*[{}] * 1000), 1000) > size
    for args, text in (((e, 2, 5, P(A), P(A), size, None), b"g_dtype"),
                       ((e, 2, 0, None, P(A), size, None), b"null"),
                       ((e, 2, 0, P(A), None, size, None), b"null"),
                       ((e, 2, 0, P(A + 4), P(A), size, None), b"aligned"),
                       ((e, 2, 0, P(A), P(A + 4), size, None), b"aligned"),
                       ((e, 2, 0, P(A), P(A), size - 8, None), b"workspace"),
                       ((e, -1, 0, P(A), P(A), size, None), b"count"),
                       ((None, 2, 0, P(A), P(A), size, None), b"null")):
        einval(lib, lib.rdt_tensors_sq_sum(*args), text)
    assert lib.rdt_tensors_sq_sum_workspace_bytes(entries(dict(n=-1)), 1) == 0


@pytest.mark.parametrize("sizes", [[1 << 40] * 400, [(1 << 40) - 5, 3] * 900, [1 << 33] * 32,
                                   [1 << 39, 1 << 40] * 16, [300] * 1203, [(1 << 40) + 0] * 3])
def test_the_workspace_of_the_squared_sum_has_room_for_every_launch(lib, sizes):
    """A launch ends at 400 entries (32 for short lists) or where the next entry's tiles of 2048
    would make it more than 2^30: then a CTA's next tile (its own, and at most 4 x 2048 chunks of
    two behind) fits 32 bits. Each launch has up to 2048 partial sums."""
    most, launches, held, tiles = 32 if len(sizes) <= 32 else 400, 1, 0, 0
    for n in sizes:
        more = -(-n // 2048)
        if held and (held == most or tiles + more > 1 << 30):
            launches, held, tiles = launches + 1, 0, 0
        held, tiles = held + 1, tiles + more
        assert tiles <= 1 << 30
    e = entries(*[dict(n=n) for n in sizes])
    size = lib.rdt_tensors_sq_sum_workspace_bytes(e, len(sizes))
    assert size >= launches * 2048 * 8
    assert size <= (3 * launches + 1) * 2048 * 8


def test_bindings_refuse_tensors_the_device_cannot_read():
    z = torch.zeros(2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        rdt.token_logprobs(z, entropy=torch.zeros(2))
    with pytest.raises(ValueError, match="CUDA"):
        rdt.OptTensors(g=[torch.zeros(4)])
    with pytest.raises(ValueError, match="gradients"):
        rdt.OptTensors(g=[torch.zeros(4, dtype=torch.float64)])
    empty = rdt.OptTensors(g=[])
    with pytest.raises(ValueError, match="seed"):
        rdt.tensors_adamw(empty, 1, 0.9, 0.95, 1e-8, seed=-1)


def test_bindings_refuse_workspaces_and_scalars_that_hold_less_than_they_seem():
    """The checks alone, on CPU tensors (device -1): an expanded workspace of one byte that
    claims a million, an empty scale that would count as none."""
    for t in (torch.empty(1, dtype=torch.uint8).expand(1 << 20),
              torch.empty(100, dtype=torch.uint8)[::2], torch.empty(4, 6).t()):
        with pytest.raises(ValueError, match="contiguous"):
            rdt._scratch(t, "ws", -1)
    ws = torch.empty(4, 6)
    assert rdt._scratch(ws, "ws", -1) == (ws.data_ptr(), 96)
    with pytest.raises(ValueError, match="no element"):
        rdt._scalar(torch.empty(0), "scale", (torch.float32,), -1)
    with pytest.raises(ValueError, match="type"):
        rdt._scalar(torch.empty(1), "skip", (torch.int32,), -1)
    one = torch.ones(1)
    assert rdt._scalar(one, "scale", (torch.float32,), -1) == one.data_ptr()


@pytest.mark.parametrize("rows,vocab", [((1 << 32) + 1, 8), (1 << 31, 8), (1, (1 << 32) + 8),
                                        (3, (1 << 30) + 1)])
def test_bindings_refuse_sizes_that_do_not_fit_the_call(rows, vocab):
    """The C call takes 32-bit sizes: 2^32 + 1 rows must not become one."""
    with pytest.raises(ValueError, match="rows"):
        rdt._rows_of(torch.empty(rows, vocab, device="meta"), "logits", -1)


def test_the_random_rounding_numbers_are_uniform():
    """The 16-bit halves that decide the rounding (the header's function of seed, step,
    entry and element, restated here): uniform, and independent of their neighbours."""
    def mix(x):
        x = x ^ (x >> 16)
        x = (x * 0x3C6EF373) & 0xFFFFFFFF
        x = x ^ (x >> 14)
        x = (x * 0xBB67AE85) & 0xFFFFFFFF
        return x ^ (x >> 16)

    n = 1 << 18
    at = torch.arange(n)
    for seed, step, entry in ((0, 1, 0), (7, 2, 3), (2 ** 32 - 1, 100000, 999)):
        key = mix((mix((mix(step) + seed) & 0xFFFFFFFF) + entry) & 0xFFFFFFFF)
        x = mix(at ^ key)
        for half in (x & 0xFFFF, x >> 16):
            u = half.double() / 65536
            # standard errors: 0.289 / sqrt(n) for the mean, 1 / sqrt(n) for a correlation
            assert abs(u.mean() - 0.5) < 5 * 0.289 / n ** 0.5
            count = torch.bincount(half >> 8, minlength=256).double()
            chi = ((count - n / 256) ** 2 / (n / 256)).sum()
            assert chi < 255 + 6 * (2 * 255) ** 0.5
            v = u - 0.5
            for lag in (1, 8, 256):
                assert abs((v[:-lag] * v[lag:]).mean() * 12) < 5 / n ** 0.5
