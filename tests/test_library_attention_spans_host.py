"""Refusals of the per-head norm with rotation and of the attention over spans: bad arguments
return RDT_EINVAL with a message before any device is touched (no GPU needed: the pointers are
never followed)."""
import ctypes

import pytest
import torch

from resident_decoder_trainer_gb300 import build, rdt

P = ctypes.c_void_p
A = 4096  # an aligned address that no call may read
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return rdt.lib()


def einval(lib, status, text):
    assert status == rdt.RDT_EINVAL, (status, lib.rdt_last_error())
    assert text in lib.rdt_last_error(), lib.rdt_last_error()


def heads(n, d=64, at=A, ts=None, hs=None):
    return ctypes.byref(rdt.Heads(at, n * d if ts is None else ts, d if hs is None else hs))


SECTIONS = (ctypes.c_int32 * 3)(8, 12, 12)
NORM = dict(tokens=5, nh=4, nkv=2, d=64, q=heads(4), k=heads(2), dtype=1, gain_q=P(A),
            gain_k=P(A), eps=1e-6, positions=P(A), axes=3, sections=SECTIONS, theta=1e4,
            q_out=heads(4, at=2 * A), k_out=heads(2, at=3 * A), out_dtype=1, stream=None)
BAD_NORM = [
    (dict(tokens=-1), b"tokens"), (dict(nh=-1), b"n_heads"), (dict(nh=0, nkv=0), b"n_heads"),
    (dict(nh=4097), b"n_heads"), (dict(d=24), b"head_dim"), (dict(d=272), b"head_dim"),
    (dict(d=0), b"head_dim"), (dict(dtype=3), b"dtypes"), (dict(out_dtype=-1), b"dtypes"),
    (dict(q=None), b"null"), (dict(k=heads(2, at=None)), b"null"),
    (dict(q=heads(4, at=A + 8)), b"aligned"), (dict(q=heads(4, ts=260)), b"multiples"),
    (dict(q=heads(4, ts=32)), b"strides"), (dict(k=heads(2, hs=32)), b"strides"),
    (dict(q=heads(4, ts=-256)), b"strides"), (dict(q=heads(4, ts=1 << 40)), b"strides"),
    (dict(q_out=heads(4, at=2 * A, ts=64)), b"overlaps itself"),
    (dict(k_out=heads(2, at=2 * A, ts=64, hs=64)), b"overlaps itself"),
    (dict(q_out=heads(4), out_dtype=0), b"place"),
    (dict(q_out=heads(4, ts=512)), b"place"),
    (dict(q_out=heads(4, at=3 * A)), b"other"), (dict(k=heads(2, at=2 * A)), b"other"),
    (dict(q=heads(4, at=3 * A)), b"other"),
    (dict(gain_q=P(A + 2)), b"aligned"), (dict(positions=P(A + 1)), b"aligned"),
    (dict(eps=-1.0), b"eps"), (dict(eps=INF), b"eps"), (dict(eps=NAN), b"eps"),
    (dict(axes=0), b"axes"), (dict(axes=5), b"axes"), (dict(sections=None), b"sections"),
    (dict(sections=(ctypes.c_int32 * 3)(8, 8, 8)), b"sections"),
    (dict(sections=(ctypes.c_int32 * 3)(-8, 20, 20)), b"section"),
    (dict(theta=0.0), b"theta"), (dict(theta=-1.0), b"theta"), (dict(theta=INF), b"theta"),
    (dict(theta=NAN), b"theta")]


@pytest.mark.parametrize("change,text", BAD_NORM)
def test_norm_refuses(lib, change, text):
    einval(lib, lib.rdt_qk_norm_rope(*{**NORM, **change}.values()), text)


GRAD = dict(tokens=5, nh=4, nkv=2, d=64, q=heads(4), k=heads(2), dtype=1, gain_q=P(A),
            gain_k=P(A), eps=1e-6, positions=P(A), axes=3, sections=SECTIONS, theta=1e4,
            d_q=heads(4, at=4 * A), d_k=heads(2, at=5 * A), d_dtype=1, dq=heads(4, at=2 * A),
            dk=heads(2, at=3 * A), out_dtype=1, d_gain_q=P(A), d_gain_k=P(A), accumulate=0,
            ws=P(A), ws_bytes=1 << 30, stream=None)


@pytest.mark.parametrize("change,text", [
    (dict(d_dtype=7), b"d_dtype"), (dict(d_q=None), b"null"), (dict(dk=None), b"null"),
    (dict(d_q=heads(4, at=4 * A + 4)), b"aligned"), (dict(gain_q=None), b"needs the gain"),
    (dict(d_gain_k=P(A + 1)), b"aligned"), (dict(ws=None), b"null"),
    (dict(ws=P(A + 64)), b"256-byte"), (dict(ws_bytes=64), b"workspace"),
    (dict(d_q=heads(4, at=2 * A, ts=512)), b"place"), (dict(d=20), b"head_dim"),
    (dict(d_q=heads(4, at=3 * A)), b"other"), (dict(d_k=heads(2, at=2 * A)), b"other"),
    (dict(dk=heads(2, at=2 * A)), b"other"),
    (dict(axes=7), b"axes"), (dict(theta=0.0), b"theta")])
def test_norm_backward_refuses(lib, change, text):
    einval(lib, lib.rdt_qk_norm_rope_backward(*{**GRAD, **change}.values()), text)


def test_no_tokens_is_fine(lib):
    assert lib.rdt_qk_norm_rope(*{**NORM, "tokens": 0, "q": None}.values()) == rdt.RDT_OK
    none = dict(tokens=0, d_gain_q=None, d_gain_k=None)
    assert lib.rdt_qk_norm_rope_backward(*{**GRAD, **none}.values()) == rdt.RDT_OK


ATTN = dict(queries=5, keys=9, nh=4, nkv=2, d=64, q=heads(4), k=heads(2), v=heads(2), lo=P(A),
            hi=P(A), scale=0.125, softcap=0.0, o=heads(4, at=2 * A), lse=P(A), ws=P(A),
            ws_bytes=1 << 40, stream=None)
BAD_SHAPES = [
    (dict(queries=-1), b"queries"), (dict(keys=-1), b"keys"), (dict(queries=(1 << 30) + 1), b"2^30"),
    (dict(nh=0), b"n_heads"), (dict(nkv=0), b"n_heads"), (dict(nkv=3), b"n_heads"),
    (dict(nh=1, nkv=2), b"n_heads"), (dict(nh=8192, nkv=4096), b"n_heads"),
    (dict(nh=258, nkv=2), b"128 query heads"), (dict(d=8), b"head_dim"), (dict(d=40), b"head_dim"),
    (dict(d=144), b"head_dim"), (dict(scale=0.0), b"scale"), (dict(scale=-1.0), b"scale"),
    (dict(scale=9e-7), b"scale"), (dict(scale=2e6), b"scale"),
    (dict(softcap=1e-6), b"softcap"), (dict(softcap=2e4), b"softcap"),
    (dict(scale=INF), b"scale"), (dict(scale=NAN), b"scale"), (dict(softcap=-1.0), b"softcap"),
    (dict(softcap=INF), b"softcap"), (dict(softcap=NAN), b"softcap"),
    (dict(lo=P(A + 2)), b"aligned"), (dict(hi=P(A + 1)), b"aligned"),
    (dict(lse=P(A + 2)), b"aligned"), (dict(q=None), b"null"), (dict(k=heads(2, at=None)), b"null"),
    (dict(v=heads(2, at=A + 2)), b"aligned"), (dict(q=heads(4, ts=252)), b"strides"),
    (dict(k=heads(2, ts=132)), b"multiples"), (dict(v=heads(2, hs=60)), b"strides")]


@pytest.mark.parametrize("change,text", BAD_SHAPES + [
    (dict(o=None), b"null"), (dict(o=heads(4, at=2 * A, ts=64)), b"overlaps itself"),
    (dict(o=heads(4)), b"at an input's place")])
def test_attention_refuses(lib, change, text):
    einval(lib, lib.rdt_attention(*{**ATTN, **change}.values()), text)


BACK = dict(queries=5, keys=9, nh=4, nkv=2, d=64, q=heads(4), k=heads(2), v=heads(2), o=heads(4),
            lse=P(A), d_o=heads(4), d_lse=None, lo=P(A), hi=P(A), scale=0.125, softcap=0.0,
            dq=heads(4, at=2 * A), dk=heads(2, at=3 * A), dv=heads(2, at=4 * A), ws=P(A),
            ws_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("change,text", BAD_SHAPES + [
    (dict(lse=None), b"null"), (dict(o=None), b"null"), (dict(d_o=None), b"null"),
    (dict(d_lse=P(A + 1)), b"aligned"), (dict(dq=heads(4, at=2 * A, ts=64)), b"overlaps itself"),
    (dict(dk=None), b"null"), (dict(dv=heads(2, at=4 * A, hs=0)), b"strides"),
    (dict(dq=heads(4)), b"at an input's place"), (dict(dk=heads(2)), b"at an input's place"),
    (dict(dv=heads(2)), b"at an input's place")])
def test_attention_backward_refuses(lib, change, text):
    einval(lib, lib.rdt_attention_backward(*{**BACK, **change}.values()), text)


def test_workspaces(lib):
    for backward in (0, 1):
        n = rdt.attention_workspace_bytes(4096, 4096, 32, 8, 128, backward=bool(backward))
        assert n % 256 == 0
        assert lib.rdt_attention_workspace_bytes(5, 9, 4, 3, 64, backward) == 0
        if n:
            call = lib.rdt_attention_backward if backward else lib.rdt_attention
            base = {**(BACK if backward else ATTN), "queries": 4096, "keys": 4096, "nh": 32,
                    "nkv": 8, "d": 128}
            for x in base:
                if base[x] is not None and x in ("q", "o", "d_o", "dq"):
                    base[x] = heads(32, 128, at=A if x == "q" else 2 * A)
                elif x in ("k", "v", "dk", "dv"):
                    base[x] = heads(8, 128, at=A if x in ("k", "v") else 3 * A)
            for change, text in ((dict(ws=None), b"null"), (dict(ws=P(A + 16)), b"256-byte"),
                                 (dict(ws_bytes=n - 1), b"workspace")):
                einval(lib, call(*{**base, **change}.values()), text)


def test_nothing_to_do_is_fine(lib):
    none = dict(queries=0, q=None, o=None, lse=None)
    assert lib.rdt_attention(*{**ATTN, **none}.values()) == rdt.RDT_OK
    none = dict(queries=0, keys=0, q=None, k=None, v=None, o=None, dq=None, dk=None, dv=None)
    assert lib.rdt_attention_backward(*{**BACK, **none}.values()) == rdt.RDT_OK


def test_bindings_refuse_what_is_not_on_the_device(lib):
    x = torch.zeros(3, 2, 16, dtype=torch.bfloat16)
    for call in (lambda: rdt.qk_norm_rope(x, x, x, x), lambda: rdt.attention(x, x, x, x),
                 lambda: rdt.qk_norm_rope_backward(x, x, x, x, x, x),
                 lambda: rdt.attention_backward(x, x, x, x, None, x, x, x, x)):
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            call()
    for q, k in ((None, None), (x[0], x), (x, x[0])):
        with pytest.raises(ValueError):
            rdt.qk_norm_rope(q, k, q, k)
