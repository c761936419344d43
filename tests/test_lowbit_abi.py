"""What the 4-bit cache's calls, the read-back and the prefill over the low-bit caches refuse on the host, before
any CUDA work (no GPU needed)."""
import ctypes

import pytest
import torch

from paged_gqa_attention_gb300 import build as pa_build
from paged_gqa_attention_gb300 import ops
from test_window_abi import Addresses, BAD_WINDOWS, REFUSED, rope_args


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return ops.load()


def cache(p, bits):
    """Arguments of the cache's tensors behind the codes: scales, and exponents in 4 bits."""
    return dict(ks=p(10), vs=p(11)) | (dict(ke=p(12), ve=p(13)) if bits == 4 else {})


def call(fn, a, kw):
    assert set(kw) <= set(a), kw
    return fn(*(a | kw).values())


def append_args(p):
    return dict(shape=ops.SHAPE, kp=p(0), vp=p(1)) | cache(p, 4) | dict(
        k=p(2), v=p(3), bt=p(4), w=1, nb=1, cu=p(5), sl=p(6), seqs=1, tokens=1, ws=p(7), ws_bytes=1024, stream=None)


def read_args(p, bits):
    return dict(shape=ops.SHAPE, k_out=p(0), v_out=p(1), kp=p(2), vp=p(3)) | cache(p, bits) | dict(
        bt=p(4), w=1, nb=1, cu=p(5), first=p(6), seqs=1, rows=1, ws=p(7), ws_bytes=1024, stream=None)


def decode_args(p):
    return dict(shape=ops.SHAPE, out=p(0), lse=None, q=p(1), kp=p(2), vp=p(3)) | cache(p, 4) | dict(
        bt=p(4), w=1, nb=1, sl=p(6), batch=1, window=4, sinks=1, scale=0.1, split=0, ws=p(7), ws_bytes=1 << 20, stream=None)


def prefill_args(p, bits):
    return dict(shape=ops.SHAPE, out=p(0), lse=None, q=p(1), kp=p(2), vp=p(3)) | cache(p, bits) | dict(
        bt=p(4), w=1, nb=1, cu=p(5), sl=p(6), seqs=1, tokens=4, max_q=4, window=4, sinks=1, scale=0.1, ws=p(7),
        ws_bytes=1024, stream=None)


def nothing_and_misaligned(p, wide, narrow=()):
    """Every pointer missing, and off its alignment: of 16 bytes (wide) or 4 (narrow)."""
    return [{n: None} for n in (*wide, *narrow)] + [{n: p(20, 8)} for n in wide] + [{n: p(20, 2)} for n in narrow]


OTHER_SHAPES = [ops.pa_shape(32, 4, 128, 256), ops.pa_shape(32, 8, 64, 256), ops.pa_shape(32, 8, 128, 128)]


def test_append_refuses(lib):
    p = Addresses()
    a = append_args(p)
    for bad in (nothing_and_misaligned(p, ("kp", "vp", "ks", "vs", "ke", "ve", "k", "v", "ws"), ("bt", "cu", "sl"))
                + [dict(seqs=-1), dict(tokens=-1), dict(seqs=0), dict(w=0), dict(nb=0), dict(ws_bytes=255)]):
        assert call(lib.kv_append_fp4, a, bad) == 1, bad
    for shape in OTHER_SHAPES:
        assert call(lib.kv_append_fp4, a, dict(shape=shape)) == 2
    assert call(lib.kv_append_fp4, a, dict(seqs=0, tokens=0)) == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_read_refuses(lib, bits):
    p = Addresses()
    a, fn = read_args(p, bits), lib.paged_kv_read_fp8 if bits == 8 else lib.paged_kv_read_fp4
    wide = ("k_out", "v_out", "kp", "vp", "ks", "vs", "ws") + (("ke", "ve") if bits == 4 else ())
    for bad in (nothing_and_misaligned(p, wide, ("bt", "cu", "first"))
                + [dict(seqs=-1), dict(rows=-1), dict(seqs=0), dict(w=0), dict(nb=0), dict(w=1 << 23), dict(ws_bytes=255),
                   dict(k_out=p(20, 16)), dict(v_out=p(20, 16))]):
        assert call(fn, a, bad) == 1, bad
    for shape in OTHER_SHAPES:
        assert call(fn, a, dict(shape=shape)) == 2
    assert call(fn, a, dict(rows=0)) == 0 and call(fn, a, dict(rows=0, seqs=0)) == 0


def test_decode_refuses(lib):
    p = Addresses()
    a, fn = decode_args(p), lib.paged_attn_decode_fp4
    for bad in (nothing_and_misaligned(p, ("out", "q", "kp", "vp", "ks", "vs", "ke", "ve", "ws"), ("bt", "sl")) + BAD_WINDOWS
                + [dict(split=100), dict(split=128), dict(split=-256), dict(batch=-1), dict(batch=8193), dict(ws_bytes=100),
                   dict(w=0), dict(nb=0), dict(w=1 << 23), dict(lse=p(20, 2)), dict(scale=float("inf"))]):   # (0 is a scale)
        assert call(fn, a, bad) == 1, bad
    for shape in OTHER_SHAPES:
        assert call(fn, a, dict(shape=shape)) == 2
    assert call(fn, a, dict(batch=0)) == 0


@pytest.mark.parametrize("bits", [8, 4])
def test_prefill_refuses(lib, bits):
    p = Addresses()
    a, fn = prefill_args(p, bits), lib.paged_attn_prefill_fp8 if bits == 8 else lib.paged_attn_prefill_fp4
    wide = ("out", "q", "kp", "vp", "ks", "vs", "ws") + (("ke", "ve") if bits == 4 else ())
    for bad in (nothing_and_misaligned(p, wide, ("bt", "cu", "sl")) + BAD_WINDOWS
                + [dict(max_q=0), dict(max_q=5), dict(out=p(0, 16)), dict(seqs=0), dict(seqs=-1), dict(tokens=-1), dict(w=0),
                   dict(nb=0), dict(w=1 << 23), dict(ws_bytes=255), dict(lse=p(20, 2))]):
        assert call(fn, a, bad) == 1, bad
    for shape in OTHER_SHAPES:
        assert call(fn, a, dict(shape=shape)) == 2
    assert call(fn, a, dict(tokens=0, max_q=0)) == 0


@pytest.mark.parametrize("change,status", REFUSED, ids=[str(c[0])[:40] for c in REFUSED])
def test_rope_append_refuses(lib, change, status):
    """What paged_rope_append refuses, its form for the 4-bit cache does."""
    p = Addresses()
    kw = {}
    for n, x in change.items():
        if n in ("q_out", "q", "k", "v", "kp", "vp", "ws", "bt", "cu", "sl") and x is not None:
            x = p(20, x)
        kw[n] = p(21) if n in ("gq", "gk") and x is not None else x
    args = rope_args(p, **kw)
    tail = [p(i) for i in (10, 11, 12, 13)]
    assert lib.paged_rope_append_fp4(*args[:17], *tail, *args[17:]) == status


def test_rope_append_refuses_missing_scales(lib):
    p = Addresses()
    args = rope_args(p)
    for i in range(4):
        for bad in (None, p(20, 8)):
            tail = [p(10 + j) if j != i else bad for j in range(4)]
            assert lib.paged_rope_append_fp4(*args[:17], *tail, *args[17:]) == 1


def low(blocks=2):
    return ops.fp4_cache(blocks, "cpu")


def test_the_python_calls_say_what_is_wrong():
    """Host tensors, other types and other shapes: TypeError and ValueError, never a launch."""
    c4 = low()
    c8 = (torch.zeros(2, 256, 8, 128, dtype=torch.uint8),) * 2 + (torch.zeros(2, 8, 256),) * 2
    row = torch.zeros(1, 8, 128, dtype=torch.bfloat16)
    q = torch.zeros(1, 32, 128, dtype=torch.bfloat16)
    table, cu, lens = (torch.zeros(*n, dtype=torch.int32) for n in ((1, 2), (2,), (1,)))
    ws = torch.zeros(1024, dtype=torch.uint8)
    calls = [lambda c=c4: ops.kv_append_fp4(*c, row, row, table, cu, lens, ws),
             lambda c=c4: ops.paged_rope_append_fp4(q, row, row, *c, table, cu, lens, ws, rope_theta=1e6),
             lambda c=c4: ops.paged_kv_read_fp4(*c, table, cu, lens, 1, ws),
             lambda c=c8: ops.paged_kv_read_fp8(*c, table, cu, lens, 1, ws),
             lambda c=c4: ops.paged_attn_decode_fp4(q, *c, table, lens, ws),
             lambda c=c4: ops.paged_attn_prefill_fp4(q, *c, table, cu, lens, 1, ws),
             lambda c=c8: ops.paged_attn_prefill_fp8(q, *c, table, cu, lens, 1, ws)]
    for f in calls:
        with pytest.raises(ValueError, match="CUDA"):
            f()
        c = f.__defaults__[0]
        with pytest.raises((TypeError, ValueError)):   # (the codes' type, or a host tensor met before)
            f((c[0].float(), *c[1:]))


def test_the_compiled_binding_leaves_odd_cases_to_the_checks(lib):
    b = ops._usual()
    t = torch.zeros(1, 32, 128, dtype=torch.bfloat16)
    for fn, n in ((b.rope_append, 21), (b.append_fp4, 12), (b.kv_read, 13), (b.decode_fp4, 16), (b.prefill_low, 17)):
        for x in (None, t, 3, "x", torch.nn.Parameter(t)):
            assert fn(*[x] * n) is None
        assert fn() is None and fn(*[t] * (n + 1)) is None


def test_an_empty_4_bit_cache_reads_as_nan():
    codes, _, scales, _, exps, _ = low(3)
    assert codes.shape == (3, 256, 8, 64) and scales.shape == (3, 8, 256, 8) and exps.shape == (3, 8, 256)
    assert (exps == 255).all()
