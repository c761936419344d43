"""What the rotated append refuses on the host, before any CUDA work (no GPU needed)."""
import ctypes

import pytest
import torch

import definitions
from paged_gqa_attention_gb300 import build as pa_build
from paged_gqa_attention_gb300 import ops


@pytest.fixture(scope="module")
def lib():
    pa_build.build()
    return ops.load()


class Addresses:
    """16-byte aligned host addresses: no call below may get past validation."""

    def __init__(self):
        self.buf = (ctypes.c_uint8 * 16384)()
        self.base = (ctypes.addressof(self.buf) + 255) // 256 * 256

    def __call__(self, i, off=0):
        return ctypes.c_void_p(self.base + 256 * i + off)


def rope_args(p, **kw):
    a = dict(shape=ops.SHAPE, theta=1e6, positions=None, axes=1, pair_axis=None, gq=None, gk=None, eps=1e-6, q_out=p(0),
             q=p(1), qs=4096, k=p(2), ks=1024, v=p(3), vs=1024, kp=p(4), vp=p(5), bt=p(6), w=1, nb=1, cu=p(7), sl=p(8),
             seqs=1, tokens=1, ws=p(9), ws_bytes=1024, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    return list(a.values())


REFUSED = [
    (dict(shape=ops.pa_shape(32, 8, 64, 256)), 2),
    (dict(theta=1.0), 1), (dict(theta=-2.0), 1), (dict(theta=float("inf")), 1), (dict(theta=float("nan")), 1),
    (dict(axes=0), 1), (dict(axes=4), 1), (dict(axes=2), 1), (dict(axes=3, pair_axis=bytes(64)), 1),
    (dict(pair_axis=bytes([1] + [0] * 63)), 1), (dict(theta=0.0, pair_axis=bytes(64)), 1),
    (dict(w=(1 << 16) + 1), 1),                               # positions past 2^24
    (dict(w=1 << 23, theta=0.0), 1),
    (dict(eps=-1.0, gq=1, gk=1), 1), (dict(eps=float("nan"), gq=1, gk=1), 1),
    (dict(gq=1), 1), (dict(gk=1), 1),
    (dict(qs=4095), 1), (dict(qs=4088), 1), (dict(ks=1020), 1), (dict(vs=1028), 1), (dict(ks=0), 1), (dict(vs=-1024), 1),
    (dict(seqs=-1), 1), (dict(tokens=-1), 1), (dict(seqs=0), 1), (dict(w=0), 1), (dict(nb=0), 1),
    (dict(ws=None), 1), (dict(ws_bytes=255), 1),
    *[({n: None}, 1) for n in ("q_out", "q", "k", "v", "kp", "vp", "bt", "cu", "sl")],
    *[({n: 8}, 1) for n in ("q_out", "q", "k", "v", "kp", "vp", "ws")],
    *[({n: 2}, 1) for n in ("bt", "cu", "sl")],
]


@pytest.mark.parametrize("change,status", REFUSED, ids=[str(c[0])[:40] for c in REFUSED])
def test_rope_append_refuses(lib, change, status):
    p = Addresses()
    names = ("q_out", "q", "k", "v", "kp", "vp", "ws", "bt", "cu", "sl")
    kw = {}
    for n, x in change.items():
        if n in names and x is not None:
            x = p(20, x)                                      # misaligned by that many bytes
        if n in ("gq", "gk") and x is not None:
            x = p(21)
        kw[n] = x
    assert lib.paged_rope_append(*rope_args(p, **kw)) == status
    args = rope_args(p, **kw)
    assert lib.paged_rope_append_fp8(*args[:17], p(22), p(23), *args[17:]) == status


def test_rope_append_refuses_in_place_over_strided_rows(lib):
    p = Addresses()
    assert lib.paged_rope_append(*rope_args(p, q=p(0), qs=6144)) == 1
    args = rope_args(p)
    assert lib.paged_rope_append_fp8(*args[:17], None, p(23), *args[17:]) == 1
    assert lib.paged_rope_append_fp8(*args[:17], p(22), p(23, 8), *args[17:]) == 1


def test_rope_append_of_no_tokens_is_done(lib):
    p = Addresses()
    assert lib.paged_rope_append(*rope_args(p, tokens=0, seqs=0, q=None, k=None)) == 0


def test_rope_pair_axes():
    assert ops.rope_pair_axes((16, 24, 24)) == bytes([0] * 16 + [1] * 24 + [2] * 24)
    assert ops.rope_pair_axes((64,)) == bytes(64)
    x = ops.rope_pair_axes((24, 20, 20), interleaved=True)
    assert x[:60] == bytes([0, 1, 2] * 20) and x[60:] == bytes(4)
    for bad in ((64, 1), (), (10, 10, 10), (16, 16, 16, 16), (-1, 65)):
        with pytest.raises(ValueError):
            ops.rope_pair_axes(bad)
    for bad in ((32, 32), (4, 30, 30), (64,)):
        with pytest.raises(ValueError):
            ops.rope_pair_axes(bad, interleaved=True)


def test_the_binding_refuses_wrong_rows():
    t = torch.zeros(2, 32, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        ops._need_rows(t.float(), "q", (2, 32, 128), t.device)
    with pytest.raises(ValueError):
        ops._need_rows(t, "q", (2, 32, 128), t.device)        # not a CUDA tensor


def test_the_rotation_written_out_keeps_lengths_and_relative_positions():
    """The definition the GPU tests compare with: a rotation keeps each pair's length, and a
    product of two rotated heads depends on the distance of their positions alone."""
    g = torch.Generator().manual_seed(1)
    x, y = torch.randn(2, 5, 2, 128, generator=g, dtype=torch.float64)
    p = torch.tensor([0, 3, 17, 400, 100000])
    a, size = definitions.rotated(x, p, 1e6)
    assert torch.allclose(a.square().sum(-1), x.square().sum(-1)) and torch.equal(a[0], x[0])
    b, _ = definitions.rotated(y, p + 9, 1e6)
    a2, _ = definitions.rotated(x, p + 1000, 1e6)
    b2, _ = definitions.rotated(y, p + 1009, 1e6)
    assert torch.allclose((a * b).sum(-1), (a2 * b2).sum(-1))
    n, _ = definitions.rotated(x, p, 0.0, gain=torch.ones(128), eps=0.0)
    assert torch.allclose(n.square().mean(-1), torch.ones(5, 2, dtype=torch.float64))
    three = torch.stack([p, p + 5, p + 7])
    c, _ = definitions.rotated(x, three, 1e6, [0] * 16 + [1] * 24 + [2] * 24)
    d, _ = definitions.rotated(x, p + 5, 1e6)
    assert torch.equal(c[..., 16:40], d[..., 16:40]) and not torch.allclose(c[..., 40:64], d[..., 40:64])


def decode_args(p, fp8, **kw):
    a = dict(shape=ops.SHAPE, out=p(0), lse=None, q=p(1), kp=p(2), vp=p(3), ks=p(4), vs=p(5), bt=p(6), w=1, nb=1, sl=p(7),
             batch=1, window=4, sinks=1, scale=0.1, split=0, ws=p(8), ws_bytes=1 << 20, stream=None)
    assert set(kw) <= set(a)
    a.update(kw)
    if not fp8:
        del a["ks"], a["vs"]
    return list(a.values())


BAD_WINDOWS = [dict(window=0), dict(window=-1), dict(window=-(2 ** 31)), dict(sinks=-1), dict(scale=float("nan"))]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("change", BAD_WINDOWS + [dict(split=100), dict(split=-64), dict(batch=-1), dict(batch=8193),
                                                  dict(out=None), dict(ws=None), dict(ws_bytes=100), dict(w=0),
                                                  dict(nb=0), dict(w=1 << 23), dict(sl=None)], ids=str)
def test_decode_window_refuses(lib, change, fp8):
    p = Addresses()
    fn = lib.paged_attn_decode_window_fp8 if fp8 else lib.paged_attn_decode_window
    assert fn(*decode_args(p, fp8, **change)) == 1
    assert fn(*decode_args(p, fp8, shape=ops.pa_shape(32, 4, 128, 256))) == 2
    assert fn(*decode_args(p, fp8, batch=0)) == 0
    if fp8:
        assert fn(*decode_args(p, fp8, split=64)) == 1
        assert fn(*decode_args(p, fp8, ks=None)) == 1


@pytest.mark.parametrize("change", BAD_WINDOWS + [dict(max_q=0), dict(max_q=5), dict(out=16), dict(q=None), dict(seqs=0),
                                                  dict(ws_bytes=255)], ids=str)
def test_prefill_window_refuses(lib, change):
    p = Addresses()

    def args(**kw):
        a = dict(shape=ops.SHAPE, out=p(0), lse=None, q=p(1), kp=p(2), vp=p(3), bt=p(4), w=1, nb=1, cu=p(5), sl=p(6),
                 seqs=1, tokens=4, max_q=4, window=4, sinks=1, scale=0.1, ws=p(7), ws_bytes=1024, stream=None)
        a.update(kw)
        return list(a.values())

    if change.get("out"):
        change = dict(out=p(0, change["out"]))
    assert lib.paged_attn_prefill_window(*args(**change)) == 1
    assert lib.paged_attn_prefill_window(*args(shape=ops.pa_shape(32, 4, 128, 256))) == 2
    assert lib.paged_attn_prefill_window(*args(tokens=0, max_q=0)) == 0


def test_the_window_written_out_is_full_attention_when_long():
    g = torch.Generator().manual_seed(2)
    q, k, v = torch.randn(3, 32, 128, generator=g), torch.randn(9, 8, 128, generator=g), torch.randn(9, 8, 128, generator=g)
    full = torch.nn.functional.scaled_dot_product_attention(
        q.double().transpose(0, 1), k.double().repeat_interleave(4, 1).transpose(0, 1),
        v.double().repeat_interleave(4, 1).transpose(0, 1),
        attn_mask=torch.ones(3, 9, dtype=torch.bool).tril(6)).transpose(0, 1)
    scale = 128 ** -0.5
    out, _ = definitions.window_attention(q, [k], [v], [3], [9], 100, 0, scale)
    assert torch.allclose(out, full)
    out, _ = definitions.window_attention(q, [k], [v], [3], [9], 1, 100, scale)
    assert torch.allclose(out, full)
    # a window of one token without sinks returns its value; with one sink, a mix of the two
    out, _ = definitions.window_attention(q, [k], [v], [3], [9], 1, 0, scale)
    assert torch.allclose(out, v[6:].double().repeat_interleave(4, 1))
    out, _ = definitions.window_attention(q, [k], [v], [3], [9], 2, 1, scale)
    few, _ = definitions.window_attention(q[1:2], [k[[0, 6, 7]]], [v[[0, 6, 7]]], [1], [3], 9, 0, scale)
    assert torch.allclose(out[1:2], few)


def test_the_compiled_binding_leaves_odd_cases_to_the_checks(lib):
    """It makes a call only for plain CUDA tensors in the right number of arguments; host tensors,
    other objects and other counts are answered with None, and ops' checks say what is wrong."""
    b = ops._usual()
    t = torch.zeros(1, 32, 128, dtype=torch.bfloat16)
    for fn, n in ((b.rope_append, 19), (b.decode_window, 15), (b.prefill_window, 13)):
        for x in (None, t, 3, "x", torch.nn.Parameter(t)):
            assert fn(*[x] * n) is None
        assert fn() is None and fn(*[t] * (n + 1)) is None
    for window in (2 ** 31, -2 ** 31 - 1, 1.5):
        with pytest.raises(ValueError, match="window must be a 32-bit integer"):
            ops.paged_attn_decode_window(t, t, t, t, t, t, window=window)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        ops.paged_attn_decode_window(t, t, t, t, t, t, window=3)
    with pytest.raises(TypeError):
        ops.paged_attn_prefill_window(t, None, t, t, t, t, 3, t, window=3)


def test_the_binding_fails_loudly_when_it_is_missing(lib, monkeypatch, tmp_path):
    monkeypatch.setattr(ops, "_binding", None)
    monkeypatch.setattr(ops, "_LIB_PATH", str(tmp_path / "missing.so"))
    with pytest.raises(RuntimeError, match="_binding.so is missing"):
        ops._usual()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("axes", [64, True, 0, -1], ids=str)
def test_pair_axis_must_name_the_axes(axes, fp8):
    """An integer is refused, not taken as that many zeros."""
    t = torch.zeros(1, 32, 128, dtype=torch.bfloat16)
    cache = [t] * (4 if fp8 else 2)
    fn = ops.paged_rope_append_fp8 if fp8 else ops.paged_rope_append
    with pytest.raises(TypeError, match="pair_axis"):
        fn(t, t, t, *cache, t, t, t, t, rope_theta=1e6, positions=t, pair_axis=axes)
    with pytest.raises(ValueError, match="pair_axis"):
        fn(t, t, t, *cache, t, t, t, t, rope_theta=1e6, positions=t, pair_axis=[0] * 63)
    with pytest.raises(ValueError, match="pair_axis"):
        fn(t, t, t, *cache, t, t, t, t, rope_theta=1e6, positions=t, pair_axis=[0] * 63 + [256])


@pytest.mark.parametrize("scale", [0.0, -0.0, -0.1, -1e-30, float("inf"), float("-inf")])
def test_prefill_refuses_a_scale_that_is_not_positive(lib, scale):
    """Its masked scores are -infinity before they are scaled."""
    p = Addresses()
    base = [p(4), 1, 1, p(5), p(6), 1, 4, 4]                          # block table .. max_q_len
    tail = [scale, p(7), 1024, None]
    assert lib.paged_attn_prefill_window(ops.SHAPE, p(0), None, p(1), p(2), p(3), *base, 4, 1, *tail) == 1
    assert lib.paged_attn_prefill(ops.SHAPE, p(0), None, p(1), p(2), p(3), *base, *tail) == 1
    assert lib.paged_attn_prefill_append(ops.SHAPE, p(0), None, p(1), p(8), p(9), p(2), p(3), *base, *tail) == 1
