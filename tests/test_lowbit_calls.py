"""The low-bit caches' Python calls are for their own cache alone, whichever path takes them."""
import pytest
import torch

from gpu_helpers import gpu, lib_ready
from paged_gqa_attention_gb300 import ops


class Taking:
    """A compiled binding that takes every call (it tells an 8-bit cache by its missing exponents)."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        def take(*args):
            self.calls.append((name, args))
            return torch.zeros(1)
        return take


def calls(dev, cache):
    """The 4-bit calls that read a cache, over `cache` (six entries), with the stream left open or given."""
    q = torch.zeros(1, 32, 128, dtype=torch.bfloat16, device=dev)
    table, cu, lens, first = (torch.tensor(x, dtype=torch.int32, device=dev) for x in ([[0]], [0, 1], [1], [0]))
    ws = torch.zeros(1 << 20, dtype=torch.uint8, device=dev)
    return [lambda **kw: ops.paged_kv_read_fp4(*cache, table, cu, first, 1, ws, **kw),
            lambda **kw: ops.paged_attn_prefill_fp4(q, *cache, table, cu, lens, 1, ws, **kw),
            lambda **kw: ops.paged_attn_decode_fp4(q, *cache, table, lens, ws, **kw)]


def eight_bits(dev):
    codes = torch.zeros(1, 256, 8, 128, dtype=torch.uint8, device=dev)
    scales = torch.ones(1, 8, 256, device=dev)
    return codes, codes.clone(), scales, scales.clone()


def test_a_4_bit_call_never_hands_an_8_bit_cache_on(monkeypatch):
    binding = Taking()
    monkeypatch.setattr(ops, "_binding", binding)
    four = ops.fp4_cache(1, "cpu")
    for cache in ((*eight_bits("cpu"), None, None), (*eight_bits("cpu"), None, four[5]), (*four[:4], None, None)):
        for f in calls("cpu", cache)[:2]:
            with pytest.raises((TypeError, ValueError)):
                f()
    assert not binding.calls
    for f in calls("cpu", four):
        f()
    assert [n for n, _ in binding.calls] == ["kv_read", "prefill_low", "decode_fp4"]


@gpu
def test_a_4_bit_call_refuses_an_8_bit_cache():
    lib_ready()
    four = ops.fp4_cache(1)
    stream = torch.cuda.Stream()
    for cache in ((*eight_bits("cuda"), None, None), (*eight_bits("cuda"), None, four[5]), (*eight_bits("cuda"), *four[4:]),
                  (*four[:4], None, None), (*four[:5], None)):
        for f in calls("cuda", cache):
            for kw in ({}, {"stream": stream}):
                with pytest.raises((TypeError, ValueError)):
                    f(**kw)
