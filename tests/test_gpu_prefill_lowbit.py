"""Prefill over the 8-bit and the 4-bit cache on the GPU against its definition in 64 bits.  What no query
sees is NaN, and blocks without a visible token are gone (lowbit_cases.py, with the tolerances)."""
import pytest
import torch

from gpu_helpers import gpu, lib_ready
from lowbit_cases import LowCache, check_lse
from paged_gqa_attention_gb300 import ops
from window_cases import check

pytestmark = gpu
HUGE = 2 ** 31 - 1
BITS = pytest.mark.parametrize("bits", [8, 4])


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def prefill(c, **kw):
    ws = kw.pop("ws", None)
    ws = ws if ws is not None else ops.make_workspace(len(c.seq_lens), c.bt.shape[1])
    lse = torch.empty(c.qd.shape[0], 32, device="cuda")
    fn = ops.paged_attn_prefill_fp8 if c.bits == 8 else ops.paged_attn_prefill_fp4
    window = {} if c.window == HUGE and c.sinks == 0 else {"window": c.window, "sinks": c.sinks}
    out = fn(c.qd, *c.pools, c.bt, c.cu, c.lens, max(c.q_lens), ws, lse=lse, **window, **kw)
    ops.check_error(ws)
    return out, lse


def compare(c, got, what=""):
    out, lse = got
    window, sinks, c.window, c.sinks = c.window, c.sinks, min(c.window, 1 << 30), min(c.sinks, 1 << 30)
    ref, ref_lse, tol, lse_tol = c.prefill_reference(ops.DEFAULT_SCALE)
    c.window, c.sinks = window, sinks
    check(out, ref, tol, f"{what} out")
    check_lse(lse, ref_lse, lse_tol, what)


@BITS
@pytest.mark.parametrize("lens,q_lens", [([1], [1]), ([300], [300]), ([1000], [129]),
                                         ([700, 64, 5, 1500, 257], [257, 64, 0, 33, 1])])
@pytest.mark.parametrize("window,sinks", [(HUGE, 0), (1, 0), (1, 3), (2, 130), (31, 4), (64, 0), (127, 128), (128, 0),
                                          (129, 64), (300, 16), (513, 200), (40, 1 << 30)])
def test_prefill(lens, q_lens, window, sinks, bits):
    c = LowCache(lens, q_lens, min(window, 1 << 30), min(sinks, 1 << 30), 23, bits).upload()
    c.window, c.sinks = window, sinks
    compare(c, prefill(c), f"{lens} {q_lens}")
