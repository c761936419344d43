"""Outputs that the compiled binding allocates are torch.empty's: filled with NaN where torch.use_deterministic_algorithms
asks for it, and seen by a dispatch mode."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from gpu_helpers import gpu, lib_ready
from paged_gqa_attention_gb300 import ops

pytestmark = gpu
LIVE, ROWS = 3, 7         # of the batch's rows, those that a sequence owns


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def calls():
    """(name, call) of the calls that leave rows behind the last sequence alone, and of the decodes; each gives its
    outputs."""
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    q = torch.ones(ROWS, 32, 128, dtype=torch.bfloat16, device="cuda")
    k = torch.ones(ROWS, 8, 128, dtype=torch.bfloat16, device="cuda")
    table, cu, lens, first = ints(0)[None], ints(0, LIVE), ints(LIVE), ints(0)
    ws = ops.make_workspace(1, 1)
    pools = [torch.zeros(1, 256, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c8, c4 = ops.fp8_cache(1), ops.fp4_cache(1)
    rope = dict(rope_theta=1e6)
    out = []
    for name, cache, append, attend, decode, read in (
            ("bf16", pools, ops.paged_rope_append, ops.paged_attn_prefill_window, ops.paged_attn_decode_window, None),
            ("8", c8, ops.paged_rope_append_fp8, ops.paged_attn_prefill_fp8, ops.paged_attn_decode_window_fp8,
             ops.paged_kv_read_fp8),
            ("4", c4, ops.paged_rope_append_fp4, ops.paged_attn_prefill_fp4, ops.paged_attn_decode_fp4, ops.paged_kv_read_fp4)):
        out.append((f"append {name}", lambda c=cache, f=append: [f(q, k, k, *c, table, cu, lens, ws, **rope)]))
        out.append((f"prefill {name}", lambda c=cache, f=attend: [f(q, *c, table, cu, lens, LIVE, ws, window=9)]))
        out.append((f"decode {name}", lambda c=cache, f=decode: [f(q[:1], *c, table, lens, ws, window=9)]))
        if read:
            out.append((f"read {name}", lambda c=cache, f=read: list(f(*c, table, cu, first, ROWS, ws))))
    return out


class Empties(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = 0

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        self.made += func.overloadpacket is torch.ops.aten.empty
        return func(*args, **(kwargs or {}))


def test_rows_left_alone_are_nan_where_new_memory_is_to_be():
    todo = calls()
    for _, f in todo:                            # memory of these sizes that holds other values
        for x in f():
            x.fill_(5.0)
    torch.use_deterministic_algorithms(True)
    try:
        for name, f in todo:
            for x in f():
                assert x[:LIVE].isfinite().all(), name
                assert x[LIVE:].isnan().all(), name
    finally:
        torch.use_deterministic_algorithms(False)


def test_a_dispatch_mode_sees_the_outputs():
    for name, f in calls():
        with Empties() as mode:
            n = len(f())
        assert mode.made == n, name
