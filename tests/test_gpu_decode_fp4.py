"""Decode over the 4-bit cache on the GPU against its definition in 64 bits.  Everything that no query sees is
NaN, and blocks without a visible token are gone (lowbit_cases.py; tolerances: window_cases.py, whose f16 bound
for the 8-bit cache holds here: codes times scales are exact, the weights times a power of two f16)."""
import pytest
import torch

from gpu_helpers import assert_lse_close, gpu, lib_ready
from lowbit_cases import LowCache
from paged_gqa_attention_gb300 import ops
from window_cases import check, tolerance

pytestmark = gpu
HUGE = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def decode(c, ws=None, **kw):
    ws = ws if ws is not None else ops.make_workspace(len(c.seq_lens), c.bt.shape[1])
    lse = torch.empty(len(c.seq_lens), 32, device="cuda")
    window = {} if c.window == HUGE and c.sinks == 0 else {"window": c.window, "sinks": c.sinks}
    out = ops.paged_attn_decode_fp4(c.qd, *c.pools, c.bt, c.lens, ws, lse=lse, **window, **kw)
    ops.check_error(ws)
    return out, lse


def compare(c, out, lse, what=""):
    window, sinks, c.window, c.sinks = c.window, c.sinks, min(c.window, 1 << 30), min(c.sinks, 1 << 30)
    c.fp8 = True                     # f16 weights
    ref, ref_lse, tol = c.reference()
    c.fp8, c.window, c.sinks = False, window, sinks
    check(out, ref, tol, what)
    assert_lse_close(lse, ref_lse.numpy(), what)


LENS = [1, 5, 64, 255, 256, 257, 300, 1000, 2000]


@pytest.mark.parametrize("window,sinks", [(HUGE, 0), (1, 0), (1, 1), (2, 64), (15, 4), (16, 16), (17, 0), (63, 65), (64, 0),
                                          (100, 130), (128, 300), (513, 1), (1000, 16), (HUGE, HUGE), (1, HUGE)])
def test_decode(window, sinks):
    c = LowCache(LENS, [1] * len(LENS), min(window, 1 << 30), min(sinks, 1 << 30), 7).upload()
    c.window, c.sinks = window, sinks
    compare(c, *decode(c), "out")


@pytest.mark.parametrize("split", [256, 512, 1024])
def test_decode_splits(split):
    c = LowCache([3000, 700, 1, 64, 2049], [1] * 5, 1 << 30, 0, 9, spare=20).upload()
    c.window = HUGE
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda")
    compare(c, *decode(c, ws, split_tokens=split), f"split {split}")


@pytest.mark.parametrize("batch", [1, 2, 5, 40])
def test_decode_batches_and_padded_rows(batch):
    """Rows with seq_len 0 give zeros and lse -inf; a NaN output buffer and dirty table do not show."""
    lens = [(977 * i + 313) % 1500 for i in range(1, batch + 1)]
    lens[batch // 2] = 0
    if batch > 4:
        lens[0] = lens[-1] = 0
    c = LowCache(lens, [1] * batch, 300, 5, 11)
    c.q_lens = [1 if n else 0 for n in lens]
    live = torch.tensor([n > 0 for n in lens])
    c.upload()
    got, lse = decode(c, out=torch.full_like(c.qd, float("nan")))
    assert (got[~live.cuda()] == 0).all() and (lse[~live.cuda()] == float("-inf")).all()
    if live.any():
        c.q = c.q[live]
        compare(c, got[live.cuda()], lse[live.cuda()], "live rows")


def test_decode_of_more_sequences_than_a_wave_holds():
    lens = [(977 * i + 313) % 2500 + 1 for i in range(44)] + [2500]
    c = LowCache(lens, [1] * 45, 1 << 30, 0, 57).upload()
    c.window = HUGE
    out, lse = decode(c)
    compare(c, out, lse, "out")
    assert torch.equal(out, decode(c)[0])


def test_decode_far_in_the_pool_and_far_in_the_context():
    """Pool offsets past 2^31 bytes and a long context of which two blocks are left."""
    n = 70000
    c = LowCache([n], [1], 200, 3, 15, far=17000).upload()       # 17000 * 131072 bytes in front
    out, lse = decode(c)
    keep = torch.cat([torch.arange(3), torch.arange(n - 200, n)])
    c.k, c.v = [c.k[0][keep]], [c.v[0][keep]]
    c.seq_lens, c.window, c.sinks = [203], 203, 0
    compare(c, out, lse, "far")


def test_decode_rows_of_very_different_size():
    """V rows whose exponents rise and fall along the context, and zero rows: the accumulator's unit moves."""
    c = LowCache([1500, 700], [1, 1], 1 << 30, 0, 31)
    for kp in (c.v_host,):
        scale = torch.exp2(torch.randint(-20, 21, kp.shape[:2], generator=torch.Generator().manual_seed(1)).float())
        kp *= scale[..., None, None].to(torch.bfloat16)
        kp[:, ::17] *= 0
    c.upload()
    c.window = HUGE
    compare(c, *decode(c), "sizes")


def test_decode_device_checks():
    c = LowCache([1000, 700], [1, 1], 300, 5, 17).upload()
    good, _ = decode(c)
    ws = ops.make_workspace(2, c.bt.shape[1])

    def call(table=None, lens=None):
        out = ops.paged_attn_decode_fp4(c.qd, *c.pools, c.bt if table is None else table, c.lens if lens is None else lens,
                                        ws, window=300, sinks=5)
        with pytest.raises(ops.PagedAttnError) as e:
            ops.check_error(ws)
        assert e.value.status == 4
        return out, e.value.detail

    for where in (0, 2, 3):                      # the sinks' block and the window's
        table = c.bt.clone()
        assert table[0, where] >= 0
        table[0, where] = c.blocks if where else -1
        out, word = call(table)
        assert word & (1 << 8) and out[0].isnan().all() and torch.equal(out[1], good[1])
    for n in (-1, c.bt.shape[1] * 256 + 1, -(2 ** 31)):
        _, word = call(lens=torch.tensor([1000, n], dtype=torch.int32, device="cuda"))
        assert word & (1 << 9)
    out = ops.paged_attn_decode_fp4(c.qd, *c.pools, c.bt, c.lens, ws, window=300, sinks=5)
    ops.check_error(ws)
    assert torch.equal(out, good)


def test_decode_of_a_visible_nan_row_is_nan_and_of_a_hidden_one_is_not():
    c = LowCache([600, 600], [1, 1], 100, 0, 19).upload()
    good, _ = decode(c)
    for which in (4, 5):
        pools = [t.clone() for t in c.pools]
        pools[which][c.bt[0, 2].long(), 3, 550 - 512] = 255
        hidden = c.pools[which].clone()
        hidden[c.bt[0, 1].long(), :, :] = 255                    # tokens 256 .. 499 are not seen
        hidden[c.bt[0, 1].long(), :, 500 - 256:] = c.pools[which][c.bt[0, 1].long(), :, 500 - 256:]
        ws = ops.make_workspace(2, c.bt.shape[1])
        out = ops.paged_attn_decode_fp4(c.qd, *pools, c.bt, c.lens, ws, window=100)
        assert out[0, 12:16].isnan().all() and not out[0, :12].isnan().any() and torch.equal(out[1], good[1])
        pools[which] = hidden
        assert torch.equal(ops.paged_attn_decode_fp4(c.qd, *pools, c.bt, c.lens, ws, window=100), good)
        ops.check_error(ws)


def test_decode_graphs_that_share_a_workspace():
    a = LowCache([1000, 0, 700], [1, 1, 1], 300, 5, 19).upload()
    b = LowCache([2000] * 45, [1] * 45, 900, 64, 21).upload()
    ws = ops.make_workspace(45, b.bt.shape[1])
    want = [decode(x, ws)[0].clone() for x in (a, b)]
    graphs, outs = [], []
    for x in (a, b):
        out = torch.empty_like(x.qd)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ops.paged_attn_decode_fp4(x.qd, *x.pools, x.bt, x.lens, ws, window=x.window, sinks=x.sinks, out=out)
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for g, out, w in zip(graphs, outs, want):
            out.fill_(float("nan"))
            g.replay()
            assert torch.equal(out, w)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = ops.paged_attn_decode_fp4(b.qd, *b.pools, b.bt, b.lens, ws, window=b.window, sinks=b.sinks, stream=st)
    st.synchronize()
    assert torch.equal(out, want[1])
    ops.check_error(ws)
