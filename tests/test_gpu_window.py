"""Attention over a sliding window with visible first tokens (decode over the bf16 and the 8-bit
cache, prefill) on the GPU against its definition in 64 bits.  Everything that no query sees is NaN,
and blocks without a visible token are gone (window_cases.py, with the tolerances)."""
import pytest
import torch

import definitions
from gpu_helpers import assert_lse_close, gpu, lib_ready, to_cpu
from paged_gqa_attention_gb300 import ops
from window_cases import Cache, check, tolerance

pytestmark = gpu
HUGE = 2 ** 31 - 1


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def decode(c, ws=None, **kw):
    ws = ws if ws is not None else ops.make_workspace(len(c.seq_lens), c.bt.shape[1])
    fn = ops.paged_attn_decode_window_fp8 if c.fp8 else ops.paged_attn_decode_window
    lse = torch.empty(len(c.seq_lens), 32, device="cuda")
    out = fn(c.qd, *c.pools, c.bt, c.lens, ws, window=c.window, sinks=c.sinks, lse=lse, **kw)
    ops.check_error(ws)
    return out, lse


LENS = [1, 5, 64, 255, 256, 257, 300, 1000, 2000]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 64), (15, 4), (16, 16), (17, 0), (63, 65), (64, 0),
                                          (65, 4), (100, 130), (128, 300), (513, 1), (1000, 16), (HUGE, 0), (HUGE, HUGE),
                                          (1, HUGE)])
def test_decode(window, sinks, fp8):
    c = Cache(LENS, [1] * len(LENS), min(window, 1 << 30), min(sinks, 1 << 30), 7, fp8).upload()
    c.window, c.sinks = window, sinks
    out, lse = decode(c)
    c.window, c.sinks = min(window, 1 << 30), min(sinks, 1 << 30)
    ref, ref_lse, tol = c.reference()
    check(out, ref, tol, "out")
    assert_lse_close(lse, ref_lse.numpy(), "window lse")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("split", [128, 256, 1024])
def test_decode_splits(split, fp8):
    c = Cache([3000, 700, 1, 64, 2049], [1] * 5, 900, 140, 9, fp8, spare=20).upload()
    ws = torch.zeros(16 << 20, dtype=torch.uint8, device="cuda")
    out, lse = decode(c, ws, split_tokens=split)
    ref, ref_lse, tol = c.reference()
    check(out, ref, tol, f"split {split}")
    assert_lse_close(lse, ref_lse.numpy(), "window lse")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch", [1, 2, 5, 40])
def test_decode_batches_and_padded_rows(batch, fp8):
    """Rows with seq_len 0 give zeros and lse -inf; a NaN output buffer and dirty table do not show."""
    lens = [(977 * i + 313) % 1500 for i in range(1, batch + 1)]
    lens[batch // 2] = 0
    if batch > 4:
        lens[0] = lens[-1] = 0
    c = Cache(lens, [1] * batch, 300, 5, 11, fp8)
    c.q_lens = [1 if n else 0 for n in lens]
    live = torch.tensor([n > 0 for n in lens])
    c.upload()
    out = torch.full_like(c.qd, float("nan"))
    got, lse = decode(c, out=out)
    assert (got[~live.cuda()] == 0).all() and (lse[~live.cuda()] == float("-inf")).all()
    if live.any():
        c.q = c.q[live]
        ref, ref_lse, tol = c.reference()
        check(got[live.cuda()], ref, tol, "live rows")
        assert_lse_close(lse[live.cuda()], ref_lse.numpy(), "window lse")


def test_decode_of_more_sequences_than_a_wave_holds():
    """39 sequences of up to 2500 tokens: 312 (sequence, KV head) pairs on 304 places, which the
    library splits (a plain workspace is enough)."""
    lens = [(977 * i + 313) % 2500 + 1 for i in range(38)] + [2500]
    c = Cache(lens, [1] * 39, 2400, 3, 57).upload()
    out, lse = decode(c)
    ref, ref_lse, tol = c.reference()
    check(out, ref, tol, "out")
    assert_lse_close(lse, ref_lse.numpy(), "window lse")
    assert torch.equal(out, decode(c)[0])


def test_decode_equals_the_full_decode_under_a_long_window():
    c = Cache([1000, 300, 2000], [1] * 3, 1 << 20, 0, 13).upload()
    ws = ops.make_workspace(3, c.bt.shape[1])
    c.bt.clamp_(min=0)
    a = ops.paged_attn_decode_window(c.qd, *c.pools, c.bt, c.lens, ws, window=1 << 20, split_tokens=2560)
    b = ops.paged_attn_decode(c.qd, *c.pools, c.bt, c.lens, ws, split_tokens=2560)
    ops.check_error(ws)
    assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_far_in_the_pool_and_far_in_the_context(fp8):
    """Pool offsets past 2^31 elements and a long context of which two blocks are left."""
    n = 70000
    c = Cache([n], [1], 200, 3, 15, fp8, far=9000).upload()      # 9000 * 262144 elements in front
    out, lse = decode(c)
    ref, ref_lse, tol = c_reference_of_long(c, n)
    check(out, ref, tol, "far")
    assert_lse_close(lse, ref_lse.numpy(), "window lse")


def c_reference_of_long(c, n):
    """The visible keys alone, as a context of their own."""
    keep = torch.cat([torch.arange(c.sinks), torch.arange(n - c.window, n)])
    c.k, c.v = [c.k[0][keep]], [c.v[0][keep]]
    c.seq_lens, c.window, c.sinks = [len(keep)], len(keep), 0
    return c.reference()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_device_checks(fp8):
    c = Cache([1000, 700], [1, 1], 300, 5, 17, fp8).upload()
    good, _ = decode(c)
    ws = ops.make_workspace(2, c.bt.shape[1])
    fn = ops.paged_attn_decode_window_fp8 if fp8 else ops.paged_attn_decode_window

    def call(table=None, lens=None):
        out = fn(c.qd, *c.pools, c.bt if table is None else table, c.lens if lens is None else lens, ws, window=300, sinks=5)
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
    assert c.bt[0, 1] == -1
    for n in (-1, c.bt.shape[1] * 256 + 1, -(2 ** 31)):
        _, word = call(lens=torch.tensor([1000, n], dtype=torch.int32, device="cuda"))
        assert word & (1 << 9)
    out = fn(c.qd, *c.pools, c.bt, c.lens, ws, window=300, sinks=5)
    ops.check_error(ws)
    assert torch.equal(out, good)


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_graphs_that_share_a_workspace(fp8):
    a = Cache([1000, 0, 700], [1, 1, 1], 300, 5, 19, fp8).upload()
    b = Cache([2000] * 45, [1] * 45, 900, 64, 21, fp8).upload()
    ws = ops.make_workspace(45, b.bt.shape[1])
    want = [decode(x, ws)[0].clone() for x in (a, b)]
    graphs, outs = [], []
    fn = ops.paged_attn_decode_window_fp8 if fp8 else ops.paged_attn_decode_window
    for x in (a, b):
        out = torch.empty_like(x.qd)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn(x.qd, *x.pools, x.bt, x.lens, ws, window=x.window, sinks=x.sinks, out=out)
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for g, out, w in zip(graphs, outs, want):
            out.fill_(float("nan"))
            g.replay()
            assert torch.equal(out, w)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = fn(b.qd, *b.pools, b.bt, b.lens, ws, window=b.window, sinks=b.sinks, stream=st)
    st.synchronize()
    assert torch.equal(out, want[1])
    ops.check_error(ws)


# ------------------------------------------------------------------ prefill

def prefill(c, **kw):
    ws = kw.pop("ws", None)
    ws = ws if ws is not None else ops.make_workspace(len(c.seq_lens), c.bt.shape[1])
    lse = torch.empty(c.qd.shape[0], 32, device="cuda")
    out = ops.paged_attn_prefill_window(c.qd, *c.pools, c.bt, c.cu, c.lens, max(c.q_lens), ws, window=c.window,
                                        sinks=c.sinks, lse=lse, **kw)
    ops.check_error(ws)
    return out, lse


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (2, 130), (31, 4), (64, 0), (100, 1), (127, 128), (128, 0),
                                          (129, 64), (300, 16), (513, 200), (1 << 30, 0), (40, 1 << 30)])
@pytest.mark.parametrize("lens,q_lens", [([1], [1]), ([300], [300]), ([1000], [129]),
                                         ([700, 64, 5, 1500, 257], [257, 64, 0, 33, 1])])
def test_prefill(lens, q_lens, window, sinks):
    c = Cache(lens, q_lens, window, sinks, 23).upload()
    out, lse = prefill(c)
    ref, ref_lse, tol = c.reference()
    check(out, ref, tol, "out")
    assert_lse_close(lse, ref_lse.numpy(), "window lse")


def test_prefill_extreme_arguments():
    c = Cache([700, 300], [257, 300], 1 << 30, 0, 25).upload()
    want, _ = prefill(c)
    for c.window, c.sinks in ((HUGE, 0), (HUGE, HUGE), (1, HUGE)):
        assert torch.equal(prefill(c)[0], want)


def test_prefill_equals_the_full_prefill_under_a_long_window():
    c = Cache([900, 300, 64], [513, 300, 1], 1 << 20, 0, 27).upload()
    out, lse = prefill(c)
    ws = ops.make_workspace(3, c.bt.shape[1])
    lse2 = torch.empty_like(lse)
    c.bt.clamp_(min=0)
    full = ops.paged_attn_prefill(c.qd, *c.pools, c.bt, c.cu, c.lens, 513, ws, lse=lse2)
    ops.check_error(ws)
    assert torch.equal(out, full) and torch.equal(lse, lse2)


def test_prefill_without_the_planning_kernel_and_on_a_stream():
    """A workspace of the error word alone: the natural order of units, the same bits."""
    c = Cache([700, 900, 300], [257, 100, 300], 200, 10, 29).upload()
    want, _ = prefill(c)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    assert torch.equal(prefill(c, ws=ws)[0], want)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        out = ops.paged_attn_prefill_window(c.qd, *c.pools, c.bt, c.cu, c.lens, 300, ws, window=200, sinks=10)
    st.synchronize()
    assert torch.equal(out, want)


def test_prefill_leaves_rows_behind_the_last_sequence():
    c = Cache([700, 300], [100, 33], 200, 10, 31).upload()
    want, _ = prefill(c)
    c.qd = torch.cat([c.qd, torch.full((70, 32, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out = torch.full_like(c.qd, 5.0)
    got, _ = prefill(c, out=out)
    assert torch.equal(got[:133], want) and (got[133:] == 5.0).all()


def test_prefill_device_checks():
    c = Cache([1000, 700], [40, 700], 300, 5, 33).upload()
    good, _ = prefill(c)
    ws = ops.make_workspace(2, c.bt.shape[1])
    assert c.bt[0, 1] == -1                      # not seen: no error above
    for table, lens in ((c.bt.clone(), c.lens), (c.bt, torch.tensor([30, 700], dtype=torch.int32, device="cuda"))):
        if lens is c.lens:
            table[0, 2] = -1
        out = ops.paged_attn_prefill_window(c.qd, *c.pools, table, c.cu, lens, 700, ws, window=300, sinks=5)
        with pytest.raises(ops.PagedAttnError) as e:
            ops.check_error(ws)
        assert e.value.status == 4
        assert torch.equal(out[40:], good[40:])


def test_prefill_captured():
    c = Cache([700, 900], [257, 100], 200, 10, 35).upload()
    want, _ = prefill(c)
    ws = ops.make_workspace(2, c.bt.shape[1])
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.paged_attn_prefill_window(c.qd, *c.pools, c.bt, c.cu, c.lens, 257, ws, window=200, sinks=10, out=out)
    for _ in range(2):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    ops.check_error(ws)


# ------------------------------------------------------------------ used together

def test_chat_with_a_window_end_to_end():
    """Two sequences served with a window: prompt chunks, then decode steps, every new token
    through paged_rope_append first and blocks given back (and overwritten with NaN) as the window passes
    them.  The cache rows against the formulas, each step's output against the
    definition over those rows."""
    window, sinks, theta = 300, 4, ops.QWEN3_ROPE_THETA
    g = torch.Generator().manual_seed(41)
    gain = [(1.0 + 0.25 * torch.randn(128, generator=g)).to(torch.bfloat16) for _ in range(2)]
    nan = float("nan")
    kp = torch.full((12, 256, 8, 128), nan, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    cache8 = ops.fp8_cache(12)
    free = list(range(12))
    table = torch.full((2, 8), -1, dtype=torch.int32)
    ws = ops.make_workspace(2, 8)
    lens = [0, 0]
    empty = torch.zeros(0, 8, 128, dtype=torch.float64)
    keys, values, keys8, values8 = ([empty, empty] for _ in range(4))
    for step, news in enumerate([(500, 130), (300, 0), (1, 1), (1, 1), (129, 400), (1, 1), (1, 1)]):
        t = sum(news)
        x = torch.randn(t, 6144, generator=g).to(torch.bfloat16)
        cu = [0, news[0], t]
        for s in (0, 1):
            lens[s] += news[s]
            for b in range((lens[s] + 255) // 256):
                dead = 256 * b >= sinks and 256 * b + 255 <= lens[s] - max(news[s], 1) - window
                if table[s, b] >= 0 and dead:
                    kp[table[s, b]] = nan
                    vp[table[s, b]] = nan
                    for buf in cache8:
                        buf[table[s, b]] = nan if buf.dtype == torch.float32 else 0x7F
                    free.append(int(table[s, b]))
                    table[s, b] = -1
                elif table[s, b] < 0 and 256 * b + 255 >= lens[s] - news[s]:
                    table[s, b] = free.pop(0)
        xd = x.cuda()
        q, k, v = (xd[:, lo:hi].view(t, -1, 128) for lo, hi in ((0, 4096), (4096, 5120), (5120, 6144)))
        args = (table.cuda(), torch.tensor(cu, dtype=torch.int32, device="cuda"),
                torch.tensor(lens, dtype=torch.int32, device="cuda"), ws)
        kw = dict(rope_theta=theta, q_norm_weight=gain[0].cuda(), k_norm_weight=gain[1].cuda())
        qr = ops.paged_rope_append(q, k, v, kp, vp, *args, **kw)
        q8 = ops.paged_rope_append_fp8(q, k, v, *cache8, *args, **kw)
        assert torch.equal(qr, q8)
        at = definitions.places(table.tolist(), news, lens)
        pos = torch.tensor([p for _, p, _, _ in at])
        blk, slot = torch.tensor([b for _, _, b, _ in at]), torch.tensor([o for _, _, _, o in at])
        k_rows, v_rows = to_cpu(kp)[blk, slot].double(), to_cpu(vp)[blk, slot].double()
        z, size = definitions.rotated(to_cpu(k), pos, theta, gain=gain[1], eps=ops.QWEN3_NORM_EPS)
        assert ((k_rows - z).abs() <= 2.0 ** -8 * z.abs() + 5e-6 * size).all() and torch.equal(v_rows, to_cpu(v).double())
        rows8 = [to_cpu(c)[blk, slot].view(torch.float8_e4m3fn).double() * to_cpu(s)[blk, :, slot].double()[..., None]
                 for c, s in zip(cache8[:2], cache8[2:])]
        for s in (0, 1):
            part = slice(cu[s], cu[s + 1])
            for known, new in ((keys, k_rows), (values, v_rows), (keys8, rows8[0]), (values8, rows8[1])):
                known[s] = torch.cat([known[s], new[part]])

        def compare(got, k, v, fp8):
            mask = (news, lens, window, sinks, ops.DEFAULT_SCALE)
            ref, _ = definitions.window_attention(to_cpu(qr), k, v, *mask)
            p_abs_v, _ = definitions.window_attention(to_cpu(qr), k, [x.abs() for x in v], *mask)
            v_max = max(float(x.abs().max()) for x in v)
            check(got, ref, tolerance(ref, p_abs_v, fp8, max(lens), v_max), f"step {step}, fp8 {fp8}")

        if max(news) > 1:
            out = ops.paged_attn_prefill_window(qr, kp, vp, *args[:3], max(news), ws, window=window, sinks=sinks)
        else:
            out = ops.paged_attn_decode_window(qr, kp, vp, args[0], args[2], ws, window=window, sinks=sinks)
            out8 = ops.paged_attn_decode_window_fp8(qr, *cache8, args[0], args[2], ws, window=window, sinks=sinks)
            compare(out8, keys8, values8, True)
        ops.check_error(ws)
        compare(out, keys, values, False)


# ------------------------------------------------------------------ the binding

def test_wrong_arguments_are_refused_with_their_names():
    """The public calls on the GPU with one argument wrong at a time: the error names it."""
    c = Cache([300, 20], [1, 1], 100, 4, 51).upload()
    ws = ops.make_workspace(2, c.bt.shape[1])
    good = dict(q=c.qd, k_pool=c.pools[0], v_pool=c.pools[1], block_table=c.bt, seq_lens=c.lens, workspace=ws)
    ops.paged_attn_decode_window(**good, window=100)
    for name, bad in (("q", c.qd.float()), ("q", c.qd[:, :8]), ("q", c.qd.transpose(0, 1)), ("k_pool", c.pools[0][:, :100]),
                      ("v_pool", c.pools[1][:2]), ("block_table", c.bt[0]), ("block_table", c.bt.long()),
                      ("seq_lens", c.lens[:1]), ("seq_lens", c.lens.cpu()), ("workspace", ws.view(torch.int32))):
        with pytest.raises((TypeError, ValueError), match=name):
            ops.paged_attn_decode_window(**{**good, name: bad}, window=100)
    for extra in (dict(out=c.qd[:1]), dict(lse=torch.empty(2, 8, device="cuda")), dict(out=c.qd.float())):
        with pytest.raises((TypeError, ValueError), match=next(iter(extra))):
            ops.paged_attn_decode_window(**good, window=100, **extra)
    for window, sinks, split in ((0, 0, 0), (-3, 0, 0), (5, -1, 0), (5, 0, 63)):
        with pytest.raises(ops.PagedAttnError) as e:
            ops.paged_attn_decode_window(**good, window=window, sinks=sinks, split_tokens=split)
        assert e.value.status == 1
    with pytest.raises(ops.PagedAttnError) as e:       # a workspace too small for the splits
        ops.paged_attn_decode_window(**{**good, "workspace": ws[:300000]}, window=4096, split_tokens=64)
    assert e.value.status == 6
    ops.check_error(ws)


def test_numbers_may_be_whole_and_the_output_given():
    c = Cache([300, 20], [1, 1], 100, 4, 53).upload()
    ws = ops.make_workspace(2, c.bt.shape[1])
    out = torch.empty_like(c.qd)
    a = ops.paged_attn_decode_window(c.qd, *c.pools, c.bt, c.lens, ws, window=100, sinks=4, scale=1, out=out)
    b = ops.paged_attn_decode_window(c.qd, *c.pools, c.bt, c.lens, ws, window=100, sinks=4, scale=1.0,
                                     stream=torch.cuda.current_stream())
    assert a.data_ptr() == out.data_ptr() and torch.equal(a, b)
    c.qd.requires_grad_()                               # the calls know no gradients: the result has none
    assert not ops.paged_attn_decode_window(c.qd, *c.pools, c.bt, c.lens, ws, window=100).requires_grad


# few tokens over a wide window: a cluster of CTAs shares each work unit (2 to 8 of them)
@pytest.mark.parametrize("window,sinks", [(1 << 30, 0), (1000, 100), (300, 4), (2000, 0)])
@pytest.mark.parametrize("lens,q_lens", [([3000], [1]), ([3000], [65]), ([2500, 40], [64, 40]), ([2000, 2000, 100], [5, 0, 70]),
                                         ([1500], [400])])
def test_prefill_of_few_tokens(lens, q_lens, window, sinks):
    c = Cache(lens, q_lens, window, sinks, 37).upload()
    out, lse = prefill(c)
    ref, ref_lse, tol = c.reference()
    check(out, ref, tol, "out")
    assert_lse_close(lse, ref_lse.numpy(), "window lse")
    again, _ = prefill(c)
    assert torch.equal(out, again)


def test_prefill_of_few_tokens_with_a_bad_block_and_captured():
    c = Cache([3000, 2000], [20, 33], 1500, 70, 39).upload()
    want, _ = prefill(c)
    ws = ops.make_workspace(2, c.bt.shape[1])
    table = c.bt.clone()
    table[1, 6] = c.blocks + 5
    out = ops.paged_attn_prefill_window(c.qd, *c.pools, table, c.cu, c.lens, 33, ws, window=1500, sinks=70)
    with pytest.raises(ops.PagedAttnError) as e:
        ops.check_error(ws)
    assert e.value.status == 4 and torch.equal(out[:20], want[:20])
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ops.paged_attn_prefill_window(c.qd, *c.pools, c.bt, c.cu, c.lens, 33, ws, window=1500, sinks=70, out=out)
    for _ in range(2):
        out.zero_()
        g.replay()
        assert torch.equal(out, want)
    ops.check_error(ws)


def test_calls_on_two_streams_at_once():
    """Decode, prefill and append on two streams, each with a workspace of its own, again and again:
    the results of the same calls made one after another."""
    a = Cache([1000, 0, 700, 2000], [1] * 4, 300, 5, 61).upload()
    b = Cache([1500, 900], [200, 70], 400, 33, 63).upload()
    g = torch.Generator(device="cuda")
    g.manual_seed(65)
    y = torch.randn(270, 6144, generator=g, device="cuda").to(torch.bfloat16)
    rows = [y[:, lo:hi].view(270, -1, 128) for lo, hi in ((0, 4096), (4096, 5120), (5120, 6144))]
    pools = [[p.clone() for p in b.pools] for _ in range(2)]
    ws = [ops.make_workspace(4, 16) for _ in range(2)]

    def calls(i):
        q = ops.paged_rope_append(*rows, *pools[i], b.bt, b.cu, b.lens, ws[i], rope_theta=1e6)
        return (ops.paged_attn_decode_window(a.qd, *a.pools, a.bt, a.lens, ws[i], window=300, sinks=5),
                ops.paged_attn_prefill_window(q, *pools[i], b.bt, b.cu, b.lens, 200, ws[i], window=400, sinks=33), q)

    want = calls(0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls(i))
    torch.cuda.synchronize()
    for out in got[0] + got[1]:
        assert all(torch.equal(x, y) for x, y in zip(out, want))
    for w in ws:
        ops.check_error(w)


# at most 32 new tokens a sequence: one of a CTA's two row tiles, or a part of one
@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (128, 0), (300, 16), (513, 200), (1 << 30, 0), (3, 1 << 30)])
@pytest.mark.parametrize("lens,q_lens", [([1], [1]), ([32], [32]), ([700], [1]), ([1500], [31]),
                                         ([129, 3000, 5, 257, 64], [32, 17, 0, 1, 32])])
def test_prefill_of_32_tokens_at_most(lens, q_lens, window, sinks):
    c = Cache(lens, q_lens, window, sinks, 67).upload()
    out, lse = prefill(c)
    ref, ref_lse, tol = c.reference()
    check(out, ref, tol, "out")
    assert_lse_close(lse, ref_lse.numpy(), "window lse")
    assert torch.equal(out, prefill(c)[0])


def test_prefill_of_32_tokens_at_most_in_more_sequences_than_sms():
    """25 sequences x 8 KV heads are more units than SMs: they are dealt to persistent CTAs."""
    lens = [(977 * i + 313) % 900 + 32 for i in range(25)]
    c = Cache(lens, [(7 * i) % 33 for i in range(25)], 200, 5, 69).upload()
    out, lse = prefill(c)
    ref, ref_lse, tol = c.reference()
    check(out, ref, tol, "out")
    assert_lse_close(lse, ref_lse.numpy(), "window lse")


# new tokens' sequences: one whose units a cluster shares each, one of many units, several in a planned order
NAN_CASES = [([300], [130], 40, 4), ([900], [700], 200, 5), ([700], [700], 1 << 30, 0), ([700], [700], 64, 100),
             ([1500, 900, 800], [700, 640, 333], 129, 17)]


def nan_rows(c, s, p, keys, values):
    """Pools with the K and / or V row of sequence s at position p set to NaN."""
    pools = [t.clone() for t in c.pools]
    for t, on in zip(pools, (keys, values)):
        if on:
            t[int(c.table[s, p // 256]), p % 256] = float("nan")
    return pools


def prefill_of(c, pools):
    ws = ops.make_workspace(len(c.seq_lens), c.bt.shape[1])
    out = ops.paged_attn_prefill_window(c.qd, *pools, c.bt, c.cu, c.lens, max(c.q_lens), ws, window=c.window, sinks=c.sinks)
    ops.check_error(ws)
    return out


@pytest.mark.parametrize("lens,q_lens,window,sinks", NAN_CASES)
def test_prefill_nan_rows_reach_no_unit_that_does_not_see_them(lens, q_lens, window, sinks):
    """K and V of one new token are NaN: the outputs of every 64 new tokens of which none sees it keep
    their bits, those of its own sequence before it and behind its window, and the other sequences'."""
    c = Cache(lens, q_lens, window, sinks, 171).upload()
    clean = prefill_of(c, c.pools)
    for s, (n, m) in enumerate(zip(lens, q_lens)):
        for i in sorted({x for x in (0, 2, 63, 64, 65, 127, 128, 191, 200, m // 2, m - 2, m - 1) if x < m}):
            p = n - m + i
            out = prefill_of(c, nan_rows(c, s, p, True, True))
            sees = torch.zeros(sum(q_lens), dtype=torch.bool)
            t0 = sum(q_lens[:s])
            for u in range(0, m, 64):
                first, last = n - m + u, n - m + min(u + 64, m) - 1
                if last >= p and (p < sinks or first < p + window):
                    sees[t0 + u:t0 + min(u + 64, m)] = True
            assert torch.equal(out[~sees.cuda()], clean[~sees.cuda()]), (s, p)
            assert out[t0 + i].isnan().all()


@pytest.mark.parametrize("lens,q_lens,window,sinks", NAN_CASES)
def test_prefill_nan_keys_reach_no_position_that_does_not_see_them(lens, q_lens, window, sinks):
    c = Cache(lens, q_lens, window, sinks, 172).upload()
    clean = prefill_of(c, c.pools)
    for s, (n, m) in enumerate(zip(lens, q_lens)):
        for i in sorted({x for x in (0, 2, 63, 64, 65, 127, 128, 191, 200, m // 2, m - 2, m - 1) if x < m}):
            p = n - m + i
            out = prefill_of(c, nan_rows(c, s, p, True, False))
            sees = torch.zeros(sum(q_lens), dtype=torch.bool)
            at = torch.arange(n - m, n)
            sees[sum(q_lens[:s]):sum(q_lens[:s + 1])] = (at >= p) & ((p < sinks) | (at < p + window))
            assert torch.equal(out[~sees.cuda()], clean[~sees.cuda()]), (s, p)
            assert out[sees.cuda()].isnan().all()
