"""Prefill over the low-bit caches beyond single tiles (many work units a CTA, long prompts, rows of very different
size, bad tables, graphs and streams), and the low-bit operators used together as a server uses them."""
import pytest
import torch

import definitions
import window_cases
from gpu_helpers import gpu, lib_ready, to_cpu
from lowbit_cases import LowCache, check_lse
from paged_gqa_attention_gb300 import ops
from test_gpu_prefill_lowbit import BITS, HUGE, compare, prefill

pytestmark = gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


@BITS
@pytest.mark.parametrize("window,sinks", [(HUGE, 0), (200, 10)])
def test_prefill_of_more_units_than_there_are_sms(bits, window, sinks):
    """Ten sequences of up to 300 new tokens, 240 units of 128 with the empty ones: planned, several a CTA."""
    q_lens = [300, 0, 129, 64, 257, 1, 128, 192, 300, 77]
    lens = [900, 5, 129, 700, 300, 1200, 128, 195, 301, 513]
    c = LowCache(lens, q_lens, min(window, 1 << 30), sinks, 41, bits).upload()
    c.window = window
    got = prefill(c)
    compare(c, got, "units")
    assert torch.equal(got[0], prefill(c)[0])


@BITS
def test_prefill_of_many_short_questions(bits):
    """No sequence has more than 64 new tokens: units of 64, more of them than SMs."""
    q_lens = [(37 * i) % 65 for i in range(27)]
    lens = [m + (91 * i) % 500 + (m == 0) for i, m in enumerate(q_lens)]
    c = LowCache(lens, q_lens, 1 << 30, 0, 43, bits).upload()
    c.window = HUGE
    compare(c, prefill(c), "questions")


@BITS
def test_prefill_of_a_long_prompt(bits):
    """One sequence, more units than pairs of SMs, no planning; the last query block is not whole."""
    c = LowCache([1500], [1409], 1 << 30, 0, 45, bits).upload()
    c.window = HUGE
    compare(c, prefill(c), "prompt")


@BITS
def test_prefill_rows_of_very_different_size(bits):
    """V rows whose scales rise and fall along the context, K rows down to 2^-20 of the others, zero rows: the unit of O
    moves, and dividing by powers of two costs no row more than the tolerance has."""
    c = LowCache([1500, 700], [200, 130], 1 << 30, 0, 47, bits)
    g = torch.Generator().manual_seed(1)
    c.v_host *= torch.exp2(torch.randint(-20, 21, c.v_host.shape[:2], generator=g).float())[..., None, None].to(torch.bfloat16)
    c.k_host *= torch.exp2(torch.randint(-20, 1, c.k_host.shape[:2], generator=g).float())[..., None, None].to(torch.bfloat16)
    if bits == 4:                                # (the 8-bit test cache divides by the row's maximum)
        c.v_host[:, ::17] *= 0
    c.upload()
    c.window = HUGE
    compare(c, prefill(c), "sizes")


@BITS
def test_prefill_far_in_the_pool_and_far_in_the_context(bits):
    """Pool offsets past 2^31 bytes, and a long context of which a few blocks are left."""
    n, far = 70000, 9000 if bits == 8 else 17000
    c = LowCache([n], [150], 200, 3, 15, bits, far=far).upload()
    got = prefill(c)
    keep = torch.cat([torch.arange(3), torch.arange(n - 149 - 200, n)])
    c.k, c.v = [c.k[0][keep]], [c.v[0][keep]]
    c.seq_lens, c.window, c.sinks = [len(keep)], 200, 3
    compare(c, got, "far")


@BITS
def test_prefill_leaves_rows_behind_the_last_sequence(bits):
    c = LowCache([700, 300], [100, 33], 200, 10, 31, bits).upload()
    want, _ = prefill(c)
    c.qd = torch.cat([c.qd, torch.full((170, 32, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    got, _ = prefill(c, out=torch.full_like(c.qd, 5.0))
    assert torch.equal(got[:133], want) and (got[133:] == 5.0).all()


@BITS
@pytest.mark.parametrize("q0", [40, 200])
def test_prefill_device_checks(bits, q0):
    c = LowCache([1000, 700], [q0, 700], 300, 5, 33, bits).upload()
    good, _ = prefill(c)
    ws = ops.make_workspace(2, c.bt.shape[1])
    fn = ops.paged_attn_prefill_fp8 if bits == 8 else ops.paged_attn_prefill_fp4
    as_int = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    bad_table, too_many = c.bt.clone(), c.bt.clone()
    bad_table[0, 2] = -1
    too_many[0, 3] = c.blocks
    for table, cu, lens in ((bad_table, c.cu, c.lens), (too_many, c.cu, c.lens), (c.bt, c.cu, as_int(q0 - 1, 700)),
                            (c.bt, c.cu, as_int(c.bt.shape[1] * 256 + 1, 700)), (c.bt, c.cu, as_int(-(2 ** 31), 700)),
                            (c.bt, as_int(-5, q0, q0 + 700), c.lens)):
        out = fn(c.qd, *c.pools, table, cu, lens, 700, ws, window=300, sinks=5)
        with pytest.raises(ops.PagedAttnError) as e:
            ops.check_error(ws)
        assert e.value.status == 4
        assert torch.equal(out[q0:], good[q0:])
    out = fn(c.qd, *c.pools, c.bt, c.cu, c.lens, 700, ws, window=300, sinks=5)
    ops.check_error(ws)
    assert torch.equal(out, good)


@BITS
def test_prefill_graphs_that_share_a_workspace_and_another_stream(bits):
    """Two captured prefills (one planned into the workspace) and an eager one on a stream of its own."""
    cases = [LowCache([700, 900, 300], [257, 100, 300], 200, 10, 29, bits).upload(),
             LowCache([400] * 12, [200] * 12, 150, 0, 30, bits).upload()]
    ws = ops.make_workspace(12, 8)
    fn = ops.paged_attn_prefill_fp8 if bits == 8 else ops.paged_attn_prefill_fp4
    want = [prefill(c, ws=ws)[0].clone() for c in cases]
    only_errors = torch.zeros(256, dtype=torch.uint8, device="cuda")     # no room to plan: the natural order, the same bits
    graphs, outs = [], []
    for c, w in zip(cases, want):
        assert torch.equal(prefill(c, ws=only_errors)[0], w)
        out = torch.empty_like(c.qd)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn(c.qd, *c.pools, c.bt, c.cu, c.lens, max(c.q_lens), ws, window=c.window, sinks=c.sinks, out=out)
        graphs.append(g)
        outs.append(out)
    for _ in range(3):
        for g, out, w in zip(graphs, outs, want):
            out.fill_(float("nan"))
            g.replay()
            assert torch.equal(out, w)
    c = cases[1]
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out = fn(c.qd, *c.pools, c.bt, c.cu, c.lens, 200, ws, window=c.window)
    st.synchronize()
    assert torch.equal(out, want[1])
    out = fn(c.qd, *c.pools, c.bt, c.cu, c.lens, 200, ws, window=c.window, stream=st)
    st.synchronize()
    assert torch.equal(out, want[1])
    ops.check_error(ws)


# ------------------------------------------------------------------ used together

def held(read, cache, table, lens, ws):
    """Every sequence's rows as the cache holds them, on the host."""
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    as_int = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    k, v = read(*cache, table, as_int(cu), as_int([0] * len(lens)), cu[-1], ws)
    return k, v, [[to_cpu(x)[a:b] for a, b in zip(cu, cu[1:])] for x in (k, v)]


@BITS
def test_a_chat_served_from_a_low_bit_cache(bits):
    """Two conversations over one layer: prompt chunks through the rotated append and the prefill, decode steps
    through the rotated append and the decode, every output against the definition over the rows that the
    cache gives back; then both move to a bf16 cache, where the next step gives the same answer."""
    g = torch.Generator().manual_seed(53)
    gain = [(1.0 + 0.25 * torch.randn(128, generator=g)).to(torch.bfloat16).cuda() for _ in range(2)]
    theta = ops.QWEN3_ROPE_THETA
    if bits == 8:
        cache = ops.fp8_cache(8)
        append, attend = ops.paged_rope_append_fp8, ops.paged_attn_prefill_fp8
        decode, read = ops.paged_attn_decode_window_fp8, ops.paged_kv_read_fp8
    else:
        cache = ops.fp4_cache(8)
        append, attend = ops.paged_rope_append_fp4, ops.paged_attn_prefill_fp4
        decode, read = ops.paged_attn_decode_fp4, ops.paged_kv_read_fp4
    table = torch.tensor([[3, 0, 7], [1, 6, 4]], dtype=torch.int32, device="cuda")
    ws = ops.make_workspace(2, 3)
    as_int = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    lens = [0, 0]
    for news in [(300, 70), (129, 0), (1, 1), (1, 1), (60, 400), (1, 1)]:
        t = sum(news)
        lens = [n + m for n, m in zip(lens, news)]
        q, k, v = (torch.randn(t, h, 128, generator=g).to(torch.bfloat16).cuda() for h in (32, 8, 8))
        cu, sl = as_int([0, news[0], t]), as_int(lens)
        q = append(q, k, v, *cache, table, cu, sl, ws, rope_theta=theta, q_norm_weight=gain[0], k_norm_weight=gain[1])
        lse = torch.empty(t, 32, device="cuda")
        if news == (1, 1):
            out = decode(q, *cache, table, sl, ws, window=HUGE, lse=lse)
        else:
            out = attend(q, *cache, table, cu, sl, max(news), ws, lse=lse)
        ops.check_error(ws)
        k_all, v_all, (keys, values) = held(read, cache, table, lens, ws)
        # The tolerance of LowCache.prefill_reference over the rows read back.  Over the 8-bit cache those were rounded to
        # bf16, 2^-8 of a value at most (a score: of sum |q k| scale, a weight by as much, a V value by 2^-8 of itself).
        c = LowCache.__new__(LowCache)
        c.q, c.k, c.v, c.q_lens, c.seq_lens, c.window, c.sinks, c.bits = to_cpu(q), keys, values, news, lens, HUGE // 2, 0, bits
        ref, ref_lse, tol, lse_tol = c.prefill_reference(ops.DEFAULT_SCALE)
        if bits == 8:
            p_abs_v, _ = definitions.window_attention(c.q, keys, [x.abs() for x in values], news, lens, HUGE // 2, 0,
                                                      ops.DEFAULT_SCALE)
            a, at = torch.zeros_like(ref_lse), 0
            for kk, m in zip(keys, news):
                if m:
                    a[at:at + m] = torch.einsum("thd,nhd->thn", c.q[at:at + m].double().abs(),
                                                kk.double().abs().repeat_interleave(4, 1)).amax(-1) * ops.DEFAULT_SCALE
                at += m
            d = 2.0 ** -8 * a
            tol, lse_tol = tol + d[..., None].expm1() * (p_abs_v + ref.abs()) + 2.0 ** -8 * p_abs_v, lse_tol + d
        window_cases.check(out, ref, tol, f"{news}")
        check_lse(lse, ref_lse, lse_tol, f"{news}")
    # the rows move to a bf16 cache of another layout
    pools = [torch.full((6, 256, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    table2 = torch.tensor([[5, 2], [0, 4]], dtype=torch.int32, device="cuda")
    ops.kv_append(*pools, k_all, v_all, table2, as_int([0, lens[0], sum(lens)]), as_int(lens), ws)
    moved = ops.paged_attn_decode(q, *pools, table2, as_int(lens), ws)
    ops.check_error(ws)
    # a decode over bf16 rows rounds its weights to bf16, 2^-8 of each in numerator and denominator
    p_abs_v, _ = definitions.window_attention(c.q, keys, [x.abs() for x in values], news, lens, HUGE // 2, 0, ops.DEFAULT_SCALE)
    window_cases.check(moved, ref, window_cases.tolerance(ref, p_abs_v), "moved")
