"""paged_rope_append and paged_rope_append_fp8 on the GPU against the formulas in 64 bits.

Tolerances.  In fp32 the kernel's cosines and sines are off by at most 1.5e-6 (the angle, reduced
from an exact product, by under 1e-6; the fast sine and cosine by 2^-21.2), the norm's factor by
1e-6 relative (a chain of 19 additions, halved by the square root: 6e-7; rsqrtf 2.4e-7; two
products 1.2e-7) and each rotation's products and sum by 2e-7.  Against an element's pair size
|y[d]| + |y[d + 64]| that is under 3e-6; FP32 = 4e-6 is used.  A bf16 result adds half a step, 2^-8
of the value; an 8-bit one 2^-4 of the value, or half the smallest step, 2^-10 of the row's scale."""
import pytest
import torch

import definitions
import oracle
from gpu_helpers import gpu, lib_ready, to_cpu
from paged_gqa_attention_gb300 import ops
from paged_gqa_attention_gb300 import workloads as wl

pytestmark = gpu

FP32 = 4e-6
THETA = ops.QWEN3_ROPE_THETA


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def operands(tokens, seed, merged):
    """q, k_new, v_new as slices of one [T, 6144] projection, or tensors of their own."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(tokens, 6144, generator=g, device="cuda") * torch.exp2(
        torch.randint(-3, 4, (tokens, 1), generator=g, device="cuda").float())
    x = x.to(torch.bfloat16)
    q, k, v = (x[:, lo:hi].view(tokens, -1, 128) for lo, hi in ((0, 4096), (4096, 5120), (5120, 6144)))
    return (q, k, v) if merged else (q.contiguous(), k.contiguous(), v.contiguous())


def gains(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return [(1.0 + 0.25 * torch.randn(128, generator=g, device="cuda")).to(torch.bfloat16) for _ in range(2)]


def batch_of(lens, q_lens, seed=5):
    return wl.build_batch("rope_append", seed, lens, q_lens, num_blocks=sum((n + 255) // 256 for n in lens) + 2,
                          device="cuda")


def check_rows(got, ref, size, what):
    got = to_cpu(got).double()
    tol = 2.0 ** -8 * ref.abs() + FP32 * (1 + 2.0 ** -8) * size
    worst = ((got - ref).abs() - tol).max().item()
    assert worst <= 0, f"{what}: {worst:.3e} over the tolerance"


def check(b, q, k, v, q_got, cache, fp8, theta, positions, pair_axis, gq, gk, eps, before):
    at = definitions.places(b.block_table.tolist(), b.q_lens_host, b.seq_lens_host)
    pos = to_cpu(positions) if positions is not None else torch.tensor([p for _, p, _, _ in at])
    blk, slot = torch.tensor([x[2] for x in at]), torch.tensor([x[3] for x in at])
    cpu = lambda t: None if t is None else to_cpu(t)
    zq, sq = definitions.rotated(to_cpu(q), pos, theta, pair_axis, cpu(gq), eps)
    zk, sk = definitions.rotated(to_cpu(k), pos, theta, pair_axis, cpu(gk), eps)
    check_rows(q_got, zq, sq, "q")
    after = [to_cpu(t) for t in cache]
    if not fp8:
        check_rows(after[0][blk, slot], zk, sk, "k")
        assert torch.equal(after[1][blk, slot].view(torch.int16), to_cpu(v).view(torch.int16)), "v"
    else:
        amax = zk.abs().amax(-1)
        ks = after[2][blk, :, slot].double()
        # the row's maximum is off by at most FP32 of its pair's size, at most 2 of the maximum
        assert ((ks * 448 - amax).abs() <= 2 * FP32 * amax + 2.0 ** -22 * amax).all(), "k scale"
        val = after[0][blk, slot].view(torch.float8_e4m3fn).double() * ks[..., None]
        tol = 2.0 ** -4 * zk.abs() + 2.0 ** -10 * ks[..., None] + (1 + 2.0 ** -4) * FP32 * sk + 3 * FP32 * amax[..., None]
        assert ((val - zk).abs() <= tol).all(), "k codes"
        # v: the rule of kv_append_fp8, bit for bit
        kc, vc, ks0, vs0 = [t.numpy().copy() for t in (before[0], before[1], before[2], before[3])]
        ref = oracle.kv_append_fp8(kc, vc, ks0, vs0, to_cpu(k).contiguous(), to_cpu(v).contiguous(),
                                   to_cpu(b.block_table), to_cpu(b.cu_q_lens), to_cpu(b.seq_lens))
        assert torch.equal(after[1], torch.from_numpy(ref[1])), "v codes"
        assert torch.equal(after[3].view(torch.int32), torch.from_numpy(ref[3]).view(torch.int32)), "v scale"
    # no other cache byte moved
    for was, now in zip(before, after):
        is_scale = now.dtype == torch.float32
        keep = torch.ones(now.shape[0], 256, dtype=torch.bool)
        keep[blk, slot] = False
        a, c = (x.transpose(1, 2)[keep] if is_scale else x[keep] for x in (was, now))
        assert torch.equal(a.contiguous().view(torch.uint8), c.contiguous().view(torch.uint8)), "cache outside the rows"


CASES = [
    # lens, q_lens
    ([1], [1]),
    ([512], [1]),
    ([255, 256, 257, 3], [1, 1, 1, 1]),
    ([700, 30, 5, 1024, 300], [257, 30, 0, 1, 44]),
    ([1500], [1500]),                       # a warp takes a whole token
    ([2000, 900], [1301, 33]),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("lens,q_lens", CASES)
def test_against_the_formulas(lens, q_lens, norm, fp8):
    b = batch_of(lens, q_lens)
    q, k, v = operands(b.total_tokens, 11, merged=True)
    gq, gk = gains(12) if norm else (None, None)
    run(b, q, k, v, fp8, THETA, None, None, gq, gk, 1e-6)


def run(b, q, k, v, fp8, theta, positions, pair_axis, gq, gk, eps, q_out=None):
    cache = list(ops.fp8_cache(b.num_blocks)) if fp8 else [b.k_pool, b.v_pool]
    before = [to_cpu(t).clone() for t in cache]
    given = [t.clone() for t in (q, k, v)]
    ws = ops.make_workspace(max(b.num_seqs, 1), b.max_blocks_per_seq)
    fn = ops.paged_rope_append_fp8 if fp8 else ops.paged_rope_append
    out = fn(q, k, v, *cache, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=theta, positions=positions,
             pair_axis=pair_axis, q_norm_weight=gq, k_norm_weight=gk, norm_eps=eps, q_out=q_out)
    ops.check_error(ws)
    check(b, *given, out, cache, fp8, theta, positions, pair_axis, gq, gk, eps, before)
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("sections,interleaved", [((16, 24, 24), False), ((24, 20, 20), True), ((40, 24), False),
                                                  ((64,), False), ((0, 0, 64), False)])
def test_positions_of_several_axes(sections, interleaved, fp8):
    b = batch_of([700, 40], [333, 7])
    q, k, v = operands(b.total_tokens, 21, merged=True)
    g = torch.Generator(device="cuda")
    g.manual_seed(22)
    axes = len(sections)
    pos = torch.randint(0, 100000, (axes, b.total_tokens), generator=g, device="cuda", dtype=torch.int32)
    run(b, q, k, v, fp8, THETA, pos, ops.rope_pair_axes(sections, interleaved), *gains(23), 1e-6)


def test_given_positions_of_one_axis_far_and_negative():
    b = batch_of([300, 20], [30, 3])
    q, k, v = operands(b.total_tokens, 31, merged=False)
    pos = torch.tensor([2 ** 24 - 1 - 400000 * i for i in range(b.total_tokens - 2)] + [-1, -(2 ** 24) + 1],
                       dtype=torch.int32, device="cuda")
    run(b, q, k, v, False, THETA, pos, None, None, None, 0.0)
    run(b, q, k, v, False, 10000.0, pos, None, *gains(3), 1e-5)


@pytest.mark.parametrize("norm", [False, True])
def test_without_a_rotation(norm):
    b = batch_of([300, 20], [30, 3])
    q, k, v = operands(b.total_tokens, 41, merged=True)
    gq, gk = gains(42) if norm else (None, None)
    out = run(b, q, k, v, False, 0.0, None, None, gq, gk, 1e-6)
    if not norm:
        assert torch.equal(out, q)


def test_infinite_values_stay_where_they_are_without_a_rotation():
    b = batch_of([20], [3])
    q, k, v = operands(3, 43, merged=False)
    q[0, 0, 5], k[1, 2, 70], v[2, 7, 0] = float("inf"), float("-inf"), float("nan")
    ws = ops.make_workspace(1, 1)
    out = ops.paged_rope_append(q, k, v, b.k_pool, b.v_pool, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=0.0)
    ops.check_error(ws)
    blk = int(b.block_table[0, 0])
    assert torch.equal(out.view(torch.int16), q.view(torch.int16))
    assert torch.equal(b.k_pool[blk, 17:20].view(torch.int16), k.view(torch.int16))
    assert torch.equal(b.v_pool[blk, 17:20].view(torch.int16), v.view(torch.int16))


@pytest.mark.parametrize("tokens", [3, 1400])
def test_in_place(tokens):
    b = batch_of([tokens + 9], [tokens])
    q, k, v = operands(tokens, 51, merged=False)
    out = run(b, q, k, v, False, THETA, None, None, *gains(52), 1e-6, q_out=q)
    assert out.data_ptr() == q.data_ptr()


@pytest.mark.parametrize("fp8", [False, True])
def test_far_in_the_pool(fp8):
    """Rows whose offset in the pool passes 2^31 elements."""
    b = batch_of([300], [100])
    q, k, v = operands(100, 55, merged=True)
    blocks = 9000                                # 9000 * 262144 elements
    table = torch.full_like(b.block_table, -1)
    table[0, 0], table[0, 1] = blocks - 1, blocks - 3
    if fp8:
        cache = [torch.zeros(blocks, 256, 8, 128, dtype=torch.uint8, device="cuda") for _ in range(2)]
        cache += [torch.zeros(blocks, 8, 256, device="cuda") for _ in range(2)]
    else:
        cache = [torch.zeros(blocks, 256, 8, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    small = [t[:b.num_blocks].clone() for t in cache]
    ws = ops.make_workspace(1, b.max_blocks_per_seq)
    fn = ops.paged_rope_append_fp8 if fp8 else ops.paged_rope_append
    fn(q, k, v, *cache, table, b.cu_q_lens, b.seq_lens, ws, rope_theta=THETA)
    fn(q, k, v, *small, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=THETA)
    ops.check_error(ws)
    for far, near in zip(cache, small):
        for j, blk in enumerate((blocks - 1, blocks - 3)):
            assert torch.equal(far[blk].view(torch.uint8), near[int(b.block_table[0, j])].view(torch.uint8))
        assert not far[:blocks - 3].any() and not far[blocks - 2].any()


def test_zero_rows_and_8_bit_scale_of_one():
    b = batch_of([20], [2])
    q, k, v = operands(2, 61, merged=True)
    q[0, 0], k[0, 3], v[1, 4] = 0.0, 0.0, 0.0
    cache = ops.fp8_cache(b.num_blocks)
    ws = ops.make_workspace(1, 1)
    out = ops.paged_rope_append_fp8(q, k, v, *cache, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=THETA)
    ops.check_error(ws)
    blk = int(b.block_table[0, 0])
    assert (out[0, 0] == 0).all()
    assert (cache[0][blk, 18, 3] & 0x7F == 0).all() and cache[2][blk, 3, 18] == 1
    assert (cache[1][blk, 19, 4] == 0).all() and cache[3][blk, 4, 19] == 1


@pytest.mark.parametrize("pad", [1, 40, 1500])
def test_tokens_behind_the_last_sequence_are_left_alone(pad):
    b = batch_of([300, 257], [5, 257])
    t = b.total_tokens
    q, k, v = operands(t + pad, 71, merged=True)
    before = [to_cpu(b.k_pool).clone(), to_cpu(b.v_pool).clone()]
    ws = ops.make_workspace(2, b.max_blocks_per_seq)
    out = torch.full((t + pad, 32, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.paged_rope_append(q, k, v, b.k_pool, b.v_pool, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=THETA,
                          q_out=out)
    ops.check_error(ws)
    assert (out[t:] == 7.0).all()
    check(b, q[:t], k[:t], v[:t], out[:t], [b.k_pool, b.v_pool], False, THETA, None, None, None, None, 0.0, before)


def test_no_tokens_is_nothing_to_do():
    b = batch_of([20], [0])
    e = lambda h: torch.empty(0, h, 128, dtype=torch.bfloat16, device="cuda")
    ws = ops.make_workspace(1, 1)
    out = ops.paged_rope_append(e(32), e(8), e(8), b.k_pool, b.v_pool, b.block_table, b.cu_q_lens, b.seq_lens, ws,
                                rope_theta=THETA)
    assert out.shape == (0, 32, 128)
    ops.check_error(ws)


def test_a_row_does_not_depend_on_its_batch():
    """One token alone, and the same token within 1500 (another split of the work): the same bits."""
    b = batch_of([1600], [1500])
    q, k, v = operands(1500, 81, merged=True)
    ws = ops.make_workspace(1, b.max_blocks_per_seq)
    gq, gk = gains(82)
    kw = dict(rope_theta=THETA, q_norm_weight=gq, k_norm_weight=gk)
    out = ops.paged_rope_append(q, k, v, b.k_pool, b.v_pool, b.block_table, b.cu_q_lens, b.seq_lens, ws, **kw)
    kp, vp = b.k_pool.clone(), b.v_pool.clone()
    i = 777
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    lens = torch.tensor([100 + i + 1], dtype=torch.int32, device="cuda")
    one = ops.paged_rope_append(q[i:i + 1], k[i:i + 1], v[i:i + 1], b.k_pool, b.v_pool, b.block_table, cu, lens, ws, **kw)
    ops.check_error(ws)
    assert torch.equal(one[0], out[i])
    same = lambda x, y: torch.equal(x.view(torch.int16), y.view(torch.int16))
    assert same(kp, b.k_pool) and same(vp, b.v_pool)


def test_device_checks_record_errors_and_write_nothing_else():
    b = batch_of([300, 300], [2, 2])
    q, k, v = operands(4, 91, merged=True)
    ws = ops.make_workspace(2, b.max_blocks_per_seq)
    same = lambda x, y: torch.equal(x.view(torch.int16), y.view(torch.int16))

    def call(table=b.block_table, cu=b.cu_q_lens, lens=b.seq_lens, **kw):
        pools = b.k_pool.clone(), b.v_pool.clone()
        out = ops.paged_rope_append(q, k, v, *pools, table, cu, lens, ws, rope_theta=THETA, **kw)
        with pytest.raises(ops.PagedAttnError) as e:
            ops.check_error(ws)
        assert e.value.status == 4
        return out, pools, e.value.detail

    good_q = ops.paged_rope_append(q, k, v, b.k_pool.clone(), b.v_pool.clone(), b.block_table, b.cu_q_lens, b.seq_lens,
                                   ws, rope_theta=THETA)
    ops.check_error(ws)
    for bad in (-1, b.num_blocks, 2 ** 31 - 1):
        table = b.block_table.clone()
        table[1, 1] = bad
        out, pools, word = call(table=table)
        assert word & (1 << 8) and torch.equal(out, good_q)
        blk, row = int(b.block_table[0, 1]), 298 % 256
        pools[0][blk, row:row + 2] = b.k_pool[blk, row:row + 2]
        pools[1][blk, row:row + 2] = b.v_pool[blk, row:row + 2]
        assert same(pools[0], b.k_pool) and same(pools[1], b.v_pool)
    for n in (1, 0, -5, 257 * 256):
        out, _, word = call(lens=torch.tensor([300, n], dtype=torch.int32, device="cuda"))
        assert word & (1 << 9) and out[2:].isnan().all() and torch.equal(out[:2], good_q[:2])
    _, _, word = call(cu=torch.tensor([0, 2, 9], dtype=torch.int32, device="cuda"))
    assert word & (1 << 10)
    _, _, word = call(cu=torch.tensor([1, 2, 4], dtype=torch.int32, device="cuda"))
    assert word & (1 << 10)
    pos = torch.tensor([5, 2 ** 24, -(2 ** 24), 6], dtype=torch.int32, device="cuda")
    out, pools, word = call(positions=pos)
    assert word & (1 << 12) and out[1:3].isnan().all() and not out[0].isnan().any() and not out[3].isnan().any()


def test_on_a_side_stream_and_in_a_graph():
    b = batch_of([300, 300], [1, 1])
    q, k, v = operands(2, 101, merged=True)
    ws = ops.make_workspace(2, b.max_blocks_per_seq)
    want = ops.paged_rope_append(q, k, v, b.k_pool, b.v_pool, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=THETA)
    pools = b.k_pool.clone(), b.v_pool.clone()
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = ops.paged_rope_append(q, k, v, *pools, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=THETA, stream=st)
    st.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    out = torch.empty_like(want)
    with torch.cuda.graph(graph):
        ops.paged_rope_append(q, k, v, *pools, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=THETA, q_out=out)
    for n in (300, 301, 302):                     # the lengths and rows move on between replays
        b.seq_lens.fill_(n)
        q.copy_(torch.roll(q, 1, 0))
        graph.replay()
        want = ops.paged_rope_append(q, k, v, b.k_pool, b.v_pool, b.block_table, b.cu_q_lens, b.seq_lens, ws,
                                     rope_theta=THETA)
        assert torch.equal(out, want)
        assert torch.equal(pools[0].view(torch.int16), b.k_pool.view(torch.int16))
    ops.check_error(ws)


def test_8_bit_rows_of_extreme_and_odd_values_are_those_of_kv_append_fp8():
    """v rows (and k rows without norm or rotation) from the smallest to the largest bf16, with
    signed zeros, infinities and NaN: the same codes and scales as kv_append_fp8, bit for bit."""
    t = 400
    b = batch_of([t], [t])
    g = torch.Generator(device="cuda")
    g.manual_seed(111)
    x = torch.randn(t, 6144, generator=g, device="cuda")
    x = x.view(t, 48, 128) * torch.exp2(torch.randint(-132, 127, (t, 48, 1), generator=g, device="cuda").float())
    x[:, :, ::7] *= 2.0 ** -9
    x[:, :, 3], x[:, :, 4] = 0.0, -0.0
    x = x.to(torch.bfloat16)
    x[5, :, 9], x[6, :, 9], x[7, :, 9] = float("inf"), float("-inf"), float("nan")
    x[8] = 0.0
    x[9] = -0.0
    q, k, v = x[:, :32], x[:, 32:40], x[:, 40:]
    ws = ops.make_workspace(1, b.max_blocks_per_seq)
    got, want = ops.fp8_cache(b.num_blocks), ops.fp8_cache(b.num_blocks)
    ops.paged_rope_append_fp8(q, k, v, *got, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=0.0)
    ops.kv_append_fp8(*want, k.contiguous(), v.contiguous(), b.block_table, b.cu_q_lens, b.seq_lens, ws)
    ops.check_error(ws)
    for a, c in zip(got, want):
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


def rows_of(cache, blk, slot, fp8):
    """The bytes of the cache's rows at (blk, slot), by tensor."""
    out = []
    for i, t in enumerate(cache):
        t = t.transpose(1, 2) if fp8 and i >= 2 else t          # scales are [block][head][slot]
        out.append(to_cpu(t)[blk, slot].contiguous().view(torch.uint8))
    return out


def random_cache(b, fp8, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if not fp8:
        return [torch.randn(t.shape, generator=g, device="cuda").to(torch.bfloat16) for t in (b.k_pool, b.v_pool)]
    codes, _, scales, _ = ops.fp8_cache(b.num_blocks)
    return ([torch.randint(0, 120, codes.shape, generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
            + [torch.rand(scales.shape, generator=g, device="cuda") for _ in range(2)])


def append_with_an_error(b, q, k, v, cache, fp8, cu=None, lens=None, **kw):
    """(q_out, error word) of a call whose device-side check records an error."""
    ws = ops.make_workspace(b.num_seqs, b.max_blocks_per_seq)
    fn = ops.paged_rope_append_fp8 if fp8 else ops.paged_rope_append
    out = fn(q, k, v, *cache, b.block_table, b.cu_q_lens if cu is None else cu, b.seq_lens if lens is None else lens,
             ws, rope_theta=THETA, **kw)
    with pytest.raises(ops.PagedAttnError) as e:
        ops.check_error(ws)
    assert e.value.status == 4
    return out, e.value.detail


def check_only_good_rows_moved(b, before, cache, want, good, fp8):
    """Rows of the good tokens are those of `want`, a cache that a call without errors wrote; every
    other byte is what it was."""
    at = definitions.places(b.block_table.tolist(), b.q_lens_host, b.seq_lens_host)
    blk, slot = torch.tensor([x[2] for x in at]), torch.tensor([x[3] for x in at])
    for got, ref in zip(rows_of(cache, blk[good], slot[good], fp8), rows_of(want, blk[good], slot[good], fp8)):
        assert torch.equal(got, ref), "a good token's row"
    for i, (was, now) in enumerate(zip(before, cache)):
        scale = fp8 and i >= 2
        was, now = (to_cpu(t).transpose(1, 2) if scale else to_cpu(t) for t in (was, now))
        keep = torch.ones(now.shape[0], 256, dtype=torch.bool)
        keep[blk[good], slot[good]] = False
        assert torch.equal(was[keep].contiguous().view(torch.uint8), now[keep].contiguous().view(torch.uint8)), \
            "bytes outside the good tokens' rows"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("tokens", [1, 4, 405, 1500])
def test_a_position_out_of_range_moves_no_cache_byte(tokens, fp8):
    """Neither the K nor the V row of such a token is written, however the batch is cut into runs
    (one group a warp up to 405 tokens; at 1500 the runs begin at every group)."""
    b = batch_of([tokens + 30], [tokens])
    q, k, v = operands(tokens, 121, merged=True)
    g = torch.Generator().manual_seed(122)
    pos = torch.randint(0, 100000, (3, tokens), generator=g, dtype=torch.int32)
    bad = torch.rand(tokens, generator=g) < 0.4
    bad[0] = True
    axis = torch.randint(0, 3, (tokens,), generator=g)
    far = torch.tensor([2 ** 24, -(2 ** 24), 2 ** 31 - 1, -(2 ** 31)], dtype=torch.int32)
    wrong = pos.clone()
    wrong[axis[bad], bad.nonzero().flatten()] = far[torch.arange(int(bad.sum())) % 4]
    kw = dict(pair_axis=ops.rope_pair_axes((16, 24, 24)))
    cache = random_cache(b, fp8, 123)
    before = [t.clone() for t in cache]
    want = [t.clone() for t in cache]
    fn = ops.paged_rope_append_fp8 if fp8 else ops.paged_rope_append
    ws = ops.make_workspace(1, b.max_blocks_per_seq)
    q_want = fn(q, k, v, *want, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=THETA, positions=pos.cuda(), **kw)
    ops.check_error(ws)
    out, word = append_with_an_error(b, q, k, v, cache, fp8, positions=wrong.cuda(), **kw)
    good = ~bad
    assert word & (1 << 12)
    assert to_cpu(out)[bad].isnan().all() and torch.equal(to_cpu(out)[good], to_cpu(q_want)[good])
    check_only_good_rows_moved(b, before, cache, want, good, fp8)


@pytest.mark.parametrize("fp8", [False, True])
def test_inconsistent_lengths_and_offsets_move_no_other_cache_byte(fp8):
    """Tokens of a sequence whose length or whose offsets are inconsistent get a NaN q row and no
    cache row; the other tokens' rows are as in a batch without errors."""
    b = batch_of([300, 300], [2, 2])
    q, k, v = operands(4, 141, merged=True)
    start = random_cache(b, fp8, 142)
    want = [t.clone() for t in start]
    fn = ops.paged_rope_append_fp8 if fp8 else ops.paged_rope_append
    ws = ops.make_workspace(2, b.max_blocks_per_seq)
    q_want = fn(q, k, v, *want, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=THETA)
    ops.check_error(ws)
    low, high = -(2 ** 31), 2 ** 31 - 1
    cases = [(dict(lens=[300, n]), 1 << 9, [True, True, False, False]) for n in (1, 0, -5, 257 * 256, low, high)]
    first, second = [False, False, True, True], [True, True, False, False]
    cases += [(dict(cu=[0, 2, 9]), 1 << 10, second), (dict(cu=[0, 2, high]), 1 << 10, second),
              (dict(cu=[-1, 2, 4]), 1 << 10, first), (dict(cu=[low, 2, 4]), 1 << 10, first),
              (dict(cu=[low, 2, 4], lens=[1, 300]), 1 << 10, first),
              (dict(cu=[low + 500, 2, 4], lens=[low + 1, 300]), 1 << 10, first)]
    for change, bit, good in cases:
        change = {n: torch.tensor(x, dtype=torch.int32, device="cuda") for n, x in change.items()}
        cache = [t.clone() for t in start]
        out, word = append_with_an_error(b, q, k, v, cache, fp8, **change)
        good = torch.tensor(good)
        assert word & bit, change
        assert to_cpu(out)[~good].isnan().all() and torch.equal(to_cpu(out)[good], to_cpu(q_want)[good]), change
        check_only_good_rows_moved(b, start, cache, want, good, fp8)


def test_a_negative_end_of_the_batch_is_an_error():
    b = batch_of([300, 300], [2, 2])
    q, k, v = operands(4, 151, merged=True)
    for last in (-1, -(2 ** 31)):
        cache = random_cache(b, False, 152)
        before = [t.clone() for t in cache]
        cu = torch.tensor([0, 0, last], dtype=torch.int32, device="cuda")
        out = torch.full((4, 32, 128), 7.0, dtype=torch.bfloat16, device="cuda")
        _, word = append_with_an_error(b, q, k, v, cache, False, cu=cu, q_out=out)
        assert word & (1 << 10)
        assert all(torch.equal(x, y) for x, y in zip(cache, before)) and (out == 7.0).all()


def test_a_k_row_too_small_for_its_scale_is_kept():
    """Normalised K rows of at most 2^-141.2, whose maximum / 448 rounds to 0 in fp32: no NaN codes.
    Such a row is quantised by the smallest scale there is, 2^-149.  A value is off by its code's
    half step, 2^-4 of it, and by fp32's at its size: y = x * factor * gain is rounded to a
    multiple of 2^-149 once, on top of FP32's relative error."""
    t = 6
    b = batch_of([t + 9], [t])
    q, k, v = operands(t, 131, merged=False)
    g = torch.Generator(device="cuda")
    g.manual_seed(132)
    size = torch.tensor([0.0, 1.0, 3.0, 30.0, 100.0, 200.0], device="cuda")     # of the largest, in 2^-149
    x = torch.rand(t, 8, 128, generator=g, device="cuda") * 2 - 1
    x[..., 5], x[..., 100], x[..., 7] = 1.0, -1.0, 0.0
    # x * 2^-120 * (1 / sqrt(eps = 1)) * 2^-29: the mean square of 2^-120 vanishes beside eps
    k.copy_((x * size[:, None, None] * 2.0 ** -120).to(torch.bfloat16))
    gain = torch.full((128,), 2.0 ** -29, dtype=torch.bfloat16, device="cuda")
    cache = ops.fp8_cache(b.num_blocks)
    ws = ops.make_workspace(1, b.max_blocks_per_seq)
    ops.paged_rope_append_fp8(q, k, v, *cache, b.block_table, b.cu_q_lens, b.seq_lens, ws, rope_theta=0.0,
                              q_norm_weight=gain, k_norm_weight=gain, norm_eps=1.0)
    ops.check_error(ws)
    at = definitions.places(b.block_table.tolist(), b.q_lens_host, b.seq_lens_host)
    blk, slot = torch.tensor([x[2] for x in at]), torch.tensor([x[3] for x in at])
    ref, _ = definitions.rotated(to_cpu(k), torch.zeros(t), 0.0, gain=to_cpu(gain), eps=1.0)
    scale = to_cpu(cache[2])[blk, :, slot].double()
    got = to_cpu(cache[0])[blk, slot].view(torch.float8_e4m3fn).double() * scale[..., None]
    assert (scale[0] == 1).all() and (scale[1:] == 2.0 ** -149).all()
    assert ((got - ref).abs() <= 2.0 ** -4 * ref.abs() + (1 + 2.0 ** -4) * (2.0 ** -150 + FP32 * ref.abs())).all()
