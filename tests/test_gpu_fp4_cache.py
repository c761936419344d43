"""The 4-bit cache written and the low-bit caches read back, on the GPU against the rule in 64 bits
(lowbit_cases.py): codes, scales and exponents bit for bit."""
import pytest
import torch

import definitions
from gpu_helpers import gpu, lib_ready, to_cpu
from lowbit_cases import pack4, quantise4, unpack4, values4
from paged_gqa_attention_gb300 import ops

pytestmark = gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    lib_ready()


def batch(q_lens, seq_lens, seed=0, spare=1, dev="cuda"):
    """(table, cu, lens) on the device and the new tokens' places."""
    g = torch.Generator().manual_seed(seed)
    width = max((n + 255) // 256 for n in seq_lens) + spare
    need = [(n + 255) // 256 for n in seq_lens]
    free = torch.randperm(sum(need) + 2, generator=g).tolist()
    table = [[free.pop() for _ in range(n)] + [-1] * (width - n) for n in need]
    cu = [0]
    for q in q_lens:
        cu.append(cu[-1] + q)
    as_int = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    return as_int(table), as_int(cu), as_int(seq_lens), definitions.places(table, q_lens, seq_lens), sum(need) + 2


def rows(t, seed, kind="normal"):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(t, 8, 128, generator=g)
    if kind == "outliers":                    # a few dims and tokens far above the rest
        x[..., 5] *= 300
        x[::3] *= 1e4
        x[1::3] *= 1e-4
    if kind == "grid":                        # quotients on and beside every midpoint
        x = torch.randint(-96, 97, (t, 8, 128), generator=g) / 4.0
    if kind == "extreme":
        x = x * torch.exp2(torch.randint(-130, 120, (t, 8, 1), generator=g).float())
        x[::5, 0] = 0.0
        x[::7, 1, 16:32] = 0.0
        x[0, 2] = torch.finfo(torch.bfloat16).max
        x[0, 3] = 2.0 ** -133
        x[0, 4] = -0.0
        x[0, 5, 0], x[0, 6, 127], x[0, 7, 64] = float("inf"), float("nan"), float("-inf")
    return x.to(torch.bfloat16)


def expect(cache, k, v, where):
    """The six tensors after appending k and v to (a host copy of) `cache`."""
    want = [to_cpu(t).clone() for t in cache]
    for i, x in enumerate((k, v)):
        codes, scale, exp = quantise4(x)
        for t, (_, _, blk, slot) in enumerate(where):
            want[i][blk, slot] = pack4(codes[t])
            want[2 + i][blk, :, slot] = scale[t]
            want[4 + i][blk, :, slot] = exp[t]
    return want


def same(got, want):
    """All six tensors alike; rows under the exponent 255 (NaN) in that exponent alone."""
    got = [to_cpu(t) for t in got]
    for i in range(2):
        assert torch.equal(got[4 + i], want[4 + i])
        live = want[4 + i] != 255
        assert torch.equal(got[2 + i][live], want[2 + i][live])
        live = live.transpose(1, 2)
        a, b = unpack4(got[i])[live], unpack4(want[i])[live]
        assert torch.equal(a, b), f"{(a != b).sum().item()} codes of {a.numel()} differ"


@pytest.mark.parametrize("kind", ["normal", "outliers", "grid", "extreme"])
@pytest.mark.parametrize("q_lens,seq_lens", [([1], [1]), ([1] * 9, [1, 5, 255, 256, 257, 300, 512, 513, 1000]),
                                             ([300, 0, 17, 257], [300, 40, 1000, 513])])
def test_append(q_lens, seq_lens, kind):
    table, cu, lens, where, blocks = batch(q_lens, seq_lens)
    cache = ops.fp4_cache(blocks)
    k, v = rows(len(where), 1, kind), rows(len(where), 2, kind)
    want = expect(cache, k, v, where)
    ws = ops.make_workspace(len(q_lens), table.shape[1])
    ops.kv_append_fp4(*cache, k.cuda(), v.cuda(), table, cu, lens, ws)
    ops.check_error(ws)
    same(cache, want)
    # and read back, from a position within each sequence's new tokens, with rows behind the last one
    first = [n - q + q // 3 for q, n in zip(q_lens, seq_lens)]
    cu2 = [0]
    for q, n, f in zip(q_lens, seq_lens, first):
        cu2.append(cu2[-1] + n - f)
    total = cu2[-1] + 3
    outs = [torch.full((total, 8, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    as_int = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    got = ops.paged_kv_read_fp4(*cache, table, as_int(cu2), as_int(first), total, ws, k_out=outs[0], v_out=outs[1])
    ops.check_error(ws)
    for i in range(2):
        w = values4(unpack4(want[i]), want[2 + i].transpose(1, 2), want[4 + i].transpose(1, 2))
        at = [(int(table[s, p // 256]), p % 256) for s, (n, f) in enumerate(zip(seq_lens, first)) for p in range(f, n)]
        blk, slot = (torch.tensor(x) for x in zip(*at))
        ref = w[blk, slot]
        have = to_cpu(got[i])
        assert torch.equal(have[cu2[-1]:], torch.full((3, 8, 128), 7.0, dtype=torch.bfloat16))
        have = have[:cu2[-1]].double()
        assert torch.equal(have.isnan(), ref.isnan())
        fine = ~ref.isnan()
        # 6 bits times a power of two: bf16 holds it, up to half a step of the smallest (2^-134) below the normal
        # range, and infinity where the codes stand for more than the largest (bf16's largest, 2040 * 2^117, takes
        # the scale 352 and the code 6: 2112 * 2^117, past 2^128)
        near = ((have - ref).abs() <= 2.0 ** -134) & (ref.abs() < 2.0 ** -126)
        assert (near | (have == ref.to(torch.bfloat16).double()))[fine].all()


@pytest.mark.parametrize("norm,theta,axes", [(True, 1e6, 1), (False, 0.0, 1), (False, 1e4, 3)])
def test_rope_append(norm, theta, axes):
    """q and k as paged_rope_append computes them; the row's rounding to 4 bits is checked against the
    64-bit row: k within half a step of its code, where the scale's own rounding is the kernel's."""
    q_lens, seq_lens = [70, 1, 200], [500, 300, 200]
    table, cu, lens, where, blocks = batch(q_lens, seq_lens)
    t = len(where)
    g = torch.Generator().manual_seed(3)
    y = torch.randn(t, 48 * 128, generator=g).to(torch.bfloat16).cuda()
    q, k, v = (y[:, lo:hi].view(t, -1, 128) for lo, hi in ((0, 4096), (4096, 5120), (5120, 6144)))
    gain = (1 + 0.25 * torch.randn(128, generator=g)).to(torch.bfloat16).cuda()
    kw = dict(rope_theta=theta)
    if norm:
        kw.update(q_norm_weight=gain, k_norm_weight=gain)
    if axes > 1:
        kw.update(positions=torch.randint(0, 5000, (axes, t), generator=g).to(torch.int32).cuda(),
                  pair_axis=ops.rope_pair_axes((16, 24, 24)))
    ws = ops.make_workspace(3, table.shape[1])
    cache = ops.fp4_cache(blocks)
    out = ops.paged_rope_append_fp4(q, k, v, *cache, table, cu, lens, ws, **kw)
    kp = torch.zeros(blocks, 256, 8, 128, dtype=torch.bfloat16, device="cuda")
    ref_q = ops.paged_rope_append(q, k, v, kp, kp.clone(), table, cu, lens, ws, **kw)
    ops.check_error(ws)
    assert torch.equal(out, ref_q)
    # v: bit for bit
    want = expect(ops.fp4_cache(blocks), to_cpu(k).contiguous(), to_cpu(v).contiguous(), where)
    same([cache[1]] * 2 + [cache[3]] * 2 + [cache[5]] * 2, [want[1]] * 2 + [want[3]] * 2 + [want[5]] * 2)
    # k: the definition's rows, 4e-6 of a pair's size off at most (test_gpu_rope_append.py)
    p = kw["positions"].cpu() if axes > 1 else torch.tensor([w[1] for w in where])
    z, size = definitions.rotated(to_cpu(k), p, theta, kw.get("pair_axis"), to_cpu(gain) if norm else None,
                                  ops.QWEN3_NORM_EPS)
    b, s = torch.tensor([w[2] for w in where]), torch.tensor([w[3] for w in where])
    codes, scale, exp = (to_cpu(cache[0])[b, s], to_cpu(cache[2])[b, :, s], to_cpu(cache[4])[b, :, s])
    off = 4e-6 * size
    low, high = quantise4(z * (1 - 2.0 ** -20)), quantise4(z * (1 + 2.0 ** -20))
    assert ((exp == low[2]) | (exp == high[2])).all()
    # the scale: within half a step of max|y| / 6, up to that error
    unit = torch.ldexp(torch.ones(exp.shape, dtype=torch.float64), exp.int() - 127)[..., None]
    top = z.unflatten(-1, (8, 16)).abs().amax(-1) / unit / 6
    err = off.unflatten(-1, (8, 16)).amax(-1) / unit / 6
    sv = scale.view(torch.float8_e4m3fn).double()
    assert ((sv - top).abs() <= torch.maximum(top * 2.0 ** -4, torch.full_like(top, 2.0 ** -10)) * (1 + 2.0 ** -4) + err).all()
    # the codes: the nearest of their neighbours, up to that error (beyond 6: clamped)
    val = values4(unpack4(codes), scale, exp)
    step = sv.repeat_interleave(16, -1) * unit
    mag = (val / torch.where(step > 0, step, 1.0)).abs()
    half = torch.where(mag < 2, 0.25, torch.where(mag < 4, 0.5, 1.0))
    over = (z.abs() - 6 * step).clamp(min=0)
    lone = torch.where(step > 0, half * step, 2.0 ** -10 * 6 * unit.expand_as(step))
    assert ((val - z).abs() <= torch.maximum(lone, over) * (1 + 1e-12) + off).all()


@pytest.mark.parametrize("lens,first,rows_", [([1], [0], [1]), ([1000], [300], [333]), ([700, 20, 2000, 256], [0, 19, 255, 256],
                                              [700, 1, 1745, 0]), ([513] * 40, list(range(40)), [3 * i % 41 for i in range(40)])])
def test_read_fp8(lens, first, rows_):
    table, _, _, _, blocks = batch([0] * len(lens), lens, seed=4)
    g = torch.Generator().manual_seed(5)
    codes = [torch.randint(0, 256, (blocks, 256, 8, 128), generator=g).to(torch.uint8) for _ in range(2)]
    scales = [torch.exp(2 * torch.randn(blocks, 8, 256, generator=g)) for _ in range(2)]
    cu = [0]
    for n in rows_:
        cu.append(cu[-1] + n)
    as_int = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = ops.make_workspace(len(lens), table.shape[1])
    cache = [t.cuda() for t in (*codes, *scales)]
    got = ops.paged_kv_read_fp8(*cache, table, as_int(cu), as_int(first), cu[-1], ws)
    ops.check_error(ws)
    where = [(int(table[s, p // 256]), p % 256) for s in range(len(lens)) for p in range(first[s], first[s] + rows_[s])]
    b, o = (torch.tensor(x) for x in zip(*where))
    for i in range(2):
        ref = (codes[i][b, o].view(torch.float8_e4m3fn).float() * scales[i][b, :, o][..., None]).to(torch.bfloat16)
        assert torch.equal(to_cpu(got[i]).view(torch.int16), ref.view(torch.int16)) or (
            torch.equal(to_cpu(got[i]).isnan(), ref.isnan()) and torch.equal(to_cpu(got[i]).nan_to_num(), ref.nan_to_num()))


@pytest.mark.parametrize("bits", [8, 4])
def test_read_device_checks(bits):
    """Rows that cannot be found are NaN, the others right, and the error is recorded."""
    table, _, _, _, blocks = batch([0] * 3, [600, 600, 600], seed=6)
    cache = ops.fp8_cache(blocks) if bits == 8 else ops.fp4_cache(blocks)
    new = rows(1800, 9).cuda()
    as_int = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = ops.make_workspace(3, table.shape[1])
    append = ops.kv_append_fp8 if bits == 8 else ops.kv_append_fp4
    read = ops.paged_kv_read_fp8 if bits == 8 else ops.paged_kv_read_fp4
    append(*cache, new, new, table, as_int([0, 600, 1200, 1800]), as_int([600] * 3), ws)
    cu, first = as_int([0, 100, 200, 300]), as_int([200, 200, 200])
    good = read(*cache, table, cu, first, 300, ws)
    ops.check_error(ws)
    assert not good[0].isnan().any()

    def bad(word, nan, **kw):
        a = dict(table=table, cu=cu, first=first)
        a.update(kw)
        got = read(*cache, a["table"], a["cu"], a["first"], 300, ws)
        with pytest.raises(ops.PagedAttnError) as e:
            ops.check_error(ws)
        assert e.value.detail & word and e.value.status == 4
        for x, y in zip(got, good):
            assert x[nan].isnan().all()
            keep = torch.ones(300, dtype=torch.bool)
            keep[nan] = False
            assert torch.equal(x[keep.cuda()], y[keep.cuda()])

    t = table.clone()
    t[1, 0] = blocks
    bad(1 << 8, slice(100, 156), table=t)
    t[1, 0] = -1
    bad(1 << 8, slice(100, 156), table=t)
    for f in (-1, -(2 ** 31), table.shape[1] * 256, 2 ** 31 - 1):
        bad(1 << 9, slice(100, 200), first=as_int([200, f, 200]))
    near = table.clone().clamp_(min=0)                       # the table ends 50 rows behind this position
    keep = read(*cache, near, cu, as_int([200, table.shape[1] * 256 - 100, 200]), 300, ws)
    ops.check_error(ws)
    got = read(*cache, near, cu, as_int([200, table.shape[1] * 256 - 50, 200]), 300, ws)
    with pytest.raises(ops.PagedAttnError):
        ops.check_error(ws)
    assert torch.equal(got[0][100:150].nan_to_num(), keep[0][150:200].nan_to_num()) and got[0][150:200].isnan().all()
    # offsets that do not increase, begin past 0 or end past the rows
    for wrong in ([5, 100, 200, 300], [0, 100, 200, 301], [0, 400, 200, 300], [-7, 100, 200, 300]):
        got = read(*cache, table, as_int(wrong), first, 300, ws)
        with pytest.raises(ops.PagedAttnError) as e:
            ops.check_error(ws)
        assert e.value.detail & (1 << 10)
    ops.check_error(ws)


@pytest.mark.parametrize("bits", [8, 4])
def test_read_far_in_the_pool(bits):
    """Code offsets past 2^31 bytes (8 bits) and past 2^31 values (4 bits)."""
    blocks = 8200 if bits == 8 else 16400
    table = torch.tensor([[blocks - 1, blocks - 2]], dtype=torch.int32, device="cuda")
    cache = ops.fp8_cache(blocks) if bits == 8 else ops.fp4_cache(blocks)
    new = rows(300, 9).cuda()
    as_int = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = ops.make_workspace(1, 2)
    append = ops.kv_append_fp8 if bits == 8 else ops.kv_append_fp4
    read = ops.paged_kv_read_fp8 if bits == 8 else ops.paged_kv_read_fp4
    append(*cache, new, -new, table, as_int([0, 300]), as_int([300]), ws)
    k, v = read(*cache, table, as_int([0, 300]), as_int([0]), 300, ws)
    ops.check_error(ws)
    assert torch.equal(k, -v)
    # half a step of the codes, and of the scale in 4 bits (the largest value of a group may be clamped)
    assert ((k - new).abs().float() <= new.abs().float().unflatten(-1, (8, 16)).amax(-1, keepdim=True).expand(-1, -1, -1, 16)
            .flatten(-2) * (2.0 ** -4 if bits == 8 else 0.25)).all()


@pytest.mark.parametrize("bits", [8, 4])
def test_append_and_read_on_another_stream_and_in_a_graph(bits):
    q_lens, seq_lens = [5, 300], [261, 300]
    table, cu, lens, where, blocks = batch(q_lens, seq_lens, seed=8)
    new = rows(len(where), 10).cuda()
    first = (lens - torch.tensor(q_lens, dtype=torch.int32, device="cuda")).contiguous()
    ws = ops.make_workspace(2, table.shape[1])
    append = ops.kv_append_fp8 if bits == 8 else ops.kv_append_fp4
    read = ops.paged_kv_read_fp8 if bits == 8 else ops.paged_kv_read_fp4
    make = lambda: ops.fp8_cache(blocks) if bits == 8 else ops.fp4_cache(blocks)
    cache = make()
    append(*cache, new, new, table, cu, lens, ws)
    want = read(*cache, table, cu, first, len(where), ws)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    other = make()
    torch.cuda.synchronize()
    append(*other, new, new, table, cu, lens, ws, stream=st)
    got = read(*other, table, cu, first, len(where), ws, stream=st)
    st.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    third = make()
    outs = [torch.empty_like(new), torch.empty_like(new)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        append(*third, new, new, table, cu, lens, ws)
        read(*third, table, cu, first, len(where), ws, k_out=outs[0], v_out=outs[1])
    for _ in range(3):
        for o in outs:
            o.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(outs, want))
    ops.check_error(ws)
