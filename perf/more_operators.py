"""What is timed of the low-bit cache's operators, and their plain forms.

Four operators around the 256-token paged KV cache of 8 KV heads x 128 dims read by 32 query heads, held
in 8 bits (E4M3 codes, an fp32 scale a row) or in 4 (E2M1 codes, an E4M3 scale for every 16 of them, a
power of two a row):

  append   the new tokens' k and v rows quantised into the 4-bit cache, and read back from it as bf16:
           what the cache now stands for;
  read     rows of ranges of sequences read back from the 8-bit or the 4-bit cache as bf16;
  decode   one query token per sequence over its context, or over the first `sinks` and the last `window`
           tokens of it, from the 4-bit cache;
  prefill  causal attention of each sequence's new tokens over its context, or over the first `sinks`
           tokens and the last `window` up to each, from the 8-bit or the 4-bit cache.

`run` computes them with elementary torch operations, or, where `own` is true, through the framework's
public calls.  A `window` of 0 is none: every earlier token is seen.
"""
import math
import random

import torch

own = False

HEADS, KV_HEADS, DIM, BLOCK = 32, 8, 128, 256
GROUP = HEADS // KV_HEADS
SCALE = 1.0 / math.sqrt(DIM)
MICRO = 16                   # values under one scale of the 4-bit cache
ROW = {8: DIM + 4, 4: DIM // 2 + DIM // MICRO + 1}      # bytes of one head of one token
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEVICE = "cuda:0"


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a decode batch's new tokens into the 4-bit cache: latency alone counts
        {"name": "append4_step128", "op": "append", "bits": 4, "seqs": 128, "q_lens": "full", "q_max": 1, "ctx": 4096,
         "lens": 1},
        # eight prompt chunks, none of them whole, as a scheduler mixes them
        {"name": "append4_chunks8", "op": "append", "bits": 4, "seqs": 8, "q_lens": "ragged", "q_max": 2048,
         "ctx": 8192, "lens": 2},
        # one short turn of a conversation handed on to another cache
        {"name": "read8_turn", "op": "read", "bits": 8, "seqs": 1, "q_lens": "full", "q_max": 333, "ctx": 1000,
         "lens": 3},
        # shared prefixes and whole conversations moved out of the 8-bit cache
        {"name": "read8_prefixes16", "op": "read", "bits": 8, "seqs": 16, "q_lens": "ragged", "q_max": 8192,
         "ctx": 8192, "lens": 4},
        # the same from the 4-bit cache
        {"name": "read4_prefixes8", "op": "read", "bits": 4, "seqs": 8, "q_lens": "ragged", "q_max": 4096,
         "ctx": 16384, "lens": 5},
        # one sequence decoding in an interactive chat
        {"name": "decode4_one", "op": "decode", "bits": 4, "batch": 1, "ctx_min": 9001, "ctx_max": 9001, "window": 0,
         "sinks": 0, "lens": 6},
        # the usual decode batch
        {"name": "decode4_batch32", "op": "decode", "bits": 4, "batch": 32, "ctx_min": 128, "ctx_max": 4096,
         "window": 0, "sinks": 0, "lens": 7},
        # many long conversations: the cache that 4 bits make room for
        {"name": "decode4_batch64_16k", "op": "decode", "bits": 4, "batch": 64, "ctx_min": 8192, "ctx_max": 16384,
         "window": 0, "sinks": 0, "lens": 8},
        # a short question after a long conversation
        {"name": "prefill8_question", "op": "prefill", "bits": 8, "seqs": 1, "q_lens": "full", "q_max": 129,
         "ctx": 4129, "window": 0, "sinks": 0, "lens": 9},
        # eight prompt chunks over contexts of different lengths, as a scheduler mixes them
        {"name": "prefill8_chunks8", "op": "prefill", "bits": 8, "seqs": 8, "q_lens": "ragged", "q_max": 512,
         "ctx": 8192, "window": 0, "sinks": 0, "lens": 10},
        # the second half of a long document
        {"name": "prefill8_prompt8192", "op": "prefill", "bits": 8, "seqs": 1, "q_lens": "full", "q_max": 8192,
         "ctx": 16384, "window": 0, "sinks": 0, "lens": 11},
        # chunks of a layer with a sliding window over the 4-bit cache
        {"name": "prefill4_window4", "op": "prefill", "bits": 4, "seqs": 4, "q_lens": "ragged", "q_max": 1024,
         "ctx": 16384, "window": 2048, "sinks": 4, "lens": 12},
    ]


def draw(rng):
    def log(lo, hi):
        return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))

    lens = rng.randrange(1 << 30)
    op = rng.choice(["append", "read", "decode", "prefill"])
    if op in ("append", "read"):
        seqs = log(1, 128)
        q_max = log(1, 16384 // seqs if op == "append" else min(16384, 65536 // seqs))
        return {"op": op, "bits": 4 if op == "append" else rng.choice([8, 4]), "seqs": seqs,
                "q_lens": rng.choice(["ragged", "full"]), "q_max": q_max, "ctx": max(q_max, log(1, 8192)), "lens": lens}
    window = rng.choice([0, log(1, 4096)])
    sinks = rng.choice([0, 1, 4, log(1, 128)]) if window else 0
    if op == "decode":
        hi = log(1, 16384)
        return {"op": op, "bits": 4, "batch": log(1, 64), "ctx_min": rng.choice([1, hi]), "ctx_max": hi,
                "window": window, "sinks": sinks, "lens": lens}
    q_max = log(1, 4096)
    ctx = max(q_max, log(1, 16384))
    seqs = log(1, max(1, min(16, (1 << 26) // (q_max * ctx))))
    return {"op": op, "bits": rng.choice([8, 4]), "seqs": seqs, "q_lens": rng.choice(["ragged", "full"]),
            "q_max": q_max, "ctx": ctx, "window": window, "sinks": sinks, "lens": lens}


def lengths(case):
    """(rows, end) of every sequence: its rows are the tokens end - rows .. end - 1 of a context that, for
    attention, ends there too; by the case alone."""
    r = random.Random(case["lens"])
    if case["op"] == "decode":
        return [(1, r.randint(case["ctx_min"], case["ctx_max"])) for _ in range(case["batch"])]
    out = []
    for _ in range(case["seqs"]):
        most = case["q_max"]
        q = most if case["q_lens"] == "full" else r.randint(max(1, most // 2), most)
        out.append((q, case["ctx"] if case["q_lens"] == "full" else r.randint(q, max(q, case["ctx"]))))
    return out


def seen_pairs(case, q_len, n):
    """(query, key) pairs within the mask."""
    w, s = case["window"] or n, case["sinks"]
    total = 0
    for p in range(n - q_len, n):
        lo = max(0, p + 1 - w)
        total += p + 1 - lo + min(s, lo)
    return total


def work(case):
    ls = lengths(case)
    t = sum(q for q, _ in ls)
    row = ROW[case["bits"]]
    if case["op"] in ("append", "read"):
        wide, low = 2 * t * KV_HEADS * DIM * 2, 2 * t * KV_HEADS * row
        # a value is scaled twice and rounded; the append reads the rows, writes the cache and gives them back
        return {"bytes": wide + low + (wide if case["op"] == "append" else 0), "flops": 4 * t * KV_HEADS * DIM}
    keys = 0
    for q, n in ls:
        lo = max(0, n - q + 1 - (case["window"] or n))
        keys += n - lo + min(case["sinks"], lo)
    pairs = sum(seen_pairs(case, q, n) for q, n in ls)
    return {"bytes": 2 * t * HEADS * DIM * 2 + 2 * keys * KV_HEADS * row, "flops": 4 * pairs * HEADS * DIM}


# ------------------------------------------------------------------ the 4-bit rows

def to_e2m1(x):
    """Codes 0 .. 15 of the nearest E2M1 values, ties to the even code, beyond 6 to 6."""
    a = x.abs()
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    return code | (torch.signbit(x).to(torch.uint8) << 3)


def two_to(n):
    """2^n in 32 bits for n in -126 .. 127, of the bits (the GPU's power is off by a last place)."""
    return ((n.int() + 127) << 23).view(torch.float32)


def quantise4(x):
    """Rows x [..., 128] in 32 bits -> (packed codes [..., 64], block scales [..., 8], exponents [...] with
    a bias of 127).  The exponent is the least that brings the row's largest magnitude to 6 * 448."""
    amax = x.abs().amax(-1)
    part, power = torch.frexp(amax)
    power = torch.where(amax > 0, (power - 12 + (part > 0.65625)).clamp(min=-126), 0)
    y = (x * two_to(-power)[..., None]).unflatten(-1, (DIM // MICRO, MICRO))
    top = y.abs().amax(-1)
    # by a tensor: by a number the GPU multiplies with the rounded reciprocal, which turns ties around
    scale = (top / torch.full_like(top, 6.0)).clamp(max=448).to(torch.float8_e4m3fn)
    m = scale.float()[..., None]
    code = to_e2m1(torch.where(m > 0, y / m, 0.0)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), scale, (power + 127).to(torch.uint8)


def values4(codes, scale, exp, table):
    """What 4-bit rows stand for, in the type of `table` (E2M1's sixteen values)."""
    x = torch.stack([table[(codes & 15).int()], table[(codes >> 4).int()]], -1)
    x = x.unflatten(-2, (DIM // MICRO, MICRO // 2)) * scale.to(table.dtype)[..., None, None]
    return x.flatten(-3) * two_to(exp.int() - 127)[..., None].to(table.dtype)


def e2m1_table(dtype):
    return torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=dtype, device=DEVICE)


# ------------------------------------------------------------------ what a server has in hand

def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    ls = lengths(case)
    t = sum(q for q, _ in ls)
    width = max((n + BLOCK - 1) // BLOCK for _, n in ls)

    # blocks that hold a row some call of this pass touches, at random places of the pool; -1 for the
    # others, which a server with a window (or one that moves part of a sequence) has elsewhere
    live = []
    for q, n in ls:
        first = n - q if case["op"] in ("append", "read") else max(0, n - q + 1 - (case["window"] or n))
        live.append([first <= b * BLOCK + BLOCK - 1 or b * BLOCK < case.get("sinks", 0)
                     for b in range((n + BLOCK - 1) // BLOCK)])
    count = sum(sum(x) for x in live)
    order = torch.randperm(count, generator=g, device=DEVICE).tolist()
    table = [[order.pop() if ok else -1 for ok in x] + [-1] * (width - len(x)) for x in live]
    cu = [0]
    for q, _ in ls:
        cu.append(cu[-1] + q)

    s = {"case": case, "tokens": t, "max_q": max(q for q, _ in ls), "max_ctx": max(n for _, n in ls),
         "table": torch.tensor(table, dtype=torch.int32, device=DEVICE),
         "cu": torch.tensor(cu, dtype=torch.int32, device=DEVICE),
         "lens": torch.tensor([n for _, n in ls], dtype=torch.int32, device=DEVICE),
         "first": torch.tensor([n - q for q, n in ls], dtype=torch.int32, device=DEVICE),
         "workspace": torch.zeros(64 << 20, dtype=torch.uint8, device=DEVICE)}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)

    # rows whose size differs by token and by dimension, as keys' and values' do
    def rows(*shape):
        return normal(*shape, DIM) * (0.5 + torch.rand(*shape, 1, generator=g, device=DEVICE)) * spread

    spread = torch.exp(0.4 * normal(DIM))
    spread = spread / spread.square().mean().sqrt()
    pool = (count, BLOCK, KV_HEADS)
    for name in ("k", "v"):
        if case["op"] == "append":
            s[name] = rows(t, KV_HEADS).to(torch.bfloat16)
            s[name + "_codes"] = torch.zeros(*pool, DIM // 2, dtype=torch.uint8, device=DEVICE)
            s[name + "_scale"] = torch.zeros(count, KV_HEADS, BLOCK, DIM // MICRO, dtype=torch.uint8, device=DEVICE)
            s[name + "_exp"] = torch.zeros(count, KV_HEADS, BLOCK, dtype=torch.uint8, device=DEVICE)
            continue
        x = rows(*pool)
        if case["bits"] == 8:
            scale = x.abs().amax(-1) / 448.0
            s[name + "_codes"] = (x / scale[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            s[name + "_scale"] = scale.transpose(1, 2).contiguous()
        else:
            s[name + "_codes"], scale, exp = quantise4(x)
            s[name + "_scale"] = scale.view(torch.uint8).transpose(1, 2).contiguous()
            s[name + "_exp"] = exp.transpose(1, 2).contiguous()
    if case["op"] in ("decode", "prefill"):
        s["q"] = normal(t, HEADS, DIM).to(torch.bfloat16)
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    if own:
        return framework(s)
    return {"append": plain_append, "read": plain_read, "decode": plain_decode,
            "prefill": plain_prefill}[s["case"]["op"]](s)


def cache(s):
    names = ("k_codes", "v_codes", "k_scale", "v_scale") + (("k_exp", "v_exp") if s["case"]["bits"] == 4 else ())
    return [s[n] for n in names]


def appended(s, k, v):
    """The rows as the cache gives them back, and the scales and exponents that it holds."""
    return (k, v, s["k_scale"].view(torch.float8_e4m3fn), s["v_scale"].view(torch.float8_e4m3fn), s["k_exp"],
            s["v_exp"])


def framework(s):
    from paged_gqa_attention_gb300 import ops

    c = s["case"]
    window = {"window": c["window"], "sinks": c["sinks"]} if c.get("window") else {}
    if c["op"] == "append":
        ops.kv_append_fp4(*cache(s), s["k"], s["v"], s["table"], s["cu"], s["lens"], s["workspace"])
        k, v = ops.paged_kv_read_fp4(*cache(s), s["table"], s["cu"], s["first"], s["tokens"], s["workspace"])
        return appended(s, k, v)
    if c["op"] == "read":
        read = ops.paged_kv_read_fp8 if c["bits"] == 8 else ops.paged_kv_read_fp4
        return read(*cache(s), s["table"], s["cu"], s["first"], s["tokens"], s["workspace"])
    if c["op"] == "decode":
        return ops.paged_attn_decode_fp4(s["q"], *cache(s), s["table"], s["lens"], s["workspace"], **window)
    prefill = ops.paged_attn_prefill_fp8 if c["bits"] == 8 else ops.paged_attn_prefill_fp4
    return prefill(s["q"], *cache(s), s["table"], s["cu"], s["lens"], s["max_q"], s["workspace"], **window)


def owners(s):
    """Sequence and absolute position of every row."""
    i = torch.arange(s["tokens"], device=DEVICE)
    cu = s["cu"].long()
    seq = torch.searchsorted(cu, i, right=True) - 1
    return seq, s["first"].long()[seq] + (i - cu[seq])


def gather(s, name, block, slot):
    """Rows [..., KV head, dim] of cache places, in 32 bits."""
    codes, scale = s[name + "_codes"][block, slot], s[name + "_scale"][block, :, slot]
    if s["case"]["bits"] == 8:
        return codes.view(torch.float8_e4m3fn).float() * scale[..., None]
    return values4(codes, scale.view(torch.float8_e4m3fn), s[name + "_exp"][block, :, slot], e2m1_table(torch.float32))


def plain_append(s):
    seq, at = owners(s)
    block, slot = s["table"][seq, at // BLOCK].long(), at % BLOCK
    for name in ("k", "v"):
        codes, scale, exp = quantise4(s[name].float())
        s[name + "_codes"][block, slot] = codes
        s[name + "_scale"][block, :, slot] = scale.view(torch.uint8)
        s[name + "_exp"][block, :, slot] = exp
    return appended(s, *(gather(s, n, block, slot).to(torch.bfloat16) for n in ("k", "v")))


def plain_read(s):
    seq, at = owners(s)
    block, slot = s["table"][seq, at // BLOCK].long(), at % BLOCK
    return tuple(gather(s, n, block, slot).to(torch.bfloat16) for n in ("k", "v"))


def plain_decode(s):
    c = s["case"]
    n = s["lens"].long()[:, None]
    lo = (n - (c["window"] or s["max_ctx"])).clamp(min=0)
    # columns: the sinks that lie before the window, then the window
    first = torch.arange(min(c["sinks"], s["max_ctx"]), device=DEVICE).expand(len(n), -1)
    last = lo + torch.arange(min(c["window"] or s["max_ctx"], s["max_ctx"]), device=DEVICE)
    at = torch.cat([first, last.clamp(max=s["max_ctx"] - 1)], 1)
    seen = torch.cat([first < lo, last < n], 1)
    block = torch.gather(s["table"].long(), 1, at // BLOCK).clamp(min=0)
    q = s["q"].float().view(-1, KV_HEADS, GROUP, DIM)
    score = torch.matmul(q, gather(s, "k", block, at % BLOCK).permute(0, 2, 3, 1)) * SCALE
    p = torch.exp_(score.masked_fill_(~seen[:, None, None], -math.inf) - score.amax(-1, keepdim=True))
    out = torch.matmul(p, gather(s, "v", block, at % BLOCK).transpose(1, 2)) / p.sum(-1, keepdim=True)
    return out.reshape(-1, HEADS, DIM).to(torch.bfloat16)


def plain_prefill(s):
    c = s["case"]
    cu, lens = s["cu"].long(), s["lens"].long()
    q_len = cu[1:] - cu[:-1]
    # every sequence's queries and keys in a row of their own, padded to the longest
    row = torch.arange(s["max_q"], device=DEVICE)
    real = row < q_len[:, None]
    token = (cu[:-1, None] + row).clamp(max=s["tokens"] - 1)
    pos = (lens - q_len)[:, None] + row                                         # [seqs, queries]
    at = torch.arange(s["max_ctx"], device=DEVICE).expand(len(lens), -1)
    block = torch.gather(s["table"].long(), 1, at // BLOCK).clamp(min=0)
    seen = at[:, None] <= pos[..., None]
    if c["window"]:
        seen &= (at[:, None] > pos[..., None] - c["window"]) | (at[:, None] < c["sinks"])
    q = s["q"][token].float().view(len(lens), -1, KV_HEADS, GROUP, DIM).permute(0, 2, 3, 1, 4)
    q = q.reshape(len(lens), KV_HEADS, GROUP * s["max_q"], DIM)
    score = torch.matmul(q, gather(s, "k", block, at % BLOCK).permute(0, 2, 3, 1)).mul_(SCALE)
    score = score.view(len(lens), KV_HEADS, GROUP, s["max_q"], -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)                         # rows past the chunk see nothing
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    # what no query of a sequence sees is not in its cache: any block stands in for it there
    out = torch.matmul(p.view(len(lens), KV_HEADS, GROUP * s["max_q"], -1),
                       gather(s, "v", block, at % BLOCK).transpose(1, 2))
    out = out.view(len(lens), KV_HEADS, GROUP, s["max_q"], DIM) / total
    return out.permute(0, 3, 1, 2, 4).reshape(len(lens), -1, HEADS, DIM)[real].to(torch.bfloat16)


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    if case["op"] in ("decode", "prefill") and work(case)["flops"] > 2.0e12:
        return None
    s = prepare(case, seed)
    ls = lengths(case)
    if case["op"] == "append":
        return exact_append(s, ls)

    def rows(name, i, lo, hi):
        """Tokens lo .. hi - 1 of sequence i as [KV head, token, dim]."""
        at = torch.arange(lo, hi, device=DEVICE)
        b, o = s["table"][i].long()[at // BLOCK], at % BLOCK
        codes, scale = s[name + "_codes"][b, o].transpose(0, 1), s[name + "_scale"][b, :, o].transpose(0, 1)
        if case["bits"] == 8:
            return codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]
        magnitude = torch.tensor(E2M1, dtype=torch.float64, device=DEVICE)
        x = torch.empty(*codes.shape[:-1], DIM, dtype=torch.float64, device=DEVICE)
        for half, nibble in enumerate((codes % 16, codes // 16)):
            x[..., half::2] = magnitude[(nibble % 8).long()] * (1 - 2 * (nibble // 8).double())
        x *= scale.view(torch.float8_e4m3fn).double().repeat_interleave(MICRO, -1)
        return x * two_to(s[name + "_exp"][b, :, o].T.int() - 127).double()[..., None]

    if case["op"] == "read":
        return tuple(torch.cat([rows(n, i, end - q, end).transpose(0, 1) for i, (q, end) in enumerate(ls)])
                     for n in ("k", "v"))
    out, done = torch.empty(s["tokens"], HEADS, DIM, dtype=torch.float64, device=DEVICE), 0
    for i, (q_len, n) in enumerate(ls):
        for p0 in range(n - q_len, n, 1024):
            p1 = min(p0 + 1024, n)
            lo = max(0, p0 + 1 - (case["window"] or n))
            k, v, j = rows("k", i, lo, p1), rows("v", i, lo, p1), torch.arange(lo, p1, device=DEVICE)
            if min(case["sinks"], lo):
                few = min(case["sinks"], lo)
                k, v = torch.cat([rows("k", i, 0, few), k], 1), torch.cat([rows("v", i, 0, few), v], 1)
                j = torch.cat([torch.arange(few, device=DEVICE), j])
            p = torch.arange(p0, p1, device=DEVICE)[:, None]
            seen = (j <= p) & ((j < case["sinks"]) | (j > p - (case["window"] or n)))
            q = s["q"][done:done + p1 - p0].double()
            for h in range(HEADS):
                a = (q[:, h] @ k[h // GROUP].T) * SCALE
                a = torch.softmax(torch.where(seen, a, -math.inf), -1)
                out[done:done + p1 - p0, h] = a @ v[h // GROUP]
            done += p1 - p0
    return out


def exact_append(s, ls):
    """The quantisation in 64 bits; what it holds in 4 and 8 bits rounded by search among the values there are."""
    grid4 = torch.tensor(E2M1, dtype=torch.float64, device=DEVICE)
    grid8 = torch.arange(127, device=DEVICE).to(torch.uint8).view(torch.float8_e4m3fn).double()

    def nearest(x, grid):
        hi = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
        down, up = x - grid[hi - 1], grid[hi] - x
        return grid[torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)]

    at = torch.cat([torch.arange(n - q, n) for q, n in ls]).to(DEVICE)
    seq = torch.cat([torch.full((q,), i) for i, (q, _) in enumerate(ls)]).to(DEVICE)
    place = s["table"].long()[seq, at // BLOCK], at % BLOCK
    count = s["k_codes"].shape[0]
    back, scales = [], []
    for name in ("k", "v"):
        x = s[name].double().view(-1, KV_HEADS, DIM // MICRO, MICRO)
        unit = two_to(torch.ceil(torch.log2(x.abs().amax((-1, -2)) / 2688))).double()[..., None, None]
        scale = nearest((x / unit).abs().amax(-1) / 6, grid8)
        z = x / unit / torch.where(scale > 0, scale, 1.0)[..., None]
        z = torch.where(scale[..., None] > 0, nearest(z.abs(), grid4) * z.sign(), 0.0)
        back.append((z * scale[..., None] * unit).flatten(-2))
        full = torch.zeros(count, BLOCK, KV_HEADS, DIM // MICRO, dtype=torch.float64, device=DEVICE)
        full[place] = scale
        scales.append(full.transpose(1, 2).contiguous())
    return (*back, *scales, None, None)
