"""Paged caches for the window tests (test side only): sequences with known K/V, placed in a pool
where everything that no query sees is NaN and every block without a visible token is given
back (table entry -1)."""
import torch

import definitions
from gpu_helpers import to_cpu
from paged_gqa_attention_gb300 import ops

# Tolerances.  The output is sum w v / sum w.  The kernels round every weight to bf16 (f16 over the
# 8-bit cache), in numerator and denominator alike, a relative error of at most d = 2^-8 (2^-11)
# each, so the quotient moves by at most d (1 + 2d) sum p |v - out| <= d (1 + 2d) (sum p |v| +
# |out|), p the exact weights.  Scores are fp32 sums of 128 exact products: off by at most
# 128 * 2^-24 of sum |q k| scale, under 4e-5 here (|q k| <= 36 over the tests' inputs), plus 2^-22
# in each exponential: FP = 1e-4 of the same sum covers both.  The bf16 output adds half a step,
# 2^-8 of the value.  Over the 8-bit cache a weight times its V scale below f16's normal range is off
# by up to 2^-25 of the largest, 448 scale: n 2^-25 of the largest |v| over n keys.
FP = 1e-4


def tolerance(out, p_abs_v, fp8=False, keys=0, v_max=0.0):
    d = 2.0 ** -11 if fp8 else 2.0 ** -8
    spread = p_abs_v + out.abs()
    tol = (d * (1 + 2 * d) + FP) * spread
    return (tol + keys * 2.0 ** -25 * v_max) * (1 + 2.0 ** -8) + 2.0 ** -8 * out.abs()


class Cache:
    """Sequences of the given lengths, the last q_lens tokens of each new, seen under a window."""

    def __init__(self, seq_lens, q_lens, window, sinks, seed, fp8=False, spare=2, far=0):
        g = torch.Generator().manual_seed(seed)
        self.seq_lens, self.q_lens, self.window, self.sinks, self.fp8 = seq_lens, q_lens, window, sinks, fp8
        randn = lambda *s: torch.randn(*s, generator=g)
        self.q = randn(sum(q_lens), 32, 128).to(torch.bfloat16)
        self.k = [randn(n, 8, 128).to(torch.bfloat16) for n in seq_lens]
        self.v = [randn(n, 8, 128).to(torch.bfloat16) for n in seq_lens]
        width = max(1, max((n + 255) // 256 for n in seq_lens)) + spare
        seen, need = [], 0
        for n, m in zip(seq_lens, q_lens):
            ok = torch.zeros(n, dtype=torch.bool)
            if m:
                ok[max(0, n - m - window + 1):] = True
                ok[:sinks] = True
            seen.append(ok)
            need += sum(bool(ok[b:b + 256].any()) for b in range(0, n, 256))
        blocks = need + 3 + far
        free = (torch.randperm(need + 3, generator=g) + far).tolist()
        self.table = torch.full((len(seq_lens), width), -1, dtype=torch.int32)
        kp = torch.full((blocks if not far else need + 3, 256, 8, 128), float("nan"), dtype=torch.bfloat16)
        vp = kp.clone()
        for s, ok in enumerate(seen):
            for b in range(0, len(ok), 256):
                part = ok[b:b + 256]
                if part.any():
                    i = free.pop()
                    self.table[s, b // 256] = i
                    kp[i - far, :len(part)][part] = self.k[s][b:b + 256][part]
                    vp[i - far, :len(part)][part] = self.v[s][b:b + 256][part]
        self.blocks, self.far = blocks, far
        self.k_host, self.v_host = kp, vp
        self.seen = seen

    def upload(self):
        cu = [0]
        for m in self.q_lens:
            cu.append(cu[-1] + m)
        self.cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(self.seq_lens, dtype=torch.int32, device="cuda")
        self.bt = self.table.cuda()
        self.qd = self.q.cuda()
        pools = []
        for x in (self.k_host, self.v_host):
            pool = torch.empty(self.blocks, 256, 8, 128, dtype=torch.bfloat16, device="cuda")
            pool[self.far:] = x.cuda()
            pools.append(pool)
        if not self.fp8:
            self.pools = pools
            return self
        # quantised rows (the rule of kv_append_fp8 need not hold: any codes and scales will do)
        self.pools, scales = [], []
        for pool in pools:
            x = pool.float()
            hidden = x[..., 0].isnan()
            scale = x.abs().amax(-1) / 448
            codes = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            codes[hidden] = 0x7F
            scale[hidden] = float("nan")
            self.pools.append(codes)
            scales.append(scale.transpose(1, 2).contiguous())
        self.pools += scales
        # what the rows stand for
        for name, codes, scale in (("k", self.pools[0], scales[0]), ("v", self.pools[1], scales[1])):
            rows = (codes[self.far:].view(torch.float8_e4m3fn).double() *
                    scale[self.far:].transpose(1, 2).double()[..., None]).cpu()
            new = []
            for s, ok in enumerate(self.seen):
                x = torch.zeros(len(ok), 8, 128, dtype=torch.float64)
                for b in range(0, len(ok), 256):
                    if self.table[s, b // 256] >= 0:
                        x[b:b + 256] = rows[int(self.table[s, b // 256]) - self.far, :len(ok[b:b + 256])]
                x[~ok] = 0.0
                new.append(x)
            setattr(self, name, new)
        return self

    def reference(self, scale=ops.DEFAULT_SCALE):
        """(out, lse, tolerance of out) in 64 bits, rows of non-empty sequences."""
        args = (self.q_lens, self.seq_lens, self.window, self.sinks, scale)
        out, lse = definitions.window_attention(self.q, self.k, self.v, *args)
        p_abs_v, _ = definitions.window_attention(self.q, self.k, [v.abs() for v in self.v], *args)
        v_max = max([float(v.double().abs().max()) for v in self.v if len(v)] + [0.0])
        keys = max(self.seq_lens)
        return out, lse, tolerance(out, p_abs_v, self.fp8, keys, v_max)


def check(got, ref, tol, what=""):
    got = to_cpu(got).double()
    assert got.shape == ref.shape
    over = (got - ref).abs() - tol
    assert not got.isnan().any() and over.max().item() <= 0, f"{what}: {over.max().item():.3e} over the tolerance"
