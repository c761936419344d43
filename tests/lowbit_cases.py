"""The 4-bit rows written out in 64 bits, and paged low-bit caches for the tests (test side only)."""
import torch

import definitions
import window_cases
from gpu_helpers import to_cpu

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()    # 0 .. 448


def nearest(x, grid):
    """Index of the value of `grid` nearest to x >= 0, ties to the even index."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    down, up = x - grid[hi - 1], grid[hi] - x
    return torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, hi - 1)


def quantise4(x):
    """x [..., 128] (bf16 or fp32 values) -> (codes [..., 128] 0 .. 15, scales [..., 8] as E4M3 bytes,
    exponent bytes [...]) by the definition, in 64 bits."""
    x = x.double()
    amax = x.abs().amax(-1)
    bad = ~torch.isfinite(x).all(-1)
    part, power = torch.frexp(torch.where(bad, 1.0, amax))     # amax = part 2^power, 0.5 <= part < 1
    e = torch.where(part * 2 <= 2688 / 2048, power - 1 - 11, power - 1 - 10).clamp(min=-126)
    e = torch.where(amax == 0, 0, e)
    y = torch.ldexp(torch.where(bad[..., None], 0.0, x), -e[..., None]).unflatten(-1, (8, 16))
    scale = nearest(y.abs().amax(-1) / 6, E4M3)
    s = E4M3[scale][..., None]
    code = nearest(torch.where(s > 0, y.abs() / torch.where(s > 0, s, 1.0), 0.0), E2M1)
    code = torch.where(s > 0, code + 8 * torch.signbit(y), 0)
    return code.flatten(-2), scale.to(torch.uint8), torch.where(bad, 255, e + 127).to(torch.uint8)


def pack4(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).to(torch.uint8)


def unpack4(packed):
    p = packed.long()
    return torch.stack([p & 15, p >> 4], -1).flatten(-2)


def values4(codes, scale, exp):
    """What rows stand for, in 64 bits."""
    m = E2M1[codes & 7] * torch.where(codes >= 8, -1.0, 1.0)
    m = m * E4M3[scale.long().clamp(max=126)].repeat_interleave(16, -1)
    e = torch.ldexp(torch.ones(exp.shape, dtype=torch.float64), exp.int() - 127)
    return m * torch.where(exp == 255, float("nan"), e)[..., None]


class LowCache(window_cases.Cache):
    """window_cases.Cache over the 8-bit or the 4-bit cache; what no query sees is NaN (4 bits: any codes and
    scales under the exponent 255)."""

    def __init__(self, seq_lens, q_lens, window, sinks, seed, bits=4, **kw):
        super().__init__(seq_lens, q_lens, window, sinks, seed, fp8=bits == 8, **kw)
        self.bits, self.seed = bits, seed

    def upload(self):
        if self.bits == 8:
            return super().upload()
        super().upload()                        # (the bf16 pools are not used)
        g = torch.Generator().manual_seed(self.seed + 1000)
        tensors = {}
        for name, host in (("k", self.k_host), ("v", self.v_host)):
            hidden = host[..., 0].isnan()
            codes, scale, exp = quantise4(torch.where(hidden[..., None], 0.0, host.double()))
            rows = values4(codes, scale, exp)
            codes[hidden] = torch.randint(0, 16, codes[hidden].shape, generator=g)
            scale[hidden] = torch.randint(0, 256, scale[hidden].shape, generator=g).to(torch.uint8)
            exp[hidden] = 255
            new = []
            for s, ok in enumerate(self.seen):
                x = torch.zeros(len(ok), 8, 128, dtype=torch.float64)
                for b in range(0, len(ok), 256):
                    if self.table[s, b // 256] >= 0:
                        x[b:b + 256] = rows[int(self.table[s, b // 256]) - self.far, :len(ok[b:b + 256])]
                x[~ok] = 0.0
                new.append(x)
            setattr(self, name, new)
            parts = [pack4(codes), scale.transpose(1, 2), exp.transpose(1, 2)]
            for what, part in zip(("codes", "scale", "exp"), parts):
                full = torch.zeros(self.blocks, *part.shape[1:], dtype=torch.uint8, device="cuda")
                full[self.far:] = part.cuda()
                tensors[name, what] = full
        self.pools = [tensors[n, w] for w in ("codes", "scale", "exp") for n in ("k", "v")]
        return self

    def prefill_reference(self, scale):
        """(out, lse, tolerance of out, tolerance of lse) in 64 bits for the prefill over this cache.

        Weights are rounded to f16, in numerator and denominator alike: 2^-11 each (half a step of f16),
        as in window_cases.  Over the 8-bit cache a key's value is code * scale rounded to f16 as well, so a score
        moves by up to 2^-11 of sum |q k| scale (A, the largest over the row's keys), a weight by as much relatively,
        and a V value by 2^-11 of itself.  (4-bit values are f16 as they are.)  P below 2^-14: keys *
        2^-25 of the largest |v|.  Scores in fp32, the exponential and q below 2^-14 in f16: FP, as in
        window_cases."""
        args = (self.q_lens, self.seq_lens, self.window, self.sinks, scale)
        out, lse = definitions.window_attention(self.q, self.k, self.v, *args)
        p_abs_v, _ = definitions.window_attention(self.q, self.k, [v.abs() for v in self.v], *args)
        a = torch.zeros_like(lse)
        if self.bits == 8:
            t = 0
            for k, m, n in zip(self.k, self.q_lens, self.seq_lens):
                if m:
                    kk = k.double().abs().repeat_interleave(4, 1)
                    a[t:t + m] = torch.einsum("thd,nhd->thn", self.q[t:t + m].double().abs(), kk).amax(-1) * scale
                t += m
        half = 2.0 ** -11
        d = half + half * a * 1.01 + window_cases.FP
        v_max = max([float(v.double().abs().max()) for v in self.v if len(v)] + [0.0])
        tol = (d * (1 + 2 * d))[..., None] * (p_abs_v + out.abs()) + max(self.seq_lens) * 2.0 ** -25 * v_max
        if self.bits == 8:
            tol = tol + half * p_abs_v
        return out, lse, tol * (1 + 2.0 ** -8) + 2.0 ** -8 * out.abs(), d * 1.01 + 1e-4


def check_lse(got, ref, tol, what=""):
    got = to_cpu(got).double()
    assert ((got - ref).abs() <= tol).all(), f"{what}: lse off by up to {((got - ref).abs() - tol).max().item():.3e} over"
