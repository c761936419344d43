"""Attention over the low-bit caches held to what it may lose row by row (test side only): the bounds go by the rows that a
query sees and by the unit that its work unit is in, not by the largest value of the batch."""
import torch

import window_cases
from gpu_helpers import to_cpu
from lowbit_cases import LowCache, check_lse, quantise4
from paged_gqa_attention_gb300 import ops

HUGE = 2 ** 31 - 1
SCALE = ops.DEFAULT_SCALE


class Rows(LowCache):
    """LowCache whose zero rows are those of the appends: codes 0 under the scale 1 in 8 bits (exponent 127 in 4)."""

    def upload(self):
        super().upload()
        self.zero_rows_as_appended()
        self.window, self.sinks = HUGE if self.window >= 1 << 30 else self.window, self.sinks
        return self

    def zero_rows_as_appended(self):
        if self.bits == 4:
            return
        for codes, scale in zip(self.pools[:2], self.pools[2:]):
            zero = scale == 0
            scale[zero] = 1.0
            codes[zero.transpose(1, 2)] = 0
        self.k, self.v = ([torch.nan_to_num(x, nan=0.0) for x in rows] for rows in (self.k, self.v))

    def aim(self, which, at):
        """Query heads `which` of every new token look at one key each: at(sequence, position) -> key.  q = 2 k, a score of
        about 2 * 128 * scale = 22.6 there and N(0, 2^2) elsewhere."""
        t = 0
        for s, (m, n) in enumerate(zip(self.q_lens, self.seq_lens)):
            for i in range(m):
                key = self.k[s][at(s, n - m + i)]
                for h in which:
                    self.q[t, h] = (2.0 * key[h // 4]).to(torch.bfloat16)
                t += 1

    def units(self, s, rows, lo, hi):
        """The largest power of two that rows lo .. hi - 1 of a sequence can make a unit, per KV head: in 8 bits the scale's
        next power of two, twice it at most, in 4 the largest 2^(e - 127) (of the rows as they came: theirs may be twice that
        of the quantised ones)."""
        x = rows[s][lo:hi].double()
        if self.bits == 8:
            amax = x.abs().amax(-1)              # (448 times the scale; a zero row has the scale 1)
            return 2 * torch.where(amax == 0, 1.0, amax / 448).amax(0)
        e = quantise4(x)[2].double() - 127
        return torch.exp2(torch.where(x.abs().amax(-1) == 0, e, e + 1).amax(0))

    def bounds(self, prefill):
        """(out, lse, tolerance of out, tolerance of lse) in 64 bits.

        out = sum w v / sum w.  What the kernels round, u = 2^-11 being half a step of f16:
          weights     to f16 for the products only: u of sum p |v|.  Those below 2^-14 (the largest is 1 at least, so p is no
                      larger than the weight) by 2^-25, and by no more than themselves: min(2^-25, p) |v| each.  In the decode
                      a weight carries its V row's power of two over the largest of the rows seen: 2^-25 of 2688 2^e, where
                      the largest row quantised is above 1344 (1 - 1/16) 2^e: 2^-25 of 2.2 times the largest |v|, and
                      p |v| at most;
          scores      fp32 sums of 128 products, 2^-24 or (truncated) 2^-23 of sum |q k| scale for each: 2^-16 a, a the
                      largest such sum of the keys seen; the exponential, its argument and the softmax scale add less than
                      2^-16 (1 + a).  A score that is off by ds moves p by as much, relatively, in numerator and
                      denominator: ds (1 + 2 ds) (sum p |v| + |out|);
          K, V        (prefill) as f16, in units of a power of two.  8 bits: u of the value, and 1.1 * 2^-25 of the unit
                      below f16's normal range.  4 bits: exact, 7 * 2^-25 of the unit below it (a scale is rounded before its
                      code, up to 6, multiplies it);
          products    fp32 sums over n keys, each addition 2^-23 at most;
          out         to bf16, 2^-8."""
        u, part = 2.0 ** -11, (1.1 if self.bits == 8 else 7.0) * 2.0 ** -25
        block = (128 if max(self.q_lens) > 64 else 64) if prefill else 1
        outs, lses, tols, lse_tols, t = [], [], [], [], 0
        for s, (m, n) in enumerate(zip(self.q_lens, self.seq_lens)):
            if m == 0:
                continue
            p = torch.arange(n - m, n)[:, None]
            j = torch.arange(n)
            window, sinks = min(self.window, 1 << 30), min(self.sinks, 1 << 30)
            seen = (j <= p) & ((j < sinks) | (j > p - window))
            q = self.q[t:t + m].double()
            k, v = (x[s].double().repeat_interleave(4, 1) for x in (self.k, self.v))
            score = torch.einsum("thd,nhd->htn", q, k) * SCALE
            score = torch.where(seen, score, float("-inf"))
            lse = torch.logsumexp(score, -1)
            w = torch.exp(score - lse[..., None])
            out, abs_v = torch.einsum("htn,nhd->thd", w, v), torch.einsum("htn,nhd->thd", w, v.abs())
            a = torch.einsum("thd,nhd->htn", q.abs(), k.abs()) * SCALE
            a = torch.where(seen, a, 0.0).amax(-1).T                                       # [t, h]
            size = v.abs().amax(-1).T[:, None]                                             # [h, 1, n]
            if prefill:
                lost = torch.minimum(w, torch.tensor(2.0 ** -25, dtype=w.dtype)) * size
            else:
                lost = torch.minimum(w * size, 2.2 * 2.0 ** -25 * torch.where(seen, size, 0.0).amax(-1, keepdim=True))
            lost = torch.where(seen, lost, 0.0).sum(-1).T                                  # [t, h]
            ds = 2.0 ** -16 * 2 * (1 + a)
            v_unit = torch.zeros(m, 32, dtype=torch.float64)
            if prefill:
                k_unit = torch.zeros_like(v_unit)
                for i in range(0, m, block):
                    first, last = n - m + i, min(n - m + i + block, n) - 1
                    live = (j <= last) & ((j < sinks) | (j > first - window))
                    lo, hi = int(live.nonzero()[0]), last + 1                              # (all that may be fetched)
                    for unit, rows in ((k_unit, self.k), (v_unit, self.v)):
                        unit[i:i + block] = self.units(s, rows, lo, hi).repeat_interleave(4)
                ds = ds + (u * a if self.bits == 8 else 0) + part * k_unit * q.abs().sum(-1) * SCALE
            ds = ds[..., None]
            tol = u * abs_v * (2 if prefill and self.bits == 8 else 1) * 1.01 + ds * (1 + 2 * ds) * (abs_v + out.abs())
            tol = tol + (lost + part * v_unit)[..., None] + n * 2.0 ** -23 * abs_v
            outs.append(out)
            lses.append(lse.T)
            tols.append(tol * (1 + 2.0 ** -8) + 2.0 ** -8 * out.abs())
            lse_tols.append(ds[..., 0] * 1.01 + 1e-5 + 2.0 ** -22 * lse.T.abs())
            t += m
        return [torch.cat(x) for x in (outs, lses, tols, lse_tols)]

    def call(self, prefill):
        ws = ops.make_workspace(len(self.seq_lens), self.bt.shape[1])
        lse = torch.empty(self.qd.shape[0], 32, device="cuda")
        kw = dict(lse=lse, window=self.window, sinks=self.sinks)
        if prefill:
            fn = ops.paged_attn_prefill_fp8 if self.bits == 8 else ops.paged_attn_prefill_fp4
            out = fn(self.qd, *self.pools, self.bt, self.cu, self.lens, max(self.q_lens), ws, **kw)
        else:
            fn = ops.paged_attn_decode_window_fp8 if self.bits == 8 else ops.paged_attn_decode_fp4
            out = fn(self.qd, *self.pools, self.bt, self.lens, ws, **kw)
        ops.check_error(ws)
        return out, lse

    def compare(self, prefill, what=""):
        self.qd = self.q.cuda()
        out, lse = self.call(prefill)
        ref, ref_lse, tol, lse_tol = self.bounds(prefill)
        assert not to_cpu(out).isnan().any(), what
        window_cases.check(out, ref, tol, what)
        check_lse(lse, ref_lse, lse_tol, what)
