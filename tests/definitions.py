"""The operators over new tokens and windows written out in 64 bits (test side only): the
rotated append and attention over a sliding window with visible first tokens, in plain torch
float64 on the host, one definition per function."""
import math

import torch

PAIRS, DIM, GROUP = 64, 128, 4


def rotated(x, positions, theta, pair_axis=None, gain=None, eps=0.0):
    """x [T, heads, 128] -> (z, scale): the normalised and rotated heads, and |y[d]| + |y[d + 64]|
    of every element's pair, the size that rounding errors of the rotation go by.  positions
    [T] or [axes, T]."""
    y = x.double()
    if gain is not None:
        y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps) * gain.double()
    a, b = y[..., :PAIRS], y[..., PAIRS:]
    size = torch.cat([a.abs() + b.abs()] * 2, -1)
    if theta == 0:
        return y, size
    p = positions.double()
    p = p[None].expand(1, -1) if p.dim() == 1 else p
    axis = torch.tensor(list(pair_axis)) if pair_axis is not None else torch.zeros(PAIRS, dtype=torch.long)
    angle = p[axis].T * theta ** (-torch.arange(PAIRS, dtype=torch.float64) / PAIRS)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    return torch.cat([a * c - b * s, b * c + a * s], -1), size


def places(table, q_lens, seq_lens):
    """(sequence, position, block, slot) of every new token, from host lists."""
    out = []
    for s, (q, n) in enumerate(zip(q_lens, seq_lens)):
        for p in range(n - q, n):
            out.append((s, p, int(table[s][p // 256]), p % 256))
    return out


def window_attention(q, keys, values, q_lens, seq_lens, window, sinks, scale):
    """q [T, 32, 128]; keys / values: per sequence [n, 8, 128], any type.  New token i of a sequence
    sees keys j <= p with j < sinks or j > p - window, p = n - q_len + i.  Returns (out [T, 32,
    128], lse [T, 32]) in 64 bits; a sequence without tokens has no rows."""
    outs, lses, t = [], [], 0
    for k, v, m, n in zip(keys, values, q_lens, seq_lens):
        if m == 0:
            continue
        p = torch.arange(n - m, n)[:, None]
        j = torch.arange(n)
        seen = (j <= p) & ((j < sinks) | (j > p - window))
        kk = k.double().repeat_interleave(GROUP, 1)
        vv = torch.where(seen.any(0)[:, None, None], v.double(), torch.zeros((), dtype=torch.float64))
        vv = vv.repeat_interleave(GROUP, 1)
        score = torch.einsum("thd,nhd->htn", q[t:t + m].double(), kk) * scale
        score = torch.where(seen, score, torch.full((), -math.inf, dtype=torch.float64))
        lse = torch.logsumexp(score, -1)
        outs.append(torch.einsum("htn,nhd->thd", torch.exp(score - lse[..., None]), vv))
        lses.append(lse.T)
        t += m
    return torch.cat(outs), torch.cat(lses)
