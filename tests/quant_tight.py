"""Attention over codes and over packed prompts in 64 bits, with bounds that a lost token breaks.

The bounds follow how an output is made, key by key, with the weights that the keys have:

* a score is off by at most STEPS roundings of its terms' size A_j = |scale| (sum of its products' magnitudes), and
  moves the output by w_j |v_j - o| times that (a shift of all scores alike moves nothing);
* a weight that is rounded for its product with V (FP16 over codes, BF16 over prompts) is off by at most half a step, each
  in a direction of its own: four standard deviations of the sum, the variance of a rounding being a third of its
  largest square.  Weights over codes that FP16 holds as subnormal numbers are off by half of its smallest step, and
  lost below that;
* sums in 32 bits, each off by half a step of a partial sum: a partial sum is no larger than the magnitudes' sum;
* one rounding to the output's type.
"""
import math

import torch

from quant_reference import HALF, unpack

# Roundings of a score: products are exact, D / 16 sums of a matrix step, each cut off by up to a step of 2^-23 where the
# tensor core aligns its terms (two roundings), the sum of a row's elements, scale and offset.
STEPS = 24
FP16 = 2.0 ** -11       # half a step
SMALLEST = 2.0 ** -25   # half of FP16's smallest number, as a part of ...
SHIFT = 7               # ... the largest weight times 2^-SHIFT


def _weights(x):
    """Softmax over the last dimension: exact weights."""
    return torch.softmax(x, -1)


def codes(q, pools, tables, lens, scale, bits):
    """(out, bound) of decode attention over codes [B, Hq, D]."""
    kc, kp, vc, vp = pools
    B, Hq, D = q.shape
    Hk, bs = kc.shape[1], kc.shape[2]
    out, bound = torch.zeros(B, Hq, D, dtype=torch.float64), torch.zeros(B, Hq, D, dtype=torch.float64)
    for b, L in enumerate(lens):
        if L <= 0:
            continue
        t = torch.arange(L)
        blk, off = tables[b].long()[t // bs], t % bs
        for h in range(Hk):
            n, c = (unpack(x[blk, h, off], bits).double() for x in (kc, vc))
            s, z, vs, vz = (p[blk, h, off].double()[:, i] for p in (kp, vp) for i in (0, 1))
            v = c * vs[:, None] + vz[:, None]
            for i in range(h * (Hq // Hk), (h + 1) * (Hq // Hk)):
                x = q[b, i].double()
                size = (s * (n @ x.abs()) + z.abs() * x.abs().sum()) * abs(scale)
                w = _weights((s * (n @ x) + z * x.sum()) * scale)
                o = w @ v
                e = STEPS * 2.0 ** -24 * ((w * size) @ (v - o).abs())
                ws = w * vs
                e = e + 4 / math.sqrt(3) * FP16 * ((ws ** 2) @ (c ** 2)).sqrt()
                small = SMALLEST * 2.0 ** -SHIFT * ws.max()
                e = e + 4 / math.sqrt(3) * small * (c ** 2).sum(0).sqrt() + (ws * (ws < small)) @ c
                e = e + (L / 64 + 32) * 2.0 ** -24 * (ws @ c + w @ vz.abs())
                out[b, i], bound[b, i] = o, e + HALF[torch.bfloat16] * (o.abs() + e)
    return out, bound


def prompts(q, k, v, q_lens, k_lens, scale):
    """(out, bound) of attention over packed rows."""
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    out, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    half = HALF[q.dtype]
    weight = half if q.dtype == torch.bfloat16 else 0.0
    iq = ik = 0
    for n, m in zip(q_lens, k_lens):
        seen = torch.arange(m)[None] <= torch.arange(n)[:, None] + (m - n)
        some = seen.any(1)
        for h in range(Hq):
            if n == 0 or not some.any():
                continue
            a, c, d = (x.double() for x in (q[iq:iq + n, h], k[ik:ik + m, h // (Hq // Hk)], v[ik:ik + m, h // (Hq // Hk)]))
            a, see = a[some], seen[some]
            w = _weights((a @ c.T * scale).masked_fill(~see, -math.inf))
            size = a.abs() @ c.abs().T * abs(scale)
            o = w @ d
            # w |v - o| <= w |v| + w |o|
            u = w * size
            e = STEPS * 2.0 ** -24 * (u @ d.abs() + u.sum(1, keepdim=True) * o.abs())
            e = e + 4 / math.sqrt(3) * weight * ((w ** 2) @ (d ** 2)).sqrt()
            e = e + (m / 16 + 32) * 2.0 ** -24 * (w @ d.abs())
            out[iq:iq + n, h][some], bound[iq:iq + n, h][some] = o, e + half * (o.abs() + e)
        iq, ik = iq + n, ik + m
    return out, bound


def check(got, want, bound):
    err = (got.cpu().double() - want).abs()
    ok = err <= bound
    assert bool(ok.all()), (float(err.max()), float((err / bound).nan_to_num(math.inf).max()), int((~ok).sum()), ok.numel())
