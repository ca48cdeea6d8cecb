"""Plain references of the quantised cache and of prompt attention: torch on
the CPU, the format's own steps in 32 bits (their results are bit for bit the
cache's), everything else in 64.  They share no code with the library."""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def quantise(x, bits):
    """(codes int64 [.., D], params bfloat16 [.., 2]) of rows x."""
    x = x.float() + 0.0
    n_max = 2 ** bits - 1
    lo, hi = x.amin(-1), x.amax(-1)  # (torch's propagate NaN)
    w = lo.contiguous().view(torch.int32)
    cut = w & -65536
    z = torch.where((lo < 0) & (cut != w), cut + 65536, cut).view(torch.float32)
    r = hi - z
    bad = ~torch.isfinite(r)
    s = torch.maximum(torch.maximum(r / torch.full_like(r, n_max), z.abs() * 2.0 ** -16), torch.full_like(r, 2.0 ** -100))
    s = torch.where(bad, torch.ones_like(s), s)
    z = torch.where(bad, torch.zeros_like(z), z)
    s = ((s.view(torch.int32) + 65535) & -65536).view(torch.float32)
    inv = (torch.ones_like(s) / s) * torch.full_like(s, 1.0 + 2.0 ** -21)
    n = ((x - z[..., None]) * inv[..., None] + 0.5).floor()
    n = torch.where(bad[..., None], torch.zeros_like(n), n).long()
    assert int(n.min()) >= 0 and int(n.max()) <= n_max
    nan = torch.full_like(s, float("nan"))
    return n, torch.stack([torch.where(bad, nan, s), torch.where(bad, nan, z)], -1).to(torch.bfloat16)


def pack(n, bits):
    return (n if bits == 8 else n[..., 0::2] + 16 * n[..., 1::2]).to(torch.uint8)


def unpack(c, bits):
    c = c.long()
    return c if bits == 8 else torch.stack([c % 16, c // 16], -1).flatten(-2)


def values(codes, params, bits):
    p = params.double()
    return p[..., 1:] + p[..., :1] * unpack(codes, bits).double()


def quant_attention(q, pools, tables, lens, scale, bits):
    """(out, bound): attention over the codes in 64 bits, and what the kernel's
    roundings may move each output by.

    Scores: tensor-core sums of 128 products and the terms of (s, z), each a
    32-bit rounding of at most 2^-23 of A_t = |scale| log2(e) (s sum |q| n + |z|
    sum |q|): an exponent off by 144 x 2^-23 A_t, and a weight by ln 2 times it,
    twice (the normaliser's share).  Weights enter the second product in FP16:
    half a step is 2^-11 of the code part s n, or 2^-25 of the row's largest s w
    where the weight is subnormal there (times the sum of the codes).  Sums over
    tokens and the correction z in 32 bits: 2^-18 of the magnitudes.  One
    rounding to BF16."""
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
            g = slice(h * (Hq // Hk), (h + 1) * (Hq // Hk))
            n = unpack(kc[blk, h, off], bits).double()
            s, z = (kp[blk, h, off].double()[:, i] for i in (0, 1))
            qh = q[b, g].double()
            x = (s * (qh @ n.T) + z * qh.sum(1, keepdim=True)) * scale
            size = (s * (qh.abs() @ n.T) + z.abs() * qh.abs().sum(1, keepdim=True)) * abs(scale) / math.log(2)
            w = torch.softmax(x, 1)
            off_w = (2 * math.log(2) * 144 * 2.0 ** -23 * size).amax(1, keepdim=True)
            c = unpack(vc[blk, h, off], bits).double()
            vs, vz = (vp[blk, h, off].double()[:, i] for i in (0, 1))
            o = w @ (c * vs[:, None] + vz[:, None])
            code, offset = (w * vs) @ c, (w * vz.abs()).sum(1, keepdim=True)
            e = 2.0 ** -11 * code + (off_w + 2.0 ** -18) * (code + offset)
            e = e + 2.0 ** -25 * (w * vs).amax(1, keepdim=True) * c.sum(0)
            out[b, g], bound[b, g] = o, e + HALF[torch.bfloat16] * (o.abs() + e)
    return out, bound


def prompt(q, k, v, q_lens, k_lens, scale):
    """(out, bound) of packed rows (no gaps), in 64 bits.

    Scores as above with 144 x 2^-23 of |scale| log2(e) |q| . |k|; with BF16
    every weight is rounded once more (half a step: 2^-8); 32-bit sums over m
    keys are off by at most (m / 16 + 64) x 2^-23 of the magnitudes (sixteen
    products a step); one rounding to the output's type."""
    Hq, Hk, D = q.shape[1], k.shape[1], q.shape[2]
    out, bound = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape, dtype=torch.float64)
    half = HALF[q.dtype]
    weight = half if q.dtype == torch.bfloat16 else 0.0
    iq = ik = 0
    for n, m in zip(q_lens, k_lens):
        seen = torch.arange(m)[None] <= torch.arange(n)[:, None] + (m - n)
        some = seen.any(1)
        for h in range(Hq):
            if n == 0 or m == 0:
                continue
            a, c, d = (x.double() for x in (q[iq:iq + n, h], k[ik:ik + m, h // (Hq // Hk)], v[ik:ik + m, h // (Hq // Hk)]))
            x = (a @ c.T * scale).masked_fill(~seen, -math.inf)
            size = (a.abs() @ c.abs().T * abs(scale) / math.log(2)).masked_fill(~seen, 0).amax(1, keepdim=True)
            w = torch.softmax(x, 1)[some]
            o, mass = w @ d, w @ d.abs()
            e = (weight + 2 * math.log(2) * 144 * 2.0 ** -23 * size[some] + (m / 16 + 64) * 2.0 ** -23) * mass
            out[iq:iq + n, h][some], bound[iq:iq + n, h][some] = o, e + half * (o.abs() + e)
        iq, ik = iq + n, ik + m
    return out, bound
