"""Plain references of the serving-step operators: 64-bit torch on the CPU and
walks over Python lists.  They share no code with the library."""
import math

import torch

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # half a step, relative


def attention(q, k_pool, v_pool, tables, lens, scale, k_scale=1.0, v_scale=1.0):
    """(out, mass, floor): softmax(scale q K^T) V per sequence in 64 bits, the
    same weights over |V| (what a relative error of each weight can move), and
    the largest weight times the sum of |V|."""
    B, Hq, D = q.shape
    k_pool, v_pool = k_pool.double(), v_pool.double()
    _, Hk, bs, _ = k_pool.shape
    out = torch.zeros(B, Hq, D, dtype=torch.float64)
    mass = torch.zeros(B, Hq, D, dtype=torch.float64)
    floor = torch.zeros(B, Hq, D, dtype=torch.float64)
    for b, L in enumerate(lens):
        if L == 0:
            continue
        t = torch.arange(L)
        blk, off = tables[b].long()[t // bs], t % bs
        for h in range(Hq):
            g = h // (Hq // Hk)
            k = k_pool[blk, g, off] * k_scale
            v = v_pool[blk, g, off] * v_scale
            w = torch.softmax(k @ q[b, h].double() * scale, 0)
            out[b, h], mass[b, h], floor[b, h] = w @ v, w @ v.abs(), w.max() * v.abs().sum(0)
    return out, mass, floor


def norm_rope(x, weight, eps, cos_sin, positions, sections, interleaved):
    """(z, size): the normed and rotated rows of x [T, H, D] in 64 bits, and
    for every element the magnitudes that were added up to it."""
    x = x.double()
    if weight is not None:
        x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * weight.double()
    half = sum(sections)
    axis = torch.tensor([a for a, n in enumerate(sections) for _ in range(n)])
    z, size = x.clone(), x.abs()
    for j in range(half):
        p = positions[axis[j]].long()
        c, s = cos_sin[p, j].double()[:, None], cos_sin[p, half + j].double()[:, None]
        a, b = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        u, w = x[:, :, a], x[:, :, b]
        z[:, :, a], z[:, :, b] = u * c - w * s, w * c + u * s
        size[:, :, a] = u.abs() * c.abs() + w.abs() * s.abs()
        size[:, :, b] = w.abs() * c.abs() + u.abs() * s.abs()
    return z, size


def grow(tables, lens, new, ring, free_state, bs, max_tokens):
    """Walk over the requests; tables is changed in place (a list of lists)."""
    head, count = free_state
    width = len(tables[0]) if tables else 0
    slots, pos, seqs = [-1] * max_tokens, [0] * max_tokens, [-1] * max_tokens
    offsets, granted, lens_out = [0], [], []
    waiting, row = False, 0
    for b, (L, n) in enumerate(zip(lens, new)):
        held, need = -(-L // bs), -(-(L + n) // bs) - -(-L // bs)
        room = L + n <= width * bs and (n == 0 or row + n <= max_tokens)
        if room and need > 0 and (waiting or need > count):
            waiting = True
        ok = room and (need == 0 or not waiting)
        if ok:
            for j in range(need):
                tables[b][held + j] = ring[head]
                head, count = (head + 1) % len(ring), count - 1
        for p in range(L, L + n):
            if row < max_tokens:
                pos[row], seqs[row] = p, b
                if ok:
                    slots[row] = tables[b][p // bs] * bs + p % bs
            row += 1
        offsets.append(min(row, max_tokens))
        granted.append(n if ok else 0)
        lens_out.append(L + n if ok else L)
    return slots, pos, seqs, offsets, granted, lens_out, [head, count]


def release(tables, lens, finished, keep, ring, free_state, bs):
    """ring is changed in place."""
    head, count = free_state
    out = list(lens)
    for b, L in enumerate(lens):
        if finished[b]:
            held = -(-L // bs)
            for blk in tables[b][min(max(keep[b], 0), held):held]:
                ring[(head + count) % len(ring)] = blk
                count += 1
            out[b] = 0
    return out, [head, count]


def attention_bound(out, mass, kv="bf16", floor=0.0):
    """|error| of the tensor-core design.  Every weight is rounded to BF16 (half
    a step: at most 2^-8 of it), with FP8 pools to two E4M3 terms (2^-4 of the
    weight, then 2^-4 of the rest: 2^-8 again, and 2^-11 for the FP16 between; at
    least 2^-15 of the row's largest weight, where the low term is subnormal:
    `floor` is that weight times the sum of |V|).  The output is rounded once to
    BF16.  Scores, sums and 2^x in fp32, and FP8's query split (exact but for
    elements below 2^-10 of a row's largest, which are off by 2^-18 of it), add
    up to well under 2^-13 of `mass` (128-term dot products of values near 4:
    128 x 2^-24 x 16 in the exponent; the split: 2^-18 x 3 x 128 x 0.09)."""
    h = HALF[torch.bfloat16]
    weight = h * mass
    if kv == "fp8":
        weight = weight + 2.0 ** -11 * mass + 2.0 ** -15 * floor
    return weight + h * (out.abs() + weight) + 2.0 ** -13 * mass


def scale_for(d):
    return 1.0 / math.sqrt(d)
