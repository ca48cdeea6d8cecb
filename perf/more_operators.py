"""The operators around a quantised cache that perf measures: their cases, inputs and plain forms.

Three groups:

* ``attend``: decode attention over a cache of 4- or 8-bit codes with a scale
  and an offset for every (token, head) row;
* ``cache`` / ``read``: rows quantised as they are written to that cache and
  read back through the block tables, and the read-back of an FP8 pool;
* ``prompt``: causal attention over whole prompts, packed one after the other,
  with grouped heads and, where rows of a cache come first, a cached prefix.

Every input comes from the seed alone.  The plain forms are elementary torch
operations in 32 bits (integers in 64).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "bf16": 2}


def _ceil(a, b):
    return -(-a // b)


# --------------------------------------------------------------------- cases
def _attend(name, seqs, lo, hi, bits, q_heads=32, kv_heads=8, dim=128, block=16):
    return {"name": name, "op": "attend", "seqs": seqs, "lo": lo, "hi": hi, "bits": bits, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "block": block}


def _cache(name, seqs, new_lo, new_hi, past_hi, bits, kv_heads=8, dim=128, block=16, inp="bf16"):
    return {"name": name, "op": "cache", "seqs": seqs, "new_lo": new_lo, "new_hi": new_hi, "past_hi": past_hi,
            "bits": bits, "kv_heads": kv_heads, "dim": dim, "block": block, "inp": inp}


def _read(name, seqs, lo, hi, kv_heads=8, dim=128, block=16):
    return {"name": name, "op": "read", "seqs": seqs, "lo": lo, "hi": hi, "kv_heads": kv_heads, "dim": dim,
            "block": block}


def _prompt(name, seqs, lo, hi, past_hi=0, q_heads=32, kv_heads=8, dim=128, inp="bf16"):
    return {"name": name, "op": "prompt", "seqs": seqs, "lo": lo, "hi": hi, "past_hi": past_hi, "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "inp": inp}


def listed():
    return [
        # four requests that have just started: latency
        _attend("attend_few", 4, 1, 512, 4),
        # the 64-sequence decode batch over a 4-bit cache
        _attend("attend_batch", 64, 128, 4096, 4),
        # the 55 full-context requests over an 8-bit cache
        _attend("attend_full", 55, 8192, 8192, 8, block=64),
        # two very long contexts: the split along the cache
        _attend("attend_long", 2, 130001, 131072, 4, block=64),
        # one decode step of 64 short requests: a row each written, the whole contexts read back
        _cache("cache_decode", 64, 1, 1, 63, 8),
        # 16 prompt chunks of up to 256 tokens behind what their requests hold already
        _cache("cache_chunks", 16, 1, 256, 1792, 4, block=32),
        # long prompts written at once, from 32-bit rows
        _cache("cache_prompts", 7, 2048, 8191, 0, 4, block=64, inp="f32"),
        # prefixes of an FP8 pool handed to the attention of the prompts that continue them
        _read("read_fp8", 9, 1000, 8192, block=32),
        # a few dozen short questions packed together
        _prompt("prompt_short", 33, 1, 127),
        # the prompts that one scheduler pass takes
        _prompt("prompt_batch", 16, 128, 4096),
        # chunks of up to 512 tokens behind long cached prefixes
        _prompt("prompt_chunks", 8, 256, 512, past_hi=8192),
        # one long document
        _prompt("prompt_long", 1, 16384, 16384),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


HEADS = [(32, 8), (32, 8), (8, 8), (16, 2), (12, 4), (5, 1), (64, 8), (16, 1)]


def draw(rng):
    op = rng.choice(["attend", "attend", "cache", "cache", "read", "prompt", "prompt", "prompt"])
    q_heads, kv_heads = rng.choice(HEADS)
    dim = rng.choice([64, 128, 128])
    block = rng.choice([16, 32, 64])
    if op == "attend":
        bits = rng.choice([4, 4, 8])
        seqs = _log(rng, 1, 256)
        # no more rows than the largest listed case
        hi = _log(rng, 1, min(131072, 55 * 8192 * 8 // (seqs * kv_heads)))
        return _attend("", seqs, rng.choice([0, 1, max(1, hi // 2)]), hi, bits, q_heads, kv_heads, dim, block)
    if op == "cache":
        seqs = _log(rng, 1, 128)
        new = _log(rng, 1, min(8192, 32768 // seqs))
        past = rng.choice([0, _log(rng, 1, max(1, 32768 // seqs))])
        return _cache("", seqs, rng.choice([0, 1, max(1, new // 2)]), new, past, rng.choice([4, 4, 8]), kv_heads, dim,
                      block, rng.choice(["bf16", "bf16", "f32"]))
    if op == "read":
        seqs = _log(rng, 1, 128)
        hi = _log(rng, 1, min(16384, 65536 // seqs))
        return _read("", seqs, rng.choice([0, 1, max(1, hi // 2)]), hi, kv_heads, dim, block)
    seqs = _log(rng, 1, 64)
    inp = rng.choice(["bf16", "bf16", "bf16", "f32"])
    # no more products than the long document
    most = int(math.sqrt(16384 * 16384 * 32 / (seqs * q_heads) / (20 if inp == "f32" else 2)))
    hi = _log(rng, 1, min(8192, most))
    past = rng.choice([0, 0, _log(rng, 1, max(1, min(16384, most)))])
    return _prompt("", seqs, rng.choice([0, 1, max(1, hi // 2)]), hi, past, q_heads, kv_heads, dim, inp)


# -------------------------------------------------------------------- inputs
def _gens(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    return g, np.random.default_rng(seed * 7919 + 19)


def _dev(x, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV, dtype)


def _offsets(n):
    return np.concatenate([[0], np.cumsum(n)])


def _lens(r, lo, hi, seqs):
    """Lengths in lo .. hi whose sum is the same for every seed: lo + x goes with hi - x."""
    x = r.integers(0, hi - lo + 1, seqs // 2)
    return r.permutation(np.concatenate([lo + x, hi - x, [(lo + hi + 1) // 2] * (seqs % 2)]).astype(np.int64))


def _tables(r, lens, block):
    """Block tables of a random order of the pool's blocks, padded with -1."""
    held = -(-np.asarray(lens) // block)
    num_blocks = max(1, int(held.sum()))
    order = r.permutation(num_blocks).astype(np.int32)
    tables = np.full((len(held), max(1, int(held.max()))), -1, np.int32)
    at = _offsets(held)
    for b, n in enumerate(held):
        tables[b, :n] = order[at[b]:at[b] + n]
    return tables, num_blocks


def _rows(g, shape, dtype, keys):
    """Rows as a projection gives them; keys have a few large channels."""
    x = torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)
    if keys:
        x[..., 3::29] *= 4.0
        x[..., 7] += 2.0
    return x.to(dtype)


# The format of a row of values x: z = lo rounded down to bfloat16, s = (hi - z) / N
# rounded up to it, codes n = (x - z) / s to the nearest (halves, which 16-bit
# inputs give often, upwards: a reciprocal that is 2^-21 too large sees to that),
# each value being z + s n.
def _down(x):
    w = x.view(torch.int32)
    cut = w & -65536
    return torch.where((w < 0) & (cut != w), cut + 65536, cut).view(torch.float32)


def _up(x):
    return ((x.view(torch.int32) + 65535) & -65536).view(torch.float32)


def _quantise(x, bits):
    """Codes [.., D] (whole numbers, float32), scale and offset [..] of rows of finite values."""
    x = x.float()
    z = _down(x.amin(-1) + 0.0)
    s = (x.amax(-1) - z) / torch.full_like(z, 2 ** bits - 1)  # (a number there would become a product with its inverse)
    s = _up(torch.maximum(s, (z.abs() * 2.0 ** -16).clamp(min=2.0 ** -100)))
    n = ((x - z[..., None]) * ((1.0 / s) * (1.0 + 2.0 ** -21))[..., None] + 0.5).floor()
    return n, s, z


def _pack(n, bits):
    n = n.to(torch.uint8)
    return n if bits == 8 else n[..., 0::2] | (n[..., 1::2] << 4)


def _unpack(c, bits):
    return c.float() if bits == 8 else torch.stack([c & 15, c >> 4], -1).flatten(-2).float()


def _quantised_pool(g, num_blocks, c):
    """Codes and (scale, offset) pairs of one of a cache's two tensors' blocks, as appends left them."""
    out = []
    for keys in (True, False):
        parts = []
        for first in range(0, num_blocks, 16384):
            n = min(16384, num_blocks - first)
            x = _rows(g, (n, c["kv_heads"], c["block"], c["dim"]), torch.bfloat16, keys)
            codes, s, z = _quantise(x, c["bits"])
            parts.append((_pack(codes, c["bits"]), torch.stack([s, z], -1).to(torch.bfloat16)))
        out += [torch.cat([p[i] for p in parts])[None] for i in (0, 1)]
    return out


def _attend_inputs(c, seed):
    g, r = _gens(seed)
    lens = _lens(r, c["lo"], c["hi"], c["seqs"])
    tables, num_blocks = _tables(r, lens, c["block"])
    kc, kp, vc, vp = _quantised_pool(g, num_blocks, c)
    q = torch.randn((c["seqs"], c["q_heads"], c["dim"]), generator=g, device=DEV).to(torch.bfloat16)
    return {"q": q, "k_codes": kc, "k_params": kp, "v_codes": vc, "v_params": vp, "tables": _dev(tables),
            "lens": _dev(lens), "host_lens": lens, "max_len": max(1, int(lens.max())), "num_blocks": num_blocks,
            "scale": 1.0 / math.sqrt(c["dim"])}


def _cache_inputs(c, seed):
    """New rows behind what the sequences hold (slots of shuffled blocks; one new token in sixteen of a larger
    batch is not stored), the tables, and the packed rows that are read back: all of every sequence."""
    g, r = _gens(seed)
    new = _lens(r, c["new_lo"], c["new_hi"], c["seqs"])
    past = _lens(r, 0, c["past_hi"], c["seqs"])
    lens = past + new
    tables, num_blocks = _tables(r, lens, c["block"])
    T, bs = int(new.sum()), c["block"]
    seq = np.repeat(np.arange(c["seqs"]), new)
    pos = np.arange(T) - _offsets(new)[seq] + past[seq]
    slots = tables[seq, pos // bs].astype(np.int64) * bs + pos % bs
    if T >= 64:
        slots[r.integers(0, T, T // 16)] = -1
    k, v = (_rows(g, (T, c["kv_heads"], c["dim"]), TORCH[c["inp"]], keys) for keys in (True, False))
    kc, kp, vc, vp = _quantised_pool(g, num_blocks, c)
    return {"k": k, "v": v, "slots": _dev(slots, torch.int64), "k_codes": kc, "k_params": kp, "v_codes": vc,
            "v_params": vp, "tables": _dev(tables), "offsets": _dev(_offsets(lens)), "rows": int(lens.sum()),
            "host_lens": lens, "num_blocks": num_blocks}


def _read_inputs(c, seed):
    g, r = _gens(seed)
    lens = _lens(r, c["lo"], c["hi"], c["seqs"])
    tables, num_blocks = _tables(r, lens, c["block"])
    shape = (1, num_blocks, c["kv_heads"], c["block"], c["dim"])
    k, v = (torch.randn(shape, generator=g, device=DEV).mul_(90.0).clamp_(-448, 448).to(torch.float8_e4m3fn)
            for _ in range(2))
    return {"k_pool": k, "v_pool": v, "k_scale": 0.0117, "v_scale": 0.0093, "tables": _dev(tables),
            "offsets": _dev(_offsets(lens)), "rows": int(lens.sum()), "host_lens": lens, "num_blocks": num_blocks}


def _prompt_inputs(c, seed):
    """Queries of packed prompts: rows of one projection, or with cached prefixes (past > 0) keys and values
    that were read back in front of the new ones."""
    g, r = _gens(seed)
    Hq, Hk, D, dt = c["q_heads"], c["kv_heads"], c["dim"], TORCH[c["inp"]]
    n = _lens(r, c["lo"], c["hi"], c["seqs"])
    past = _lens(r, 0, c["past_hi"], c["seqs"])
    T, Tk = int(n.sum()), int((n + past).sum())
    s = {"host_q": n, "host_k": n + past, "q_offsets": _dev(_offsets(n)), "k_offsets": _dev(_offsets(n + past)),
         "scale": 1.0 / math.sqrt(D)}
    if c["past_hi"]:
        s["q"], s["k"], s["v"] = (torch.randn((t, h, D), generator=g, device=DEV).to(dt)
                                  for t, h in ((T, Hq), (Tk, Hk), (Tk, Hk)))
    else:
        qkv = torch.randn((T, (Hq + 2 * Hk) * D), generator=g, device=DEV).to(dt)
        s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hk * D, Hk * D], 1))
    return s


INPUTS = {"attend": _attend_inputs, "cache": _cache_inputs, "read": _read_inputs, "prompt": _prompt_inputs}


def prepare(case, seed):
    c = case
    s = INPUTS[c["op"]](c, seed)
    s["case"] = c
    if c["op"] in ("cache", "read"):
        s["k_rows"], s["v_rows"] = (torch.empty((s["rows"], c["kv_heads"], c["dim"]), dtype=torch.bfloat16, device=DEV)
                                    for _ in range(2))
    if not own:
        return s
    from paged_kv_cache_194_gb300 import binding as pk
    s["pk"] = pk
    if c["op"] in ("attend", "cache"):
        pool = pk.QuantKVPool(1, s["num_blocks"], c["block"], c["kv_heads"], c["dim"], c["bits"])
        for name in ("k_codes", "k_params", "v_codes", "v_params"):
            getattr(pool, name).copy_(s.pop(name))
        s["pool"] = pool
    if c["op"] == "attend":
        s["out"] = torch.empty_like(s["q"])
        s["workspace"] = pk.quant_decode_workspace(pool, c["seqs"], c["q_heads"], s["max_len"])
    elif c["op"] == "read":
        pool = s["pool"] = pk.KVPool(1, s["num_blocks"], c["block"], c["kv_heads"], c["dim"], "fp8", s["k_scale"],
                                     s["v_scale"])
        pool.k.copy_(s.pop("k_pool").view(torch.uint8))
        pool.v.copy_(s.pop("v_pool").view(torch.uint8))
    elif c["op"] == "prompt":
        s["out"] = torch.empty(s["q"].shape, dtype=s["q"].dtype, device=DEV)
        s["workspace"] = pk.prompt_attention_workspace(s["q"], c["seqs"], c["kv_heads"])
    return s


# ----------------------------------------------------------------------- run
def run(state):
    return (RUN_OWN if own else RUN_PLAIN)[state["case"]["op"]](state)


def _own_attend(s):
    return s["pk"].paged_quant_decode_attention(s["q"], s["pool"], 0, s["tables"], s["lens"], s["max_len"], s["scale"],
                                                out=s["out"], workspace=s["workspace"])


def _own_cache(s):
    s["pk"].kv_quant_append(s["pool"], 0, s["k"], s["v"], s["slots"])
    return _own_read(s)


def _own_read(s):
    return s["pk"].kv_read(s["pool"], 0, s["tables"], s["offsets"], s["rows"], k_out=s["k_rows"], v_out=s["v_rows"])


def _own_prompt(s):
    return s["pk"].prompt_attention(s["q"], s["k"], s["v"], s["q_offsets"], s["k_offsets"], s["scale"], out=s["out"],
                                    workspace=s["workspace"])


def _values(codes, params, bits):
    """What codes [.., D * bits / 8] and pairs [.., 2] stand for."""
    p = params.float()
    return _unpack(codes, bits) * p[..., :1] + p[..., 1:]


def _plain_attend(s):
    """All sequences at once, padded to the longest: gather through the tables, softmax, weighted sum."""
    c, q = s["case"], s["q"]
    B, Hk, D, bs, L = c["seqs"], c["kv_heads"], c["dim"], c["block"], s["max_len"]
    blocks = s["tables"][:, :_ceil(L, bs)].long().clamp(min=0)
    k, v = (_values(s[x + "_codes"][0][blocks], s[x + "_params"][0][blocks], c["bits"])
            .transpose(1, 2).reshape(B, Hk, -1, D)[:, :, :L] for x in ("k", "v"))
    gone = (torch.arange(L, device=DEV)[None] >= s["lens"].long()[:, None])[:, None, None]
    z = (q.float().view(B, Hk, -1, D) @ k.transpose(2, 3)) * s["scale"]
    z = z.masked_fill(gone, -math.inf)
    p = (z - z.amax(3, keepdim=True).clamp(min=-3e38)).exp()
    out = (p @ v) / p.sum(3, keepdim=True).clamp(min=1e-30)
    return out.view(q.shape).to(q.dtype)


def _token_slots(s):
    """Block and place in it of every packed row."""
    row = torch.arange(s["rows"], device=DEV)
    offsets = s["offsets"].long()
    seq = torch.searchsorted(offsets[1:], row, right=True)
    pos = row - offsets[seq]
    bs = s["case"]["block"]
    return s["tables"][seq, pos // bs].long(), pos % bs


def _plain_cache(s):
    c = s["case"]
    keep = s["slots"] >= 0
    slot = s["slots"][keep]
    blk, off = slot // c["block"], slot % c["block"]
    for x in ("k", "v"):
        n, sc, z = _quantise(s[x][keep], c["bits"])
        s[x + "_codes"][0][blk, :, off] = _pack(n, c["bits"])
        s[x + "_params"][0][blk, :, off] = torch.stack([sc, z], -1).to(torch.bfloat16)
    blk, off = _token_slots(s)
    for x in ("k", "v"):
        s[x + "_rows"].copy_(_values(s[x + "_codes"][0][blk, :, off], s[x + "_params"][0][blk, :, off], c["bits"]))
    return s["k_rows"], s["v_rows"]


def _plain_read(s):
    blk, off = _token_slots(s)
    for x in ("k", "v"):  # indexed loads of bytes
        rows = s[x + "_pool"][0].view(torch.uint8)[blk, :, off].view(torch.float8_e4m3fn)
        s[x + "_rows"].copy_(rows.float() * s[x + "_scale"])
    return s["k_rows"], s["v_rows"]


def _padded(x, offsets, lens, longest):
    """Packed rows [T, H, D] as [B, H, longest, D], and which of them are there."""
    at = torch.arange(longest, device=DEV)[None]
    there = at < lens[:, None]
    row = (offsets[:-1, None] + at).clamp(max=max(0, x.shape[0] - 1))
    return x[row].float().masked_fill(~there[:, :, None, None], 0.0).transpose(1, 2), there


def _plain_prompt(s):
    """All prompts at once, padded to the longest, one KV head after the other."""
    c, q = s["case"], s["q"]
    Hk, g = c["kv_heads"], c["q_heads"] // c["kv_heads"]
    out = torch.empty(q.shape, dtype=q.dtype, device=DEV)
    if q.shape[0] == 0:
        return out
    qo, ko = s["q_offsets"].long(), s["k_offsets"].long()
    n, m = qo.diff(), ko.diff()
    N, M = int(s["host_q"].max()), int(s["host_k"].max())
    ahead = (m - n)[:, None, None]  # keys before the first query
    seen = torch.arange(M, device=DEV)[None, None] <= torch.arange(N, device=DEV)[None, :, None] + ahead
    for h in range(Hk):
        qh, there = _padded(q[:, h * g:(h + 1) * g], qo, n, N)
        kh, vh = (_padded(x[:, h:h + 1], ko, m, M)[0] for x in (s["k"], s["v"]))
        z = (qh @ kh.transpose(2, 3)).mul_(s["scale"]).masked_fill_(~seen[:, None], -math.inf)
        p = z.sub_(z.amax(3, keepdim=True)).exp_()
        o = (p @ vh) / p.sum(3, keepdim=True)
        out[:, h * g:(h + 1) * g] = o.transpose(1, 2)[there].to(q.dtype)
    return out


RUN_PLAIN = {"attend": _plain_attend, "cache": _plain_cache, "read": _plain_read, "prompt": _plain_prompt}
RUN_OWN = {"attend": _own_attend, "cache": _own_cache, "read": _own_read, "prompt": _own_prompt}


# ---------------------------------------------------------------------- work
def work(case):
    c = case
    D = c["dim"]
    if c["op"] == "prompt":
        n, past = (c["lo"] + c["hi"]) / 2, c["past_hi"] / 2
        var = ((c["hi"] - c["lo"] + 1) ** 2 - 1) / 12
        pairs = c["seqs"] * ((n * n + var + n) / 2 + n * past)  # (query, key) pairs seen
        rows = c["seqs"] * (2 * n * c["q_heads"] + 2 * (n + past) * c["kv_heads"])
        return {"bytes": int(rows * D * BYTES[c["inp"]]) + 1, "flops": int(4 * D * c["q_heads"] * pairs)}
    if c["op"] == "read":
        rows = c["seqs"] * (c["lo"] + c["hi"]) / 2 * c["kv_heads"] * 2
        return {"bytes": int(rows * D * 3) + 1, "flops": int(rows * D)}
    stored = D * c["bits"] // 8 + 4  # bytes of a row
    if c["op"] == "attend":
        tokens = c["seqs"] * (c["lo"] + c["hi"]) / 2
        return {"bytes": int(tokens * c["kv_heads"] * 2 * stored + 4 * c["seqs"] * c["q_heads"] * D),
                "flops": int(4 * c["q_heads"] * D * tokens)}
    new = c["seqs"] * (c["new_lo"] + c["new_hi"]) / 2 * c["kv_heads"] * 2
    rows = new + c["seqs"] * c["past_hi"] / 2 * c["kv_heads"] * 2
    # new rows read and stored, all of them read (the new ones as they are written) and given out
    return {"bytes": int(new * (D * BYTES[c["inp"]] + stored) + (rows - new) * stored + rows * D * 2) + 1,
            "flops": int(3 * new * D + 2 * rows * D)}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    return {"attend": _exact_attend, "cache": _exact_cache, "read": _exact_read,
            "prompt": _exact_prompt}[case["op"]](case, INPUTS[case["op"]](case, seed))


def _exact_values(codes, params, bits):
    """Rows in 64 bits, the codes taken apart by whole-number arithmetic."""
    c = codes.long()
    if bits == 4:
        both = torch.empty(c.shape[:-1] + (2 * c.shape[-1],), dtype=torch.int64, device=DEV)
        both[..., 0::2], both[..., 1::2] = c % 16, c // 16
        c = both
    p = params.double()
    return p[..., 1:2] + c.double() * p[..., 0:1]


def _exact_attend(c, s):
    """One sequence and KV head at a time over slots."""
    bs, group = c["block"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros((c["seqs"], c["q_heads"], c["dim"]), dtype=torch.float64, device=DEV)
    for b in range(c["seqs"]):
        t = torch.arange(int(s["host_lens"][b]), device=DEV)
        if not len(t):
            continue
        blk, off = s["tables"][b].long()[t // bs], t % bs
        for h in range(c["kv_heads"]):
            k, v = (_exact_values(s[x + "_codes"][0, blk, h, off], s[x + "_params"][0, blk, h, off], c["bits"])
                    for x in ("k", "v"))
            w = s["q"][b, h * group:(h + 1) * group].double() @ k.T * s["scale"]
            out[b, h * group:(h + 1) * group] = (w - torch.logsumexp(w, 1, keepdim=True)).exp() @ v
    return out


def _bf16_at(x, upward):
    """The nearest bfloat16 value on one side of x, in 64 bits."""
    m, e = torch.frexp(x)
    m = torch.ceil(m * 256) if upward else torch.floor(m * 256)
    return torch.ldexp(m / 256, e)


def _exact_cache(c, s):
    bs, N = c["block"], 2 ** c["bits"] - 1
    rows = []
    where = [(s["tables"][b].long()[t // bs], t % bs) for b, n in enumerate(s["host_lens"])
             for t in [torch.arange(int(n), device=DEV)]]
    for name in ("k", "v"):
        pool = _exact_values(s[name + "_codes"][0], s[name + "_params"][0], c["bits"])
        keep = s["slots"] >= 0
        x = s[name][keep].double()
        z = _bf16_at(x.min(-1, keepdim=True).values, False)
        step = (x.max(-1, keepdim=True).values - z) / N
        step = torch.maximum(step, torch.maximum(z.abs() / 65536, torch.full_like(z, 2.0 ** -100)))
        step = _bf16_at(step, True)
        n = torch.floor((x - z) / step + 0.5)
        slot = s["slots"][keep]
        pool[slot // bs, :, slot % bs] = z + n * step
        rows.append(torch.cat([pool[blk, :, off] for blk, off in where]))
    return rows[0], rows[1]


def _exact_read(c, s):
    bs = c["block"]
    where = [(s["tables"][b].long()[t // bs], t % bs) for b, n in enumerate(s["host_lens"])
             for t in [torch.arange(int(n), device=DEV)]]
    return tuple(torch.cat([(p[0].float()[blk, :, off]).double() for blk, off in where]) * sc
                 for p, sc in ((s["k_pool"], s["k_scale"]), (s["v_pool"], s["v_scale"])))


def _exact_prompt(c, s):
    """One sequence and KV head at a time, a thousand queries after the other, over the keys that they see."""
    g = c["q_heads"] // c["kv_heads"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    qa, ka = _offsets(s["host_q"]), _offsets(s["host_k"])
    for b in range(c["seqs"]):
        n, m = int(s["host_q"][b]), int(s["host_k"][b])
        for h in range(c["kv_heads"]):
            k, v = (s[x][ka[b]:ka[b + 1], h].double() for x in ("k", "v"))
            for i in range(0, n, 1024):
                j = min(n, i + 1024)
                last = m - n + j  # keys before this one are seen by the last of these queries
                w = torch.einsum("nhd,md->hnm", s["q"][qa[b] + i:qa[b] + j, h * g:(h + 1) * g].double(), k[:last])
                hide = torch.ones((j - i, last), dtype=torch.bool, device=DEV).triu(m - n + i + 1)
                w = torch.softmax((w * s["scale"]).masked_fill(hide, -math.inf), 2)
                out[qa[b] + i:qa[b] + j, h * g:(h + 1) * g] = torch.einsum("hnm,md->nhd", w, v[:last])
    return out
