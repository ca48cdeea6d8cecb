"""The serving-step operators that perf measures: their cases, inputs and plain forms.

Three groups of operators around the paged KV cache:

* ``prefix``: decode attention of a batch whose sequences share long prefixes
  (system prompts, few-shot examples, forked requests);
* ``rope``: the step between the QKV projection and attention: per-head RMS
  norm, rotary positions and the append to the paged cache in one pass;
* ``grow`` / ``release``: block tables, slot maps and the free list kept on
  the GPU from request lengths.

Every input comes from the seed alone.  The plain forms are elementary torch
operations in 32 bits (integers in 64).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
ELEM = {"f32": 4, "bf16": 2, "fp8": 1}
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
FP8_MAX = 448.0


def _ceil(a, b):
    return -(-a // b)


# --------------------------------------------------------------------- cases
def _prefix(name, groups, prefix, own_tokens, q_heads=32, kv_heads=8, dim=128, block=16, pool="bf16"):
    return {"name": name, "op": "prefix", "groups": groups, "prefix_lo": prefix[0], "prefix_hi": prefix[1],
            "seqs": own_tokens[0], "own_lo": own_tokens[1], "own_hi": own_tokens[2], "q_heads": q_heads,
            "kv_heads": kv_heads, "dim": dim, "block": block, "pool": pool}


def _rope(name, tokens, q_heads=32, kv_heads=8, dim=128, rotary=128, axes=1, interleaved=False, norm=True,
          block=16, pool="bf16", inp="bf16", max_pos=8192):
    return {"name": name, "op": "rope", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim,
            "rotary": rotary, "axes": axes, "interleaved": interleaved, "norm": norm, "block": block, "pool": pool,
            "inp": inp, "max_pos": max_pos}


def _tables(name, op, seqs, len_hi, block=16, prompts=0, chunk=0, finished=0.25):
    return {"name": name, "op": op, "seqs": seqs, "len_hi": len_hi, "block": block, "prompts": prompts,
            "chunk": chunk, "finished": finished}


def listed():
    return [
        # four requests of one short system prompt, just started: latency
        _prefix("prefix_few", 1, (512, 512), (4, 1, 64)),
        # the 64-sequence decode batch, half of whose context is one shared prompt
        _prefix("prefix_batch", 1, (2048, 2048), (64, 128, 2048)),
        # one long document asked about by 64 requests
        _prefix("prefix_document", 1, (32768, 32768), (64, 1, 1024), block=64),
        # eight prompts of odd lengths shared by 55 requests over an FP8 pool
        _prefix("prefix_groups_fp8", 8, (1024, 8192), (55, 1, 1024), block=64, pool="fp8"),
        # the small fp32 geometry: a handful of tokens, partial rotation
        _rope("rope_tiny_f32", 33, q_heads=2, kv_heads=1, dim=64, rotary=32, pool="f32", inp="f32", max_pos=512),
        # one decode step of 64 sequences
        _rope("rope_decode", 64),
        # 16 prompt chunks of 256 tokens
        _rope("rope_chunks", 4096, block=32),
        # a long multi-modal prompt: three position axes, FP8 pool, an odd token count
        _rope("rope_axes_fp8", 32771, axes=3, interleaved=True, block=64, pool="fp8"),
        # one decode step of the 256-sequence in-flight batch
        _tables("grow_decode", "grow", 256, 8192, block=32),
        # prompt chunks mixed into a large decode batch
        _tables("grow_chunks", "grow", 1024, 4096, prompts=128, chunk=2048),
        # a quarter of the in-flight batch finishes
        _tables("release_quarter", "release", 256, 8192, block=32),
        # a large batch is dropped at once
        _tables("release_all", "release", 4096, 4096, finished=1.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prefix", "prefix", "rope", "rope", "grow", "release"])
    if op == "prefix":
        pool = rng.choice(["bf16", "bf16", "bf16", "fp8", "fp8", "f32"])
        dim = rng.choice([64, 128, 128, 128])
        q_heads, kv_heads = rng.choice([(32, 8), (32, 8), (8, 8), (16, 2), (12, 4), (5, 1), (64, 8)])
        seqs = _log(rng, 1, 64)
        groups = rng.randint(1, min(seqs, 8))
        # no more tokens to read, nor products to form, than the largest listed case
        small = 16 if pool == "f32" else 1
        hi = min(32768 // groups, 32768 * 64 * 32 // (seqs * q_heads)) // small
        lo = _log(rng, 16, hi)
        return _prefix("", groups, (lo, rng.randint(lo, hi)), (seqs, 0, _log(rng, 1, min(1024, hi))), q_heads,
                       kv_heads, dim, rng.choice([16, 32, 64]), pool)
    if op == "rope":
        dim = rng.choice([64, 128, 128])
        pool = rng.choice(["bf16", "bf16", "fp8", "f32"])
        inp = "f32" if pool == "f32" else rng.choice(["bf16", "bf16", "f32"])
        q_heads, kv_heads = rng.choice([(32, 8), (8, 8), (16, 2), (12, 4), (5, 1)])
        return _rope("", _log(rng, 1, 8192), q_heads, kv_heads, dim,
                     rng.choice([dim, dim, dim // 2, dim - 16, 16]), rng.choice([1, 1, 2, 3]),
                     rng.random() < 0.5, rng.random() < 0.75, rng.choice([16, 32, 64]), pool, inp,
                     rng.choice([1000, 8192, 131072]))
    seqs = _log(rng, 1, 4096)
    block = rng.choice([16, 32, 64])
    if op == "release":
        return _tables("", "release", seqs, _log(rng, 1, 4096), block, finished=rng.choice([0.1, 0.25, 0.5, 1.0]))
    prompts = rng.choice([0, rng.randint(1, max(1, seqs // 8))])
    return _tables("", "grow", seqs, _log(rng, 16, 8192), block, min(prompts, 128), _log(rng, 2, 2048))


# -------------------------------------------------------------------- inputs
def _gens(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 11)
    return g, np.random.default_rng(seed * 7919 + 13)


def _inverse(scale):
    """1 / scale, rounded once to 32 bits."""
    return float(np.float32(1.0) / np.float32(scale))


def _prefix_inputs(c, seed):
    """Groups of consecutive sequences; the first prefix_lens[g] tokens of a
    group's sequences lie in the same (whole) blocks, as the block manager's
    prefix matching shares them.  Tables are a random order of the pool."""
    g, r = _gens(seed)
    B, G, bs = c["seqs"], c["groups"], c["block"]
    cuts = np.sort(r.choice(np.arange(1, B), G - 1, replace=False)) if G > 1 else np.zeros(0, np.int64)
    offsets = np.concatenate([[0], cuts, [B]]).astype(np.int64)
    prefix = r.integers(c["prefix_lo"], c["prefix_hi"] + 1, G) // bs * bs
    lens = np.zeros(B, np.int64)
    for i in range(G):
        n = offsets[i + 1] - offsets[i]
        lens[offsets[i]:offsets[i + 1]] = prefix[i] + r.integers(c["own_lo"], c["own_hi"] + 1, n)
    own_blocks = [_ceil(int(lens[b] - prefix[i]), bs) for i in range(G) for b in range(offsets[i], offsets[i + 1])]
    num_blocks = max(1, int(sum(prefix) // bs + sum(own_blocks)))
    width = max(1, _ceil(int(lens.max()), bs))
    order = r.permutation(num_blocks).astype(np.int32)
    tables = np.full((B, width), -1, np.int32)
    at = 0
    for i in range(G):
        p = int(prefix[i]) // bs
        for b in range(offsets[i], offsets[i + 1]):
            tables[b, :p] = order[at:at + p]
        at += p
        for b in range(offsets[i], offsets[i + 1]):
            n = own_blocks[b]
            tables[b, p:p + n] = order[at:at + n]
            at += n
    shape = (1, num_blocks, c["kv_heads"], bs, c["dim"])
    wide = torch.float32 if c["pool"] == "f32" else torch.bfloat16
    kv, scales = [], []
    for _ in range(2):
        x = torch.randn(shape, generator=g, device=DEV, dtype=wide)
        s = 1.0
        if c["pool"] == "fp8":
            s = float(x.abs().max().float() / FP8_MAX)
            x = (x.float() * _inverse(s)).clamp(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
        kv.append(x)
        scales.append(s)
    q = torch.randn((B, c["q_heads"], c["dim"]), generator=g, device=DEV, dtype=wide)
    return {"q": q, "k": kv[0], "v": kv[1], "k_scale": scales[0], "v_scale": scales[1],
            "tables": torch.from_numpy(tables).to(DEV), "host_lens": [int(x) for x in lens],
            "lens": torch.from_numpy(lens.astype(np.int32)).to(DEV),
            "offsets": torch.from_numpy(offsets.astype(np.int32)).to(DEV),
            "prefix": torch.from_numpy(prefix.astype(np.int32)).to(DEV),
            "scale": 1.0 / math.sqrt(c["dim"]), "max_len": max(1, int(lens.max()))}


def _sections(c):
    """Rotated pairs per position axis (time, height, width: the first axis
    takes what the others leave)."""
    half, a = c["rotary"] // 2, c["axes"]
    rest = half // (a + 1) if a > 1 else 0
    return [half - rest * (a - 1)] + [rest] * (a - 1)


def _angles(c):
    """cos | sin of the standard frequencies, from 64-bit angles: [max_pos, rotary]."""
    j = torch.arange(c["rotary"] // 2, dtype=torch.float64, device=DEV)
    a = torch.arange(c["max_pos"], dtype=torch.float64, device=DEV)[:, None] * 10000.0 ** (-2.0 * j / c["rotary"])
    return torch.cat([a.cos(), a.sin()], 1).to(torch.float32)


def _rope_inputs(c, seed):
    """Rows of a QKV projection [tokens, q | k | v], positions, slots of
    shuffled blocks (one token in sixteen of a larger batch has no slot)."""
    g, r = _gens(seed)
    T, Hq, Hk, D, bs = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"], c["block"]
    dt = TORCH[c["inp"]]
    qkv = torch.randn((T, (Hq + 2 * Hk) * D), generator=g, device=DEV, dtype=torch.float32).to(dt)
    num_blocks = _ceil(T, bs) + 1
    order = r.permutation(num_blocks)
    t = np.arange(T)
    slots = (order[t // bs] * bs + t % bs).astype(np.int64)
    if T >= 16:
        slots[r.integers(0, T, T // 16)] = -1
    pos = r.integers(0, c["max_pos"], (c["axes"], T)).astype(np.int32)
    weights = [None, None]
    if c["norm"]:
        weights = [(1.0 + 0.1 * torch.randn(D, generator=g, device=DEV)).to(dt) for _ in range(2)]
    scale = float(np.float32(5.0 / FP8_MAX)) if c["pool"] == "fp8" else 1.0
    return {"q": qkv[:, :Hq * D].unflatten(1, (Hq, D)), "k": qkv[:, Hq * D:(Hq + Hk) * D].unflatten(1, (Hk, D)),
            "v": qkv[:, (Hq + Hk) * D:].unflatten(1, (Hk, D)), "num_blocks": num_blocks,
            "slots": torch.from_numpy(slots).to(DEV), "pos": torch.from_numpy(pos).to(DEV), "cos_sin": _angles(c),
            "q_weight": weights[0], "k_weight": weights[1], "k_scale": scale, "v_scale": scale, "eps": 1e-6}


def _table_inputs(c, seed):
    """Tables of a running batch and a free ring that wraps.  Growing: one new
    token per sequence, a prompt chunk for the first few, and a free list that
    just covers about nine in ten of the blocks asked for."""
    _, r = _gens(seed)
    B, bs = c["seqs"], c["block"]
    lens = np.clip(np.exp(r.normal(math.log(max(1.0, c["len_hi"] / 8)), 1.0, B)).astype(np.int64), 0, c["len_hi"])
    new = np.ones(B, np.int64)
    new[r.random(B) < 0.05] = 0
    if c["prompts"]:
        who = r.choice(B, min(B, c["prompts"]), replace=False)
        new[who] = r.integers(1, c["chunk"] + 1, len(who))
        lens[who] = r.integers(0, max(1, c["len_hi"] // 4), len(who))
    if c["op"] == "release":
        new[:] = 0
    held = -(-lens // bs)
    need = -(-(lens + new) // bs) - held
    longest = c["len_hi"] + max(1, c["chunk"])
    width = _ceil(longest, bs)
    total = B * _ceil(c["len_hi"] + 1, bs) + c["prompts"] * _ceil(c["chunk"], bs)  # the pool's blocks
    asked = math.ceil(0.9 * need.sum())
    order = r.permutation(total).astype(np.int32)
    tables = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    ring = np.full(total, -1, np.int32)
    head = int(r.integers(0, total))
    free = order[at:] if c["op"] == "release" else order[at:at + asked]
    ring[(head + np.arange(len(free))) % total] = free
    done = (r.random(B) < c["finished"]).astype(np.int32)
    keep = np.minimum(held, r.integers(0, 3, B)).astype(np.int32)
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    return {"tables": dev(tables), "lens": dev(lens.astype(np.int32)), "new": dev(new.astype(np.int32)),
            "ring": dev(ring), "free": dev(np.array([head, len(free)], np.int32)), "done": dev(done),
            "keep": dev(keep), "max_tokens": _ceil(B + c["prompts"] * c["chunk"], 64) * 64, "num_blocks": total,
            "bs": bs}


INPUTS = {"prefix": _prefix_inputs, "rope": _rope_inputs, "grow": _table_inputs, "release": _table_inputs}


def prepare(case, seed):
    c = case
    s = INPUTS[c["op"]](c, seed)
    s["case"] = c
    if c["op"] == "rope":
        s["k_pool"], s["v_pool"] = (torch.zeros((1, s["num_blocks"], c["kv_heads"], c["block"], c["dim"]),
                                                dtype=TORCH[c["pool"]], device=DEV) for _ in range(2))
    if not own:
        return s
    from paged_kv_cache_194_gb300 import binding as pk
    s["pk"] = pk
    raw = lambda x: x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x
    if c["op"] == "prefix":
        pool = pk.KVPool(1, s["k"].shape[1], c["block"], c["kv_heads"], c["dim"], c["pool"], s["k_scale"],
                         s["v_scale"])
        pool.k.copy_(raw(s.pop("k")))
        pool.v.copy_(raw(s.pop("v")))
        s["out"] = torch.empty_like(s["q"])
        s["workspace"] = pk.prefix_decode_workspace(pool, c["seqs"], c["groups"], c["q_heads"], s["max_len"])
    elif c["op"] == "rope":
        pool = pk.KVPool(1, s["num_blocks"], c["block"], c["kv_heads"], c["dim"], c["pool"], s["k_scale"],
                         s["v_scale"], fill=0)
        s["k_pool"], s["v_pool"] = (x.view(TORCH[c["pool"]]) if c["pool"] == "fp8" else x for x in (pool.k, pool.v))
        s["rope"] = pk.RopeTable(s["cos_sin"], sections=_sections(c), interleaved=c["interleaved"])
        s["out"] = torch.empty((c["tokens"], c["q_heads"], c["dim"]), device=DEV,
                               dtype=torch.float32 if c["pool"] == "f32" else torch.bfloat16)
    else:
        pool = pk.KVPool(1, s["num_blocks"], c["block"], 1, 64, "fp8")
        if c["op"] == "grow":
            s["step"] = pk.StepTables.empty(c["seqs"], s["max_tokens"], device=DEV)
        s["lens_out"], s["free_out"] = torch.empty_like(s["lens"]), torch.empty_like(s["free"])
    s["pool"] = pool
    return s


# ----------------------------------------------------------------------- run
def run(state):
    return (RUN_OWN if own else RUN_PLAIN)[state["case"]["op"]](state)


def _own_prefix(s):
    return s["pk"].paged_prefix_decode_attention(s["q"], s["pool"], 0, s["tables"], s["lens"], s["max_len"],
                                                 s["offsets"], s["prefix"], s["scale"], out=s["out"],
                                                 workspace=s["workspace"])


def _own_rope(s):
    s["pk"].kv_append_norm_rope(s["pool"], 0, s["q"], s["k"], s["v"], s["pos"], s["slots"], s["rope"],
                                q_weight=s["q_weight"], k_weight=s["k_weight"], eps=s["eps"], out=s["out"])
    return s["out"], s["k_pool"], s["v_pool"]


def _own_grow(s):
    st = s["pk"].kv_tables_grow(s["pool"], s["tables"], s["lens"], s["new"], s["ring"], s["free"], s["max_tokens"],
                                out=s["step"])
    return (s["tables"], st.slot_mapping, st.positions, st.token_seqs, st.token_offsets, st.granted, st.seq_lens,
            st.free_state)


def _own_release(s):
    s["pk"].kv_tables_release(s["pool"], s["tables"], s["lens"], s["done"], s["ring"], s["free"],
                              keep_blocks=s["keep"], seq_lens_out=s["lens_out"], free_state_out=s["free_out"])
    return s["ring"], s["lens_out"], s["free_out"]


def _plain_prefix(s):
    """Every sequence on its own: gather its tokens through the table, softmax, weighted sum."""
    c, q = s["case"], s["q"]
    Hk, D, bs = c["kv_heads"], c["dim"], c["block"]
    out = torch.zeros(q.shape, dtype=torch.float32, device=DEV)
    for b, L in enumerate(s["host_lens"]):
        if L == 0:
            continue
        blocks = s["tables"][b, :_ceil(L, bs)].long()
        k, v = ((s[x][0][blocks].float() * s[x + "_scale"]).transpose(0, 1).reshape(Hk, -1, D)[:, :L]
                for x in ("k", "v"))
        z = (q[b].float().view(Hk, -1, D) @ k.transpose(1, 2)) * s["scale"]
        p = (z - z.amax(2, keepdim=True)).exp()
        out[b] = ((p @ v) / p.sum(2, keepdim=True)).view(-1, D)
    return out.to(q.dtype)


def _rotate(x, cos, sin, interleaved):
    """x [T, H, D] rotated in its first 2 * cos.shape[-1] columns."""
    n = cos.shape[-1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., 2 * n:]], -1)


def _axis_rows(s, c):
    """cos and sin [T, rotary / 2] of each token, every pair from its own axis' position."""
    axis = torch.repeat_interleave(torch.arange(c["axes"], device=DEV), torch.tensor(_sections(c), device=DEV),
                                   output_size=c["rotary"] // 2)
    at = s["pos"].long()[axis].T                           # [T, pairs]
    pair = torch.arange(c["rotary"] // 2, device=DEV)[None]
    return s["cos_sin"][at, pair], s["cos_sin"][at, pair + c["rotary"] // 2]


def _plain_rope(s):
    c = s["case"]
    cos, sin = _axis_rows(s, c)

    def norm_rotate(x, w):
        x = x.float()
        if w is not None:
            x = x * (1.0 / ((x * x).mean(-1, keepdim=True) + s["eps"]).sqrt()) * w.float()
        return _rotate(x, cos, sin, c["interleaved"])

    q = norm_rotate(s["q"], s["q_weight"])
    k = norm_rotate(s["k"], s["k_weight"])
    keep = s["slots"] >= 0
    slot = s["slots"][keep]
    for x, name in ((k, "k"), (s["v"].float(), "v")):
        if c["pool"] == "fp8":
            x = (x * _inverse(s[name + "_scale"])).clamp(-FP8_MAX, FP8_MAX)
        dst = s[name + "_pool"]
        if c["pool"] == "fp8":  # indexed stores of bytes
            dst[0].view(torch.uint8)[slot // c["block"], :, slot % c["block"]] = \
                x[keep].to(dst.dtype).view(torch.uint8)
        else:
            dst[0][slot // c["block"], :, slot % c["block"]] = x[keep].to(dst.dtype)
    return q.to(torch.float32 if c["pool"] == "f32" else torch.bfloat16), s["k_pool"], s["v_pool"]


def _plain_grow(s):
    """Requests are served in order while the free list lasts; a request that
    it cannot cover gets nothing, and its tokens no slot."""
    tables, bs, cap = s["tables"], s["bs"], s["ring"].numel()
    L, n = s["lens"].long(), s["new"].long()
    head, count = s["free"].long()[0], s["free"].long()[1]
    held = (L + bs - 1) // bs
    need = (L + n + bs - 1) // bs - held
    cum = need.cumsum(0)
    served = (need == 0) | (cum <= count)
    first = cum - need
    # new table entries
    col = torch.arange(tables.shape[1], device=DEV)[None]
    j = col - held[:, None]
    fresh = (j >= 0) & (j < need[:, None]) & served[:, None]
    at = ((head + first[:, None] + j) % cap).clamp(0, cap - 1)
    tables.copy_(torch.where(fresh, s["ring"][at], tables))
    # token rows
    ends = n.cumsum(0)
    row = torch.arange(s["max_tokens"], device=DEV)
    seq = torch.searchsorted(ends, row, right=True)
    pad = seq >= len(L)
    q = seq.clamp(max=len(L) - 1)
    pos = L[q] + row - (ends - n)[q]
    block = tables[q, (pos // bs).clamp(0, tables.shape[1] - 1)].long()
    slots = torch.where(pad | ~served[q], -1, block * bs + pos % bs)
    granted = torch.where(served, n, 0)
    taken = torch.where(served, need, 0).sum()
    return (tables, slots, torch.where(pad, 0, pos).int(), torch.where(pad, -1, seq).int(),
            torch.cat([torch.zeros_like(ends[:1]), ends]).int(), granted.int(), (L + granted).int(),
            torch.stack([(head + taken) % cap, count - taken]).int())


def _plain_release(s):
    """The blocks of finished sequences, but for the first keep[b], go behind the free ring's tail in order."""
    tables, bs, cap = s["tables"], s["bs"], s["ring"].numel()
    L, done = s["lens"].long(), s["done"] != 0
    held = (L + bs - 1) // bs
    keep = s["keep"].long()
    rel = torch.where(done, held - keep, 0)
    cum = rel.cumsum(0)
    col = torch.arange(tables.shape[1], device=DEV)[None]
    go = done[:, None] & (col >= keep[:, None]) & (col < held[:, None])
    at = (s["free"].long().sum() + (cum - rel)[:, None] + col - keep[:, None]) % cap
    s["ring"][at[go]] = tables[go]
    total = rel.sum().int()
    return s["ring"], torch.where(done, 0, s["lens"]), torch.stack([s["free"][0], s["free"][1] + total])


RUN_PLAIN = {"prefix": _plain_prefix, "rope": _plain_rope, "grow": _plain_grow, "release": _plain_release}
RUN_OWN = {"prefix": _own_prefix, "rope": _own_rope, "grow": _own_grow, "release": _own_release}


# ---------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] == "prefix":
        own_mean = (c["own_lo"] + c["own_hi"]) / 2
        pre_mean = (c["prefix_lo"] + c["prefix_hi"]) / 2
        tokens = c["groups"] * pre_mean + c["seqs"] * own_mean     # each read once
        row = c["q_heads"] * c["dim"]
        return {"bytes": int(2 * tokens * c["kv_heads"] * c["dim"] * ELEM[c["pool"]]
                             + 2 * c["seqs"] * row * (4 if c["pool"] == "f32" else 2)),
                "flops": int(4 * row * c["seqs"] * (pre_mean + own_mean))}
    if c["op"] == "rope":
        T, rows = c["tokens"], c["q_heads"] + 2 * c["kv_heads"]
        out_q = 4 if c["pool"] == "f32" else 2
        per = c["dim"] * (rows * ELEM[c["inp"]] + c["q_heads"] * out_q + 2 * c["kv_heads"] * ELEM[c["pool"]])
        table = min(c["max_pos"], T * c["axes"]) * c["rotary"] * 4
        return {"bytes": int(T * (per + 4 * c["axes"] + 8) + table),
                "flops": int(T * (c["q_heads"] + c["kv_heads"]) * (4 * c["dim"] + 3 * c["rotary"]))}
    # a log-normal length with median len_hi / 8, sigma 1
    blocks = c["seqs"] * (c["len_hi"] / 8 * math.exp(0.5) / c["block"] + 0.5)
    if c["op"] == "release":
        return {"bytes": int(c["seqs"] * 16 + c["finished"] * blocks * 8 + 16), "flops": 0}
    tokens = c["seqs"] + c["prompts"] * c["chunk"] / 2
    return {"bytes": int(c["seqs"] * 24 + tokens * 16 + tokens / c["block"] * 8 + 16), "flops": 0}


# --------------------------------------------------------------------- exact
def exact(case, seed):
    return {"prefix": _exact_prefix, "rope": _exact_rope, "grow": _exact_grow,
            "release": _exact_release}[case["op"]](case, INPUTS[case["op"]](case, seed))


def _exact_prefix(c, s):
    """One KV head and sequence at a time over slots, in 64 bits."""
    bs, group = c["block"], c["q_heads"] // c["kv_heads"]
    out = torch.zeros((c["seqs"], c["q_heads"], c["dim"]), dtype=torch.float64, device=DEV)
    for h in range(c["kv_heads"]):
        keys, values = (s[x][0, :, h].reshape(-1, c["dim"]).double() for x in ("k", "v"))
        for b in range(c["seqs"]):
            t = torch.arange(s["host_lens"][b], device=DEV)
            if not len(t):
                continue
            slot = s["tables"][b].long()[t // bs] * bs + t % bs
            kk, vv = keys[slot], values[slot]
            for g in range(group):
                w = torch.mv(kk, s["q"][b, h * group + g].double()) * (s["scale"] * s["k_scale"])
                w = (w - torch.logsumexp(w, 0)).exp()
                out[b, h * group + g] = torch.mv(vv.T, w) * s["v_scale"]
    return out


def _exact_rope(c, s):
    T, half = c["tokens"], c["rotary"] // 2
    bounds = np.cumsum(_sections(c))
    axis = np.searchsorted(bounds, np.arange(half), side="right")
    phase = torch.empty((T, half), dtype=torch.complex128, device=DEV)
    for j in range(half):
        row = s["cos_sin"][s["pos"][int(axis[j])].long()].double()
        phase[:, j] = torch.complex(row[:, j], row[:, j + half])

    def turn(x, w):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt(x.square().sum(-1, keepdim=True) / c["dim"] + s["eps"]) * w.double()
        y = x.clone()
        lo = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["interleaved"] else \
            (slice(0, half), slice(half, 2 * half))
        z = torch.complex(x[..., lo[0]], x[..., lo[1]]) * phase[:, None]
        y[..., lo[0]], y[..., lo[1]] = z.real, z.imag
        return y

    pools = []
    keep = s["slots"] >= 0
    slot = s["slots"][keep]
    for x, sc in ((turn(s["k"], s["k_weight"]), s["k_scale"]), (s["v"].double(), s["v_scale"])):
        if c["pool"] == "fp8":
            x = (x / sc).clamp(-FP8_MAX, FP8_MAX)
        flat = torch.zeros((s["num_blocks"] * c["block"], c["kv_heads"], c["dim"]), dtype=torch.float64, device=DEV)
        flat[slot] = x[keep]
        pools.append(flat.view(1, s["num_blocks"], c["block"], c["kv_heads"], c["dim"]).transpose(2, 3).contiguous())
    return turn(s["q"], s["q_weight"]), pools[0], pools[1]


def _exact_grow(c, s):
    """The same by a walk over the requests on the host."""
    bs = c["block"]
    tables, ring = s["tables"].cpu().numpy().copy(), s["ring"].cpu().numpy()
    lens, new = s["lens"].tolist(), s["new"].tolist()
    head, count = s["free"].tolist()
    slots = np.full(s["max_tokens"], -1, np.int64)
    pos = np.zeros(s["max_tokens"], np.int32)
    seqs = np.full(s["max_tokens"], -1, np.int32)
    offsets, granted, blocked, row = [0], [], False, 0
    for b, (L, n) in enumerate(zip(lens, new)):
        need = _ceil(L + n, bs) - _ceil(L, bs)
        blocked = blocked or need > count
        ok = need == 0 or not blocked
        if ok:
            for j in range(need):
                tables[b, _ceil(L, bs) + j] = ring[head]
                head, count = (head + 1) % len(ring), count - 1
        p = np.arange(L, L + n)
        pos[row:row + n], seqs[row:row + n] = p, b
        if ok and n:
            slots[row:row + n] = tables[b, p // bs].astype(np.int64) * bs + p % bs
        row += n
        offsets.append(row)
        granted.append(n if ok else 0)
    back = lambda x, dt=torch.int32: torch.tensor(np.asarray(x), dtype=dt, device=DEV)
    return (back(tables), back(slots, torch.int64), back(pos), back(seqs), back(offsets), back(granted),
            back(np.array(lens) + np.array(granted)), back([head, count]))


def _exact_release(c, s):
    bs = c["block"]
    tables, ring = s["tables"].cpu().numpy(), s["ring"].cpu().numpy().copy()
    lens, done, keep = s["lens"].tolist(), s["done"].tolist(), s["keep"].tolist()
    head, count = s["free"].tolist()
    for b, L in enumerate(lens):
        if done[b]:
            mine = tables[b, keep[b]:_ceil(L, bs)]
            ring[(head + count + np.arange(len(mine))) % len(ring)] = mine
            count += len(mine)
            lens[b] = 0
    back = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)
    return back(ring), back(lens), back([head, count])
