"""GPU tests of the step's other operators: norm + rotation + append, tables
and slots on the device, and a run of all of them as a decode loop uses them."""
import numpy as np
import pytest
import torch

import step_reference as ref
from paged_kv_cache_194_gb300 import binding as pk
from paged_kv_cache_194_gb300.block_manager import BlockManager

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
I32 = torch.int32


def dev(x, dtype=I32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


# ------------------------------------------------------- norm, rotation, append
def _rope_case(T, Hq, Hk, D, rotary, sections, interleaved, normed, kv, inp, bs=16, max_pos=300, seed=0, fused=True,
               weight="f32", wide=1.0):
    g = torch.Generator().manual_seed(seed)
    dt = DT[inp]
    if fused:  # rows of one projection
        qkv = (torch.randn(T, (Hq + 2 * Hk) * D, generator=g) * wide).to(dt).cuda()
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([Hq * D, Hk * D, Hk * D], 1))
    else:
        q, k, v = ((torch.randn(T, h, D, generator=g) * wide).to(dt).cuda() for h in (Hq, Hk, Hk))
    nb = -(-T // bs) + 2
    slots = torch.randperm(nb * bs, generator=g)[:T]
    slots[torch.rand(T, generator=g) < 0.1] = -1
    pos = torch.randint(0, max_pos, (len(sections), T), generator=g).to(I32)
    rope = pk.RopeTable.create(max_pos, rotary, sections=sections, interleaved=interleaved)
    w = [(1 + 0.2 * torch.randn(D, generator=g)).to(DT[weight]).cuda() for _ in range(2)] if normed else [None, None]
    ks, vs = (0.031, 0.027) if kv == "fp8" else (1.0, 1.0)
    pool = pk.KVPool(2, nb, bs, Hk, D, kv, ks, vs, fill=0x35)
    return dict(q=q, k=k, v=v, slots=slots, pos=pos, rope=rope, w=w, pool=pool, sections=sections)


def _rope_call(c, out=None, **kw):
    return pk.kv_append_norm_rope(c["pool"], 1, c["q"], c["k"], c["v"], c["pos"].cuda(), c["slots"].cuda(), c["rope"],
                                  q_weight=c["w"][0], k_weight=c["w"][1], eps=1e-5, out=out, **kw)


def _rope_check(c, out):
    pool, rope = c["pool"], c["rope"]
    args = (1e-5, rope.cos_sin.cpu(), c["pos"], c["sections"], rope.interleaved)
    cpu = lambda x: None if x is None else x.cpu()
    zq, size = ref.norm_rope(c["q"].cpu(), cpu(c["w"][0]), *args)
    # fp32: 128 squares, a reciprocal root, two products and a two-term sum are
    # below 32 roundings of 2^-24 of the magnitudes; then the stored type's one
    fp32 = 2.0 ** -19
    err = (out.cpu().double() - zq).abs()
    assert (err <= ref.HALF[out.dtype] * (zq.abs() + fp32 * size) + fp32 * size).all(), float(err.max())
    zk, ksize = ref.norm_rope(c["k"].cpu(), cpu(c["w"][1]), *args)
    keep = c["slots"] >= 0
    blk, off = c["slots"][keep] // pool.block_size, c["slots"][keep] % pool.block_size
    raw = pool.k[1].cpu()
    if pool.kv_dtype == "fp8":
        got = raw[blk, :, off].view(torch.float8_e4m3fn).double()
        want, slack = (zk[keep] / pool.k_scale), fp32 * ksize[keep] / pool.k_scale
        lim = want.clamp(-448, 448)
        # E4M3: half a step is 2^-4 of the value, 2^-10 below the smallest normal
        assert ((got - lim).abs() <= 2.0 ** -4 * (lim.abs() + slack) + 2.0 ** -10 + slack).all()
    else:
        got = raw[blk, :, off].double()
        half = ref.HALF[raw.dtype]
        assert ((got - zk[keep]).abs() <= half * (zk[keep].abs() + fp32 * ksize[keep]) + fp32 * ksize[keep]).all()
    # V, and every slot that no token names, are exactly what kv_append leaves
    other = pk.KVPool(2, pool.num_blocks, pool.block_size, pool.num_kv_heads, pool.head_dim, pool.kv_dtype,
                      pool.k_scale, pool.v_scale, fill=0x35)
    pk.kv_append(other, 1, c["k"].contiguous(), c["v"].contiguous(), c["slots"].cuda())
    assert torch.equal(other.v.view(torch.uint8), pool.v.view(torch.uint8))
    unused = torch.ones(pool.num_blocks * pool.block_size, dtype=torch.bool)
    unused[c["slots"][keep]] = False
    u = unused.nonzero()[:, 0]
    assert (raw[u // pool.block_size, :, u % pool.block_size].contiguous().view(torch.uint8) == 0x35).all()
    assert (pool.k[0].view(torch.uint8) == 0x35).all()


ROPE = [  # T, Hq, Hk, D, rotary, sections, interleaved, normed
    (1, 32, 8, 128, 128, (64,), False, True),
    (3, 2, 1, 64, 32, (16,), False, True),
    (64, 32, 8, 128, 128, (64,), False, False),
    (33, 5, 1, 128, 112, (56,), False, True),
    (33, 5, 1, 128, 112, (56,), True, True),
    (17, 8, 8, 64, 64, (32,), True, True),
    (20, 16, 2, 128, 128, (16, 24, 24), False, True),      # whole vectors of pairs
    (20, 16, 2, 128, 128, (22, 21, 21), False, True),      # axes that change inside one
    (20, 12, 4, 128, 96, (20, 28), True, True),
    (21, 12, 4, 64, 48, (7, 0, 17), True, False),
    (2, 1, 1, 64, 16, (8,), False, True),
    (700, 4, 4, 64, 64, (32,), False, True),
    (2500, 32, 8, 128, 64, (8, 12, 12), True, True),
]


@pytest.mark.parametrize("case", ROPE, ids=str)
@pytest.mark.parametrize("kv,inp", [("bf16", "bf16"), ("fp8", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("fp8", "f32")])
def test_norm_rope_append(case, kv, inp):
    c = _rope_case(*case, kv, inp, bs=(16, 32, 64)[case[0] % 3], seed=case[0], fused=case[0] % 2 == 0,
                   weight=("f32", "bf16")[case[0] % 2])
    _rope_check(c, _rope_call(c))
    assert c["pool"].errors() == 0


def test_norm_rope_no_norm_equals_plain_append_where_nothing_turns():
    """Positions 0: rotation by nothing, no norm: K is kv_append's, bit for bit, and q is q."""
    for kv, inp in (("bf16", "bf16"), ("fp8", "bf16"), ("f32", "f32")):
        c = _rope_case(50, 8, 2, 128, 128, (64,), False, False, kv, inp, seed=3)
        c["pos"].zero_()
        out = _rope_call(c)
        other = pk.KVPool(2, c["pool"].num_blocks, 16, 2, 128, kv, c["pool"].k_scale, c["pool"].v_scale, fill=0x35)
        pk.kv_append(other, 1, c["k"].contiguous(), c["v"].contiguous(), c["slots"].cuda())
        assert torch.equal(other.k.view(torch.uint8), c["pool"].k.view(torch.uint8))
        assert torch.equal(out.float(), c["q"].float())


def test_norm_rope_in_place_and_on_a_stream():
    c = _rope_case(40, 8, 2, 128, 128, (64,), False, True, "bf16", "bf16", seed=4, fused=False)
    want = _rope_call(c)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c["q"] = c["q"].clone()
    got = _rope_call(c, out=c["q"], stream=side)
    side.synchronize()
    assert got.data_ptr() == c["q"].data_ptr() and torch.equal(got, want)


def test_norm_rope_wide_values_and_zero_rows():
    c = _rope_case(30, 4, 2, 128, 128, (64,), False, True, "bf16", "f32", seed=5, wide=1e4)
    c["q"][3] = 0
    c["k"][4] = 0
    out = _rope_call(c)
    assert (out[3] == 0).all()
    _rope_check(c, out)


def test_norm_rope_flags_bad_positions_and_slots():
    c = _rope_case(24, 8, 2, 128, 128, (32, 32), False, True, "bf16", "bf16", seed=6)
    slots = c["slots"].clone()
    slots[slots < 0] = c["pool"].num_blocks * 16 - 1  # (only one token left out below)
    c["slots"] = slots.unique()[torch.randperm(len(slots.unique()), generator=torch.Generator().manual_seed(1))]
    T = len(c["slots"])
    for n in ("q", "k", "v"):
        c[n] = c[n][:T]
    c["pos"] = c["pos"][:, :T].contiguous()
    c["pos"][1, 2], c["pos"][0, 5], c["pos"][0, 7] = 300, -1, 2 ** 31 - 1
    good = c["slots"].clone()
    c["slots"][9] = c["pool"].num_blocks * 16
    c["slots"][10] = -2
    out = _rope_call(c)
    assert c["pool"].errors() == pk.ERRBIT_POSITION | pk.ERRBIT_SLOT
    assert (out[[2, 5, 7]] == 0).all() and (out[[9, 10]] != 0).any()
    left = [2, 5, 7, 9, 10]
    raw = c["pool"].k[1].view(torch.uint8).cpu()
    assert (raw[good[left] // 16, :, good[left] % 16] == 0x35).all()
    c["slots"][left] = -1
    c["pos"].clamp_(0, 299)
    want = out.clone()
    want[[2, 5, 7]] = _rope_call(c)[[2, 5, 7]]
    _rope_check(c, want)


def test_norm_rope_long_batch_past_32_bits():
    """Rows whose element offsets pass 2^31 (a broadcast row apart from the last ones)."""
    T, Hq, Hk, D = 350_000, 32, 8, 128  # 350000 x 6144 elements
    row = torch.zeros(T, (Hq + 2 * Hk) * D, dtype=torch.bfloat16, device="cuda")
    row[-3:] = torch.randn(3, (Hq + 2 * Hk) * D, generator=torch.Generator().manual_seed(7)).to(torch.bfloat16).cuda()
    q, k, v = (x.unflatten(1, (-1, D)) for x in row.split([Hq * D, Hk * D, Hk * D], 1))
    pool = pk.KVPool(1, 1, 16, Hk, D, "bf16", fill=0)
    slots = torch.full((T,), -1, dtype=torch.int64)
    slots[-3:] = torch.tensor([5, 0, 15])
    pos = torch.zeros(T, dtype=I32)
    pos[-3:] = torch.tensor([1, 2, 3], dtype=I32)
    rope = pk.RopeTable.create(8, 128)
    out = pk.kv_append_norm_rope(pool, 0, q, k, v, pos.cuda(), slots.cuda(), rope)
    small = pk.KVPool(1, 1, 16, Hk, D, "bf16", fill=0)
    want = pk.kv_append_norm_rope(small, 0, q[-3:], k[-3:], v[-3:], pos[-3:].cuda(), slots[-3:].cuda(), rope)
    assert torch.equal(out[-3:], want) and (out[:-3] == 0).all()
    assert torch.equal(pool.k, small.k) and torch.equal(pool.v, small.v)


# ------------------------------------------------------------ tables and slots
def _pool(num_blocks, bs):
    return pk.KVPool(1, num_blocks, bs, 1, 64, "fp8")


def _grow_inputs(B, bs, len_hi, new_hi, share, seed, width=None, slack=0, every=1):
    """Random lengths and tables; the ring holds `share` of the blocks asked
    for.  every: only each so manieth request has more than one new token."""
    r = np.random.default_rng(seed)
    lens = r.integers(0, len_hi + 1, B)
    new = r.integers(0, new_hi + 1, B)
    new = np.where(np.arange(B) % every == every - 1, new, np.minimum(new, 1))
    held, need = -(-lens // bs), -(-(lens + new) // bs) - -(-lens // bs)
    width = width or int(max(1, (held + need).max(initial=1)))
    total = int(held.sum() + need.sum()) + 5
    order = r.permutation(total)
    tables = np.full((B, width), -1)
    at = 0
    for b in range(B):
        n = min(held[b], width)
        tables[b, :n] = order[at:at + n]
        at += held[b]
    count = int(share * need.sum())
    ring = np.full(count + slack + 1, -1)
    head = int(r.integers(0, len(ring)))
    ring[(head + np.arange(count)) % len(ring)] = order[at:at + count]
    return total, tables, lens, new, ring, [head, count]


def _check_grow(B, bs, len_hi, new_hi, share, seed, extra_rows=3, in_place=False, errors=0, **kw):
    total, tables, lens, new, ring, state = _grow_inputs(B, bs, len_hi, new_hi, share, seed, **kw)
    T = int(new.sum()) + extra_rows
    want_tables = tables.tolist()
    want = ref.grow(want_tables, lens.tolist(), new.tolist(), ring.tolist(), state, bs, T)
    pool = _pool(total, bs)
    t, L, n, rg, st = dev(tables).reshape(tables.shape), dev(lens), dev(new), dev(ring), dev(state)
    out = None
    if in_place:
        out = pk.StepTables.empty(B, T)._replace(seq_lens=L, free_state=st)
    got = pk.kv_tables_grow(pool, t, L, n, rg, st, T, out=out)
    assert t.tolist() == want_tables
    for name, x, y in zip(got._fields, got, want):
        assert x.tolist() == y, name
    assert pool.errors() == errors
    assert rg.tolist() == ring.tolist()
    if not in_place:
        assert L.tolist() == lens.tolist() and st.tolist() == state
    return got


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("B,len_hi,new_hi", [(1, 0, 1), (1, 100, 1), (7, 40, 1), (64, 300, 1), (256, 200, 1), (257, 64, 3),
                                             (1024, 100, 1), (1025, 90, 2), (2500, 60, 4), (40, 500, 150), (5, 0, 3000)])
@pytest.mark.parametrize("share", [1.0, 0.6, 0.0])
def test_grow_matches_a_walk(B, len_hi, new_hi, share, bs):
    _check_grow(B, bs, len_hi, new_hi, share, seed=B + bs)


def test_grow_long_slot_maps():
    """More token rows than the scanning CTA fills itself."""
    _check_grow(100, 16, 500, 400, 0.9, seed=1)
    _check_grow(3, 64, 10, 30000, 1.0, seed=2, extra_rows=1000)
    _check_grow(1500, 16, 50, 40, 0.5, seed=3, in_place=True)


@pytest.mark.parametrize("B,every,new_hi,len_hi", [(1024, 97, 600, 100), (1024, 1024, 3000, 16), (2200, 31, 200, 300),
                                                   (700, 350, 2500, 0), (256, 5, 40, 64)])
@pytest.mark.parametrize("share", [1.0, 0.5])
def test_grow_few_long_requests_among_short_ones(B, every, new_hi, len_hi, share):
    _check_grow(B, 16, len_hi, new_hi, share, seed=B, every=every)
    _check_grow(B, 64, len_hi, new_hi, share, seed=B + 1, every=every, in_place=True)


@pytest.mark.parametrize("big", [2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30])
def test_grow_sums_past_32_bits(big):
    """New tokens whose sum passes 2^31: those requests wait, ones before them do not."""
    pool = _pool(64, 16)
    B = 1100
    lens, new = [5] * B, [0] * B
    new[0], new[7], new[1050] = 20, 1, 1
    for b in (40, 41, 42, 1060, 1099):
        new[b] = big
    ring, T = list(range(10)), 30
    tables = [[20 + b % 40, -1, -1] for b in range(B)]
    # (the walk goes row by row: 40 tokens pass max_tokens as well)
    want = ref.grow([list(x) for x in tables], lens, [min(n, 40) for n in new], ring, [3, 5], 16, T)
    t = dev(tables)
    got = pk.kv_tables_grow(pool, t, dev(lens), dev(new), dev(ring), dev([3, 5]), T)
    for name, x, y in zip(got._fields, got, want):
        assert x.tolist() == y, name
    assert got.granted.tolist()[:8] == [20, 0, 0, 0, 0, 0, 0, 1] and sum(got.granted.tolist()) == 21
    assert t[0].tolist() == [20, 3, -1] and pool.errors() == pk.ERRBIT_STEP


@pytest.mark.parametrize("B,new_hi", [(200, 1), (1100, 2), (30, 100)])
def test_grow_in_place(B, new_hi):
    _check_grow(B, 16, 100, new_hi, 0.8, seed=B, in_place=True)


def test_grow_without_rows_or_requests():
    _check_grow(9, 16, 100, 0, 1.0, seed=1, extra_rows=0)
    pool = _pool(4, 16)
    e = torch.empty(0, dtype=I32, device="cuda")
    got = pk.kv_tables_grow(pool, torch.empty(0, 3, dtype=I32, device="cuda"), e, e, dev([3, 2]), dev([1, 1]), 5)
    assert got.slot_mapping.tolist() == [-1] * 5 and got.token_offsets.tolist() == [0] and got.free_state.tolist() == [1, 1]


def test_grow_full_table_rows_wait():
    """A request past its table row waits and takes no block; the others go
    on.  Lengths go up to 70, past the row's 64 positions: those are flagged."""
    _check_grow(60, 16, 70, 20, 1.0, seed=5, width=4, errors=pk.ERRBIT_SEQ_LEN)


def test_grow_flags_what_cannot_be():
    pool = _pool(32, 16)
    t = torch.full((5, 4), -1, dtype=I32)
    t[0, 0], t[2, :2], t[4, 0] = 7, torch.tensor([8, 9], dtype=I32), 99
    lens, new = [10, -3, 20, 65, 5], [2, 1, -1, 1, 1]
    ring = [20, 21, 22, 23]
    got = pk.kv_tables_grow(pool, t.cuda(), dev(lens), dev(new), dev(ring), dev([0, 4]), 6)
    assert pool.errors() == pk.ERRBIT_SEQ_LEN | pk.ERRBIT_STEP | pk.ERRBIT_BLOCK_ID
    assert got.granted.tolist() == [2, 0, 0, 0, 1]
    assert got.seq_lens.tolist() == [12, -3, 20, 65, 6]
    assert got.slot_mapping.tolist() == [7 * 16 + 10, 7 * 16 + 11, -1, -1, -1, -1]  # (the last: block 99)
    assert got.token_offsets.tolist() == [0, 2, 3, 3, 4, 5]
    pool.clear_errors()
    # a bad ring entry: no slot, and -1 in the table
    t = torch.full((2, 4), -1, dtype=I32).cuda()
    got = pk.kv_tables_grow(pool, t, dev([0, 0]), dev([1, 1]), dev([32, 5]), dev([0, 2]), 2)
    assert pool.errors() == pk.ERRBIT_BLOCK_ID and got.slot_mapping.tolist() == [-1, 80] and t[:, 0].tolist() == [-1, 5]
    pool.clear_errors()
    for state in ([4, 1], [-1, 1], [0, 5], [0, -1]):  # no such ring state: nothing free
        got = pk.kv_tables_grow(pool, t, dev([0, 16]), dev([1, 0]), dev(ring), dev(state), 2)
        assert got.granted.tolist() == [0, 0] and got.free_state.tolist() == state
        assert pool.errors() == pk.ERRBIT_STEP
        pool.clear_errors()


@pytest.mark.parametrize("max_tokens", [0, 1, 5, 9000])
def test_grow_rows_past_the_limit_wait(max_tokens):
    pool = _pool(4000, 16)
    B = 8
    new = [1, 2, 3, 4000, 5000, 1, 0, 2] if max_tokens == 9000 else [1, 2, 3, 1, 1, 1, 0, 2]
    lens = [16 * i for i in range(B)]
    width = 400
    tables = [[-1] * width for _ in range(B)]
    for b in range(B):
        tables[b][:b] = [100 + 10 * b + i for i in range(b)]
    t = dev(tables)
    ring = list(range(1000, 2000))
    want = ref.grow(tables, lens, new, ring, [0, 1000], 16, max_tokens)
    got = pk.kv_tables_grow(pool, t, dev(lens), dev(new), dev(ring), dev([0, 1000]), max_tokens)
    for name, x, y in zip(got._fields, got, want):
        assert x.tolist() == y, name
    assert t.tolist() == tables
    assert pool.errors() == pk.ERRBIT_STEP


@pytest.mark.parametrize("B,width,finished", [(1, 3, 1.0), (50, 20, 0.3), (1024, 9, 0.5), (1500, 7, 0.9),
                                              (3000, 120, 0.5), (5000, 60, 1.0), (2, 200000, 1.0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_release_matches_a_walk(B, width, finished, in_place):
    """One CTA, and (from a quarter million table entries on) the grid form."""
    r = np.random.default_rng(B)
    bs = 16
    lens = r.integers(0, width * bs + 1, B)
    held = -(-lens // bs)
    total = int(held.sum()) + 10
    order = r.permutation(total)
    tables = np.full((B, width), -1)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    head, count = int(r.integers(0, total)), total - at
    ring = np.full(total, -1)
    ring[(head + np.arange(count)) % total] = order[at:]
    done = (r.random(B) < finished).astype(int)
    keep = r.integers(-1, 4, B)
    pool = _pool(total, bs)
    for kept in (keep, None):
        want_ring = ring.tolist()
        want_lens, want_state = ref.release(tables.tolist(), lens.tolist(), done.tolist(),
                                            kept.tolist() if kept is not None else [0] * B, want_ring, [head, count], bs)
        L, st, rg, t = dev(lens), dev([head, count]), dev(ring), dev(tables)
        a, f = pk.kv_tables_release(pool, t, L, dev(done), rg, st, keep_blocks=dev(kept) if kept is not None else None,
                                    **(dict(seq_lens_out=L, free_state_out=st) if in_place else {}))
        assert rg.tolist() == want_ring and a.tolist() == want_lens and f.tolist() == want_state
        assert torch.equal(t, dev(tables))
        assert pool.errors() == 0


@pytest.mark.parametrize("B", [3, 3000])
def test_release_refuses_an_overfull_ring(B):
    pool = _pool(B * 100, 16)
    t = torch.arange(B * 100, dtype=I32).view(B, 100).cuda()
    lens, done = dev([1600] * B), dev([1] * B)
    for state, size in (([0, 1], B * 100), ([5, 0], 5), ([0, -1], B * 200)):
        ring = torch.full((size,), -7, dtype=I32, device="cuda")
        a, f = pk.kv_tables_release(pool, t, lens, done, ring, dev(state))
        assert a.tolist() == [1600] * B and f.tolist() == state and (ring == -7).all()
        assert pool.errors() == pk.ERRBIT_STEP
        pool.clear_errors()
    # a bad length is left alone and flagged, the others go
    lens = dev([1601] + [16] * (B - 1))
    ring = torch.full((B * 100,), -7, dtype=I32, device="cuda")
    a, f = pk.kv_tables_release(pool, t, lens, done, ring, dev([0, 0]))
    assert a.tolist() == [1601] + [0] * (B - 1) and f.tolist() == [0, B - 1]
    assert ring[:B - 1].tolist() == t[1:, 0].tolist() and pool.errors() == pk.ERRBIT_SEQ_LEN


def test_grow_and_release_follow_the_block_manager():
    """A decode loop of grow and release hands out the host block manager's
    blocks and slots, pauses included, step by step."""
    r = np.random.default_rng(11)
    B, bs, nb, width = 24, 16, 40, 6
    order = r.permutation(nb)
    bm = BlockManager(nb, bs, width, free_order=order.tolist())
    pool = _pool(nb, bs)
    t, L = torch.full((B, width), -1, dtype=I32, device="cuda"), dev([0] * B)
    ring, st = dev(order), dev([0, nb])
    for s in range(B):
        bm.add(s)
    for step in range(120):
        want = bm.decode_slots(range(B))
        got = pk.kv_tables_grow(pool, t, L, dev([1] * B), ring, st, B,
                                out=pk.StepTables.empty(B, B)._replace(seq_lens=L, free_state=st))
        assert got.slot_mapping.tolist() == list(want), step
        assert L.tolist() == [bm.seq_len(s) for s in range(B)]
        if step % 7 == 6:
            done = r.random(B) < 0.3
            for s in np.flatnonzero(done):
                bm.free_sequence(int(s))
                bm.add(int(s))
            pk.kv_tables_release(pool, t, L, dev(done.astype(int)), ring, st, seq_lens_out=L, free_state_out=st)
        assert int(st[1]) == bm.num_free
        # the free lists agree entry by entry
        h, c = st.tolist()
        assert [int(ring[(h + i) % nb]) for i in range(c)] == list(bm.free)
    assert pool.errors() == 0


# ---------------------------------------------------------- the step as a whole
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("captured", [False, True])
def test_decode_loop_of_the_step_operators(captured, kv):
    """A group of requests forks from one cached prompt; every step grows the
    tables, norms, rotates and appends the new token, and attends with the
    prompt read once; one request finishes half way.  Every step's output is
    compared with 64-bit attention over the tokens appended so far.  captured:
    one step is captured and replayed."""
    B, Hq, Hk, D, bs, prompt, steps = 6, 8, 2, 128, 16, 208, 24
    g = torch.Generator().manual_seed(1)
    width, nb = 20, 80
    shared = prompt // bs
    scale = ref.scale_for(D)
    pool = pk.KVPool(1, nb, bs, Hk, D, kv, *((0.02, 0.02) if kv == "fp8" else (1.0, 1.0)), fill=0xFF)
    rope = pk.RopeTable.create(1024, D)
    w = (1 + 0.1 * torch.randn(D, generator=g)).cuda()
    ring, st = dev(list(range(shared, nb))), dev([0, nb - shared])
    tables = torch.full((B, width), -1, dtype=I32, device="cuda")
    tables[:, :shared] = torch.arange(shared, dtype=I32)  # the prompt's blocks, in every table
    L = dev([prompt] * B)
    # the prompt: its rows go through the same norm, rotation and append
    qkv = torch.randn(prompt, (Hq + 2 * Hk) * D, generator=g).to(torch.bfloat16).cuda()
    cut = lambda x: [y.unflatten(1, (-1, D)) for y in x.split([Hq * D, Hk * D, Hk * D], 1)]
    pk.kv_append_norm_rope(pool, 0, *cut(qkv), torch.arange(prompt, dtype=I32).cuda(),
                           torch.arange(prompt).cuda(), rope, w, w)
    offsets, prefix, new = dev([0, B]), dev([prompt]), dev([1] * B)
    out_tables = pk.StepTables.empty(B, B)._replace(seq_lens=L, free_state=st)
    rows = torch.empty(B, (Hq + 2 * Hk) * D, dtype=torch.bfloat16, device="cuda")
    q_rot = torch.empty(B, Hq, D, dtype=torch.bfloat16, device="cuda")
    attn = torch.empty_like(q_rot)
    ws = pk.prefix_decode_workspace(pool, B, 1, Hq, width * bs)

    def step():
        s = pk.kv_tables_grow(pool, tables, L, new, ring, st, B, out=out_tables)
        pk.kv_append_norm_rope(pool, 0, *cut(rows), s.positions, s.slot_mapping, rope, w, w, out=q_rot)
        pk.paged_prefix_decode_attention(q_rot, pool, 0, tables, L, width * bs, offsets, prefix, scale, out=attn,
                                         workspace=ws)

    graph = None
    for i in range(steps):
        rows.copy_(torch.randn(rows.shape, generator=g).to(torch.bfloat16))
        if captured and i == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        if graph is not None:
            graph.replay()
        else:
            step()
        lens = L.tolist()
        want_lens = [prompt + i + 1 if i < 12 or b != 2 else i - 11 for b in range(B)]
        assert lens == want_lens and pool.errors() == 0
        raw = (lambda x: x.view(torch.float8_e4m3fn)) if kv == "fp8" else (lambda x: x)
        want, mass, floor = ref.attention(q_rot.cpu(), raw(pool.k[0].cpu()), raw(pool.v[0].cpu()), tables.cpu(), lens, scale,
                                   pool.k_scale, pool.v_scale)
        bound = ref.attention_bound(want, mass, kv, floor)
        ok = (attn.cpu().double() - want).abs() <= bound
        assert bool(ok.all()), i
        if i == 11:  # request 2 finishes (its prompt's blocks stay) and a new one starts from nothing
            pk.kv_tables_release(pool, tables, L, dev([0, 0, 1, 0, 0, 0]), ring, st, keep_blocks=dev([shared] * B),
                                 seq_lens_out=L, free_state_out=st)
            tables[2] = -1
