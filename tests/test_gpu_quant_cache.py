"""GPU tests of the quantised cache: rows as they are written (bit for bit),
as they are read back, and decode attention over them."""
import itertools

import numpy as np
import pytest
import torch

import quant_reference as ref
from paged_kv_cache_194_gb300 import binding as pk

pytestmark = pytest.mark.gpu

I32, BF = torch.int32, torch.bfloat16
DT = {"f32": torch.float32, "bf16": BF}


def dev(x, dtype=I32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


def raw(pool):
    return [x.cpu().view(torch.uint8) for x in (pool.k_codes, pool.k_params, pool.v_codes, pool.v_params)]


def tables_of(lens, bs, g, spare=3):
    held = [-(-max(0, n) // bs) for n in lens]
    nb = sum(held) + spare
    order = torch.randperm(nb, generator=g).to(I32)
    t = torch.full((len(lens), max(held + [1]) + 1), -1, dtype=I32)
    at = 0
    for b, n in enumerate(held):
        t[b, :n] = order[at:at + n]
        at += n
    return t, nb


# ---------------------------------------------------------------------- append
def expect_append(want, layer, k, v, slots, bs, bits):
    """What an append leaves in a pool's tensors (as raw() gives them)."""
    for i, x in ((0, k), (2, v)):
        n, p = ref.quantise(x.cpu(), bits)
        c, p = ref.pack(n, bits), p.contiguous().view(torch.uint8)
        for t, s in enumerate(slots.tolist()):
            if s >= 0:
                want[i][layer, s // bs, :, s % bs] = c[t]
                want[i + 1][layer, s // bs, :, s % bs] = p[t]
    return want


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("T,Hk,D,bs", [(1, 1, 64, 16), (1, 8, 128, 16), (7, 3, 128, 32), (33, 2, 64, 64), (65, 5, 64, 16),
                                       (300, 8, 128, 64), (1001, 1, 128, 32)])
def test_append_bit_for_bit(bits, inp, T, Hk, D, bs):
    g = torch.Generator().manual_seed(T + D)
    nb = -(-T // bs) + 2
    slots = torch.randperm(nb * bs, generator=g)[:T]
    slots[torch.rand(T, generator=g) < 0.1] = -1
    rows = (torch.randn(T, 3 * Hk * D, generator=g) * 3).to(DT[inp])  # slices of a projection's rows
    k, v = rows[:, Hk * D:2 * Hk * D].unflatten(1, (Hk, D)), rows[:, 2 * Hk * D:].unflatten(1, (Hk, D))
    d = rows.cuda()
    pool = pk.QuantKVPool(2, nb, bs, Hk, D, bits, fill=0x35)
    want = expect_append(raw(pool), 1, k, v, slots, bs, bits)
    pk.kv_quant_append(pool, 1, d[:, Hk * D:2 * Hk * D].unflatten(1, (Hk, D)), d[:, 2 * Hk * D:].unflatten(1, (Hk, D)),
                       slots.cuda())
    for name, x, y in zip(("k_codes", "k_params", "v_codes", "v_params"), raw(pool), want):
        assert torch.equal(x, y), name
    assert pool.errors() == 0


def special_rows(D, dt):
    g = torch.Generator().manual_seed(3)
    x = torch.randn(24, D, generator=g)
    x[0] = 0.0
    x[1] = -0.0
    x[2] = 3.25
    x[3] = -1e-30
    x[4, 5] = float("inf")
    x[5, 7] = float("-inf")
    x[6, D - 1] = float("nan")
    x[7] = x[7] * 1e38
    x[8, 0], x[8, 1] = 3e38, -3e38           # the range is not finite
    x[9] = 3e38
    x[10] = x[10] * 1e-39                    # subnormal in 32 bits
    x[11] = x[11] * 1e-4 + 1000.0
    x[12] = -x[12].abs()
    x[13] = x[13].abs() + 1
    x[14] = torch.arange(D) % 16
    x[15] = torch.arange(D) / 2.0            # halves between codes
    x[16] = torch.where(torch.arange(D) % 2 == 0, 1e30, -1e-30)
    x[17, 3] = 1e20
    x[18] = torch.finfo(torch.float32).max
    x[19] = -torch.finfo(torch.float32).max
    x[20] = float("inf")
    return x.to(dt)


@pytest.mark.parametrize("bits,inp,D", list(itertools.product([4, 8], ["bf16", "f32"], [64, 128])))
def test_append_special_rows(bits, inp, D):
    x = special_rows(D, DT[inp])
    T = x.shape[0]
    k, v = x[:, None].contiguous(), x.flip(0)[:, None].contiguous()
    pool = pk.QuantKVPool(1, 2, 16, 1, D, bits, fill=0x11)
    slots = torch.arange(T)
    want = expect_append(raw(pool), 0, k, v, slots, 16, bits)
    pk.kv_quant_append(pool, 0, k.cuda(), v.cuda(), slots.cuda())
    for name, a, b in zip(("k_codes", "k_params", "v_codes", "v_params"), raw(pool), want):
        if "params" in name:  # (a NaN is a NaN)
            a, b = a.view(BF), b.view(BF)
            assert torch.equal(a.isnan(), b.isnan()), name
            a, b = a.nan_to_num(0.5), b.nan_to_num(0.5)
        assert torch.equal(a, b), name


def test_append_slots_outside_the_pool_are_flagged():
    pool = pk.QuantKVPool(1, 2, 16, 2, 64, 4, fill=7)
    x = torch.ones(4, 2, 64, dtype=BF, device="cuda")
    pk.kv_quant_append(pool, 0, x, x, dev([-1, -2, 32, 2 ** 40], torch.int64))
    assert pool.errors() == pk.ERRBIT_SLOT and all((r == 7).all() for r in raw(pool))
    pool.clear_errors()
    pk.kv_quant_append(pool, 0, x[:0], x[:0], dev([], torch.int64))
    pk.kv_quant_append(pool, 0, x[:1], x[:1], dev([31], torch.int64))
    assert pool.errors() == 0 and (raw(pool)[0][0, 1, :, 15] == 0).all() and (raw(pool)[0][0, 1, :, 14] == 7).all()


# ------------------------------------------------------------------- read back
def fill_pool(kind, nb, bs, Hk, D, g, layers=2):
    """A pool of random contents, and its K and V in 64 bits [layers, nb, Hk, bs, D]."""
    shape = (layers, nb, Hk, bs, D)
    if kind in ("q4", "q8"):
        bits = int(kind[1])
        pool = pk.QuantKVPool(layers, nb, bs, Hk, D, bits)
        out = []
        for codes, params in ((pool.k_codes, pool.k_params), (pool.v_codes, pool.v_params)):
            n, p = ref.quantise((torch.randn(shape, generator=g) + 0.3).to(BF), bits)
            codes.copy_(ref.pack(n, bits))
            params.copy_(p)
            out.append(ref.values(ref.pack(n, bits), p, bits))
        return pool, out
    scales = (0.031, 0.027) if kind == "fp8" else (1.0, 1.0)
    pool = pk.KVPool(layers, nb, bs, Hk, D, kind, *scales)
    out = []
    for x, sc in ((pool.k, scales[0]), (pool.v, scales[1])):
        y = torch.randn(shape, generator=g) * (30 if kind == "fp8" else 1)
        y = y.to({"f32": torch.float32, "bf16": BF, "fp8": torch.float8_e4m3fn}[kind])
        x.copy_(y.view(torch.uint8) if kind == "fp8" else y)
        out.append(y.double() * float(np.float32(sc)))
    return pool, out


def expect_rows(values, tables, lens, bs):
    rows = []
    for b, n in enumerate(lens):
        t = torch.arange(n)
        rows.append(values[tables[b].long()[t // bs], :, t % bs])
    return torch.cat(rows)


def check_rows(got, want):
    # the value in 32 bits (one rounding, or none) and one to the output's type
    half = ref.HALF[got.dtype]
    err = (got.cpu().double() - want).abs()
    assert (err <= (half + 2.0 ** -23) * want.abs()).all(), float(err.max())


@pytest.mark.parametrize("kind", ["q4", "q8", "fp8", "bf16", "f32"])
@pytest.mark.parametrize("lens,Hk,D,bs", [((1,), 1, 64, 16), ((0, 0), 2, 128, 16), ((5, 0, 16, 17, 1), 2, 128, 16),
                                          ((64, 63, 65, 200), 8, 128, 32), ((130, 0, 1, 31), 3, 64, 64),
                                          (tuple(range(60)), 1, 128, 16), ((1500, 2, 700), 4, 64, 32)])
def test_read_back(kind, lens, Hk, D, bs):
    g = torch.Generator().manual_seed(sum(lens) + D)
    tables, nb = tables_of(lens, bs, g)
    pool, (k, v) = fill_pool(kind, nb, bs, Hk, D, g)
    offsets = np.concatenate([[0], np.cumsum(lens)])
    got = pk.kv_read(pool, 1, tables.cuda(), dev(offsets), int(offsets[-1]))
    assert got[0].dtype == (torch.float32 if kind == "f32" else BF)
    for x, y in zip(got, (k, v)):
        check_rows(x, expect_rows(y[1], tables, lens, bs))
    assert pool.errors() == 0


@pytest.mark.parametrize("kind", ["q4", "q8", "fp8", "bf16"])
def test_read_leaves_other_rows_and_flags_bad_entries(kind):
    g = torch.Generator().manual_seed(1)
    lens, bs, Hk, D = (20, 3, 40, 0, 9), 16, 2, 128
    tables, nb = tables_of(lens, bs, g)
    pool, (k, _) = fill_pool(kind, nb, bs, Hk, D, g, layers=1)
    offsets = np.concatenate([[0], np.cumsum(lens)]) + 5
    rows = int(offsets[-1]) + 4
    outs = [torch.full((rows, Hk, D), 77.0, dtype=BF, device="cuda") for _ in range(2)]
    got, _ = pk.kv_read(pool, 0, tables.cuda(), dev(offsets), rows, k_out=outs[0], v_out=outs[1])
    assert got.data_ptr() == outs[0].data_ptr()
    check_rows(got[5:-4], expect_rows(k[0], tables, lens, bs))
    assert (got[:5] == 77).all() and (got[-4:] == 77).all() and (outs[1][-4:] == 77).all() and pool.errors() == 0
    # a table entry outside the pool, and a table that is too short: zero rows
    bad = tables.clone()
    bad[0, 1] = nb
    got, _ = pk.kv_read(pool, 0, bad.cuda(), dev(offsets - 5), rows - 9)
    assert pool.errors() == pk.ERRBIT_BLOCK_ID and (got[16:20] == 0).all()
    check_rows(got[20:], expect_rows(k[0], tables, lens, bs)[20:])
    pool.clear_errors()
    got, _ = pk.kv_read(pool, 0, tables[:, :2].contiguous().cuda(), dev(offsets - 5), rows - 9)
    assert pool.errors() == pk.ERRBIT_SEQ_LEN and (got[23 + 32:63] == 0).all()
    check_rows(got[:23 + 32], expect_rows(k[0], tables, lens, bs)[:23 + 32])
    pool.clear_errors()
    # offsets that cannot be: those sequences are left out, the others are read
    for bad, lost in (([0, 20, 23, 22, 63, 72], slice(22, 63)), ([-1, 20, 23, 63, 63, 72], slice(0, 20)),
                      ([0, 20, 23, 63, 63, 73], slice(63, 72))):
        outs[0].fill_(77.0)
        pk.kv_read(pool, 0, tables.cuda(), dev(bad), 72, k_out=outs[0][:72], v_out=outs[1][:72])
        assert pool.errors() & pk.ERRBIT_OFFSETS
        pool.clear_errors()
        keep = torch.ones(72, dtype=torch.bool)
        keep[lost] = False
        if bad[3] != 22:
            check_rows(outs[0][:72][keep.cuda()], expect_rows(k[0], tables, lens, bs)[keep])
        else:  # (sequence 3 then claims rows 22 .. 62, and has no table there)
            check_rows(outs[0][:22], expect_rows(k[0], tables, lens, bs)[:22])
        assert (outs[0][72:] == 77).all()


# ------------------------------------------------------------ decode attention
class Quantised:
    """A batch over a quantised cache whose blocks hold codes of 0xFF and NaN
    pairs wherever no token lies."""

    def __init__(self, lens, Hq=8, Hk=2, D=128, bs=16, bits=4, seed=0, wide=1.0, dtype=BF):
        g = torch.Generator().manual_seed(seed + sum(lens))
        self.lens, self.bits, self.bs, self.scale = list(lens), bits, bs, D ** -0.5
        self.tables, nb = tables_of(lens, bs, g)
        self.pool = pk.QuantKVPool(2, nb, bs, Hk, D, bits, fill=0xFF)
        self.q = (torch.randn(len(lens), Hq, D, generator=g) * wide).to(BF)
        slots = torch.cat([torch.zeros(0, dtype=torch.int64)] + [
            self.tables[b].long()[torch.arange(n) // bs] * bs + torch.arange(n) % bs for b, n in enumerate(lens)])
        x = torch.randn(2, len(slots), Hk, D, generator=g)
        x[0, ..., 3::29] *= 4
        x[0, ..., 7] += 2
        x = x.to(dtype)
        pk.kv_quant_append(self.pool, 1, x[0].cuda(), x[1].cuda(), slots.cuda())
        self.max_len = max(list(lens) + [1])

    def pools(self):
        return [x[1].cpu() for x in (self.pool.k_codes, self.pool.k_params, self.pool.v_codes, self.pool.v_params)]

    def run(self, **kw):
        out = pk.paged_quant_decode_attention(self.q.cuda(), self.pool, 1, self.tables.cuda(), dev(self.lens),
                                              kw.pop("max_len", self.max_len), self.scale, **kw)
        torch.cuda.synchronize()
        return out

    def check(self, out=None, rows=slice(None)):
        out = self.run() if out is None else out
        want, bound = ref.quant_attention(self.q, self.pools(), self.tables, self.lens, self.scale, self.bits)
        err = (out.cpu().double() - want).abs()[rows]
        ok = err <= bound[rows]
        assert bool(ok.all()), (float(err.max()), int((~ok).sum()))
        return out


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hk,D,bs", [(8, 2, 128, 16), (4, 4, 128, 32), (5, 1, 128, 64), (16, 2, 64, 16), (12, 4, 64, 64),
                                        (16, 1, 128, 16), (17, 1, 128, 32), (40, 1, 64, 16), (3, 3, 64, 32)])
def test_attention_heads_and_lengths(bits, Hq, Hk, D, bs):
    b = Quantised((1, 0, 2, 15, 16, 17, 31, 63, 64, 65, 100, 127, 128, 129, 300, 1000), Hq, Hk, D, bs, bits)
    b.check()
    assert b.pool.errors() == 0


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lens", [(1,), (0,), (7,), (20000,), (5000, 1, 9000), (0, 0, 3, 0), tuple([40] * 200),
                                  (3000, 0, 1, 64, 2500, 700) * 6])
def test_attention_batches(bits, lens):
    b = Quantised(lens, bits=bits, bs=(16, 64)[len(lens) % 2])
    b.check()
    assert b.pool.errors() == 0


@pytest.mark.parametrize("bits", [4, 8])
def test_attention_repeats_bit_for_bit_and_leaves_its_counters(bits):
    b = Quantised((3000, 17, 0, 900, 4097, 64), bits=bits)
    ws = pk.quant_decode_workspace(b.pool, 6, 8, b.max_len)
    first = b.check(b.run(workspace=ws))
    for _ in range(3):
        assert torch.equal(b.run(workspace=ws), first)
    assert torch.equal(b.run(max_len=b.tables.shape[1] * 16), first)  # (the bound is no part of the result)


@pytest.mark.parametrize("wide", [1e-6, 1.0, 50.0, 1e6])
def test_attention_query_magnitudes(wide):
    Quantised((100, 257, 1), wide=wide, seed=5).check()


def test_attention_of_rows_of_very_different_scales():
    """V rows from 1e-20 to 1e20, constant ones among them: the weights stay relative to what they weigh."""
    b = Quantised((64, 200), Hq=2, Hk=1, seed=6)
    g = torch.Generator().manual_seed(9)
    p = b.pool.v_params[1].cpu().float()
    size = 10.0 ** torch.randint(-20, 21, p.shape[:-1], generator=g).float()
    size[torch.rand(size.shape, generator=g) < 0.2] = 0
    fine = ~p.isnan()
    q = torch.where(fine, p * size[..., None], p)
    q[..., 0] = torch.where(fine[..., 0], q[..., 0].clamp(min=2.0 ** -100), q[..., 0])
    b.pool.v_params[1].copy_(q.to(BF))
    b.check()


@pytest.mark.parametrize("bits", [4, 8])
def test_attention_zero_rows_constant_rows_and_nan_rows(bits):
    b = Quantised((40, 40, 40), bits=bits, seed=2)
    slot = lambda s, t: (int(b.tables[s, t // 16]), t % 16)
    x = torch.zeros(3, 2, 128, dtype=BF)
    x[1] = 2.5
    x[2, :, 9] = float("nan")
    at = [slot(0, 3), slot(0, 4), slot(1, 39)]
    slots = torch.tensor([blk * 16 + off for blk, off in at])
    pk.kv_quant_append(b.pool, 1, x.cuda(), x.cuda(), slots.cuda())
    out = b.run().cpu()
    assert out[1].isnan().all()
    b.check(out, rows=[0, 2])
    # one token, a row of zeros: exactly zero
    z = Quantised((1,), bits=bits)
    pk.kv_quant_append(z.pool, 1, x[:1].cuda(), x[:1].cuda(), z.tables[0, :1].long().cuda() * 16)
    assert (z.run() == 0).all()
    pk.kv_quant_append(z.pool, 1, x[:1].cuda(), x[1:2].cuda(), z.tables[0, :1].long().cuda() * 16)
    assert (z.run() == 2.5).all()


def test_attention_flags_lengths_and_blocks():
    b = Quantised((40, 70, 20, 33))
    good = b.run().cpu()
    t = b.tables.clone()
    t[1, 2], t[2, 0] = b.pool.num_blocks, -1
    lens = dev([40, 70, 20, -5])
    out = pk.paged_quant_decode_attention(b.q.cuda(), b.pool, 1, t.cuda(), lens, 80, b.scale).cpu()
    assert b.pool.errors() == pk.ERRBIT_BLOCK_ID | pk.ERRBIT_SEQ_LEN
    assert torch.equal(out[0], good[0]) and (out[3] == 0).all()
    b.pool.clear_errors()
    # longer than the caller's bound: cut there
    out = pk.paged_quant_decode_attention(b.q.cuda(), b.pool, 1, b.tables.cuda(), dev([40, 70, 2 ** 31 - 1, 33]), 70,
                                          b.scale)
    assert b.pool.errors() & pk.ERRBIT_SEQ_LEN
    assert torch.equal(out.cpu()[:2], good[:2])


def test_attention_captured_with_other_lengths_and_on_a_stream():
    b = Quantised((300, 5, 0, 1000), bits=8)
    ws = pk.quant_decode_workspace(b.pool, 4, 8, 1100)
    q, t, lens = b.q.cuda(), b.tables.cuda(), dev(b.lens)
    out = torch.empty_like(q)
    call = lambda **kw: pk.paged_quant_decode_attention(q, b.pool, 1, t, lens, 1000, b.scale, out=out, workspace=ws, **kw)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for new in ((300, 5, 0, 1000), (1, 0, 0, 17), (0, 0, 0, 0), (299, 4, 0, 64)):
        lens.copy_(dev(new))
        b.lens = list(new)
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        b.check(out)
    side = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    call(stream=side)
    side.synchronize()
    b.check(out)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lens", [(512,), (513,), (1024,), (1025,), (1024, 700) * 60, (1025, 700) * 60, (64,) * 152,
                                  (2048, 1, 1), (1, 30) * 500], ids=lambda x: "%dx%d" % (len(x), max(x)))
def test_attention_short_units_and_many(bits, lens):
    """Units that are a CTA's own, and ones that are cut: both sides of the rule."""
    b = Quantised(lens, bits=bits, bs=32, seed=11)
    b.check()
    assert b.pool.errors() == 0


@pytest.mark.parametrize("bits", [4, 8])
def test_attention_workspace_serves_calls_of_all_sizes(bits):
    """One workspace, the largest call's, for calls of other batches and heads: each leaves it as the next needs it."""
    calls = [Quantised(lens, Hq, Hk, D, 16, bits, seed=12) for lens, Hq, Hk, D in
             [((9000, 5000), 8, 2, 128), ((3000, 0, 1, 64, 2500, 700) * 8, 8, 2, 128), ((20000,), 16, 1, 128),
              ((4000,) * 30, 8, 4, 64), ((7000, 1), 40, 1, 64), ((2000,) * 70, 8, 2, 128)]]
    sizes = [pk.quant_decode_workspace(b.pool, len(b.lens), b.q.shape[1], b.max_len).numel() for b in calls]
    ws = torch.zeros(max(sizes), dtype=torch.uint8, device="cuda")
    first = [b.check(b.run(workspace=ws)) for b in calls]
    for i in (5, 0, 3, 1, 4, 2, 1, 5):
        assert torch.equal(calls[i].run(workspace=ws), first[i]), i


def test_attention_two_graphs_share_a_workspace():
    a, b = Quantised((6000, 40), bits=4, seed=13), Quantised((900,) * 20, bits=4, seed=14)
    ws = max((pk.quant_decode_workspace(x.pool, len(x.lens), 8, x.max_len) for x in (a, b)), key=lambda w: w.numel())
    graphs = []
    for x in (a, b):
        args = (x.q.cuda(), x.pool, 1, x.tables.cuda(), dev(x.lens), x.max_len, x.scale)
        out = torch.empty_like(args[0])
        pk.paged_quant_decode_attention(*args, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pk.paged_quant_decode_attention(*args, out=out, workspace=ws)
        graphs.append((graph, out, x, args))
    for _ in range(3):
        for graph, out, x, _ in graphs:
            out.fill_(9.0)
            graph.replay()
        torch.cuda.synchronize()
        for _, out, x, _ in graphs:
            x.check(out)


def test_attention_on_two_streams_at_once():
    a, b = Quantised((6000, 40), bits=4, seed=15), Quantised((900,) * 20, bits=8, seed=16)
    want = [a.check(), b.check()]
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    args = [(x.q.cuda(), x.pool, 1, x.tables.cuda(), dev(x.lens), x.max_len, x.scale) for x in (a, b)]
    ws = [pk.quant_decode_workspace(x.pool, len(x.lens), 8, x.max_len) for x in (a, b)]
    outs = [torch.empty_like(x[0]) for x in args]
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            pk.paged_quant_decode_attention(*args[i], out=outs[i], workspace=ws[i], stream=side[i])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want[0]) and torch.equal(outs[1], want[1])


@pytest.mark.parametrize("kind", ["q4", "q8", "bf16"])
def test_read_back_of_many_sequences(kind):
    """More sequences than a CTA keeps offsets of, most of them empty or one row long."""
    g = torch.Generator().manual_seed(21)
    lens = torch.randint(0, 4, (3000,), generator=g).tolist()
    lens[7], lens[2999] = 50, 33
    tables, nb = tables_of(lens, 16, g)
    pool, values = fill_pool(kind, nb, 16, 2, 128, g)
    off = np.concatenate([[0], np.cumsum(lens)])
    k, v = pk.kv_read(pool, 1, tables.cuda(), dev(off), int(off[-1]))
    check_rows(k, expect_rows(values[0][1], tables, lens, 16))
    check_rows(v, expect_rows(values[1][1], tables, lens, 16))
    assert pool.errors() == 0


@pytest.mark.parametrize("bits,inp", list(itertools.product([4, 8], ["bf16", "f32"])))
def test_append_one_row_to_many_slots(bits, inp):
    """A token stride of zero: one row, stored at every slot."""
    dt = BF if inp == "bf16" else torch.float32
    x = torch.randn(2, 1, 3, 64, generator=torch.Generator().manual_seed(22)).to(dt)
    pool = pk.QuantKVPool(1, 3, 16, 3, 64, bits, fill=0xFF)
    slots = torch.tensor([0, 17, 33, -1, 47])
    pk.kv_quant_append(pool, 0, x[0].cuda().expand(5, 3, 64), x[1].cuda().expand(5, 3, 64), slots.cuda())
    want = raw(pk.QuantKVPool(1, 3, 16, 3, 64, bits, fill=0xFF))
    expect_append(want, 0, x[0].expand(5, 3, 64), x[1].expand(5, 3, 64), slots, 16, bits)
    for got, w in zip(raw(pool), want):
        assert torch.equal(got, w)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 2, 128), (16, 2, 64), (32, 2, 128), (5, 1, 64), (40, 2, 128)])
def test_attention_many_short_sequences(bits, Hq, Hk, D):
    """Units that are a warp's own: empty sequences between, one token, whole and cut steps and tiles, one longer unit."""
    g = torch.Generator().manual_seed(23)
    lens = torch.randint(0, 100, (1200 // Hk,), generator=g).tolist()
    lens[:12] = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 65, 130]
    lens[-3:] = [0, 97, 0]
    b = Quantised(lens, Hq, Hk, D, 16, bits, seed=24)
    first = b.check()
    assert b.pool.errors() == 0 and torch.equal(b.run(), first)
