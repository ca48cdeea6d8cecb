"""GPU parity of decode attention over shared prefixes against 64-bit softmax
attention of every sequence on its own, and against paged_decode_attention."""
import itertools
import time

import pytest
import torch

import step_reference as ref
from parity import TOL
from paged_kv_cache_194_gb300 import binding as pk

pytestmark = pytest.mark.gpu

RAW = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


class Batch:
    """Sequences of the given lengths; groups [(first, last + 1, prefix)] share
    whole blocks of their prefix and hold equal copies of a partial one.  Every
    slot no sequence uses holds NaN."""

    def __init__(self, lens, groups, q_heads=8, kv_heads=2, dim=128, bs=16, kv="bf16", seed=0, spread=1.0, extra=3,
                 offsets=None, prefix=None):
        g = torch.Generator().manual_seed(seed)
        B = len(lens)
        need = [-(-n // bs) for n in lens]
        width = max(1, max(need)) + extra
        free = iter(torch.randperm(sum(need) + 4, generator=g).tolist())
        tables = torch.full((B, width), -1, dtype=torch.int32)
        k = torch.full((sum(need) + 4, kv_heads, bs, dim), float("nan"))
        v = k.clone()
        lead = {}
        for first, last, p in groups:
            for b in range(first, last):
                # the group's longest sequence provides the prefix of the others
                lead[b] = (max(range(first, last), key=lambda x: lens[x]), p)
        order = sorted(range(B), key=lambda b: -lens[b])
        for b in order:
            src, p = lead.get(b, (b, 0))
            for i in range(need[b]):
                if src != b and (i + 1) * bs <= min(p, lens[b]):
                    tables[b, i] = tables[src, i]
                    continue
                blk = next(free)
                tables[b, i] = blk
                n = min(bs, lens[b] - i * bs)
                k[blk, :, :n] = torch.randn(kv_heads, n, dim, generator=g) * spread
                v[blk, :, :n] = torch.randn(kv_heads, n, dim, generator=g)
                if src != b and i * bs < p:
                    c = min(p, lens[b]) - i * bs
                    k[blk, :, :c], v[blk, :, :c] = k[tables[src, i], :, :c], v[tables[src, i], :, :c]
        self.k_scale, self.v_scale = (0.013, 0.011) if kv == "fp8" else (1.0, 1.0)
        # (values past 448 scales would become NaN in an E4M3 cast)
        self.k, self.v = (((x / s).clamp(-448, 448) if kv == "fp8" else x).to(RAW[kv])
                          for x, s in ((k, self.k_scale), (v, self.v_scale)))
        qd = torch.float32 if kv == "f32" else torch.bfloat16
        self.q = torch.randn(B, q_heads, dim, generator=g).to(qd)
        self.tables, self.lens, self.kv = tables, lens, kv
        self.scale = ref.scale_for(dim)
        self.max_len = max(1, max(lens))
        layers = 2
        self.pool = pk.KVPool(layers, k.shape[0], bs, kv_heads, dim, kv, self.k_scale, self.v_scale, fill=0xFF)
        for dst, src in ((self.pool.k, self.k), (self.pool.v, self.v)):
            dst[1].copy_(src.view(torch.uint8) if kv == "fp8" else src)
        self.offsets = torch.tensor(offsets if offsets is not None else
                                    ([x[0] for x in groups] + [groups[-1][1]] if groups else [0]), dtype=torch.int32)
        self.prefix = torch.tensor(prefix if prefix is not None else [x[2] for x in groups], dtype=torch.int32)

    def run(self, algo="auto", **kw):
        args = dict(out=torch.full_like(self.q, 7.0).cuda())
        args.update(kw)
        return pk.paged_prefix_decode_attention(self.q.cuda(), self.pool, 1, self.tables.cuda(),
                                                torch.tensor(self.lens, dtype=torch.int32).cuda(), self.max_len,
                                                self.offsets.cuda(), self.prefix.cuda(), self.scale, algo=algo, **args)

    def reference(self):
        return ref.attention(self.q, self.k, self.v, self.tables, self.lens, self.scale, self.k_scale, self.v_scale)

    def check(self, out, design):
        want, mass, floor = self.reference()
        err = (out.cpu().double() - want).abs()
        if design == "tc":
            bound = ref.attention_bound(want, mass, self.kv, floor)
        else:  # the designs of decode attention, within its own tolerance
            bound = TOL[self.kv] * (1.0 + want.abs())
        bad = ~(err <= bound)
        assert not bad.any(), "%d of %d outside; worst %g of the bound at %s" % (
            int(bad.sum()), bad.numel(), float((err / bound.clamp(min=1e-30)).max()), bad.nonzero()[:4].tolist())
        for b, n in enumerate(self.lens):
            if n == 0:
                assert (out[b] == 0).all()

    def design(self, algo="auto"):
        return pk.prefix_decode_algo(self.pool, len(self.lens), len(self.prefix), self.q.shape[1], self.max_len, algo)


SHAPES = {
    "one_group": ((700, 640, 641, 655, 704, 1000, 66, 900), [(0, 8, 640)]),
    "exact_tiles": ((128, 128, 128, 128), [(0, 4, 128)]),           # nothing behind the prefix
    "short_prefix": ((70, 90, 64, 65), [(0, 4, 50)]),               # below one tile: all own
    "one_tile": ((64, 65, 300), [(0, 3, 64)]),
    "odd_prefix": ((500, 333, 420, 299), [(0, 4, 297)]),            # not a multiple of tile or block
    "shorter_members": ((500, 0, 100, 450, 1, 447, 448), [(0, 7, 448)]),
    "single_members": ((300, 200, 100), [(0, 1, 256), (1, 2, 128), (2, 3, 64)]),
    "outside_groups": ((90, 300, 310, 0, 64), [(1, 3, 256)]),
    "no_groups": ((1, 63, 64, 65, 0, 500), []),
    "empty_batch_rows": ((0, 0, 0), [(0, 3, 64)]),
    "length_one": ((1, 1), [(0, 2, 1)]),
    "many": (tuple(130 + 7 * i for i in range(40)), [(0, 40, 128)]),
}


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("kv,dim", [("bf16", 128), ("fp8", 128), ("f32", 64), ("bf16", 64)])
def test_prefix_parity(shape, kv, dim):
    lens, groups = SHAPES[shape]
    bt = Batch(lens, groups, dim=dim, kv=kv, seed=len(shape))
    bt.check(bt.run(), bt.design())
    assert bt.pool.errors() == 0


@pytest.mark.parametrize("bs", [16, 32, 64])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (8, 8), (5, 1), (12, 4), (16, 2), (40, 1), (64, 2), (128, 1)])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_heads_and_blocks(q_heads, kv_heads, bs, kv):
    """Row tiles: 128 / (query heads per KV head) sequences each, the last one ragged."""
    lens = (400, 385, 384, 390, 700, 420)
    bt = Batch(lens, [(0, 5, 384), (5, 6, 384)], q_heads, kv_heads, bs=bs, kv=kv, seed=q_heads)
    try:
        design = bt.design()
    except pk.PkvError:  # no design takes so many query heads on this pool: refused
        with pytest.raises(pk.PkvError):
            bt.run()
        return
    bt.check(bt.run(), design)
    assert bt.pool.errors() == 0


@pytest.mark.parametrize("q_heads,kv_heads", [(12, 4), (5, 1), (16, 2), (7, 1), (34, 2), (130, 1)])
@pytest.mark.parametrize("kv,dim", [("f32", 64), ("f32", 128), ("bf16", 64), ("fp8", 64), ("bf16", 128), ("fp8", 128)])
def test_prefix_and_decode_any_number_of_heads(q_heads, kv_heads, kv, dim):
    """Numbers of query heads per KV head without a launch of their own: for
    every pool, with one split and with several, for one query and for three."""
    bt = Batch((400, 65, 0, 700, 1), [(0, 2, 64), (3, 5, 640)], q_heads, kv_heads, dim, kv=kv, seed=q_heads)
    bt.check(bt.run(), bt.design())
    lens = torch.tensor(bt.lens, dtype=torch.int32).cuda()
    args = (bt.pool, 1, bt.tables.cuda())
    for split in (0, 1024, 128):
        bt.check(pk.paged_decode_attention(bt.q.cuda(), *args, lens, bt.max_len, bt.scale, split_tokens=split), "decode")
    bt.check(pk.paged_decode_attention(bt.q.cuda(), *args, lens, bt.max_len, bt.scale, algo="simt"), "decode")
    # three queries: each as a decode call over the tokens that it sees
    q = torch.stack([bt.q.flip(0), bt.q.flip(1), bt.q], 1).contiguous().cuda()
    out = pk.paged_multi_query_attention(q, *args, lens, bt.max_len, bt.scale, algo="simt")
    for c in range(3):
        one = pk.paged_decode_attention(q[:, c].contiguous(), *args, (lens - 2 + c).clamp(min=0), bt.max_len, bt.scale,
                                        algo="simt")
        for b, n in enumerate(bt.lens):
            if n - 2 + c > 0:
                assert ((out[b, c] - one[b]).abs() <= TOL[kv] * (1 + one[b].abs())).all()
    assert bt.pool.errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_many_groups(kv):
    groups = [(0, 9, 320), (9, 9, 64), (9, 12, 1024), (12, 13, 128), (13, 50, 64), (50, 52, 100)]
    lens = tuple(1024 + 13 * (i % 7) if 9 <= i < 12 else 320 + 11 * (i % 5) for i in range(53))
    bt = Batch(lens, groups, seed=5, kv=kv)
    bt.check(bt.run(), bt.design())
    assert bt.pool.errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_long_split_over_ctas(kv):
    """One KV head and two sequences: every CTA has a piece of one unit."""
    bt = Batch((20000, 19990), [(0, 2, 19968)], 4, 1, bs=64, seed=3, kv=kv)
    bt.check(bt.run(), bt.design())
    assert bt.pool.errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_growing_scores_rescale(kv):
    """Wide scores: the running maximum moves by more than its slack often."""
    bt = Batch((900, 960, 930), [(0, 3, 832)], seed=9, kv=kv, spread=1.0)
    with torch.no_grad():
        bt.q = (bt.q.float() * 6).to(bt.q.dtype)
    out = bt.run()
    want, mass, floor = bt.reference()
    if bt.design() == "tc":
        # scores six times as wide: 6 x the exponent's error
        bound = ref.attention_bound(want, mass, kv, floor) + 5 * 2.0 ** -13 * mass
        assert ((out.cpu().double() - want).abs() <= bound).all()
    else:
        assert ((out.cpu().double() - want).abs() <= 6 * TOL[kv] * (1 + want.abs())).all()


@pytest.mark.parametrize("size", [2.0 ** -100, 1e-6, 1.0, 1e6, 2.0 ** 100])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_query_magnitudes(kv, size):
    """Queries of any size (the scale takes it back): FP8 pools scale each row into FP16's range."""
    bt = Batch((300, 333, 290, 70), [(0, 3, 256)], seed=14, kv=kv)
    rows = torch.tensor([1.0, 0.5, 3.0, 0.01]).view(4, 1, 1)  # (other sizes from row to row)
    bt.q = (bt.q.float() * rows * size).to(torch.bfloat16)
    bt.q[1, 2] = 0
    bt.scale = bt.scale / size
    bt.check(bt.run(), "tc")


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_negative_and_zero_scale(kv):
    bt = Batch((300, 333, 290), [(0, 3, 256)], seed=2, kv=kv)
    for scale in (-0.07, 0.0):
        bt.scale = scale
        bt.check(bt.run(), bt.design())


@pytest.mark.parametrize("shape", ["one_group", "odd_prefix", "shorter_members", "outside_groups"])
def test_prefix_agrees_with_decode_attention(shape):
    lens, groups = SHAPES[shape]
    bt = Batch(lens, groups, seed=21)
    out = bt.run()
    dec = pk.paged_decode_attention(bt.q.cuda(), bt.pool, 1, bt.tables.cuda(),
                                    torch.tensor(lens, dtype=torch.int32).cuda(), bt.max_len, bt.scale)
    want, mass, floor = bt.reference()
    # both within their own bounds of the same value
    assert ((out.double() - dec.double()).abs().cpu() <= ref.attention_bound(want, mass) + TOL["bf16"] * (1 + want.abs())).all()
    for algo in ("mma", "simt"):
        assert torch.equal(bt.run(algo=algo), pk.paged_decode_attention(
            bt.q.cuda(), bt.pool, 1, bt.tables.cuda(), torch.tensor(lens, dtype=torch.int32).cuda(), bt.max_len,
            bt.scale, algo=algo))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_bad_groups_still_give_right_results(kv):
    lens = (300, 310, 320, 330)
    for offsets, prefix, bit in (([0, 3, 1, 4], [256, 256, 256], pk.ERRBIT_GROUP), ([-1, 4], [256], pk.ERRBIT_GROUP),
                                 ([0, 9], [256], pk.ERRBIT_GROUP), ([0, 4], [-5], pk.ERRBIT_GROUP),
                                 ([0, 4], [10 ** 6], 0)):  # longer than every member: shares nothing
        bt = Batch(lens, [(0, 4, 256)], seed=4, kv=kv, offsets=offsets, prefix=prefix)
        bt.check(bt.run(algo="tc"), "tc")
        assert bt.pool.errors() == bit, (offsets, prefix)


def test_prefix_fp8_nan_codes_stay_nan():
    """A NaN code in a value a sequence attends to makes its output NaN there,
    and touches no other sequence or column."""
    bt = Batch((300, 310, 320), [(0, 3, 256)], seed=4, kv="fp8")
    good = bt.run()
    blk = int(bt.tables[1, 18])  # an own block of sequence 1
    bt.pool.v[1, blk, 0, 3, 7] = 0x7F
    out = bt.run()
    assert out[1, :4, 7].isnan().all()
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1, :4, 7] = False
    assert torch.equal(out[keep], good[keep])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_prefix_infinite_queries_stay_in_their_row(kv, bad):
    bt = Batch((300, 310, 320), [(0, 3, 256)], seed=4, kv=kv)
    good = bt.run()
    bt.q[1, 2, 5] = bad
    out = bt.run()
    assert out[1, 2].isnan().all()
    keep = torch.ones_like(out, dtype=torch.bool)
    keep[1, 2] = False
    assert torch.equal(out[keep], good[keep])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_reports_bad_lengths_and_blocks(kv):
    bt = Batch((300, 310, 320), [(0, 3, 256)], seed=4, kv=kv)
    good = bt.run()
    lens = bt.lens
    bt.lens = (300, 310, -2)
    out = bt.run()
    assert bt.pool.errors() == pk.ERRBIT_SEQ_LEN and (out[2] == 0).all()
    bt.pool.clear_errors()
    # fewer members, other pieces: equal up to rounding
    bt.lens = (300, 310, 0)
    bt.check(out, "tc")
    bt.lens = lens
    bt.tables[1, 18] = 10 ** 6  # an own block of sequence 1
    out = bt.run()
    assert bt.pool.errors() == pk.ERRBIT_BLOCK_ID
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_repeats_exactly_and_leaves_other_rows(kv):
    lens, groups = SHAPES["many"]
    bt = Batch(lens, groups, seed=8, kv=kv)
    B = len(lens)
    big = torch.full((B + 5,) + bt.q.shape[1:], 3.0, dtype=bt.q.dtype, device="cuda")
    ws = pk.prefix_decode_workspace(bt.pool, B, 1, bt.q.shape[1], bt.max_len)
    first = bt.run(out=big[:B], workspace=ws).clone()
    assert (big[B:] == 3.0).all()
    for _ in range(3):
        assert torch.equal(bt.run(out=big[:B], workspace=ws), first)


def test_prefix_shares_a_workspace_with_decode_attention():
    """Alternating calls of the sharing design and of decode attention (whose
    counters must stay zero) on one workspace."""
    lens = tuple([2000, 1900, 1950, 2100] * 2)
    a = Batch(lens, [(0, 8, 1856)], 32, 8, seed=1)
    b = Batch(lens, [(0, 8, 1856)], 32, 8, seed=2)
    ws = pk.prefix_decode_workspace(a.pool, 8, 1, 32, a.max_len)
    want_a, want_b = a.run(), b.run(algo="mma")
    for _ in range(3):
        assert torch.equal(a.run(workspace=ws), want_a)
        assert torch.equal(b.run(algo="mma", workspace=ws), want_b)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_captured_call_follows_lengths_and_groups(kv):
    """One captured call replayed over other lengths, groups and queries."""
    bt = Batch((900, 800, 850, 700, 720), [(0, 3, 768), (3, 5, 640)], seed=6, kv=kv)
    dev = dict(q=bt.q.cuda(), t=bt.tables.cuda(), n=torch.tensor(bt.lens, dtype=torch.int32).cuda(),
               o=bt.offsets.cuda(), p=bt.prefix.cuda())
    ws = pk.prefix_decode_workspace(bt.pool, 5, 2, 8, bt.max_len)
    out = torch.zeros_like(dev["q"])

    def call():
        pk.paged_prefix_decode_attention(dev["q"], bt.pool, 1, dev["t"], dev["n"], bt.max_len, dev["o"], dev["p"],
                                         bt.scale, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lens, offsets, prefix in (((900, 800, 850, 700, 720), [0, 3, 5], [768, 640]),
                                  ((800, 790, 820, 650, 0), [0, 2, 4], [512, 0]),
                                  ((64, 1, 850, 300, 720), [0, 0, 5], [64, 10])):
        bt.lens = lens
        dev["n"].copy_(torch.tensor(lens, dtype=torch.int32))
        dev["o"].copy_(torch.tensor(offsets, dtype=torch.int32))
        # the second shape groups sequences 2 and 3, which hold different blocks: it shares 0 tokens
        dev["p"].copy_(torch.tensor(prefix, dtype=torch.int32))
        out.fill_(5.0)
        graph.replay()
        torch.cuda.synchronize()
        bt.check(out, "tc")
    assert bt.pool.errors() == 0


def test_prefix_two_streams_at_once():
    a = Batch(SHAPES["many"][0], SHAPES["many"][1], seed=30)
    b = Batch(SHAPES["one_group"][0], SHAPES["one_group"][1], seed=31)
    want = a.run(), b.run()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        got.append((a.run(stream=s1), b.run(stream=s2)))
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, want[0]) and torch.equal(y, want[1])


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_more_sequences_than_ctas(kv):
    """Many short sequences: a CTA walks over many units, some empty."""
    lens = tuple(itertools.islice(itertools.cycle((64, 70, 0, 65, 130, 64, 1)), 700))
    bt = Batch(lens, [(0, 350, 64), (350, 700, 64)], 4, 2, seed=12, bs=64, kv=kv)
    bt.check(bt.run(), "tc")
    assert bt.pool.errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_many_segments_of_many_tiles(kv):
    """Every CTA walks over several units of several tiles: the copies of K, V
    and the next unit's Q run ahead across their borders."""
    lens = tuple(600 + 37 * (i % 11) for i in range(56))
    bt = Batch(lens, [(0, 30, 320), (30, 56, 448)], 16, 8, bs=64, seed=40, kv=kv)
    bt.check(bt.run(), "tc")
    bt.prefix.zero_()  # nothing shared: own units only
    bt.check(bt.run(), "tc")
    assert bt.pool.errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("cta", [0, 7, 200, -1])
def test_prefix_expired_waits(kv, cta):
    """The failure path on demand: one CTA's first wait for a tile (or every
    one's) gives up.  The call returns with the timeout bit set, rows that the
    CTA took part in are NaN and all others right; the next call is right."""
    # (long enough that every CTA of a full GPU has a tile: its range is longer than the cost of a unit's end)
    bt = Batch((12000, 10500, 8192, 8400, 11600, 70, 0), [(0, 5, 8192)], 32, 8, bs=64, kv=kv, seed=9)
    ws = pk.prefix_decode_workspace(bt.pool, len(bt.lens), 1, 32, bt.max_len)
    good = bt.run(workspace=ws)
    bt.check(good, "tc")
    try:
        pk.set_first_wait_limit_for_testing(0, cta)
        t0 = time.perf_counter()
        out = bt.run(workspace=ws)
        torch.cuda.synchronize()
        dt = time.perf_counter() - t0
    finally:
        pk.set_first_wait_limit_for_testing(-1)
    assert dt < 5.0
    assert bt.pool.errors() == pk.ERRBIT_TIMEOUT
    lost = torch.isnan(out).any(2)
    assert torch.isnan(out[lost]).all() and torch.equal(out[~lost], good[~lost])
    assert lost.any() and (lost[:6].all() if cta < 0 else not lost.all()) and not lost[6].any()
    bt.pool.clear_errors()
    assert torch.equal(bt.run(workspace=ws), good) and bt.pool.errors() == 0
