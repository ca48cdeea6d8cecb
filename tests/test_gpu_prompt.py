"""GPU tests of attention over packed prompts, and of the operators around the
quantised cache as a serving loop uses them."""
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


def offsets(n, first=0):
    return np.concatenate([[0], np.cumsum(n)]) + first


def case(q_lens, k_lens, Hq, Hk, D, inp, fused, seed=0, wide=1.0):
    g = torch.Generator().manual_seed(seed + sum(k_lens) + D)
    T, Tk = sum(q_lens), sum(k_lens)
    if fused:
        rows = (torch.randn(T, (Hq + 2 * Hk) * D, generator=g) * wide).to(DT[inp])
        d = rows.cuda()
        return tuple([x.unflatten(1, (-1, D)) for x in y.split([Hq * D, Hk * D, Hk * D], 1)] for y in (rows, d))
    x = [(torch.randn(t, h, D, generator=g) * wide).to(DT[inp]) for t, h in ((T, Hq), (Tk, Hk), (Tk, Hk))]
    return x, [y.cuda() for y in x]


def check(got, cpu, q_lens, k_lens, scale):
    want, bound = ref.prompt(*cpu, q_lens, k_lens, scale)
    err = (got.cpu().double() - want).abs()
    ok = err <= bound
    assert bool(ok.all()), (float(err.max()), int((~ok).sum()), ok.numel())


LENS = [(1,), (2,), (127,), (128,), (129,), (64, 1, 0, 31, 33, 32), (0, 0, 5), (300, 513, 7), tuple(range(40))]
HEADS = [(8, 2, 128), (4, 4, 128), (5, 1, 128), (3, 1, 64), (16, 2, 64), (12, 4, 128), (17, 1, 64), (64, 2, 128)]


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk,D", HEADS)
@pytest.mark.parametrize("lens", LENS, ids=lambda x: "%dx%d" % (len(x), max(x)))
def test_whole_prompts(inp, Hq, Hk, D, lens):
    cpu, gpu = case(lens, lens, Hq, Hk, D, inp, fused=True)
    err = torch.zeros(1, dtype=I32, device="cuda")
    o = dev(offsets(lens))
    out = pk.prompt_attention(*gpu, o, o, D ** -0.5, error_word=err)
    check(out, cpu, lens, lens, D ** -0.5)
    assert int(err) == 0


CHUNKS = [((1,), (1000,)), ((5, 3, 0, 70), (5, 300, 20, 71)), ((130, 200), (131, 900)), ((33, 1, 64), (500, 129, 128)),
          ((40, 10), (7, 0)), ((200,), (100,)), ((1, 1, 1), (127, 128, 129))]


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk,D", [(8, 2, 128), (3, 1, 64), (4, 4, 128)])
@pytest.mark.parametrize("q_lens,k_lens", CHUNKS, ids=str)
def test_chunks_behind_a_prefix(inp, Hq, Hk, D, q_lens, k_lens):
    """More keys than queries, and fewer (queries that see nothing get zero rows)."""
    cpu, gpu = case(q_lens, k_lens, Hq, Hk, D, inp, fused=False)
    out = pk.prompt_attention(*gpu, dev(offsets(q_lens)), dev(offsets(k_lens)), 0.11)
    check(out, cpu, q_lens, k_lens, 0.11)


@pytest.mark.parametrize("Hq,Hk,lens", [(32, 8, (1500, 40, 2047)), (8, 8, (1025, 3)), (16, 1, (700, 1100))])
def test_long_prompts(Hq, Hk, lens):
    cpu, gpu = case(lens, lens, Hq, Hk, 128, "bf16", fused=True, seed=3)
    o = dev(offsets(lens))
    first = pk.prompt_attention(*gpu, o, o, 128 ** -0.5)
    check(first, cpu, lens, lens, 128 ** -0.5)
    for _ in range(3):  # and bit for bit again
        assert torch.equal(pk.prompt_attention(*gpu, o, o, 128 ** -0.5), first)


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("scale,wide", [(0.0, 1.0), (-0.2, 1.0), (5.0, 1.0), (1e-4, 30.0), (0.3, 4.0)])
def test_scales(inp, scale, wide):
    lens = (200, 77)
    cpu, gpu = case(lens, lens, 4, 2, 128, inp, fused=True, seed=4, wide=wide)
    o = dev(offsets(lens))
    check(pk.prompt_attention(*gpu, o, o, scale), cpu, lens, lens, scale)


@pytest.mark.parametrize("inp", ["bf16", "f32"])
def test_rows_of_no_sequence(inp):
    """Padding between the sequences' rows holds NaN and infinities, and its output rows are left alone."""
    lens, pad = (70, 1, 130, 20), 9
    cpu, _ = case(lens, lens, 4, 2, 128, inp, fused=False, seed=5)
    starts = [sum(lens[:b]) + pad * (b + 1) for b in range(4)]
    rows = sum(lens) + pad * 5
    gpu = []
    for x, bad in zip(cpu, (float("nan"), float("inf"), float("nan"))):
        y = torch.full((rows,) + x.shape[1:], bad, dtype=x.dtype)
        for b, s in enumerate(starts):
            y[s:s + lens[b]] = x[sum(lens[:b]):sum(lens[:b + 1])]
        gpu.append(y.cuda())
    # one call for each sequence (rows in front and behind are others'), into one output
    out = torch.full_like(gpu[0], 77.0)
    for b, s in enumerate(starts):
        o = dev([s, s + lens[b]])
        pk.prompt_attention(*gpu, o, o, 0.1, out=out)
    there = torch.zeros(rows, dtype=torch.bool)
    for b, s in enumerate(starts):
        there[s:s + lens[b]] = True
    check(out[there.cuda()], cpu, lens, lens, 0.1)
    assert (out[~there.cuda()] == 77).all()


@pytest.mark.parametrize("inp", ["bf16", "f32"])
def test_values_that_are_not_finite_stay_with_their_sequence(inp):
    """A key that is not finite is seen only behind its place; a value reaches at most 255 positions more."""
    lens = (300, 300, 300)
    cpu, gpu = case(lens, lens, 4, 2, 128, inp, fused=False, seed=6)
    o = dev(offsets(lens))
    want = pk.prompt_attention(*gpu, o, o, 0.1)
    gpu[1][300 + 200, 0, 5] = float("nan")
    gpu[2][300 + 290, 1, 7] = float("inf")
    got = pk.prompt_attention(*gpu, o, o, 0.1)
    assert torch.equal(got[:300], want[:300]) and torch.equal(got[600:], want[600:])
    assert torch.equal(got[300:500, :2], want[300:500, :2])      # before the key, its heads
    assert got[500:600, :2].isnan().all()
    assert torch.equal(got[300:300 + 290 - 255, 2:], want[300:300 + 290 - 255, 2:])
    assert not got[590:600, 2:, 7].isfinite().any()


@pytest.mark.parametrize("inp", ["bf16", "f32"])
def test_offsets_that_cannot_be(inp):
    lens = (50, 60, 70)
    cpu, gpu = case(lens, lens, 4, 2, 128, inp, fused=False, seed=7)
    good = dev(offsets(lens))
    want = pk.prompt_attention(*gpu, good, good, 0.1)
    err = torch.zeros(1, dtype=I32, device="cuda")
    for bad, lost in (([0, 50, 110, 181], (110, 180)), ([-1, 50, 110, 180], (0, 50)), ([0, 50, 40, 40], (50, 180)),
                      ([0, 50, 2 ** 31 - 1, 180], (50, 180))):
        for q_bad in (True, False):
            out = torch.full_like(want, 77.0)
            o = (dev(bad), good) if q_bad else (good, dev(bad))
            if bad[1:3] == [50, 40]:
                o = (dev(bad), dev(bad))
            err.zero_()
            pk.prompt_attention(*gpu, *o, 0.1, out=out, error_word=err)
            assert int(err) == pk.ERRBIT_OFFSETS
            lo, hi = lost
            assert (out[lo:hi] == 77).all()
            keep = torch.ones(180, dtype=torch.bool, device="cuda")
            keep[lo:hi] = False
            assert torch.equal(out[keep], want[keep])
    # no error word: the same, unsaid
    out = torch.full_like(want, 77.0)
    pk.prompt_attention(*gpu, dev([0, 50, 110, 181]), good, 0.1, out=out)
    assert torch.equal(out[:110], want[:110]) and (out[110:] == 77).all()


@pytest.mark.parametrize("inp", ["bf16", "f32"])
def test_no_rows_and_no_sequences(inp):
    z = lambda t, h: torch.zeros(t, h, 128, dtype=DT[inp], device="cuda")
    assert pk.prompt_attention(z(0, 4), z(0, 2), z(0, 2), dev([0, 0]), dev([0, 0]), 1.0).shape == (0, 4, 128)
    out = torch.full((3, 4, 128), 5.0, dtype=DT[inp], device="cuda")
    pk.prompt_attention(z(3, 4), z(3, 2), z(3, 2), dev([0]), dev([0]), 1.0, out=out)
    pk.prompt_attention(z(3, 4), z(3, 2), z(3, 2), dev([1, 1, 1]), dev([0, 3, 3]), 1.0, out=out)
    assert (out == 5).all()
    # queries without keys: zero rows, also with no key rows at all
    pk.prompt_attention(z(3, 4), z(0, 2), z(0, 2), dev([0, 2]), dev([0, 0]), 1.0, out=out)
    assert (out[:2] == 0).all() and (out[2] == 5).all()


@pytest.mark.parametrize("inp", ["bf16", "f32"])
def test_captured_with_other_offsets_and_on_a_stream(inp):
    T = 400
    cpu, gpu = case((T,), (T,), 8, 2, 128, inp, fused=True, seed=8)
    o = dev([0, 100, 250, 400])
    out = torch.empty((T, 8, 128), dtype=DT[inp], device="cuda")
    ws = pk.prompt_attention_workspace(gpu[0], 3, 2)
    call = lambda **kw: pk.prompt_attention(*gpu, o, o, 0.1, out=out, workspace=ws, **kw)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for cuts in ([0, 100, 250, 400], [0, 0, 1, 400], [0, 400, 400, 400], [0, 128, 256, 400]):
        o.copy_(dev(cuts))
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        lens = np.diff(cuts).tolist()
        check(out, cpu, lens, lens, 0.1)
    side = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    call(stream=side)
    side.synchronize()
    check(out, cpu, lens, lens, 0.1)


# ------------------------------------------------------------------- all of them
@pytest.mark.parametrize("bits", [4, 8])
def test_prompts_then_decode_then_a_chunk_on_the_cached_rows(bits):
    """Prompts are attended and quantised into the cache, a few tokens are
    decoded over it (one step captured and replayed), then a second chunk of
    every request attends to the rows read back in front of its own."""
    g = torch.Generator().manual_seed(bits)
    Hq, Hk, D, bs, scale = 8, 2, 128, 16, 128 ** -0.5
    lens, B, steps = [37, 1, 130, 64], 4, 5
    width = 16
    nb = B * width
    pool = pk.QuantKVPool(1, nb, bs, Hk, D, bits, fill=0xFF)
    plain = pk.KVPool(1, nb, bs, Hk, D, "bf16")  # (tables and slots on the device go by a pool's geometry)
    tables = torch.full((B, width), -1, dtype=I32, device="cuda")
    ring, st, L = dev(np.random.default_rng(1).permutation(nb)), dev([0, nb]), dev([0] * B)
    grow = lambda n, T: pk.kv_tables_grow(plain, tables, L, dev(n), ring, st, T,
                                          out=pk.StepTables.empty(B, T)._replace(seq_lens=L, free_state=st))
    cut = lambda x: [y.unflatten(1, (-1, D)) for y in x.split([Hq * D, Hk * D, Hk * D], 1)]
    draw = lambda t: torch.randn(t, (Hq + 2 * Hk) * D, generator=g).to(BF).cuda()

    # the prompts
    T = sum(lens)
    step = grow(lens, T)
    q, k, v = cut(draw(T))
    out = pk.prompt_attention(q, k, v, step.token_offsets, step.token_offsets, scale)
    check(out, [x.cpu() for x in (q, k, v)], lens, lens, scale)
    pk.kv_quant_append(pool, 0, k, v, step.slot_mapping)

    # decode
    rows, attn = draw(B), torch.empty(B, Hq, D, dtype=BF, device="cuda")
    ws = pk.quant_decode_workspace(pool, B, Hq, width * bs)
    buf, one = pk.StepTables.empty(B, B)._replace(seq_lens=L, free_state=st), dev([1] * B)

    def decode():
        s = pk.kv_tables_grow(plain, tables, L, one, ring, st, B, out=buf)
        q, k, v = cut(rows)
        pk.kv_quant_append(pool, 0, k, v, s.slot_mapping)
        pk.paged_quant_decode_attention(q.contiguous(), pool, 0, tables, L, width * bs, scale, out=attn, workspace=ws)

    graph = None
    for i in range(steps):
        rows.copy_(draw(B))
        if i == 1:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                decode()
        graph.replay() if graph is not None else decode()
        now = [n + i + 1 for n in lens]
        assert L.tolist() == now
        pools = [x[0].cpu() for x in (pool.k_codes, pool.k_params, pool.v_codes, pool.v_params)]
        want, bound = ref.quant_attention(cut(rows)[0].cpu(), pools, tables.cpu(), now, scale, bits)
        assert ((attn.cpu().double() - want).abs() <= bound).all(), i

    # a second chunk: its rows go to the cache, and all of them are read back for its attention
    new, past = [20, 3, 0, 50], [n + steps for n in lens]
    T, now = sum(new), [a + b for a, b in zip(new, past)]
    step = grow(new, T)
    q, k, v = cut(draw(T))
    pk.kv_quant_append(pool, 0, k, v, step.slot_mapping)
    k_off = dev(offsets(now))
    kr, vr = pk.kv_read(pool, 0, tables, k_off, sum(now))
    out = pk.prompt_attention(q, kr, vr, step.token_offsets, k_off, scale)
    check(out, [x.cpu() for x in (q, kr, vr)], new, now, scale)
    # the rows read back are what the codes stand for
    pools = [x[0].cpu() for x in (pool.k_codes, pool.k_params, pool.v_codes, pool.v_params)]
    for rows_back, c, p in ((kr, pools[0], pools[1]), (vr, pools[2], pools[3])):
        at = 0
        for b, n in enumerate(now):
            t = torch.arange(n)
            blk = tables[b].cpu().long()[t // bs]
            want = ref.values(c[blk, :, t % bs], p[blk, :, t % bs], bits)
            err = (rows_back[at:at + n].cpu().double() - want).abs()
            assert (err <= (2.0 ** -8 + 2.0 ** -23) * want.abs()).all()
            at += n
    assert pool.errors() == 0 and plain.errors() == 0


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("Hq,Hk", [(130, 1), (128, 1), (3, 3)])
def test_many_sequences_and_many_heads(inp, Hq, Hk):
    """Past what the tensor-core design plans for: more than 128 query heads to a KV head, more than 2048 sequences."""
    g = torch.Generator().manual_seed(Hq)
    lens = torch.randint(0, 4, (2100,), generator=g).tolist() if Hq == 3 else [5, 0, 70, 129]
    lens[1], lens[-1] = 0, 131
    cpu, gpu = case(lens, lens, Hq, Hk, 64, inp, fused=True, seed=30)
    o = dev(offsets(lens))
    err = torch.zeros(1, dtype=I32, device="cuda")
    check(pk.prompt_attention(*gpu, o, o, 0.125, error_word=err), cpu, lens, lens, 0.125)
    assert int(err) == 0
    o[-2:] += 1  # (the last sequence now ends behind the rows)
    pk.prompt_attention(*gpu, o, o, 0.125, error_word=err)
    assert int(err) == pk.ERRBIT_OFFSETS


@pytest.mark.parametrize("lens", [(20,) * 250, (20,) * 300, (1,) * 2048], ids=lambda x: "%dx%d" % (len(x), max(x)))
def test_as_many_sequences_as_are_planned(lens):
    cpu, gpu = case(lens, lens, 8, 4, 128, "bf16", fused=False, seed=31)
    o = dev(offsets(lens))
    check(pk.prompt_attention(*gpu, o, o, 0.1), cpu, lens, lens, 0.1)


def test_two_graphs_share_a_workspace_and_two_streams_do_not():
    g = []
    ws = pk.prompt_attention_workspace(torch.zeros(1264, 8, 128, dtype=BF, device="cuda"), 3, 2)
    for seed, lens in ((32, (700, 3)), (33, (64, 200, 1000))):
        cpu, gpu = case(lens, lens, 8, 2, 128, "bf16", fused=True, seed=seed)
        o = dev(offsets(lens))
        out = pk.prompt_attention(*gpu, o, o, 0.1, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            pk.prompt_attention(*gpu, o, o, 0.1, out=out, workspace=ws)
        g.append((graph, out, cpu, gpu, o, lens))
    for _ in range(3):
        for graph, out, *_ in g:
            out.fill_(9.0)
            graph.replay()
        torch.cuda.synchronize()
        for _, out, cpu, _, _, lens in g:
            check(out, cpu, lens, lens, 0.1)
    assert (ws[:256] == 0).all()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    own = [pk.prompt_attention_workspace(x[3][0], len(x[5]), 2) for x in g]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, (_, out, _, gpu, o, _) in enumerate(g):
            pk.prompt_attention(*gpu, o, o, 0.1, out=out, workspace=own[i], stream=side[i])
    torch.cuda.synchronize()
    for _, out, cpu, _, _, lens in g:
        check(out, cpu, lens, lens, 0.1)


def test_scores_that_rise_tile_by_tile():
    """Each tile's scores are far above (and below) the tile's before: the base of the weights moves at every tile, by
    more than the weights' range, in some rows of a warp and in one half of a tile's keys."""
    lens, D = (900,), 128
    cpu, _ = case(lens, lens, 4, 1, D, "bf16", fused=False, seed=34)
    q, k, v = cpu
    q[..., 0] = 8.0
    steps = torch.arange(900) // 64
    for up in (steps.float() * 20, (14 - steps).float() * 20, (steps % 3).float() * 30, (steps == 9).float() * 400):
        k[:, 0, 0] = up.to(BF)
        for rows in (slice(None), slice(0, 900, 2)):
            qq = q.clone()
            qq[rows, :, 0] = -8.0 if rows != slice(None) else 8.0
            gpu = [x.cuda() for x in (qq, k, v)]
            o = dev(offsets(lens))
            check(pk.prompt_attention(*gpu, o, o, 1.0), (qq, k, v), lens, lens, 1.0)


PIECES = [((1,), (5000,)), ((300,), (8300,)), ((40, 7), (3000, 9001)), ((130, 0, 1, 64), (1500, 700, 2049, 64)),
          ((200, 3), (150, 4000)), ((1,), (512,)), ((1,), (513,)), ((2000,), (2000,))]


@pytest.mark.parametrize("Hq,Hk,D", [(8, 2, 128), (5, 1, 128), (16, 1, 64), (128, 1, 128)])
@pytest.mark.parametrize("q_lens,k_lens", PIECES, ids=str)
def test_few_queries_behind_long_prefixes(Hq, Hk, D, q_lens, k_lens):
    """Fewer units than SMs: their keys are cut into pieces, which are joined in one order."""
    cpu, gpu = case(q_lens, k_lens, Hq, Hk, D, "bf16", fused=False, seed=40)
    qo, ko = dev(offsets(q_lens)), dev(offsets(k_lens))
    ws = pk.prompt_attention_workspace(gpu[0], len(q_lens), Hk)
    out = pk.prompt_attention(*gpu, qo, ko, D ** -0.5, workspace=ws)
    check(out, cpu, q_lens, k_lens, D ** -0.5)
    for _ in range(3):
        assert torch.equal(pk.prompt_attention(*gpu, qo, ko, D ** -0.5, workspace=ws), out)


def test_pieces_whose_scores_are_far_apart():
    """Pieces that weigh nothing next to others, keys and values that are not finite behind what a query sees."""
    q_lens, k_lens = (70,), (6000,)
    (q, k, v), _ = case(q_lens, k_lens, 8, 2, 128, "bf16", fused=False, seed=41)
    q[..., 0] = 8.0
    o = [dev(offsets(x)) for x in (q_lens, k_lens)]
    for at in (0, 700, 3100, 5900):
        k[:, :, 0] = 0
        k[at:at + 50, :, 0] = 60.0
        check(pk.prompt_attention(*[x.cuda() for x in (q, k, v)], *o, 1.0), (q, k, v), q_lens, k_lens, 1.0)
    want = pk.prompt_attention(*[x.cuda() for x in (q, k, v)], *o, 1.0)
    k[5999, 1] = float("nan")
    got = pk.prompt_attention(*[x.cuda() for x in (q, k, v)], *o, 1.0)
    assert torch.equal(got[:69], want[:69]) and got[69, 4:].isnan().all() and torch.equal(got[69, :4], want[69, :4])


def test_captured_from_whole_units_to_pieces_and_back():
    Tq, Tk = 3000, 9000
    cpu, gpu = case((Tq,), (Tk,), 8, 2, 128, "bf16", fused=False, seed=42)
    qo, ko = dev([0, 1000, 2000, 3000]), dev([0, 3000, 6000, 9000])
    out = torch.empty(Tq, 8, 128, dtype=BF, device="cuda")
    ws = pk.prompt_attention_workspace(gpu[0], 3, 2)
    call = lambda: pk.prompt_attention(*gpu, qo, ko, 0.1, out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for q_cuts, k_cuts in (([0, 1000, 2000, 3000], [0, 3000, 6000, 9000]), ([0, 20, 20, 21], [0, 8000, 8000, 9000]),
                           ([0, 0, 3000, 3000], [0, 0, 3000, 3000]), ([0, 3, 6, 9], [0, 3000, 3001, 9000])):
        qo.copy_(dev(q_cuts))
        ko.copy_(dev(k_cuts))
        out.fill_(9.0)
        graph.replay()
        torch.cuda.synchronize()
        n, m = np.diff(q_cuts).tolist(), np.diff(k_cuts).tolist()
        check(out[:q_cuts[-1]], [x[:t] for x, t in zip(cpu, (q_cuts[-1], k_cuts[-1], k_cuts[-1]))], n, m, 0.1)
        assert (out[q_cuts[-1]:] == 9).all()


@pytest.mark.parametrize("Hq,Hk,D,q_lens,k_lens", [
    (32, 8, 64, (300,) * 4, (2300, 2300, 2301, 2150)),     # 160 units on 152 SMs: a round, and eight in pieces
    (32, 8, 128, (1290,), (5100,)),                        # the units of one sequence: some whole, some not
    (16, 16, 64, (130,) * 10 + (70,) * 3, (1500,) * 12 + (1000,)),
    (32, 8, 64, (2600,), (8000,)), (5, 1, 64, (4100, 3), (12500, 1200))], ids=str)
def test_units_behind_the_last_full_round(Hq, Hk, D, q_lens, k_lens):
    cpu, gpu = case(q_lens, k_lens, Hq, Hk, D, "bf16", fused=False, seed=43)
    qo, ko = dev(offsets(q_lens)), dev(offsets(k_lens))
    ws = pk.prompt_attention_workspace(gpu[0], len(q_lens), Hk)
    out = pk.prompt_attention(*gpu, qo, ko, D ** -0.5, workspace=ws)
    check(out, cpu, q_lens, k_lens, D ** -0.5)
    assert torch.equal(pk.prompt_attention(*gpu, qo, ko, D ** -0.5, workspace=ws), out)


def test_sequences_that_overlap_are_not_counted_past_their_rows():
    """Offsets that go back and forth: half of the sequences ascend and are the same rows, more queries together than
    there are rows.  Their units would not be countable in 32 bits in a large call: none is taken."""
    T, B = 64, 300
    cpu, gpu = case((T,), (T,), 128, 1, 64, "bf16", fused=False, seed=44)
    o = dev([0, T] * (B // 2) + [0])
    err = torch.zeros(1, dtype=I32, device="cuda")
    out = torch.full_like(gpu[0], 77.0)
    ws = pk.prompt_attention_workspace(gpu[0], B, 1)
    pk.prompt_attention(*gpu, o, o, 0.1, out=out, error_word=err, workspace=ws)
    assert int(err) == pk.ERRBIT_OFFSETS and (out == 77).all() and not ws[:65536].any()
    o = dev([0, T] + [T] * (B - 1))  # and right offsets again
    err.zero_()
    pk.prompt_attention(*gpu, o, o, 0.1, out=out, error_word=err, workspace=ws)
    check(out, cpu, (T,), (T,), 0.1)
    assert int(err) == 0
