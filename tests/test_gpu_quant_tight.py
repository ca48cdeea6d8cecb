"""GPU tests of attention over codes and over packed prompts in which a lost, doubled or misplaced token shows: bounds
that go by each key's weight, values that tell tokens apart, and single keys that outweigh all others."""
import pytest
import torch

import quant_reference as ref
import quant_tight as tight
from paged_kv_cache_194_gb300 import binding as pk
from test_gpu_prompt import case, offsets
from test_gpu_quant_cache import BF, Quantised, dev

pytestmark = pytest.mark.gpu

# one CTA a unit, cut, a warp a unit, empty ones between; groups of up to 4, 8, 16 and more heads
BATCHES = [((20000,), 8, 2, 128), ((5000, 1, 9000), 8, 2, 128), ((3000, 0, 1, 64, 2500, 700) * 4, 4, 1, 128),
           ((700, 300) * 9, 16, 2, 64), ((40,) * 200, 8, 2, 128), ((6000, 17), 16, 1, 128), ((2500, 2600, 5), 20, 1, 64),
           ((512, 16, 1024), 8, 1, 128), ((257,) * 30, 12, 4, 64)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lens,Hq,Hk,D", BATCHES, ids=lambda x: "%dx%d" % (len(x), max(x)) if isinstance(x, tuple) else str(x))
def test_codes(bits, lens, Hq, Hk, D):
    b = Quantised(lens, Hq, Hk, D, 16, bits, seed=70)
    tight.check(b.run(), *tight.codes(b.q, b.pools(), b.tables, b.lens, b.scale, bits))
    assert b.pool.errors() == 0


def put(b, k, v):
    """Rows [T, Hk, D] of all sequences, one after the other, in the places of b's tokens."""
    slots = torch.cat([b.tables[s].long()[torch.arange(n) // b.bs] * b.bs + torch.arange(n) % b.bs
                       for s, n in enumerate(b.lens)])
    pk.kv_quant_append(b.pool, 1, k.cuda(), v.cuda(), slots.cuda())


def marks(tokens, Hk, D, step):
    """Rows of 0 and a 1 whose place says which `step` tokens they are of, another one for each head."""
    v = torch.zeros(tokens, Hk, D)
    for h in range(Hk):
        v[torch.arange(tokens), h, (torch.arange(tokens) // step * 7 + 3 * h) % D] = 1
    return v.to(BF)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("step", [1, 16])
@pytest.mark.parametrize("lens,Hq,Hk,D", BATCHES, ids=lambda x: "%dx%d" % (len(x), max(x)) if isinstance(x, tuple) else str(x))
def test_every_token_counts_once(bits, step, lens, Hq, Hk, D):
    """All weights alike: an output says how many of the tokens have their mark there."""
    b = Quantised(lens, Hq, Hk, D, 16, bits, seed=71)
    v = torch.cat([marks(n, Hk, D, step) for n in lens])
    put(b, v, v)
    b.scale = 0.0
    want, bound = tight.codes(b.q, b.pools(), b.tables, b.lens, 0.0, bits)
    tight.check(b.run(), want, bound)


def dominant(b, targets, big=4.0):
    """Keys close to zero but for one in each sequence, values at random; what attention must give: the target's row."""
    g = torch.Generator().manual_seed(72)
    T, Hk, D = sum(b.lens), b.pool.num_kv_heads, b.pool.head_dim
    k = (torch.randn(T, Hk, D, generator=g) * 0.01).to(BF)
    v = torch.randn(T, Hk, D, generator=g).to(BF)
    at = torch.tensor(offsets(b.lens)[:-1]) + torch.tensor(targets)
    k[at] = big
    put(b, k, v)
    c, p = b.pools()[2:]
    blk, off = [], []
    for s, t in enumerate(targets):
        blk.append(int(b.tables[s, t // b.bs]))
        off.append(t % b.bs)
    rows = ref.values(c[blk, :, off], p[blk, :, off], b.bits)
    return rows.repeat_interleave(b.q.shape[1] // Hk, 1)


BORDERS = [0, 1, 15, 16, 31, 63, 64, 127, 128, 1023, 1024, 1535, 2047, 2048, 2559, 2990, 2991, 2998, 2999]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("Hq,Hk,D", [(4, 1, 128), (8, 1, 64), (16, 1, 128), (8, 2, 128)])
def test_one_key_outweighs_the_others(bits, Hq, Hk, D):
    """Each sequence's at another place; weights of the others are below 2^-40."""
    b = Quantised((3000,) * len(BORDERS), Hq, Hk, D, 16, bits, seed=73)
    b.q = torch.ones_like(b.q)
    want = dominant(b, BORDERS)
    err = (b.run().cpu().double() - want).abs()
    assert (err <= (2.0 ** -8 + 2.0 ** -10) * want.abs() + 2.0 ** -10 * 6).all(), float(err.max())


@pytest.mark.parametrize("bits", [4, 8])
def test_one_key_of_a_long_sequence_outweighs_the_others(bits):
    """The key wanders over places that ranges of the list, tiles and steps may end at."""
    b = Quantised((40000, 33000), 4, 1, 128, 32, bits, seed=74)
    b.q = torch.ones_like(b.q)
    want = dominant(b, [0, 0])
    c, p = b.pools()[2:]
    small = torch.full((1, 1, 128), 0.01, dtype=BF).cuda()
    big = torch.full((1, 1, 128), 4.0, dtype=BF).cuda()
    slot = lambda s, t: int(b.tables[s, t // 32]) * 32 + t % 32
    keep = b.pool.v_codes.clone(), b.pool.v_params.clone()
    last = [0, 0]
    for i in range(60):
        for s, n in ((0, 40000), (1, 33000)):
            pk.kv_quant_append(b.pool, 1, small, small, dev([slot(s, last[s])], torch.int64))
            last[s] = (i * 661 + (i % 3 - 1) + 64 * s) % n
            pk.kv_quant_append(b.pool, 1, big, big, dev([slot(s, last[s])], torch.int64))
        b.pool.v_codes.copy_(keep[0])
        b.pool.v_params.copy_(keep[1])
        out = b.run().cpu().double()
        for s in range(2):
            blk, off = slot(s, last[s]) // 32, slot(s, last[s]) % 32
            want = ref.values(c[blk, :, off], p[blk, :, off], bits)
            assert ((out[s] - want).abs() <= (2.0 ** -8 + 2.0 ** -10) * want.abs() + 2.0 ** -10 * 6).all(), (i, s)


# --------------------------------------------------------------------- prompts
PROMPTS = [((300, 513, 7), (300, 513, 7), 8, 2, 128), ((1,), (5000,), 8, 2, 128), ((300,), (8300,), 8, 2, 128),
           ((40, 7), (3000, 9001), 16, 1, 64), ((130, 0, 1, 64), (1500, 700, 2049, 64), 5, 1, 128),
           ((300,) * 4, (2300, 2300, 2301, 2150), 32, 8, 64), ((1025, 3), (1025, 3), 8, 8, 128),
           (tuple(range(60)), tuple(range(60)), 8, 4, 128), ((200, 3), (150, 4000), 8, 2, 64)]
ids = lambda x: "%dx%d" % (len(x), max(x)) if isinstance(x, tuple) else str(x)


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("q_lens,k_lens,Hq,Hk,D", PROMPTS, ids=ids)
def test_prompts(inp, q_lens, k_lens, Hq, Hk, D):
    cpu, gpu = case(q_lens, k_lens, Hq, Hk, D, inp, fused=False, seed=75)
    out = pk.prompt_attention(*gpu, dev(offsets(q_lens)), dev(offsets(k_lens)), D ** -0.5)
    tight.check(out, *tight.prompts(*cpu, q_lens, k_lens, D ** -0.5))


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("step", [1, 16])
@pytest.mark.parametrize("q_lens,k_lens,Hq,Hk,D", PROMPTS, ids=ids)
def test_every_key_counts_once(inp, step, q_lens, k_lens, Hq, Hk, D):
    (q, k, v), _ = case(q_lens, k_lens, Hq, Hk, D, inp, fused=False, seed=76)
    v = torch.cat([marks(m, Hk, D, step) for m in k_lens]).to(q.dtype)
    out = pk.prompt_attention(*[x.cuda() for x in (q, k, v)], dev(offsets(q_lens)), dev(offsets(k_lens)), 0.0)
    want, _ = tight.prompts(q, k, v, q_lens, k_lens, 0.0)
    # weights of 1: whole numbers' sums, one quotient, one rounding
    half = 2.0 ** -8 if inp == "bf16" else 2.0 ** -23
    err = (out.cpu().double() - want).abs()
    assert (err <= (half + 2.0 ** -22) * want).all(), float(err.max())


def picks(inp, q_lens, k_lens, Hq, Hk, D, wide=1.0):
    """Keys of signs, each query in the direction of one key that it sees, first, last and tiles' borders among them: q, k,
    v, and the output, which is that key's value."""
    g = torch.Generator().manual_seed(77)
    (q, k, v), _ = case(q_lens, k_lens, Hq, Hk, D, inp, fused=False, seed=78)
    k = (torch.randint(0, 2, k.shape, generator=g) * 2 - 1).to(k.dtype) * 2
    want = torch.zeros(q.shape, dtype=torch.float64)
    iq = ik = 0
    for n, m in zip(q_lens, k_lens):
        for i in range(n):
            sees = m - n + i + 1
            if sees <= 0:
                continue
            pick = torch.randint(0, sees, (Hq,), generator=g)
            border = [0, sees - 1, max(0, sees - 2), sees // 128 * 128 % sees, (sees // 128 * 128 - 1) % sees, 63 % sees,
                      64 % sees][i % 7]
            pick[i % Hq] = border
            j = ik + pick
            h = torch.arange(Hq) // (Hq // Hk)
            q[iq + i], want[iq + i] = k[j, h] * (8 * wide), v[j, h].double()
        iq, ik = iq + n, ik + m
    return q, k, v, want


def check_picks(inp, out, want):
    # The key's weight is 2^x with x within 8 of 0 (the base of weights need not be their maximum): BF16 rounds it for its
    # product with V by up to half a step, 2^-8, and the sum that the output is divided by is of weights that are not
    # rounded.  The output is rounded by as much again: (1 + 2^-8)^2 = 1 + 2^-7 + 2^-16, and the quotient's 2^-22.
    err = 2.0 ** -7 + 2.0 ** -16 + 2.0 ** -22 if inp == "bf16" else 2.0 ** -22
    assert ((out.cpu().double() - want).abs() <= err * want.abs()).all()


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("q_lens,k_lens,Hq,Hk,D", PROMPTS, ids=ids)
def test_every_query_picks_a_key(inp, q_lens, k_lens, Hq, Hk, D):
    # a key's own score is 32 D, another's 32 times a sum of D signs: at most 0.7 D of 10^4 keys and as many queries
    # (beyond ten standard deviations), so that others weigh less than 2^-100 with a scale of 1/4
    q, k, v, want = picks(inp, q_lens, k_lens, Hq, Hk, D)
    out = pk.prompt_attention(*[x.cuda() for x in (q, k, v)], dev(offsets(q_lens)), dev(offsets(k_lens)), 0.25)
    check_picks(inp, out, want)
