"""GPU tests of decode attention over codes where magnitudes are far from one: values near the largest numbers, scores
far from zero, weights far below the largest one."""
import pytest
import torch

import quant_reference as ref
import quant_tight as tight
from paged_kv_cache_194_gb300 import binding as pk
from test_gpu_quant_cache import BF, Quantised
from test_gpu_quant_tight import put

pytestmark = pytest.mark.gpu

# a CTA a unit, cut units, a warp a unit; two steps at a time and one
SHAPES = [((300, 5), 8, 2, 128), ((6000, 40), 8, 2, 128), ((60,) * 200, 8, 2, 128), ((300, 5), 16, 2, 64),
          ((6000, 40), 16, 1, 128)]


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("lens,Hq,Hk,D", SHAPES, ids=str)
def test_value_rows_of_large_scales(bits, lens, Hq, Hk, D):
    """Scales above 2^104, which times the codes' 2^24 are past 32 bits, beside rows of small ones."""
    b = Quantised(lens, Hq, Hk, D, 16, bits, seed=80)
    g = torch.Generator().manual_seed(81)
    T = sum(lens)
    k = torch.randn(T, Hk, D, generator=g).to(BF)
    v = (torch.rand(T, Hk, D, generator=g) * 2 - 1) * 3e33
    v[torch.rand(T, generator=g) < 0.1] *= 1e-30
    v[torch.rand(T, generator=g) < 0.1] = 2e33  # (rows of one value: codes of zero)
    v[..., ::7] = 0
    put(b, k, v.to(BF))
    out = b.run()
    assert out.isfinite().all()
    tight.check(out, *tight.codes(b.q, b.pools(), b.tables, b.lens, b.scale, bits))


@pytest.mark.parametrize("bits", [4, 8])
def test_one_token_of_the_largest_values(bits):
    """A weight of one: the row itself, with a scale of up to 2^124."""
    b = Quantised((1, 1, 1), bits=bits, seed=82)
    g = torch.Generator().manual_seed(83)
    v = ((torch.rand(3, 2, 128, generator=g) - 0.5) * 3.3e38).to(BF)
    v[1] = 3e38
    put(b, v * 1e-38, v)
    p, c = b.pools()[3], b.pools()[2]
    blk = b.tables[:, 0].long()
    want = ref.values(c[blk, :, 0], p[blk, :, 0], bits).repeat_interleave(4, 1)
    err = (b.run().cpu().double() - want).abs()
    assert (err <= (2.0 ** -8 + 2.0 ** -10) * want.abs() + 2.0 ** -11 * 3.3e38).all()


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("wide", [-1e3, 1e5, -1e7, 1e9])
@pytest.mark.parametrize("lens,Hq,Hk,D", SHAPES, ids=str)
def test_scores_far_from_zero(bits, wide, lens, Hq, Hk, D):
    """Keys that are all alike, so that all weights are, with scores of up to 10^12 that leave no room for the
    logarithms of the values' scales: the mean of the values."""
    b = Quantised(lens, Hq, Hk, D, 16, bits, seed=84)
    g = torch.Generator().manual_seed(85)
    T = sum(lens)
    v = torch.randn(T, Hk, D, generator=g) * 10.0 ** torch.randint(-2, 3, (T, 1, 1), generator=g)
    put(b, (torch.randn(1, Hk, D, generator=g) + 1).expand(T, Hk, D).to(BF).contiguous(), v.to(BF))
    b.q = (torch.rand(b.q.shape, generator=g) * wide).to(BF)
    tight.check(b.run(), *tight.codes(b.q, b.pools(), b.tables, b.lens, 0.0, bits))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("lens,Hq,Hk,D", SHAPES, ids=str)
def test_scores_of_the_largest_magnitude(bits, sign, lens, Hq, Hk, D):
    """All scores at -10^36 (10^36): far below any that stands for no key."""
    b = Quantised(lens, Hq, Hk, D, 16, bits, seed=86)
    T = sum(lens)
    v = torch.randn(T, Hk, D, generator=torch.Generator().manual_seed(87)).to(BF)
    put(b, torch.full((T, Hk, D), 1e17).to(BF), v)
    b.q = torch.full(b.q.shape, sign * 1e18).to(BF)
    tight.check(b.run(), *tight.codes(b.q, b.pools(), b.tables, b.lens, 0.0, bits))


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("nats", [12.0, 17.7, 19.0])
def test_many_keys_far_below_one(bits, nats):
    """In each warp's part of a long unit one key outweighs each of the others by up to 2^27; together they matter all the
    same: values of 0 at the one (but for one element, which gives its row a scale), of 1 to 2 at the others."""
    L, B, Hk = 131072, 60, 8
    b = Quantised((L,), 4 * Hk, Hk, 128, 64, bits, seed=88)
    g = torch.Generator().manual_seed(89)
    k = (torch.randn(L, Hk, 128, generator=g) * 0.05).to(BF)
    v = (1 + torch.rand(L, Hk, 128, generator=g)).to(BF)
    v[..., 0] = 0  # (an offset of 0: the values are all in the codes)
    for t in range(L // 3, L // 3 + 64, 16):  # (four warps take 16 tokens each in turns)
        k[t], v[t], v[t, :, 0] = nats / 128 ** 0.5, 0, 2
    put(b, k, v)
    b.q = torch.ones_like(b.q)
    want, bound = tight.codes(b.q, b.pools(), b.tables, b.lens, b.scale, bits)
    b.q, b.tables, b.lens = (x.repeat_interleave(B, 0) for x in (b.q, b.tables, torch.tensor(b.lens)))  # (the same blocks)
    tight.check(b.run(), want.expand(B, -1, -1), bound.expand(B, -1, -1))


@pytest.mark.parametrize("bits,ratio", [(4, 27), (8, 31)])
@pytest.mark.parametrize("D", [64, 128])
def test_small_elements_of_a_query_row_count(bits, ratio, D):
    """Scores that depend on elements 2^-ratio of their row's largest alone, which meets codes of zero."""
    N = 2 ** bits - 1
    lens = (200, 3000)
    b = Quantised(lens, 4, 1, D, 16, bits, seed=92)
    g = torch.Generator().manual_seed(93)
    k = torch.randint(0, N + 1, (sum(lens), 1, D), generator=g).to(BF)
    k[..., 0], k[..., 1] = 0, N  # (an offset of 0, a scale of 1)
    put(b, k, torch.randn(k.shape, generator=g).to(BF))
    q = (1 + torch.rand(b.q.shape, generator=g)) * (torch.randint(0, 2, b.q.shape, generator=g) * 2 - 1) * 2.0 ** -ratio
    q[..., 0] = 1.0
    b.q, b.scale = q.to(BF), 2.0 ** ratio / (N * D ** 0.5)
    tight.check(b.run(), *tight.codes(b.q, b.pools(), b.tables, b.lens, b.scale, bits))
