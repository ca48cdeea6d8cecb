"""Shared-prefix decode attention where one key far above thousands of others
leaves its weight to a single token, and the output to the long tail: every
weight has to keep its relative precision, however small it is."""
import pytest
import torch

import step_reference as ref
from test_gpu_prefix import RAW, Batch

pytestmark = pytest.mark.gpu

TOKENS = 8192
SIZES = (1.0, 0.75, 0.875, 0.5)  # of the four query heads: gaps of that many times the largest


def _sink_batch(kv, unit, where, gap, noise, seed=1):
    """Keys c_t e with e = +-1: head h scores them scale * 128 * size_h * c_t.
    One key scores `gap` nats (for size 1), all others `noise` nats around 0;
    the values of the others are near 0.125, its own is 0."""
    if unit == "shared":
        bt = Batch((TOKENS + 70, TOKENS + 1, TOKENS), [(0, 3, TOKENS)], 4, 1, bs=64, kv=kv, seed=seed)
    else:
        bt = Batch((TOKENS, TOKENS - 37), [(0, 2, 0)], 4, 1, bs=64, kv=kv, seed=seed)
    g = torch.Generator().manual_seed(seed)
    e = torch.where(torch.rand(128, generator=g) < 0.5, -1.0, 1.0)
    per_nat = 1.0 / (bt.scale * 128)
    c = noise * per_nat * torch.randn(bt.k.shape[:3], generator=g)
    v = 0.125 + 0.05 * torch.randn(bt.v.shape, generator=g)
    at = {"first": 5, "middle": 4000, "last": TOKENS - 40}[where]
    for b in range(len(bt.lens)):
        blk = int(bt.tables[b, at // 64])
        c[blk, 0, at % 64] = gap * per_nat
        v[blk, 0, at % 64] = 0.0
    k = c[..., None] * e
    bt.k, bt.v = (((x / s).clamp(-448, 448) if kv == "fp8" else x).to(RAW[kv])
                  for x, s in ((k, bt.k_scale), (v, bt.v_scale)))
    for dst, src in ((bt.pool.k, bt.k), (bt.pool.v, bt.v)):
        dst[1].copy_(src.view(torch.uint8) if kv == "fp8" else src)
    bt.q = (torch.tensor(SIZES).view(1, 4, 1) * e).expand(len(bt.lens), 4, 128).contiguous().to(torch.bfloat16)
    return bt


def _bound(want, mass, kv):
    """|error| relative to what the weights really are.  A weight is rounded once,
    by half a step: 2^-8 of it in BF16, 2^-11 in FP16 (FP8 pools; the smallest here
    are 2^-21 of the largest, normal numbers there).  A score is a 128-term sum
    in fp32, off by at most 128 x 2^-24 of the magnitudes added, which are up to 14
    nats: 2^-13 of each weight, once above and once in the sum below.  2^x and the
    sums add less than 2^-18.  The output is rounded once to BF16."""
    half = ref.HALF[torch.bfloat16]
    weights = ((half if kv == "bf16" else 2.0 ** -11) + 2.0 ** -12 + 2.0 ** -17) * mass
    return weights + half * (want.abs() + weights)


@pytest.mark.parametrize("noise", [0.3, 0.0])
@pytest.mark.parametrize("gap", [8.0, 11.0, 13.0])
@pytest.mark.parametrize("where", ["first", "middle", "last"])
@pytest.mark.parametrize("unit", ["shared", "own"])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_tail_behind_one_key(kv, unit, where, gap, noise):
    bt = _sink_batch(kv, unit, where, gap, noise)
    out = bt.run(algo="tc").cpu().double()
    want, mass, _ = bt.reference()
    # (the tail counts: 8192 x 0.125 x e^-13, next to the key of weight 1, is 0.0023)
    assert (mass[:, 0] > 0.002).all()
    err, bound = (out - want).abs(), _bound(want, mass, kv)
    assert (err <= bound).all(), "off by up to %g of the bound, %g of the output" % (
        float((err / bound).max()), float((err / want.abs()).max()))
    assert bt.pool.errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_tail_in_another_piece_than_the_key(kv):
    """The key in a sequence's own tokens, the tail in its group's prefix."""
    bt = _sink_batch(kv, "shared", "first", 0.0, 0.3, seed=2)
    own = int(bt.tables[0, TOKENS // 64])  # sequence 0 has 70 tokens of its own
    raw = bt.pool.k[1, own, 0, 3]
    e = bt.q[0, 0].float()
    key = (e * 11.0 / (bt.scale * 128) / bt.k_scale).to(RAW[kv])
    bt.k[own, 0, 3] = key
    raw.copy_(key.view(torch.uint8) if kv == "fp8" else key)
    out = bt.run(algo="tc").cpu().double()
    want, mass, _ = bt.reference()
    assert ((out - want).abs() <= _bound(want, mass, kv)).all()
