"""Shared-prefix decode attention at the limits of its plan: more sequences and
groups than the caches of a CTA hold, ranges that pass thousands of sequences
with no tiles of their own; which design takes which batch."""
import time

import pytest
import torch

import step_reference as ref
from paged_kv_cache_194_gb300 import binding as pk
from test_gpu_prefix import SHAPES, Batch

pytestmark = pytest.mark.gpu


def _check(bt, algo="tc"):
    out = bt.run(algo=algo).cpu().double()
    want, mass, floor = ref.attention(bt.q.cuda(), bt.k.cuda(), bt.v.cuda(), bt.tables, bt.lens, bt.scale, bt.k_scale,
                                      bt.v_scale)
    bad = ~((out - want).abs() <= ref.attention_bound(want, mass, bt.kv, floor))
    assert not bad.any(), bad.nonzero()[:4].tolist()
    for b, n in enumerate(bt.lens):
        if n == 0:
            assert (out[b] == 0).all()
    assert bt.pool.errors() == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("B,G", [(1024, 128), (1025, 129), (1025, 1), (1500, 512), (2500, 300), (4096, 512), (4096, 1), (4096, 128)])
def test_prefix_many_sequences_and_groups(B, G, kv):
    """Groups of no, one and many members, sequences of no length, of their
    prefix alone and with tokens of their own."""
    g = torch.Generator().manual_seed(B + G)
    cuts = torch.randint(0, B + 1, (G - 1,), generator=g).sort().values.tolist()
    offsets = [0] + cuts + [B]
    prefix = (torch.randint(0, 3, (G,), generator=g) * 64 + torch.randint(0, 20, (G,), generator=g)).tolist()
    own = torch.randint(0, 90, (B,), generator=g) * (torch.rand(B, generator=g) < 0.5)
    none = torch.rand(B, generator=g) < 0.05
    groups = [(offsets[i], offsets[i + 1], prefix[i]) for i in range(G)]
    lens = [0 if none[b] else p + int(own[b]) for first, last, p in groups for b in range(first, last)]
    bt = Batch(tuple(lens), groups, 2, 1, bs=32, kv=kv, seed=B, offsets=offsets, prefix=prefix)
    _check(bt)


@pytest.mark.parametrize("prefix", [640, 704, 1280])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_ranges_over_thousands_of_sequences_without_own_tiles(kv, prefix):
    """One range holds own tiles of the first and of the last sequences, or
    begins among the shared ones, with four thousand empty places between."""
    B, tail = 4096, 6
    lens = [prefix] * B
    lens[0], lens[1], lens[B - tail - 1] = prefix + 10, prefix + 1, prefix + 100
    lens[B - tail:] = [70, 0, 64, 1, 130, 65]
    _check(Batch(tuple(lens), [(0, B - tail, prefix)], 2, 1, bs=64, kv=kv, seed=prefix))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_groups_behind_the_cache_share(kv):
    """Two hundred groups of five, all of them with shared and own tiles."""
    G, n = 200, 5
    groups = [(n * i, n * i + n, 64 * (1 + i % 3)) for i in range(G)]
    lens = tuple(64 * (1 + b // n % 3) + (0, 1, 64, 30, 65)[b % n] for b in range(G * n))
    _check(Batch(lens, groups, 4, 1, bs=16, kv=kv, seed=3))


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("q_heads,kv_heads", [(1, 1), (8, 8), (5, 1), (12, 4), (16, 2), (40, 1), (64, 2), (128, 1)])
def test_prefix_groups_take_the_sharing_design(q_heads, kv_heads, kv):
    """No head count within the limits may be refused or left to another design."""
    for bs in (16, 32, 64):
        pool = pk.KVPool(1, 4, bs, kv_heads, 128, kv)
        for seqs, groups, longest in ((1, 1, 64), (6, 2, 700), (4096, 512, 131072)):
            for algo in ("auto", "tc"):
                assert pk.prefix_decode_algo(pool, seqs, groups, q_heads, longest, algo) == "tc"


@pytest.mark.parametrize("shape", [s for s in SHAPES if SHAPES[s][1]], ids=str)
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_shapes_take_the_sharing_design(shape, kv):
    lens, groups = SHAPES[shape]
    assert Batch(lens, groups, kv=kv).design() == "tc"


@pytest.mark.parametrize("q_heads", [2, 8, 14, 16, 40, 128])
@pytest.mark.parametrize("kv", ["bf16", "fp8"])
def test_prefix_without_groups(kv, q_heads):
    """Nothing to share: over FP8 pools calls of less than 8 query heads per KV
    head are decode attention, bit for bit; asked for by name, and for more
    heads, the sharing design takes them."""
    bt = Batch((900, 1, 0, 64, 2000), [], q_heads, 2, kv=kv, seed=6)
    left = kv == "fp8" and q_heads < 16
    assert bt.design() == ("mma" if left else "tc") and bt.design("tc") == "tc"
    if left:
        assert torch.equal(bt.run(), bt.run(algo="mma"))
    _check(bt)


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("cta", [0, 1, 151, 152, 303, -1])
def test_prefix_expired_waits_in_many_segments(kv, cta):
    """A CTA with several segments of several tiles gives up at its first tile:
    all of its roles leave, whatever is still to come in its range."""
    lens = tuple(600 + 37 * (i % 11) for i in range(56))
    bt = Batch(lens, [(0, 30, 320), (30, 56, 448)], 16, 8, bs=64, seed=40, kv=kv)
    ws = pk.prefix_decode_workspace(bt.pool, len(lens), 2, 16, bt.max_len)
    good = bt.run(workspace=ws)
    try:
        pk.set_first_wait_limit_for_testing(0, cta)
        t0 = time.perf_counter()
        out = bt.run(workspace=ws)
        torch.cuda.synchronize()
        took = time.perf_counter() - t0
    finally:
        pk.set_first_wait_limit_for_testing(-1)
    assert took < 5.0 and bt.pool.errors() == pk.ERRBIT_TIMEOUT
    lost = torch.isnan(out).any(2)
    assert torch.isnan(out[lost]).all() and torch.equal(out[~lost], good[~lost])
    assert lost.all() if cta < 0 else lost.any() and not lost.all()
    bt.pool.clear_errors()
    assert torch.equal(bt.run(workspace=ws), good) and bt.pool.errors() == 0
