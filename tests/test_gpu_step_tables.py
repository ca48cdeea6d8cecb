"""Tables and slots on the device: the same results on both sides of every size
at which another launch takes over."""
import numpy as np
import pytest
import torch

from paged_kv_cache_194_gb300 import binding as pk
from test_gpu_step import I32, _check_grow, _pool, dev, test_release_matches_a_walk as release_matches_a_walk

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_tokens", [6, 256, 257, 4096, 4097, 9000])
def test_grow_flags_and_rows_whatever_the_limit(max_tokens):
    """Bad lengths, counts, blocks and ring entries give the same rows, flags
    and tables however many rows the slot map has."""
    pool = _pool(32, 16)
    t = torch.full((7, 4), -1, dtype=I32)
    t[0, 0], t[2, :2], t[4, 0], t[5, 0] = 7, torch.tensor([8, 9], dtype=I32), 99, 3
    lens, new = [10, -3, 20, 65, 5, 16, 0], [2, 1, -1, 1, 0, 1, 2]
    t = t.cuda()
    got = pk.kv_tables_grow(pool, t, dev(lens), dev(new), dev([20, 32, 22, 23]), dev([0, 4]), max_tokens)
    # request 5 takes ring entry 20; request 6 entry 32, which is no block; its second row is past a limit of 6
    wide = max_tokens > 6
    assert pool.errors() == pk.ERRBIT_SEQ_LEN | pk.ERRBIT_STEP | (pk.ERRBIT_BLOCK_ID if wide else 0)
    assert got.granted.tolist() == [2, 0, 0, 0, 0, 1, 2 if wide else 0]
    assert got.seq_lens.tolist() == [12, -3, 20, 65, 5, 17, 2 if wide else 0]
    assert got.token_offsets.tolist() == [0, 2, 3, 3, 4, 4, 5, 7 if wide else 6]
    rows = 7 if wide else 6
    pad = max_tokens - rows
    assert got.slot_mapping.tolist() == [7 * 16 + 10, 7 * 16 + 11, -1, -1, 20 * 16, -1, -1][:rows] + [-1] * pad
    assert got.positions.tolist() == [10, 11, 0, 65, 16, 0, 1][:rows] + [0] * pad
    assert got.token_seqs.tolist() == [0, 0, 1, 3, 5, 6, 6][:rows] + [-1] * pad
    assert t[5].tolist() == [3, 20, -1, -1] and t[6].tolist() == [-1] * 4
    assert got.free_state.tolist() == ([2, 2] if wide else [1, 3])


@pytest.mark.parametrize("rows_more", [0, 1])
@pytest.mark.parametrize("B,rows", [(1, 256), (127, 256), (129, 258), (256, 512), (257, 514), (1024, 2048), (1025, 2050),
                                    (2048, 4096), (2049, 4096), (4096, 4096)])
def test_grow_at_the_borders_of_the_launches(B, rows, rows_more):
    """As many token rows as the scanning CTA still fills, and one more."""
    new = np.full(B, rows // B)
    new[:rows - int(new.sum())] += 1
    r = np.random.default_rng(B)
    bs, lens = 16, r.integers(0, 40, B)
    held, need = -(-lens // bs), -(-(lens + new) // bs) - -(-lens // bs)
    total = int((held + need).sum())
    order = r.permutation(total)
    width = int((held + need).max())
    tables = np.full((B, width), -1)
    at = 0
    for b in range(B):
        tables[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    t, T = dev(tables).reshape(tables.shape), rows + rows_more
    got = pk.kv_tables_grow(_pool(total, bs), t, dev(lens), dev(new), dev(order[at:]), dev([0, total - at]), T)
    t = t.cpu().numpy()
    seqs = np.repeat(np.arange(B), new)
    pos = np.concatenate([np.arange(L, L + n) for L, n in zip(lens, new)])
    slots = t[seqs, pos // bs] * bs + pos % bs
    assert sorted(t[t >= 0].tolist()) == list(range(total))
    assert t[:, 0].min() >= 0 and [int((x >= 0).sum()) for x in t] == (held + need).tolist()
    assert got.slot_mapping.tolist() == slots.tolist() + [-1] * rows_more
    assert got.positions.tolist() == pos.tolist() + [0] * rows_more
    assert got.token_seqs.tolist() == seqs.tolist() + [-1] * rows_more
    assert got.granted.tolist() == new.tolist() and got.free_state[1] == 0


@pytest.mark.parametrize("share", [1.0, 0.6])
@pytest.mark.parametrize("B,new_hi", [(30, 17), (200, 3), (250, 40)])
def test_grow_second_kernel_behind_the_small_scan(B, new_hi, share):
    _check_grow(B, 16, 200, new_hi, share, seed=B)
    _check_grow(B, 32, 200, new_hi, share, seed=B, in_place=True, extra_rows=600)


@pytest.mark.parametrize("B,width,finished", [(127, 40, 0.5), (128, 3000, 0.5), (129, 40, 0.5), (129, 3000, 1.0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_release_at_the_border_of_the_launches(B, width, finished, in_place):
    release_matches_a_walk(B, width, finished, in_place)
