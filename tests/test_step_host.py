"""Refusals of the serving-step operators, without a GPU: every call here is
rejected on the host before anything is enqueued."""
import ctypes

import pytest
import torch

from paged_kv_cache_194_gb300 import binding as pk

FAKE = 0x100000  # aligned, never dereferenced
P = ctypes.c_void_p


@pytest.fixture()
def pool():
    handles = []

    def make(**kw):
        d = dict(num_layers=1, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=128, kv_dtype=1, k_scale=1.0,
                 v_scale=1.0, k_base=FAKE, v_base=FAKE, error_word=None)
        d.update(kw)
        h = ctypes.c_void_p()
        assert pk.lib().kv_pool_create(ctypes.byref(pk.PoolDesc(**d)), ctypes.byref(h)) == 0
        handles.append(h)
        return h

    yield make
    for h in handles:
        pk.lib().kv_pool_destroy(h)


def test_prefix_attention_refusals(pool):
    h = pool()
    ws = ctypes.c_size_t()
    assert pk.lib().paged_prefix_decode_plan(h, 2, 1, 8, 64, ctypes.byref(ws)) == 0 and ws.value > 0

    def call(**k):
        return pk.lib().paged_prefix_decode_attention(
            P(k.get("q", FAKE)), k.get("dt", 1), k.get("h", h), k.get("layer", 0), P(k.get("t", FAKE)), k.get("mb", 4),
            P(k.get("lens", FAKE)), k.get("B", 2), k.get("Hq", 8), k.get("maxlen", 64), P(k.get("off", FAKE)),
            P(k.get("pre", FAKE)), k.get("G", 1), k.get("scale", 0.1), k.get("algo", 0), P(k.get("ws", FAKE)),
            k.get("wsb", ws.value), P(k.get("out", FAKE)), None)

    assert call(h=None) == 1
    assert call(layer=1) == 1 and call(layer=-1) == 1
    assert call(q=None) == 1 and call(q=FAKE + 2) == 1 and call(out=None) == 1 and call(out=FAKE + 8) == 1
    assert call(t=None) == 1 and call(lens=None) == 1 and call(lens=FAKE + 2) == 1
    assert call(off=None) == 1 and call(pre=None) == 1 and call(off=FAKE + 1) == 1
    assert call(G=-1) == 1 and call(B=-1) == 1 and call(Hq=0) == 1 and call(Hq=7) == 1
    assert call(maxlen=65) == 1 and call(maxlen=-1) == 1 and call(mb=0) == 1
    assert call(scale=float("nan")) == 1 and call(algo=9) == 1
    assert call(dt=0) == 2
    assert call(B=0) == 0
    if pk.lib().paged_prefix_decode_algo(h, 2, 1, 8, 64, 0) > 0:
        assert call(ws=None) == 3 and call(wsb=ws.value - 1) == 3 and call(ws=FAKE + 16) == 3
    # what the sharing design does not serve, asked for by name
    assert call(h=pool(kv_dtype=0), dt=0, algo=3) == 2
    assert call(h=pool(head_dim=64), algo=3) == 2
    assert pk.lib().paged_prefix_decode_algo(h, 4097, 1, 8, 64, 3) == -1
    assert pk.lib().paged_prefix_decode_algo(h, 2, 513, 8, 64, 3) == -1
    assert pk.lib().paged_prefix_decode_algo(h, 2, 1, 2 * 129, 64, 3) == -1
    assert pk.lib().paged_prefix_decode_algo(h, 4096, 1, 8, 2 ** 31 - 1, 3) == -1
    assert pk.lib().paged_prefix_decode_algo(None, 2, 1, 8, 64, 0) == -1
    assert pk.lib().paged_prefix_decode_plan(h, 2, -1, 8, 64, ctypes.byref(ws)) == 1
    assert pk.lib().paged_prefix_decode_plan(None, 2, 1, 8, 64, ctypes.byref(ws)) == 1


def test_prefix_workspace_covers_decode_attention(pool):
    """A workspace of the plan also serves decode attention, and grows with
    everything it is sized by."""
    h = pool()
    size = lambda *a: (lambda w: (pk.lib().paged_prefix_decode_plan(h, *a, ctypes.byref(w)), w.value)[1])(ctypes.c_size_t())
    w = ctypes.c_size_t()
    assert pk.lib().paged_decode_plan(h, 64, 8, 64, 0, None, None, ctypes.byref(w)) == 0
    assert size(64, 1, 8, 64) >= w.value
    assert size(64, 1, 8, 64) < size(128, 1, 8, 64) and size(64, 1, 8, 64) < size(64, 1, 16, 64)
    assert size(64, 1, 8, 64) < size(64, 65, 8, 64)


def _rope(**kw):
    d = dict(cos_sin=FAKE, max_pos=64, rotary_dim=128, interleaved=0, num_axes=1, q_weight=None, k_weight=None,
             weight_dtype=0, eps=1e-6)
    sections = kw.pop("sections", (64, 0, 0))
    d.update(kw)
    r = pk.NormRopeDesc(**d)
    for i, n in enumerate(sections):
        r.sections[i] = n
    return r


def test_norm_rope_refusals(pool):
    h = pool()
    Q, K, V, O = FAKE, 2 * FAKE, 3 * FAKE, 4 * FAKE

    def call(**k):
        rope = k["rope"] if "rope" in k else _rope()
        return pk.lib().kv_append_norm_rope(
            k.get("h", h), k.get("layer", 0), P(k.get("q", Q)), P(k.get("k", K)), P(k.get("v", V)), k.get("dt", 1),
            k.get("qs", 1024), k.get("ks", 256), k.get("vs", 256), P(k.get("pos", FAKE)), P(k.get("slots", FAKE)),
            k.get("T", 4), k.get("Hq", 8), ctypes.byref(rope) if rope is not None else None, P(k.get("out", O)), None)

    assert call(T=0) == 0
    assert call(h=None) == 1 and call(rope=None) == 1 and call(layer=1) == 1 and call(T=-1) == 1 and call(Hq=0) == 1
    assert call(dt=2) == 1 and call(h=pool(kv_dtype=0), dt=1) == 2
    for n in ("q", "k", "v", "pos", "slots", "out"):
        assert call(**{n: None}) == 1, n
    for n, p in (("q", Q), ("k", K), ("v", V), ("out", O)):
        assert call(**{n: p + 8}) == 1, n
    assert call(pos=FAKE + 2) == 1 and call(slots=FAKE + 4) == 1
    for n in ("qs", "ks", "vs"):
        assert call(**{n: -8}) == 1 and call(**{n: 1028}) == 1 and call(**{n: 2 ** 62}) == 1
    for bad in (dict(rotary_dim=0, sections=(0, 0, 0)), dict(rotary_dim=144, sections=(72, 0, 0)),
                dict(rotary_dim=24, sections=(12, 0, 0)), dict(max_pos=0), dict(interleaved=2), dict(num_axes=0),
                dict(num_axes=4), dict(sections=(63, 0, 0)), dict(num_axes=2, sections=(65, -1, 0)),
                dict(cos_sin=None), dict(cos_sin=FAKE + 4), dict(q_weight=FAKE), dict(k_weight=FAKE),
                dict(q_weight=FAKE, k_weight=FAKE, weight_dtype=2), dict(q_weight=FAKE, k_weight=FAKE, eps=0.0),
                dict(q_weight=FAKE, k_weight=FAKE, eps=1e-40), dict(q_weight=FAKE, k_weight=FAKE, eps=-1e-6),
                dict(q_weight=FAKE, k_weight=FAKE, eps=float("inf")), dict(q_weight=FAKE + 4, k_weight=FAKE)):
        assert call(rope=_rope(**bad)) == 1, bad
    # overlap of the output with an input, but for q itself laid out alike
    assert call(out=Q + 16) == 1 and call(out=K) == 1 and call(out=V - 16) == 1
    assert call(out=Q, qs=1032) == 1
    assert call(out=Q, dt=0) == 1  # fp32 rows into BF16 ones in place


def test_tables_refusals(pool):
    h = pool()

    def grow(**k):
        g = lambda n: P(k.get(n, FAKE))
        return pk.lib().kv_tables_grow(k.get("h", h), g("t"), k.get("mb", 4), g("lens"), g("new"), k.get("B", 2),
                                       g("ring"), k.get("size", 8), g("st"), k.get("T", 4), g("slots"), g("pos"),
                                       g("seqs"), g("off"), g("granted"), g("lo"), g("so"), None)

    def release(**k):
        g = lambda n: P(k.get(n, FAKE))
        return pk.lib().kv_tables_release(k.get("h", h), g("t"), k.get("mb", 4), g("lens"), g("done"), g("keep"),
                                          k.get("B", 2), g("ring"), k.get("size", 8), g("st"), g("lo"), g("so"), None)

    for f, names in ((grow, ("t", "lens", "new", "ring", "st", "slots", "pos", "seqs", "off", "granted", "lo", "so")),
                     (release, ("t", "lens", "done", "ring", "st", "lo", "so"))):
        assert f(h=None) == 1 and f(mb=0) == 1 and f(size=0) == 1 and f(B=-1) == 1
        assert f(mb=2 ** 31 // 16) == 2  # positions past 2^31 - 1
        assert f(size=2 ** 30 + 1) == 2
        for n in names:
            assert f(**{n: None}) == 1, n
            assert f(**{n: FAKE + (4 if n == "slots" else 2)}) == 1, n
    assert grow(T=-1) == 1 and release(keep=FAKE + 2) == 1 and grow(T=2 ** 30 + 1) == 2


def test_binding_checks_shapes_types_and_devices():
    pool = pk.KVPool(1, 8, 16, 2, 128, "bf16", device="cpu")
    z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)
    bf = torch.bfloat16
    rope = pk.RopeTable.create(16, 128, device="cpu")
    q, k, v = z(4, 8, 128, dtype=bf), z(4, 2, 128, dtype=bf), z(4, 2, 128, dtype=bf)
    good = dict(q=q, k=k, v=v, positions=z(4), slot_mapping=z(4, dtype=torch.int64), rope=rope)
    for bad in (dict(q=z(4, 8, 64, dtype=bf)), dict(k=z(4, 3, 128, dtype=bf)), dict(v=z(5, 2, 128, dtype=bf)),
                dict(k=k.float()), dict(positions=z(5)), dict(positions=z(2, 4)), dict(positions=z(4, dtype=torch.int64)),
                dict(slot_mapping=z(4)), dict(q=q.transpose(0, 1).contiguous().transpose(0, 1)),
                dict(q=z(4, 8, 256, dtype=bf)[..., ::2]), dict(q_weight=torch.ones(128)),
                dict(q_weight=torch.ones(64), k_weight=torch.ones(64)),
                dict(q_weight=torch.ones(128), k_weight=torch.ones(128, dtype=bf)),
                dict(out=z(4, 8, 128, dtype=torch.float32)), dict(q=q.to("meta"))):
        with pytest.raises(ValueError):
            pk.kv_append_norm_rope(pool, 0, **{**good, **bad})
    for args in ((torch.zeros(4, 128), (63,)), (torch.zeros(4, 128), (16, 16, 16, 16)), (torch.zeros(4, 128), (65, -1)),
                 (torch.zeros(4, 128, dtype=torch.float64), None), (torch.zeros(128), None)):
        with pytest.raises(ValueError):
            pk.RopeTable(*args)
    t, n = z(3, 4), z(3)
    for bad in (dict(block_tables=z(2, 4)), dict(block_tables=t.long()), dict(seq_lens=n.long()), dict(new_tokens=z(2)),
                dict(free_state=z(3)), dict(free_ring=z(8)[::2]), dict(block_tables=z(4, 3).T)):
        with pytest.raises(ValueError):
            pk.kv_tables_grow(**{**dict(pool=pool, block_tables=t, seq_lens=n, new_tokens=n, free_ring=z(8),
                                        free_state=z(2), max_tokens=5), **bad})
    for bad in (dict(finished=n.bool()), dict(keep_blocks=z(2)), dict(seq_lens_out=z(2)), dict(block_tables=z(3))):
        with pytest.raises(ValueError):
            pk.kv_tables_release(**{**dict(pool=pool, block_tables=t, seq_lens=n, finished=n, free_ring=z(8),
                                           free_state=z(2)), **bad})
    qa = z(3, 8, 128, dtype=bf)
    for bad in (dict(group_offsets=z(3)), dict(seq_lens=z(2)), dict(block_tables=z(2, 4)), dict(out=qa[:2]),
                dict(prefix_lens=z(1, dtype=torch.int64)), dict(q=z(3, 8, 64, dtype=bf)),
                dict(q=z(8, 3, 128, dtype=bf).transpose(0, 1)),
                dict(workspace=torch.zeros(8, device="meta"))):
        with pytest.raises(ValueError):
            pk.paged_prefix_decode_attention(**{**dict(q=qa, pool=pool, layer=0, block_tables=t, seq_lens=n,
                                                       max_seq_len=64, group_offsets=z(2), prefix_lens=z(1), scale=1.0),
                                                **bad})

    # every call reaches its last check with right arguments, and stops there: no GPU
    for f, k in ((pk.kv_tables_grow, dict(block_tables=t, seq_lens=n, new_tokens=n, free_ring=z(8), free_state=z(2),
                                          max_tokens=5, out=pk.StepTables.empty(3, 5, device="cpu"))),
                 (pk.kv_tables_release, dict(block_tables=t, seq_lens=n, finished=n, free_ring=z(8), free_state=z(2),
                                             keep_blocks=n)),
                 (pk.paged_prefix_decode_attention, dict(q=qa, layer=0, block_tables=t, seq_lens=n, max_seq_len=64,
                                                         group_offsets=z(2), prefix_lens=z(1), scale=1.0))):
        with pytest.raises(ValueError, match="not on a GPU"):
            f(pool=pool, **k)
        # wrong kinds of arguments, and integers past 32 bits
        for name, bad in (("seq_lens", [1, 2, 3]), ("block_tables", None), ("free_state", 7), ("layer", 2 ** 40),
                          ("max_seq_len", "64"), ("scale", None), ("max_tokens", 2 ** 31)):
            if name in k:
                with pytest.raises((TypeError, ValueError, AttributeError, pk.PkvError, ctypes.ArgumentError)):
                    f(pool=pool, **{**k, name: bad})


def test_rope_table_angles_are_64_bit():
    t = pk.RopeTable.create(70001, 16, device="cpu").cos_sin
    j = torch.arange(8, dtype=torch.float64)
    a = 70000.0 * 10000.0 ** (-2.0 * j / 16)
    want = torch.cat([a.cos(), a.sin()])
    assert ((t[70000].double() - want).abs() <= 2.0 ** -24).all()
