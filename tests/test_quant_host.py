"""The quantised cache and prompt attention without a GPU: the format's
arithmetic, and refusals (every call here is rejected on the host before
anything is enqueued)."""
import ctypes

import pytest
import torch

import quant_reference as ref
from paged_kv_cache_194_gb300 import binding as pk

FAKE = 0x100000  # aligned, never dereferenced
P = ctypes.c_void_p


def _desc(**kw):
    d = dict(num_layers=1, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=128, bits=4, k_codes=FAKE, v_codes=FAKE,
             k_params=FAKE, v_params=FAKE, error_word=None)
    d.update(kw)
    return pk.QuantPoolDesc(**d)


@pytest.fixture()
def pool():
    handles = []

    def make(**kw):
        h = ctypes.c_void_p()
        assert pk.lib().kv_quant_pool_create(ctypes.byref(_desc(**kw)), ctypes.byref(h)) == 0
        handles.append(h)
        return h

    yield make
    for h in handles:
        pk.lib().kv_quant_pool_destroy(h)


@pytest.mark.parametrize("bits", [4, 8])
@pytest.mark.parametrize("kind", ["normal", "offset", "tiny", "huge", "constant", "steps"])
def test_format_errs_by_half_a_scale(bits, kind):
    """Every value reads back within half a scale (and the reciprocal's excess)."""
    g = torch.Generator().manual_seed(bits)
    x = torch.randn(500, 128, generator=g)
    x = {"normal": x, "offset": x * 0.01 + 7, "tiny": x * 1e-36, "huge": x * 1e36, "constant": x[:, :1].expand(-1, 128),
         "steps": torch.randint(-8, 8, x.shape, generator=g) / 4.0}[kind].contiguous()
    for dt in (torch.float32, torch.bfloat16):
        y = x.to(dt)
        n, p = ref.quantise(y, bits)
        s = p[..., :1].double()
        err = (ref.values(ref.pack(n, bits), p, bits) - y.double()).abs()
        # 32-bit difference and products: 4 roundings of a quotient below 256, and the 2^-21 excess
        assert (err <= s * (0.5 + 256 * (4 * 2.0 ** -24 + 2.0 ** -21))).all()


def test_pool_refusals():
    def create(**kw):
        h = ctypes.c_void_p()
        rc = pk.lib().kv_quant_pool_create(ctypes.byref(_desc(**kw)), ctypes.byref(h))
        assert not h.value or rc == 0
        pk.lib().kv_quant_pool_destroy(h)
        return rc

    assert create() == 0
    for bad in (dict(num_layers=0), dict(num_blocks=0), dict(num_kv_heads=-1), dict(k_codes=None), dict(v_codes=FAKE + 8),
                dict(k_params=None), dict(v_params=FAKE + 4), dict(error_word=FAKE + 2)):
        assert create(**bad) == 1, bad
    for bad in (dict(block_size=8), dict(head_dim=96), dict(bits=2), dict(bits=5), dict(num_blocks=2 ** 27)):
        assert create(**bad) == 2, bad
    L = pk.lib()
    assert L.kv_quant_pool_create(None, ctypes.byref(P())) == 1 and L.kv_quant_pool_create(ctypes.byref(_desc()), None) == 1
    c, p = ctypes.c_size_t(), ctypes.c_size_t()
    assert L.kv_quant_pool_bytes(ctypes.byref(_desc(num_layers=3)), ctypes.byref(c), ctypes.byref(p)) == 0
    assert (c.value, p.value) == (3 * 8 * 2 * 16 * 64, 3 * 8 * 2 * 16 * 4)
    assert L.kv_quant_pool_bytes(ctypes.byref(_desc(bits=8, head_dim=64)), ctypes.byref(c), None) == 0
    assert c.value == 8 * 2 * 16 * 64
    assert L.kv_quant_pool_bytes(None, None, None) == 1 and L.kv_quant_pool_bytes(ctypes.byref(_desc(bits=3)), None, None) == 2
    with pytest.raises(pk.PkvError):
        pk.QuantKVPool(1, 8, 16, 2, 128, 6, device="cpu")


def test_append_refusals(pool):
    h = pool()

    def call(**k):
        return pk.lib().kv_quant_append(k.get("h", h), k.get("layer", 0), P(k.get("k", FAKE)), P(k.get("v", FAKE)),
                                        k.get("dt", 1), k.get("ks", 256), k.get("vs", 256), P(k.get("slots", FAKE)),
                                        k.get("T", 4), None)

    assert call(T=0) == 0
    assert call(h=None) == 1 and call(layer=1) == 1 and call(layer=-1) == 1 and call(T=-1) == 1 and call(dt=2) == 1
    for n in ("k", "v", "slots"):
        assert call(**{n: None}) == 1 and call(**{n: FAKE + 4}) == 1, n
    for n in ("ks", "vs"):
        assert call(**{n: -8}) == 1 and call(**{n: 260}) == 1 and call(**{n: 2 ** 62}) == 1


def test_read_refusals(pool):
    h = pool()
    plain = ctypes.c_void_p()
    d = pk.PoolDesc(num_layers=1, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=128, kv_dtype=1, k_scale=1.0,
                    v_scale=1.0, k_base=FAKE, v_base=FAKE, error_word=None)
    assert pk.lib().kv_pool_create(ctypes.byref(d), ctypes.byref(plain)) == 0
    for f, pl in ((pk.lib().kv_quant_read, h), (pk.lib().kv_read, plain)):
        def call(**k):
            return f(k.get("h", pl), k.get("layer", 0), P(k.get("t", FAKE)), k.get("mb", 4), P(k.get("off", FAKE)),
                     k.get("B", 2), k.get("rows", 9), P(k.get("ko", FAKE)), P(k.get("vo", FAKE)), None)

        assert call(B=0) == 0 and call(rows=0) == 0
        assert call(h=None) == 1 and call(layer=1) == 1 and call(mb=0) == 1 and call(B=-1) == 1 and call(rows=-1) == 1
        for n in ("t", "off", "ko", "vo"):
            assert call(**{n: None}) == 1 and call(**{n: FAKE + 2}) == 1, n
        assert call(ko=FAKE + 8) == 1
    pk.lib().kv_pool_destroy(plain)


def test_quant_decode_refusals(pool):
    h = pool()
    ws = ctypes.c_size_t()
    assert pk.lib().paged_quant_decode_plan(h, 2, 8, 64, ctypes.byref(ws)) == 0

    def call(**k):
        return pk.lib().paged_quant_decode_attention(
            P(k.get("q", FAKE)), k.get("dt", 1), k.get("h", h), k.get("layer", 0), P(k.get("t", FAKE)), k.get("mb", 4),
            P(k.get("lens", FAKE)), k.get("B", 2), k.get("Hq", 8), k.get("maxlen", 64), k.get("scale", 0.1),
            P(k.get("ws", FAKE)), k.get("wsb", ws.value), P(k.get("out", FAKE)), None)

    assert call(B=0) == 0
    assert call(h=None) == 1 and call(layer=1) == 1 and call(mb=0) == 1 and call(B=-1) == 1 and call(Hq=0) == 1
    assert call(Hq=7) == 1 and call(maxlen=65) == 1 and call(maxlen=-1) == 1 and call(scale=float("inf")) == 1
    assert call(dt=0) == 2 and call(B=65536) == 2 and call(Hq=65536) == 2
    for n in ("q", "t", "lens", "out"):
        assert call(**{n: None}) == 1 and call(**{n: FAKE + 2}) == 1, n
    if ws.value:
        assert call(ws=None) == 3 and call(wsb=ws.value - 1) == 3 and call(ws=FAKE + 16) == 3
    assert pk.lib().paged_quant_decode_plan(None, 2, 8, 64, ctypes.byref(ws)) == 1


def test_prompt_refusals():
    Q, K, V, O = FAKE, 2 * FAKE, 3 * FAKE, 4 * FAKE

    def call(**k):
        return pk.lib().prompt_attention(
            P(k.get("q", Q)), P(k.get("k", K)), P(k.get("v", V)), k.get("dt", 1), k.get("qs", 1024), k.get("ks", 256),
            k.get("vs", 256), P(k.get("qo", FAKE)), P(k.get("ko", FAKE)), k.get("B", 2), k.get("T", 9), k.get("Tk", 9),
            k.get("Hq", 8), k.get("Hk", 2), k.get("D", 128), k.get("scale", 0.1), P(k.get("ws", FAKE)),
            k.get("wsb", 2 ** 40), P(k.get("out", O)), P(k.get("err", None)), None)

    assert call(B=0) == 0 and call(T=0) == 0
    assert call(B=-1) == 1 and call(T=-1) == 1 and call(Tk=-1) == 1 and call(Hq=0) == 1 and call(Hk=0) == 1
    assert call(Hq=7) == 1 and call(dt=2) == 1 and call(D=96) == 2 and call(scale=float("nan")) == 1
    assert call(Hq=65536, Hk=65536, qs=2 ** 23, ks=2 ** 23, vs=2 ** 23) == 2
    for n, p in (("q", Q), ("k", K), ("v", V), ("out", O)):
        assert call(**{n: None}) == 1 and call(**{n: p + 8}) == 1, n
    for n in ("qo", "ko"):
        assert call(**{n: None}) == 1 and call(**{n: FAKE + 2}) == 1, n
    for n in ("qs", "ks", "vs"):  # too narrow, not whole chunks, negative, past 64 bits
        for s in (128, 1028, -8, 2 ** 62):
            assert call(**{n: s}) == 1, (n, s)
    assert call(err=FAKE + 2) == 1
    assert call(out=Q) == 1 and call(out=Q + 16) == 1 and call(out=K) == 1 and call(out=V - 16) == 1
    ws = ctypes.c_size_t()
    assert pk.lib().prompt_attention_plan(2, 9, 8, 2, 128, 1, ctypes.byref(ws)) == 0
    if ws.value:
        assert call(ws=None) == 3 and call(wsb=ws.value - 1) == 3 and call(ws=FAKE + 16) == 3
    for bad in ((-1, 9, 8, 2, 128, 1), (2, -1, 8, 2, 128, 1), (2, 9, 8, 3, 128, 1), (2, 9, 8, 2, 128, 2)):
        assert pk.lib().prompt_attention_plan(*bad, ctypes.byref(ws)) == 1, bad
    assert pk.lib().prompt_attention_plan(2, 9, 8, 2, 80, 1, ctypes.byref(ws)) == 2


def test_binding_checks_shapes_types_and_devices():
    bf = torch.bfloat16
    z = lambda *s, dtype=torch.int32: torch.zeros(s, dtype=dtype)
    pool = pk.QuantKVPool(1, 8, 16, 2, 128, 4, device="cpu")
    assert pool.k_codes.shape == (1, 8, 2, 16, 64) and pool.v_params.shape == (1, 8, 2, 16, 2)
    plain = pk.KVPool(1, 8, 16, 2, 128, "fp8", device="cpu")
    kv = z(4, 2, 128, dtype=bf)
    good = dict(k=kv, v=kv, slot_mapping=z(4, dtype=torch.int64))
    for bad in (dict(k=z(4, 2, 64, dtype=bf)), dict(v=z(4, 2, 128, dtype=torch.float32)), dict(v=z(5, 2, 128, dtype=bf)),
                dict(slot_mapping=z(4)), dict(slot_mapping=z(5, dtype=torch.int64)), dict(k=z(4, 2, 256, dtype=bf)[..., ::2]),
                dict(k=kv.half(), v=kv.half()), dict(k=z(2, 4, 128, dtype=bf).transpose(0, 1)), dict(k=kv.to("meta"))):
        with pytest.raises(ValueError):
            pk.kv_quant_append(pool, 0, **{**good, **bad})
    t, off = z(3, 4), z(4)
    for p in (pool, plain):
        for bad in (dict(block_tables=z(2, 4)), dict(block_tables=t.long()), dict(offsets=z(0)), dict(offsets=off.long()),
                    dict(k_out=z(6, 2, 128, dtype=torch.float32)), dict(v_out=z(7, 2, 128, dtype=bf)),
                    dict(k_out=z(6, 2, 256, dtype=bf)[..., :128]), dict(num_rows=-1)):
            with pytest.raises((ValueError, RuntimeError)):
                pk.kv_read(p, 0, **{**dict(block_tables=t, offsets=off, num_rows=6), **bad})
    q = z(3, 8, 128, dtype=bf)
    attend = dict(q=q, layer=0, block_tables=t, seq_lens=z(3), max_seq_len=64, scale=1.0)
    for bad in (dict(q=z(3, 8, 64, dtype=bf)), dict(seq_lens=z(2)), dict(block_tables=z(2, 4)), dict(out=q[:2]),
                dict(q=z(8, 3, 128, dtype=bf).transpose(0, 1)), dict(workspace=torch.zeros(8, device="meta")),
                dict(seq_lens=z(3, dtype=torch.int64))):
        with pytest.raises(ValueError):
            pk.paged_quant_decode_attention(pool=pool, **{**attend, **bad})
    qp, kp = z(6, 8, 128, dtype=bf), z(7, 2, 128, dtype=bf)
    prompt = dict(q=qp, k=kp, v=kp, q_offsets=off, k_offsets=off, scale=1.0)
    for bad in (dict(q=qp.half()), dict(k=kp.float()), dict(v=z(6, 2, 128, dtype=bf)), dict(v=z(7, 1, 128, dtype=bf)),
                dict(q_offsets=z(5)), dict(q_offsets=off.long()), dict(k_offsets=z(8)[::2]), dict(out=z(6, 8, 64, dtype=bf)),
                dict(out=qp.float()), dict(error_word=z(2)), dict(q=z(6, 128, dtype=bf)), dict(k=z(7, 128, dtype=bf)),
                dict(q=z(8, 6, 128, dtype=bf).transpose(0, 1))):
        with pytest.raises((ValueError, pk.PkvError)):
            pk.prompt_attention(**{**prompt, **bad})
    # every call reaches its last check with right arguments, and stops there: no GPU
    for f, k in ((pk.kv_quant_append, dict(pool=pool, layer=0, **good)),
                 (pk.kv_read, dict(pool=pool, layer=0, block_tables=t, offsets=off, num_rows=6)),
                 (pk.kv_read, dict(pool=plain, layer=0, block_tables=t, offsets=off, num_rows=6)),
                 (pk.paged_quant_decode_attention, dict(pool=pool, **attend)), (pk.prompt_attention, prompt)):
        with pytest.raises(ValueError, match="not on a GPU"):
            f(**k)
        for name, bad in (("k", [1]), ("block_tables", None), ("layer", 2 ** 40), ("max_seq_len", "64"), ("scale", None),
                          ("num_rows", 2 ** 31), ("q_offsets", 3)):
            if name in k:
                with pytest.raises((TypeError, ValueError, AttributeError, RuntimeError, ctypes.ArgumentError)):
                    f(**{**k, name: bad})


def test_lengths_past_32_bits_of_tiles_are_refused(pool):
    ws = ctypes.c_size_t()
    h = pool()
    assert pk.lib().paged_quant_decode_plan(h, 1, 8, 2 ** 31 - 64, ctypes.byref(ws)) == 0
    for n in (2 ** 31 - 63, 2 ** 31 - 1):
        assert pk.lib().paged_quant_decode_plan(h, 1, 8, n, ctypes.byref(ws)) == 2


def test_workspaces_grow_with_what_they_serve(pool):
    """A workspace of a larger call serves the smaller ones: sizes depend on neither the batch nor the lengths."""
    ws, h = ctypes.c_size_t(), pool()
    sizes = set()
    for B, n in ((1, 1), (4, 100), (65535, 2 ** 31 - 64)):
        assert pk.lib().paged_quant_decode_plan(h, B, 8, n, ctypes.byref(ws)) == 0
        sizes.add(ws.value)
    assert len(sizes) == 1 and sizes.pop() > 65536
    prompts = set()
    for B, T in ((1, 1), (2048, 2048), (7, 100000)):
        assert pk.lib().prompt_attention_plan(B, T, 8, 2, 128, 1, ctypes.byref(ws)) == 0
        prompts.add(ws.value)
    assert len(prompts) == 1 and prompts.pop() > 65536
    for B, T, Hq, Hk, dt in ((2049, 5000, 8, 2, 1), (2, 9, 258, 2, 1), (2, 9, 8, 2, 0)):  # the CUDA cores' design needs none
        assert pk.lib().prompt_attention_plan(B, T, Hq, Hk, 128, dt, ctypes.byref(ws)) == 0
        assert ws.value == 0
