"""Read-back without a GPU: refusals, with outputs that do not overlap and ones that do (every call here is rejected on
the host before anything is enqueued)."""
import ctypes

import pytest
import torch

from paged_kv_cache_194_gb300 import binding as pk

FAKE = 0x100000  # aligned, never dereferenced
P = ctypes.c_void_p


@pytest.fixture(params=["q4", "q8", "bf16", "f32", "fp8"])
def pool(request):
    """(reads, handle, bytes of a packed row of two heads of 64)"""
    h = ctypes.c_void_p()
    if request.param[0] == "q":
        d = pk.QuantPoolDesc(num_layers=1, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=64, bits=int(request.param[1]),
                             k_codes=FAKE, v_codes=FAKE, k_params=FAKE, v_params=FAKE, error_word=None)
        assert pk.lib().kv_quant_pool_create(ctypes.byref(d), ctypes.byref(h)) == 0
        yield pk.lib().kv_quant_read, h, 256
        pk.lib().kv_quant_pool_destroy(h)
    else:
        d = pk.PoolDesc(num_layers=1, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=64,
                        kv_dtype={"f32": 0, "bf16": 1, "fp8": 2}[request.param], k_scale=1.0, v_scale=1.0, k_base=FAKE,
                        v_base=FAKE, error_word=None)
        assert pk.lib().kv_pool_create(ctypes.byref(d), ctypes.byref(h)) == 0
        yield pk.lib().kv_read, h, 512 if request.param == "f32" else 256
        pk.lib().kv_pool_destroy(h)


def test_read_refusals(pool):
    f, h, row = pool
    K, V, rows = FAKE, 2 * FAKE, 9

    def call(**k):
        return f(k.get("h", h), k.get("layer", 0), P(k.get("t", FAKE)), k.get("mb", 4), P(k.get("off", FAKE)),
                 k.get("B", 2), k.get("rows", rows), P(k.get("ko", K)), P(k.get("vo", V)), None)

    assert call(B=0) == 0 and call(rows=0) == 0 and call(rows=0, vo=K) == 0
    assert call(h=None) == 1 and call(layer=1) == 1 and call(mb=0) == 1 and call(B=-1) == 1 and call(rows=-1) == 1
    for n in ("t", "off", "ko", "vo"):
        assert call(**{n: None}) == 1 and call(**{n: V + FAKE + 2}) == 1, n
    assert call(ko=K + 8) == 1
    # outputs that overlap, by one row or all of them
    if not torch.cuda.is_available():
        assert call() == 4 and call(vo=K + rows * row) == 4  # (apart: refused by nothing but the missing GPU)
    for v in (K, K + 16, K + (rows - 1) * row, K - 16, K - (rows - 1) * row):
        assert call(vo=v) == 1, v - K
