"""GPU: codes of values next to the border between two codes, where a product and a sum that are rounded once together give
another code than the format's steps, each of which is rounded."""
import numpy as np
import pytest
import torch

import quant_reference as ref
from paged_kv_cache_194_gb300 import binding as pk
from test_gpu_quant_cache import raw, expect_append

pytestmark = pytest.mark.gpu


def rows(bits, D, count):
    """Rows from 0 to a maximum, one value of each between the borders of the two ways of rounding."""
    r = np.random.default_rng(bits * D)
    out = []
    while len(out) < count:
        x = np.zeros(D, np.float32)
        x[1:] = r.random(D - 1, dtype=np.float32)
        x[1] = 1.0 + r.random(dtype=np.float32)
        s = ref.quantise(torch.from_numpy(x)[None], bits)[1][0, 0].float().numpy()
        inv = np.float32(np.float32(1) / s * np.float32(1 + 2.0 ** -21))
        near = np.float32(0.5) / inv
        tries = near + np.arange(-64, 65, dtype=np.float32) * np.spacing(near)
        apart = np.floor((tries * inv).astype(np.float32) + np.float32(0.5))
        fused = np.floor((tries.astype(np.float64) * np.float64(inv) + 0.5).astype(np.float32))
        found = tries[apart != fused]
        if len(found):
            x[2:2 + min(len(found), D - 2)] = found[:D - 2]
            out.append(x)
    return torch.from_numpy(np.stack(out))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bits", [4, 8])
def test_each_step_is_rounded(bits, D):
    x = rows(bits, D, 64)[:, None]
    pool = pk.QuantKVPool(1, 4, 16, 1, D, bits, fill=0)
    slots = torch.arange(64)
    want = expect_append(raw(pool), 0, x, x, slots, 16, bits)
    pk.kv_quant_append(pool, 0, x.cuda(), x.cuda(), slots.cuda())
    for a, b in zip(raw(pool), want):
        assert torch.equal(a, b), int((a != b).sum())
