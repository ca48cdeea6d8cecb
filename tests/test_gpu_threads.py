"""Calls on one pool from several host threads."""
import threading

import pytest
import torch

from paged_kv_cache_194_gb300 import binding as pk
from test_gpu_prefix import Batch

pytestmark = pytest.mark.gpu


def in_new_thread(f):
    got = []
    t = threading.Thread(target=lambda: got.append(f()))
    t.start()
    t.join()
    return got[0]


@pytest.mark.parametrize("kv", ["bf16", "fp8"])
@pytest.mark.parametrize("used", [False, True])
def test_first_call_of_a_host_thread(kv, used):
    """A thread whose first CUDA call is this one runs what others run, on a
    new pool and on one that has served calls."""
    make = lambda: Batch((300, 333, 290, 70), [(0, 3, 256)], seed=14, kv=kv)
    want = make().run()
    bt = make()
    dev = [x.cuda() for x in (bt.q, bt.tables, torch.tensor(bt.lens, dtype=torch.int32), bt.offsets, bt.prefix)]
    out, dec = torch.zeros_like(dev[0]), torch.zeros_like(dev[0])
    ws = pk.prefix_decode_workspace(bt.pool, 4, 1, 8, bt.max_len)
    dws = pk.workspace_for(bt.pool, 4, 8, bt.max_len)
    if used:
        bt.run()
    torch.cuda.synchronize()

    def first():
        return pk.paged_prefix_decode_attention(dev[0], bt.pool, 1, dev[1], dev[2], bt.max_len, dev[3], dev[4], bt.scale,
                                                out=out, workspace=ws, algo="tc")

    def decode():
        return pk.paged_decode_attention(dev[0], bt.pool, 1, dev[1], dev[2], bt.max_len, bt.scale, out=dec,
                                         workspace=dws, algo="mma")

    for f in (first, decode) if used else (decode, first):
        in_new_thread(f)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(dec, make().run(algo="mma"))


def test_first_calls_of_a_pool_from_several_threads():
    """A pool's first calls may come at once: each finds the pool's descriptors complete."""
    n = 8
    for _ in range(100):
        pool = pk.KVPool(1, 4, 16, 2, 128, "bf16")
        gate, got = threading.Barrier(n), []

        def first(i):
            gate.wait()
            if i % 2:
                got.append(pk.lib().paged_prefix_decode_algo(pool.handle, 4, 1, 8, 64, 3))
            else:
                got.append(pk.lib().paged_multi_query_algo(pool.handle, 64, 8, 0, 3))

        threads = [threading.Thread(target=first, args=(i,)) for i in range(n)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert got == [3] * n
