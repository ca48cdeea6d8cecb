"""GPU: a wait of prompt attention's tensor-core design that runs out, made to happen on demand (no fault, no hang):
the error bit, NaN in every row that is lost, the other rows bit for bit, and a workspace that needs no clearing."""
import time

import numpy as np
import pytest
import torch

import quant_reference as ref
from paged_kv_cache_194_gb300 import binding as pk
from test_gpu_prompt import case, offsets

pytestmark = pytest.mark.gpu

CASES = {  # query heads, KV heads, head_dim, queries, keys
    "many_units": (32, 8, 128, (1500, 40, 700, 1, 900), (1500, 40, 700, 1, 900)),
    "short": (8, 2, 64, tuple(range(1, 120, 4)), tuple(range(1, 120, 4))),
    "pieces": (8, 2, 128, (300,), (8300,)),
    "pieces_of_some": (32, 8, 64, (300,) * 4, (2300, 2300, 2301, 2150)),
}


@pytest.mark.parametrize("cta", [0, 1, 77, -1])
@pytest.mark.parametrize("name", list(CASES))
def test_a_cta_gives_up(name, cta):
    Hq, Hk, D, q_lens, k_lens = CASES[name]
    cpu, gpu = case(q_lens, k_lens, Hq, Hk, D, "bf16", fused=False, seed=60)
    args = (*gpu, *(torch.as_tensor(offsets(x)).to(torch.int32).cuda() for x in (q_lens, k_lens)), D ** -0.5)
    ws = pk.prompt_attention_workspace(gpu[0], len(q_lens), Hk)
    good = pk.prompt_attention(*args, workspace=ws)
    want, bound = ref.prompt(*cpu, q_lens, k_lens, D ** -0.5)
    assert ((good.cpu().double() - want).abs() <= bound).all()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    for word in (err, None):  # (the rows say it, too)
        out = torch.full_like(good, 7.0)
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        try:
            pk.set_first_wait_limit_for_testing(0, cta)
            pk.prompt_attention(*args, out=out, error_word=word, workspace=ws)
            torch.cuda.synchronize()
        finally:
            pk.set_first_wait_limit_for_testing(-1)
        assert time.perf_counter() - t0 < 5.0
        lost = out.isnan().any(2)
        assert (out.isnan().all(2) == lost).all()
        assert torch.equal(out[~lost], good[~lost])
        units = {"pieces": 2 * 5}.get(name, 1000)  # (of fewer units than CTAs some CTA has none)
        assert lost.all() if cta < 0 else lost.any() or cta >= units
        if cta >= 0 and name in ("many_units", "pieces_of_some"):
            assert float(lost.float().mean()) < 0.1
        assert not ws[:65536].any()
    assert int(err) in ((pk.ERRBIT_TIMEOUT,) if lost.any() else (0,))
    again = torch.full_like(good, 7.0)
    err.zero_()
    pk.prompt_attention(*args, out=again, error_word=err, workspace=ws)
    assert torch.equal(again, good) and int(err) == 0 and not ws[:65536].any()


def test_other_calls_and_other_threads_are_not_limited():
    """The limit is the calling thread's, and off again afterwards; a captured call keeps what it was captured with."""
    Hq, Hk, D, lens, _ = CASES["short"]
    _, gpu = case(lens, lens, Hq, Hk, D, "bf16", fused=False, seed=61)
    o = torch.as_tensor(np.asarray(offsets(lens))).to(torch.int32).cuda()
    ws = pk.prompt_attention_workspace(gpu[0], len(lens), Hk)
    out = torch.empty_like(gpu[0])
    call = lambda: pk.prompt_attention(*gpu, o, o, 0.1, out=out, workspace=ws)
    want = call().clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    try:
        pk.set_first_wait_limit_for_testing(0, -1)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        assert call().isnan().all()
    finally:
        pk.set_first_wait_limit_for_testing(-1)
    assert torch.equal(call(), want)
