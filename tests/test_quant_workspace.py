"""Workspaces of the quantised cache's decode attention and of prompt attention: what calls leave behind lies past
the first 64 KB, which stay zero, so that both operators' calls may share one."""
import ctypes

import numpy as np
import pytest
import torch

import quant_reference as ref
from paged_kv_cache_194_gb300 import binding as pk

FAKE = 0x100000  # aligned, never dereferenced
ZEROS = 65536


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,columns", [(1, 8), (8, 8), (9, 16), (40, 16)])
def test_partial_results_lie_behind_the_zeros(D, group, columns):
    """Sizes: the zeros, then (maximum, sum) and the output of two pieces for each of 1024 CTAs."""
    desc = pk.QuantPoolDesc(num_layers=1, num_blocks=8, block_size=16, num_kv_heads=2, head_dim=D, bits=4, k_codes=FAKE,
                            v_codes=FAKE, k_params=FAKE, v_params=FAKE, error_word=None)
    h, n = ctypes.c_void_p(), ctypes.c_size_t()
    assert pk.lib().kv_quant_pool_create(ctypes.byref(desc), ctypes.byref(h)) == 0
    try:
        assert pk.lib().paged_quant_decode_plan(h, 5, 2 * group, 100, ctypes.byref(n)) == 0
        assert n.value >= ZEROS + 1024 * 2 * columns * (2 + D) * 4
        assert pk.lib().prompt_attention_plan(3, 100, 2 * group, 2, D, 1, ctypes.byref(n)) == 0
        pieces = 2 * 16 * 32 * (2 + D // 2) * 4  # an SM's two pieces: 16 warps' (maximum, sum) and half rows
        assert (n.value - ZEROS) % pieces == 0 and (n.value - ZEROS) // pieces >= 100
    finally:
        pk.lib().kv_quant_pool_destroy(h)


def dev(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x)).to(dtype).cuda()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [4, 8])
def test_decode_and_prompts_share_a_workspace(bits):
    """Cut calls of both in turns, on one workspace: each one's result is bit for bit that of a workspace of its own."""
    from test_gpu_prompt import case, offsets
    from test_gpu_quant_cache import Quantised

    decode = [Quantised(lens, Hq, Hk, D, 16, bits, seed=51) for lens, Hq, Hk, D in
              (((9000, 5000), 8, 2, 128), ((3000, 0, 1, 64, 2500, 700) * 6, 8, 2, 128), ((7000, 1), 40, 1, 64))]
    prompts = []
    for Hq, Hk, D, q_lens, k_lens in ((8, 2, 128, (300,), (8300,)), (16, 1, 64, (40, 7), (3000, 9001)),
                                      (32, 8, 64, (300,) * 4, (2300, 2300, 2301, 2150))):
        cpu, gpu = case(q_lens, k_lens, Hq, Hk, D, "bf16", fused=False, seed=52)
        args = (*gpu, dev(offsets(q_lens)), dev(offsets(k_lens)), D ** -0.5)
        prompts.append((args, cpu, q_lens, k_lens, pk.prompt_attention_workspace(gpu[0], len(q_lens), Hk)))
    own = [pk.quant_decode_workspace(b.pool, len(b.lens), b.q.shape[1], b.max_len) for b in decode]
    ws = torch.zeros(max(w.numel() for w in own + [p[4] for p in prompts]), dtype=torch.uint8, device="cuda")
    calls = [lambda w, b=b: b.run(workspace=w) for b in decode]
    calls += [lambda w, p=p: pk.prompt_attention(*p[0], workspace=w) for p in prompts]
    want = [f(w) for f, w in zip(calls, own + [p[4] for p in prompts])]
    for b, o in zip(decode, want):
        b.check(o)
    for (args, cpu, q_lens, k_lens, _), o in zip(prompts, want[3:]):
        exact, bound = ref.prompt(*cpu, q_lens, k_lens, args[5])
        assert ((o.cpu().double() - exact).abs() <= bound).all()
    for i in (0, 3, 0, 4, 1, 5, 2, 3, 1, 4, 0, 5, 5, 2):
        assert torch.equal(calls[i](ws), want[i]), i
        assert not ws[:ZEROS].any(), i
