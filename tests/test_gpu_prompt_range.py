"""GPU tests of prompt attention where magnitudes are far from one: large values under rising scores, large scores, keys
that are not finite among pieces that weigh nothing."""
import pytest
import torch

import quant_tight as tight
from paged_kv_cache_194_gb300 import binding as pk
from test_gpu_prompt import case, offsets
from test_gpu_quant_cache import dev
from test_gpu_quant_tight import PROMPTS, check_picks, ids, picks

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("q_lens,k_lens", [((900,), (900,)), ((200,), (5000,))], ids=str)
@pytest.mark.parametrize("rise", [12.0, 30.0, 55.0])
def test_large_values_under_rising_scores(inp, q_lens, k_lens, rise):
    """Scores that rise by 2^rise from one tile of keys to the next, so that the weights' base lags behind them, and
    values of 2^96: sums of weights and values stay within 32 bits."""
    (q, k, v), _ = case(q_lens, k_lens, 4, 2, 128, inp, fused=False, seed=90)
    q = q * 0.01
    q[..., 0] = 1.0
    k[..., 0] = (torch.arange(k.shape[0]) // 128 * rise * 0.6931)[:, None].to(k.dtype)
    v = v * 2.0 ** 96
    out = pk.prompt_attention(*[x.cuda() for x in (q, k, v)], dev(offsets(q_lens)), dev(offsets(k_lens)), 1.0)
    assert out.isfinite().all()
    tight.check(out, *tight.prompts(q, k, v, q_lens, k_lens, 1.0))


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("bad", [slice(100, 101), slice(128, 256), slice(0, 640)], ids=str)
@pytest.mark.parametrize("heavy", [3100, 5900])
def test_keys_that_are_nan_where_nothing_weighs(inp, bad, heavy):
    """A query that sees a key of NaN is NaN, whatever the other keys of its tile or piece weigh beside the rest."""
    (q, k, v), _ = case((70,), (6000,), 8, 2, 128, inp, fused=False, seed=91)
    q[..., 0] = 8.0
    k[:, :, 0] = 0
    k[heavy:heavy + 50, :, 0] = 60.0
    o = [dev(offsets(x)) for x in ((70,), (6000,))]
    want = pk.prompt_attention(*[x.cuda() for x in (q, k, v)], *o, 1.0)
    tight.check(want, *tight.prompts(q, k, v, (70,), (6000,), 1.0))
    k[bad, 1] = float("nan")
    got = pk.prompt_attention(*[x.cuda() for x in (q, k, v)], *o, 1.0)
    assert got[:, 4:].isnan().all() and torch.equal(got[:, :4], want[:, :4])


@pytest.mark.parametrize("inp", ["bf16", "f32"])
@pytest.mark.parametrize("wide", [-2.0 ** 12, 2.0 ** 20, 2.0 ** 30, 2.0 ** 50])
@pytest.mark.parametrize("q_lens,k_lens,Hq,Hk,D", [PROMPTS[0], PROMPTS[2], PROMPTS[4], PROMPTS[7]], ids=ids)
def test_large_scores(inp, wide, q_lens, k_lens, Hq, Hk, D):
    """Scores of up to 10^19: 32 bits have steps of many units there, and the largest still outweighs the others."""
    q, k, v, want = picks(inp, q_lens, k_lens, Hq, Hk, D, abs(wide))
    sign = -1.0 if wide < 0 else 1.0  # (a negative scale: every score turned around, twice)
    out = pk.prompt_attention(*[x.cuda() for x in (q * sign, k, v)], dev(offsets(q_lens)), dev(offsets(k_lens)), 0.25 * sign)
    check_picks(inp, out, want)
