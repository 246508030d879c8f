"""The decoder with the rotating append, shaped scores and sampled speculation: turning and
appending, attention over the cache, and the verification of drafts run together, as a serving
step uses them."""
import math

import numpy as np
import pytest
import torch

from invariant_bi_matmul_gb300 import inputs

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")
from invariant_bi_matmul_gb300.decoder import GreedyDecoder, lookup_drafter  # noqa: E402
from invariant_bi_matmul_gb300.decoder import random_drafter, reference_drafter  # noqa: E402

CFG = inputs.TINY_DECODER


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def weights(dev):
    w = inputs.decoder_weights(CFG, 800, std=0.05, norm_std=0.1)
    return {k: v.to(dev) for k, v in w.items()}


def decoder(dev, weights, batch=4, **kw):
    return GreedyDecoder(CFG, weights, max_batch=batch, max_len=400, max_width=4, device=dev,
                         page_seed=3, prefill_width=64, **kw)


def prompts(n, length=150):
    return [inputs.decoder_prompt(CFG, s, 801, length) for s in range(n)]


KINDS = {"plain": {}, "fused": dict(fused_append=True),
         "fused q8": dict(fused_append=True, kv_cache="q8"),
         "shaped": dict(softcap=5.0, window=60, fused_append=True)}


@pytest.mark.parametrize("kind", KINDS)
def test_temperature_0_is_greedy_decoding(dev, weights, kind):
    """The same tokens and log-probabilities as token-by-token decoding, from wrong drafts, right
    ones and a mixture; and the same caches' bits, whichever way the tokens came."""
    steps = 40
    dec = decoder(dev, weights, logprobs=True, **KINDS[kind])
    dec.prefill(prompts(4))
    want = dec.decode(steps)
    want_lp = dec.trace_logprobs
    for width, drafter, share in ((4, random_drafter(CFG.vocab, 5), 0.0),
                                  (4, reference_drafter(want, 0.3, CFG.vocab), None),
                                  (3, reference_drafter(want, 0.0, CFG.vocab), 1.0)):
        dec.prefill(prompts(4), width=7 if width == 3 else 64)
        got, blocks, accepted = dec.speculate_sampled(steps, width, drafter, 0.0)
        assert got == want
        # (both are log p at temperature 1: fp32 sums of 512 entries, by different trees)
        np.testing.assert_allclose(dec.trace_logprobs, want_lp, rtol=2e-6, atol=2e-6)
        if share is not None:
            assert (accepted == 0) == (share == 0.0) and (blocks == steps) == (share == 0.0)
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("kind", KINDS)
def test_sampled_traces_do_not_depend_on_the_batch(dev, weights, kind):
    steps = 30
    dec = decoder(dev, weights, **KINDS[kind])
    dec.prefill(prompts(4))
    want, _, accepted = dec.speculate_sampled(steps, 4, lookup_drafter, 0.8, seed=11)
    lp = dec.trace_logprobs
    assert all(len(t) == steps for t in want) and len({tuple(t) for t in want}) == 4
    for some in ([2], [3, 0], [1, 2, 3]):
        dec.prefill([prompts(4)[i] for i in some])
        got, _, _ = dec.speculate_sampled(steps, 4, lookup_drafter, 0.8, seed=11, seq_ids=some)
        assert got == [want[i] for i in some]
        assert dec.trace_logprobs == [lp[i] for i in some]
    dec.prefill(prompts(4))
    other, _, _ = dec.speculate_sampled(steps, 4, lookup_drafter, 0.8, seed=12)
    assert other != want
    assert bi.device_status() == bi.BI_OK


def test_log_probabilities_of_sampled_tokens(dev, weights):
    """Those of the logits that the block was verified with, at the temperature, in 64 bits."""
    dec = decoder(dev, weights)
    dec.prefill(prompts(2))
    seen = []
    forward = dec.forward
    dec.forward = lambda *a, **k: (forward(*a, **k), seen.append(dec.logits.clone()))[0]
    traces, blocks, _ = dec.speculate_sampled(12, 1, lookup_drafter, 1.3, seed=3)
    assert blocks == 12
    for i in range(12):
        logp = torch.log_softmax(seen[i][:2].double() / 1.3, -1)
        for b in range(2):
            want = float(logp[b, traces[b][i]])
            assert abs(dec.trace_logprobs[b][i] - want) <= 2e-6 * max(1.0, abs(want))


def test_fused_append_is_near_the_separate_one(dev, weights):
    """Angles of positions below 200 agree to 2^-16; a turned value is rounded to bf16 either way,
    a possible step of 2^-8 of it in each of two layers' queries and keys."""
    a, b = decoder(dev, weights), decoder(dev, weights, fused_append=True)
    for d in (a, b):
        d.prefill(prompts(4))
        d.forward(d.last, [1] * 4)
    x, y = a.logits[:4].double(), b.logits[:4].double()
    assert float((x - y).norm() / x.norm()) < 2.0 ** -8 * math.sqrt(31)


def test_window_hides_the_start(dev, weights):
    """With a window no longer than the last block's tokens see, what lies in front of it through
    all layers changes nothing: prompts that differ only there decode alike."""
    window = 20
    reach = CFG.layers * (window - 1)               # what a token's logits depend on
    dec = decoder(dev, weights, window=window)
    p = prompts(2, 150)
    q = [t[:] for t in p]
    for t in q:
        t[:150 - reach - 1] = reversed(t[:150 - reach - 1])
    dec.prefill(p)
    want = dec.decode(8)
    first = dec.logits[:2].clone()
    dec.prefill(q)
    assert dec.decode(8) == want and torch.equal(dec.logits[:2], first)


def test_refusals(dev, weights):
    for bad in (dict(softcap=5.0), dict(window=10)):
        with pytest.raises(ValueError):
            decoder(dev, weights, kv_cache="q8", **bad)
    dec = decoder(dev, weights)
    dec.prefill(prompts(2))
    for bad in (dict(width=0), dict(width=5), dict(seq_ids=[1])):
        with pytest.raises(ValueError):
            dec.speculate_sampled(3, **(dict(width=2, drafter=lookup_drafter, temperature=1.0)
                                        | bad))


def test_a_temperature_and_logits_without_a_distribution_are_reported(dev, weights):
    dec = decoder(dev, weights)
    dec.prefill(prompts(2))
    for bad in (-1.0, float("inf"), float("nan")):
        with pytest.raises(ValueError, match="temperature"):
            dec.speculate_sampled(3, 2, lookup_drafter, bad)
    dec.w = {k: torch.full_like(v, float("nan")) if v.dim() == 1 else v
             for k, v in weights.items()}
    with pytest.raises(RuntimeError, match="no distribution"):
        dec.speculate_sampled(3, 2, lookup_drafter, 1.0)
