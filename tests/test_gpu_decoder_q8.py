"""The decoder with 8-bit caches, token log-probabilities and forks: append, attention over the
cache, log-probabilities and page copies run together, as a serving step uses them."""
import math

import numpy as np
import pytest
import torch

from invariant_bi_matmul_gb300 import inputs
from tolerance import bits_equal

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")
from invariant_bi_matmul_gb300.decoder import GreedyDecoder, random_drafter  # noqa: E402
from invariant_bi_matmul_gb300.decoder import reference_drafter  # noqa: E402

CFG = inputs.TINY_DECODER


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def weights(dev):
    w = inputs.decoder_weights(CFG, 700, std=0.05, norm_std=0.1)
    return {k: v.to(dev) for k, v in w.items()}


def decoder(dev, weights, kv="q8", batch=4, **kw):
    return GreedyDecoder(CFG, weights, max_batch=batch, max_len=400, max_width=4, device=dev,
                         page_seed=3, prefill_width=64, kv_cache=kv, logprobs=True, **kw)


def prompts(n, length=150):
    return [inputs.decoder_prompt(CFG, s, 701, length) for s in range(n)]


@pytest.mark.parametrize("kv", ["bf16", "q8"])
def test_traces_and_logprobs_do_not_depend_on_batch_or_width(dev, weights, kv):
    """Token by token in a batch, alone, and in verify blocks with wrong and right drafts: the
    same tokens and the same log-probability bits; prefill in blocks of 64, 5 and 1."""
    steps = 40
    dec = decoder(dev, weights, kv)
    dec.prefill(prompts(4))
    want = dec.decode(steps)
    want_lp = dec.trace_logprobs
    assert all(len(t) == steps for t in want_lp) and all(x <= 0 for t in want_lp for x in t)
    for width, drafter in ((4, random_drafter(CFG.vocab, 5)),
                           (4, reference_drafter(want, 0.3, CFG.vocab)),
                           (3, reference_drafter(want, 0.0, CFG.vocab))):
        dec.prefill(prompts(4), width=5 if width == 3 else 64)
        got, _, _ = dec.speculate(steps, width, drafter)
        assert got == want and dec.trace_logprobs == want_lp
    dec.prefill(prompts(4)[2:3], width=1)
    assert dec.decode(steps) == want[2:3] and dec.trace_logprobs == want_lp[2:3]
    assert bi.device_status() == bi.BI_OK


def test_q8_logits_are_near_the_bf16_ones(dev, weights):
    """E4M3 holds a value to 2^-4 of itself; keys and values enter the logits through averages
    over the context: the logits of the two caches differ by less than that."""
    a, b = decoder(dev, weights, "bf16"), decoder(dev, weights, "q8")
    for d in (a, b):
        d.prefill(prompts(4))
        d.forward(d.last, [1] * 4)
    x, y = a.logits[:4].double(), b.logits[:4].double()
    assert float((x - y).norm() / x.norm()) < 2.0 ** -4
    assert not torch.equal(x, y)


@pytest.mark.parametrize("kv", ["bf16", "q8"])
@pytest.mark.parametrize("length", [64, 65, 129, 150])
def test_forks_continue_as_copies_do(dev, weights, kv, length):
    """Forked sequences (full pages shared, the open page copied) decode, each from a token of its
    own, exactly as sequences whose prompts were computed apart; then the pool is compacted and
    decoding goes on unchanged."""
    firsts = [5, 77, 900]
    prompt = prompts(1, length)[0]
    apart = decoder(dev, weights, kv)
    apart.prefill([prompt] * 4)
    apart.last[1:] = firsts
    want = apart.decode(30)
    want_lp = apart.trace_logprobs
    dec = decoder(dev, weights, kv)
    dec.prefill([prompt])
    dec.fork(0, 3, firsts)
    shared = (length - 1) // 64
    assert all(dec.tables[j][:shared] == dec.tables[0][:shared] for j in range(4))
    got = dec.decode(12)
    lp = dec.trace_logprobs
    used = dec.compact()
    assert used == dec.num_pages - 3 * shared
    assert max(p for t in dec.tables for p in t) == used - 1
    got = [a + b for a, b in zip(got, dec.decode(18))]
    assert got == want
    assert [a + b for a, b in zip(lp, dec.trace_logprobs)] == want_lp
    # a snapshot of shared pages, and a new start after forks
    snap = dec.snapshot()
    more = dec.decode(5)
    dec.prefill([prompt] * 4)
    assert len({p for t in dec.tables for p in t}) == dec.num_pages
    dec.restore(snap)
    assert dec.decode(5) == more
    assert bi.device_status() == bi.BI_OK


def test_fork_refusals(dev, weights):
    dec = decoder(dev, weights)
    dec.prefill(prompts(2, 70))
    for bad in (dict(slot=2, n=1), dict(slot=-1, n=1), dict(slot=0, n=3), dict(slot=0, n=-1),
                dict(slot=0, n=1, first_tokens=[1, 2])):
        with pytest.raises(ValueError):
            dec.fork(**bad)
    dec.fork(1, 0)
    with pytest.raises(ValueError):
        GreedyDecoder(CFG, weights, max_batch=1, max_len=400, device=dev, kv_cache="int8")


def test_logprobs_gradient_of_a_decoded_block(dev, weights):
    """The trainer's side: the decoder's logits, its tokens' log-probabilities recomputed in one
    batch (the sampler's bits), and their gradient against differences of the definition."""
    dec = decoder(dev, weights)
    dec.prefill(prompts(4))
    rows, toks, lps = [], [], []
    for _ in range(6):
        t = dec.forward(dec.last, [1] * 4)
        rows.append(dec.logits[:4].clone())
        toks.append(t.clone())
        lps.append(dec.token_stats.logprobs.clone())
        dec.last = t.tolist()
        dec.cached = [c + 1 for c in dec.cached]
    x, tok = torch.cat(rows), torch.cat(toks)
    r = bi.token_logprobs(x, tok, top=3)
    assert bits_equal(r.logprobs, torch.cat(lps))
    assert torch.equal(r.top_ids[:, 0], tok) and bits_equal(r.top_logprobs[:, 0].contiguous(),
                                                            r.logprobs)
    g = torch.linspace(-1, 1, len(tok), device=dev)
    d = bi.token_logprobs_backward(x, tok, r.lse, r.entropy, g).double().cpu()
    x64, eps = x.double().cpu(), 1e-4
    for i, j in ((0, 0), (5, int(tok[5])), (23, 17), (11, int(tok[11]))):
        e = torch.zeros_like(x64[i])
        e[j] = eps
        t = int(tok[i])
        up, down = (torch.log_softmax(x64[i] + s * e, -1)[t] for s in (1, -1))
        assert abs(float(g[i]) * float(up - down) / (2 * eps) - float(d[i, j])) < 1e-6
