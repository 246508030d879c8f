"""Sampled speculation at temperature 0 leaves the caches that token-by-token decoding leaves: the
same bits in every row of a token that both came to, whatever blocks the tokens came in."""
import pytest
import torch

from test_gpu_decoder_sampled import CFG, KINDS, decoder, prompts, weights  # noqa: F401
from invariant_bi_matmul_gb300.decoder import random_drafter, reference_drafter

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def planes(dec):
    names = ("k_cache", "v_cache") + (("k_scale", "v_scale") if dec.kv_cache == "q8" else ())
    return [getattr(dec, name) for name in names]


def rows(dec, b, n):
    """The first n tokens' rows of sequence b, in every layer and plane."""
    page = torch.tensor([dec.tables[b][p // 64] for p in range(n)], device=dec.dev)
    slot = torch.arange(n, device=dec.dev) % 64
    return [layer[page, :, slot].clone() for plane in planes(dec) for layer in plane]


@pytest.mark.parametrize("kind", list(KINDS) + ["q8"])
def test_the_same_rows(dev, weights, kind):  # noqa: F811
    steps, length = 40, 150
    dec = decoder(dev, weights, **(KINDS | {"q8": dict(kv_cache="q8")})[kind])
    dec.prefill(prompts(4, length))
    want = dec.decode(steps)
    n = dec.cached[0]                            # the prompt and every token that was fed back
    assert dec.cached == [n] * 4 and n >= length + steps - 1
    kept = [rows(dec, b, n) for b in range(4)]
    assert all(bool((r.float() != 0).any()) for r in kept[0])
    for width, drafter in ((4, random_drafter(CFG.vocab, 5)),
                           (4, reference_drafter(want, 0.3, CFG.vocab)),
                           (3, reference_drafter(want, 0.0, CFG.vocab)),
                           (1, random_drafter(CFG.vocab, 6))):
        for plane in planes(dec):
            for layer in plane:
                layer.zero_()
        dec.prefill(prompts(4, length), width=7 if width == 3 else 64)
        got, _, _ = dec.speculate_sampled(steps, width, drafter, 0.0)
        assert got == want
        for b in range(4):
            assert dec.cached[b] >= n
            for x, y in zip(rows(dec, b, n), kept[b]):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert bi.device_status() == bi.BI_OK
