"""Verification of drafts at temperature 0 where rows have no distribution: the block ends there,
as at any other temperature."""
import pytest
import torch

from test_gpu_verify_drafts import Batch

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")
from invariant_bi_matmul_gb300 import inputs  # noqa: E402
from invariant_bi_matmul_gb300.decoder import GreedyDecoder, lookup_drafter  # noqa: E402


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def greedy(widths, n, dtype, draft):
    """A batch whose drafts are the largest entries of their rows."""
    b = Batch(widths, n, dtype, draft, seed=n, temps=[0.0] * len(widths))
    d = 0
    for s, w in enumerate(widths):
        for j in range(w - 1):
            b.drafts[d] = int(b.logits[int(b.cu[s]) + j].float().argmax())
            d += 1
    return b


@pytest.mark.parametrize("draft", ["logits", "tokens"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n,batch", [(1, 1), (700, 4), (700, 320), (40003, 4), (150001, 1)])
@pytest.mark.parametrize("bad", ["nan", "inf", "-inf"])
def test_rows_without_a_distribution(dev, n, batch, dtype, draft, bad):
    if draft == "logits" and batch == 320 and dtype != "bf16":
        return
    W = 4
    b = greedy([W] * batch, n, dtype, draft)
    r = b.run(dev)
    assert r.accepted.tolist() == [W - 1] * batch and bool(r.logprobs.isfinite().all())
    for j in range(W):                                # the row of the block that is bad
        c = greedy([W] * batch, n, dtype, draft)
        rows = torch.arange(batch) * W + j
        if bad == "-inf":
            c.logits[rows] = -float("inf")
        else:
            c.logits[rows, torch.arange(batch) % n] = float(bad)
        got = c.run(dev)
        assert got.accepted.tolist() == [j] * batch
        assert torch.equal(got.tokens[:, :j], r.tokens[:, :j])
        assert torch.equal(got.logprobs[:, :j], r.logprobs[:, :j])
        assert bool((got.tokens[:, j:] == -1).all())
        assert bool(got.logprobs[:, j].isnan().all()) and not bool(got.logprobs[:, j + 1:].any())
    if b.near is not None:                            # draft rows take no part
        b.near[:] = float("nan")
        assert all(torch.equal(x, y) for x, y in zip(b.run(dev), r))
    assert bi.device_status() == bi.BI_OK


def test_entries_of_minus_infinity_and_the_lowest_value(dev):
    for dtype in ("fp32", "bf16", "fp16"):
        b = greedy([3] * 2, 900, dtype, "tokens")
        for mask in (-float("inf"), torch.finfo(b.dtype).min):
            b.logits[:, ::2] = mask
            b.logits[:, 7] = 30.0
            b.drafts[:] = 7
            r = b.run(dev)
            assert r.accepted.tolist() == [2, 2] and r.tokens.tolist() == [[7] * 3] * 2


def test_the_decoder_reports_them(dev):
    cfg = inputs.TINY_DECODER
    w = {k: v.to(dev) for k, v in inputs.decoder_weights(cfg, 800, std=0.05, norm_std=0.1).items()}
    dec = GreedyDecoder(cfg, w, max_batch=2, max_len=400, max_width=4, device=dev, page_seed=3,
                        prefill_width=64)
    dec.prefill([inputs.decoder_prompt(cfg, s, 801, 150) for s in range(2)])
    dec.w = {k: torch.full_like(v, float("nan")) if v.dim() == 1 else v for k, v in w.items()}
    with pytest.raises(RuntimeError, match="no distribution"):
        dec.speculate_sampled(3, 2, lookup_drafter, 0.0)
