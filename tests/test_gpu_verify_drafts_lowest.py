"""Log-probabilities of kept drafts whose entry is the type's lowest value (a mask): finite where
fp32 holds them, -inf where not, never NaN.  A uniform of 0 keeps every draft that p can say."""
import numpy as np
import pytest
import torch

from test_gpu_verify_drafts import Batch, softmax

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.mark.parametrize("draft", ["logits", "tokens"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("temperature", [1.0, 0.25, 0.75, 1.25, 8.0])
@pytest.mark.parametrize("n", [40, 5003])
def test_masked_drafts(n, temperature, dtype, draft):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    b = Batch([3, 2], n, dtype, draft, seed=3, temps=[temperature] * 2)
    lowest = torch.finfo(b.dtype).min
    b.logits[:, 1::2] = lowest
    b.drafts[:] = torch.tensor([1, 3, 39])
    b.u[:] = 0.0
    r = b.run("cuda:0")
    assert bi.device_status() == bi.BI_OK
    assert r.accepted.tolist() == [2, 1]
    assert r.tokens[0, :2].tolist() == [1, 3] and int(r.tokens[1, 0]) == 39
    for s, j in ((0, 0), (0, 1), (1, 0)):
        row = b.logits[int(b.cu[s]) + j].double().numpy()
        want = softmax(row, temperature)[1][int(b.drafts[int(b.cu[s]) - s + j])]
        got = float(r.logprobs[s, j])
        # (three roundings of 2^-24, and 1/T's own)
        if want < -float(np.finfo(np.float32).max):
            assert got == -float("inf")
        else:
            assert abs(got - want) <= 2.0 ** -22 * abs(want)
    assert bool(r.logprobs[0, 2:].isfinite().all()) and float(r.logprobs[1, 1]) > -50
