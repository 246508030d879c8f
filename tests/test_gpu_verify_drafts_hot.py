"""Every finite temperature is served: at fp32's largest, entries of ordinary size weigh alike."""
import numpy as np
import pytest
import torch

from test_gpu_verify_drafts import Batch, check

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.mark.parametrize("draft", ["logits", "tokens"])
@pytest.mark.parametrize("temperature", [3.4e38, 3.4015e38, float(np.finfo(np.float32).max)])
def test_the_largest_temperatures(temperature, draft):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    b = Batch([3, 1, 4], 600, "bf16", draft, seed=6, temps=[temperature] * 3)
    b.logits[:, ::5] = -float("inf")
    b.drafts[:] = torch.tensor([1, 2, 3, 4, 6])
    r = b.run("cuda:0")
    assert all(torch.equal(x, y) for x, y in zip(r, b.run("cuda:0", temps=temperature)))
    if draft == "tokens":  # (with p = q throughout but the masked entries, borders lie on one another)
        check(b, r)
    assert bi.device_status() == bi.BI_OK and bool((r.tokens[:, 0] >= 0).all())
