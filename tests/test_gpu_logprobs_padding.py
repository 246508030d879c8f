"""The gradient of rows that carry none (padding, masked tokens): zeros, whatever the logits are."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [7, 1000, 1001, 40000])
@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("other", [False, True])
def test_rows_without_a_gradient(dtype, n, entropy, other):
    """Token -1, or a token whose gradients are 0, in rows of NaN, infinities, nothing but -inf
    and ordinary numbers; the other rows keep theirs.  other: dx not aligned as x is."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    x = torch.randn(9, n, generator=torch.Generator().manual_seed(n)).to(dtype).cuda()
    x[0] = math.nan
    x[1] = -math.inf
    x[2, n // 2] = math.inf
    x[3, :2] = math.nan
    tok = torch.tensor([-1, -1, -1, 2, -1, 4, 5, 1, -1], dtype=torch.int32, device="cuda")
    gl = torch.ones(9, device="cuda")
    gl[3] = gl[5] = 0
    ge = torch.zeros(9, device="cuda") if entropy else None
    if entropy:
        ge[7] = 0.5
    r = bi.token_logprobs(x, tok)
    out = torch.full((9, n + 5), 3.0, dtype=dtype, device="cuda")[:, 3:n + 3] if other else None
    d = bi.token_logprobs_backward(x, tok, r.lse, r.entropy if entropy else None, gl, ge, out=out)
    assert bool((d[[0, 1, 2, 3, 4, 5, 8]] == 0).all())
    assert bool((d[[6, 7]] != 0).any(-1).all()) and bool(torch.isfinite(d).all())
    assert bi.device_status() == bi.BI_OK
