"""Token log-probabilities of rows of the type's lowest and largest finite values (a mask that
left nothing, or wrote the lowest value in place of -inf)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n", [1, 3, 9, 1000, 4097, 50001, 700001])
@pytest.mark.parametrize("rows", [1, 400])
def test_rows_of_the_lowest_value(dtype, n, rows):
    """log s is that of n equal entries, or of those that are not masked."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if rows * n > 10 ** 8:
        rows = 8
    f = torch.finfo(dtype)
    x = torch.full((rows, n), f.min, dtype=dtype, device="cuda")
    seen = n
    tok = torch.zeros(rows, dtype=torch.int32, device="cuda")
    for fill in (f.min, f.max, f.min / 2):
        x.fill_(fill)
        r = bi.token_logprobs(x, tok, top=min(3, n))
        assert bool((r.logprobs + math.log(n)).abs().le(2.0 ** -16 * (1 + math.log(n))).all())
        assert bool((r.entropy - math.log(n)).abs().le(2.0 ** -15 * (1 + math.log(n))).all())
        assert bool(((r.lse - float(x[0, 0])).abs() <= 1e-6 * abs(fill) + 1.1 * math.log(n)).all())
        assert bool((r.top_ids == torch.arange(min(3, n), device="cuda")).all())
    x.fill_(f.min)
    x[:, ::3] = 1.5
    x[:, n // 2:] = f.min
    seen = max(1, len(range(0, max(n // 2, 1), 3)))
    if n > 1:
        r = bi.token_logprobs(x, tok)
        assert bool((r.logprobs + math.log(seen)).abs().le(2.0 ** -16 * (1 + math.log(n))).all())
        assert bool((r.entropy - math.log(seen)).abs().le(2.0 ** -15 * (1 + math.log(n))).all())
    assert bi.device_status() == bi.BI_OK
