"""Token log-probabilities of many rows of several parts: a CTA takes one part of its row, some of
them or all, as the number of rows has it, and that changes no bit."""
import numpy as np
import pytest
import torch

from test_gpu_token_logprobs import check, ranked
from tolerance import bits_equal

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")

TYPES = [torch.float32, torch.bfloat16, torch.float16]


# rows for a cluster of as many CTAs as parts (4 and 8), for divisors of that, and for one
# CTA a row, on a GPU of 152 multiprocessors
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [50001, 65536, 100000, 128256, 128255])
@pytest.mark.parametrize("rows", [30, 50, 100, 200, 320])
def test_rows_of_several_parts(dtype, n, rows):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    g = torch.Generator(device="cuda").manual_seed(n + rows)
    x = (torch.randn(rows, n, generator=g, device="cuda") * 2.5).to(dtype)
    x[1, ::2] = -float("inf")                                   # the second pass over the sums
    x[2] = (torch.arange(n, device="cuda") % 3).to(dtype)       # ties beyond the candidates' list
    x[3] = 1.5
    x[4, 5:] = -float("inf")
    x[5, n - 3:] = 9.0                                          # the top in the last part
    x[6, 17], x[6, n // 2] = 20.0, 20.0
    tok = torch.randint(0, n, (rows,), generator=g, device="cuda", dtype=torch.int32)
    tok[1], tok[4] = 1, 3
    every = bi.token_logprobs(x, tok, top=20)
    sample = [0, 1, 2, 3, 4, 5, 6, rows // 2, rows - 1]
    for r in sample:
        one = bi.token_logprobs(x[r:r + 1].clone(), tok[r:r + 1], top=20)
        for a, b in zip(one[:4], every[:4]):
            assert bits_equal(a[0], b[r]), r
        assert torch.equal(one.top_ids[0], every.top_ids[r]), r
    plain = bi.token_logprobs(x, tok)
    for a, b in zip(plain[:3], every[:3]):
        assert bits_equal(a, b)
    ids = every.top_ids.cpu().numpy()
    assert np.array_equal(ids[[1, 2, 3, 4, 6]], ranked(x[[1, 2, 3, 4, 6]].cpu(), 20))
    for r in (0, rows - 1):
        check(bi.TokenLogprobs(*(t[r:r + 1] for t in every)), x[r:r + 1].cpu(), tok[r:r + 1].cpu(),
              20)
    assert bi.device_status() == bi.BI_OK
