"""Block offsets whose sums or differences pass 2^31 are reported, and nothing is read or written
for them: the bf16 and the 8-bit cache's appends and attention."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")

OFFSETS = [(0, 2 ** 31 - 1, -2 ** 31), (-2 ** 31, 2, 3), (-2 ** 31, 2 ** 31 - 1, -2 ** 31)]


@pytest.mark.parametrize("offsets", OFFSETS)
@pytest.mark.parametrize("D", [64, 128])
def test_offsets_that_wrap(offsets, D):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev, Hq, Hkv, pages = "cuda", 8, 2, 4
    i32 = dict(dtype=torch.int32, device=dev)
    table = torch.arange(pages, **i32).view(2, 2)
    sl, cu = torch.tensor([70, 70], **i32), torch.tensor(offsets, **i32)
    q = torch.ones(3, Hq, D, dtype=torch.bfloat16, device=dev)
    new = torch.ones(3, Hkv, D, dtype=torch.bfloat16, device=dev)
    k, v = (torch.ones(pages, Hkv, 64, D, dtype=torch.bfloat16, device=dev) * 2 for _ in range(2))
    codes = [torch.full((pages, Hkv, 64, D), 3, dtype=torch.uint8, device=dev) for _ in range(2)]
    scales = [torch.full((pages, Hkv, 64), 100, dtype=torch.uint8, device=dev) for _ in range(2)]
    assert bi.device_status() == bi.BI_OK

    # the sequences that are whole: the rows of (2, 3) in the second list
    whole = offsets[1:] == (2, 3)
    bi.kv_append(new, new, k, v, table, sl, cu)
    assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
    bi.kv_append_q8(new, new, *codes, *scales, table, sl, cu)
    assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
    written = (k != 2).flatten(1).any(1).tolist()
    assert written == [False, False, False, whole] == (scales[0] != 100).flatten(1).any(1).tolist()

    rest = dict(max_q=2, max_seq_len=70, scale=0.1)
    for call in (lambda o: bi.verify_block(q, k, v, table, sl, cu, out=o, **rest),
                 lambda o: bi.prefill_attn(q, k, v, table, sl, cu, out=o, **rest),
                 lambda o: bi.verify_block_q8(q, *codes, *scales, table, sl, cu, out=o, **rest),
                 lambda o: bi.prefill_attn_q8(q, *codes, *scales, table, sl, cu, out=o, **rest)):
        out = torch.full_like(q, 7.0)
        call(out)
        assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
        assert bool((out[:2] == 7).all()) and bool((out[2] == 7).all()) != whole
    assert bi.device_status() == bi.BI_OK
