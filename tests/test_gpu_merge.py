"""The merge of chunk partials: which of its kernels and windows runs follows the call's rows and
chunks, and changes no bit."""
import pytest
import torch

import invariant_bi_matmul_gb300 as bi

pytestmark = pytest.mark.gpu


def bits(t):
    return t.view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


# 1 to 42 chunks of 512 keys: windows of 4, 8 and 9 partials for a warp per row, of 5 and 17 for
# a CTA per row, and their limits
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("L", [400, 2048, 2049, 4096, 4097, 4609, 8704, 8705, 20480, 20481, 21505])
def test_rows_of_a_large_batch_and_alone(D, L):
    dev, B, Hq, Hkv, pages = "cuda", 40, 32, 4, 400
    g = torch.Generator().manual_seed(L + D)
    # the last sequence is the longest: its length sizes the windows of both calls
    lens = [int(x) for x in torch.randint(1, L + 1, (B - 1,), generator=g)] + [L]
    table = torch.randint(0, pages, (B, -(-L // 64)), generator=g).int().to(dev)
    q = (torch.randn(B, Hq, D, generator=g) * 3).to(torch.bfloat16).to(dev)
    shape = (pages, Hkv, 64, D)
    k, v = (torch.randn(shape, generator=g).to(torch.bfloat16).to(dev) for _ in range(2))
    kc, vc = (torch.randint(0, 120, shape, generator=g).to(torch.uint8).to(dev) for _ in range(2))
    ks, vs = (torch.randint(118, 124, shape[:3], generator=g).to(torch.uint8).to(dev)
              for _ in range(2))
    sl = torch.tensor(lens, dtype=torch.int32, device=dev)

    def both(sel):
        rest = dict(max_seq_len=max(lens[b] for b in sel), scale=D ** -0.5)
        tab, s, x = (t[sel].contiguous() for t in (table, sl, q))
        return (*bi.decode_attn(x, k, v, tab, s, **rest),
                *bi.decode_attn_q8(x, kc, vc, ks, vs, tab, s, **rest))

    every = both(list(range(B)))                     # 1,280 rows: a warp each
    for b in (0, 13, B - 1):                         # 32 rows: a CTA each
        for got, want in zip(every, both([b])):
            assert torch.equal(bits(got[b]), bits(want[0]))
    assert bi.device_status() == bi.BI_OK
