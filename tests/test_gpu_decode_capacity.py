"""Decode calls whose buffers hold more sequences than they serve: q's rows say how many, and
nothing behind them is read or written."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.mark.parametrize("own_workspace", [False, True])
@pytest.mark.parametrize("active", [1, 3, 6])
def test_the_rows_of_q_are_served(active, own_workspace):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev, hq, hkv, D, seqs, pages = "cuda:0", 8, 2, 64, 6, 4
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(seqs * pages, hkv, 64, D, generator=g).bfloat16().to(dev) for _ in "kv")
    table = torch.randperm(seqs * pages, generator=g).int().reshape(seqs, pages).to(dev)
    lens = torch.tensor([200, 1, 64, 130, 255, 17], dtype=torch.int32, device=dev)
    q = torch.randn(seqs, hq, D, generator=g).bfloat16().to(dev)
    kw = dict(max_seq_len=256, scale=0.125)
    want, want_lse = bi.decode_attn(q, k, v, table, lens, **kw)
    # the capacity's buffers, of which the call gets the first rows
    out = torch.full((seqs, hq, D), 7.0, dtype=torch.bfloat16, device=dev)
    lse = torch.full((seqs, hq), 7.0, device=dev)
    if own_workspace:
        kw["workspace"] = torch.empty(bi.attn_workspace_size(seqs, hq, D, 256), dtype=torch.uint8,
                                      device=dev)
    bi.decode_attn(q[:active], k, v, table, lens, out=out[:active], lse=lse[:active], **kw)
    assert bi.device_status() == bi.BI_OK
    assert torch.equal(out[:active], want[:active]) and torch.equal(lse[:active], want_lse[:active])
    assert (out[active:] == 7.0).all() and (lse[active:] == 7.0).all()


def test_more_queries_than_sequences_are_refused():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = "cuda:0"
    k = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16, device=dev)
    i32 = dict(dtype=torch.int32, device=dev)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=dev)
    for seqs, rows in ((2, 3), (3, 2)):
        with pytest.raises(ValueError):
            bi.decode_attn(q, k, k, torch.zeros(rows, 2, **i32), torch.ones(seqs, **i32),
                           max_seq_len=64, scale=1.0)
