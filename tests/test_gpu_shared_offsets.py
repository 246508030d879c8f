"""Prefill with first keys where token offsets fall so far that two sequences share their tiles'
places: the sequences apart from them get what they get alone, however often the call is made."""
import pytest
import torch

from test_gpu_shaped_scores import Paged, i32

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.mark.parametrize("fall", [21, 20, 15])
@pytest.mark.parametrize("total", [180, 1700])
def test_the_others_keep_their_results(total, fall):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev = "cuda:0"
    # tokens 0..19, 20..89, a fall, tokens from there on to total - 30, and the last 30
    lens, cu = [300, 200, 64, 5000, 700], [0, 20, 90, fall, total - 30, total]
    p = Paged(dev, lens, [20, 70, 1, total - 121, 30], 8, 2, 64, seed=31)
    assert p.T == total
    first = torch.full((total,), 4600, dtype=torch.int32)
    first[:90] = torch.arange(90, dtype=torch.int32)
    first[-30:] = 640
    first = first.to(dev)
    tables = p.table.to(dev), i32(lens, dev)
    kw = dict(max_seq_len=5000, scale=p.scale, max_q=total)
    apart = {slice(0, min(20, fall)): (0, 20), slice(total - 30, total): (4, 30)}
    want = {}
    for rows, (b, n) in apart.items():
        at = slice(0, n) if b == 0 else rows
        r = bi.prefill_attn(p.q[at].contiguous(), p.k, p.v, *(x[b:b + 1] for x in tables),
                            i32([0, n], dev), first_key=first[at].contiguous(), **kw)
        want[rows] = [x[:rows.stop - rows.start] for x in r]
    assert bi.device_status() == bi.BI_OK
    for fill in (0, 0x7f, 0xff, 0x3f):
        ws = torch.full((bi.attn_workspace_size(total, 8, 64, 5000),), fill, dtype=torch.uint8,
                        device=dev)
        out, lse = bi.prefill_attn(p.q, p.k, p.v, *tables, i32(cu, dev), first_key=first,
                                   workspace=ws, **kw)
        assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
        for rows, (o, l) in want.items():
            assert torch.equal(out[rows].view(torch.int16), o.view(torch.int16))
            assert torch.equal(lse[rows], l)
