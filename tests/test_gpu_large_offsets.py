"""The rotating append, shaped attention and draft verification where offsets pass 32 bits: caches
of more than 2^32 bytes and 2^31 values, logits of more than 2^31 entries."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    return torch.device("cuda:0")


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("bits", [16, 8])
def test_append_and_attend_in_a_large_cache(dev, bits):
    """Sequences whose pages lie at the ends of the cache, and one cache's worth of them apart;
    the same bits as in a small cache."""
    hq, hkv, D, pages = 8, 8, 128, 70000          # 4.6e9 values a cache
    near, far = [0, 1, 2, 3], [pages - 1, 5, pages // 2, pages - 3]
    g = torch.Generator().manual_seed(1)
    lens, qs = [120, 65], [100, 65]
    q, k, v = (torch.randn(165, h, D, generator=g).to(torch.bfloat16).to(dev)
               for h in (hq, hkv, hkv))
    args = (i32(lens, dev), i32([0, 100, 165], dev))
    got = []
    for n, at in ((4, near), (pages, far)):
        dtype = torch.bfloat16 if bits == 16 else torch.uint8
        cache = [torch.empty(n, hkv, 64, D, dtype=dtype, device=dev) for _ in range(2)]
        if bits == 8:
            cache += [torch.empty(n, hkv, 64, dtype=dtype, device=dev) for _ in range(2)]
        for c in cache:
            c[at] = 0
        table = i32([at[:2], at[2:]], dev)
        fn = bi.rope_kv_append if bits == 16 else bi.rope_kv_append_q8
        turned = fn(q, k, v, *cache, table, *args)
        rows = [c[at].clone() for c in cache]
        if bits == 16:
            o, l = bi.prefill_attn(turned, *cache, table, *args, max_q=100, max_seq_len=120,
                                   scale=D ** -0.5, softcap=20.0, window=50)
            rows += [o[20:], l[20:]]              # (positions below 20 hold zeros in front)
        assert bi.device_status() == bi.BI_OK
        got.append([turned] + rows)
        del cache
        torch.cuda.empty_cache()
    for a, b in zip(*got):
        assert torch.equal(a, b)


def test_drafts_of_a_large_batch_of_logits(dev):
    """17,000 rows of 131,072 entries (2.2e9): every sequence has the same two rows, so all decide
    and draw as one does alone."""
    B, n = 8500, 131072
    g = torch.Generator().manual_seed(2)
    two = (torch.randn(2, n, generator=g) * 2).to(torch.bfloat16).to(dev)
    draft = (two[:1].float() + 0.5).to(torch.bfloat16)
    draft[0, ::2] = two[0, ::2]
    logits = two.repeat(B, 1)
    near = draft.repeat(B, 1)
    u = torch.rand(2, generator=g)
    tok = i32([int(two[0].argmax())], dev)
    r = bi.verify_drafts(logits, tok.repeat(B), u.repeat(B).to(dev),
                         (torch.arange(B + 1, dtype=torch.int32) * 2).to(dev), max_q=2,
                         draft_logits=near, temperature=0.9)
    one = bi.verify_drafts(two, tok, u.to(dev), i32([0, 2], dev), max_q=2, draft_logits=draft,
                           temperature=0.9)
    assert bi.device_status() == bi.BI_OK
    for x, y in zip(r, one):
        assert bool((x == y[0]).all()), (x[0], y[0])
    assert int(one.accepted[0]) in (0, 1) and np.isfinite(one.logprobs.cpu().numpy()).all()
