"""bi_kv_copy_pages on the GPU: bytes move whole, in every plane, and nothing else changes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def planes(n, pages, dev, seed=0):
    """Planes of unlike page types: bf16 caches, 8-bit caches, scale bytes, one 16-byte page."""
    g = torch.Generator(device=dev).manual_seed(seed)
    shapes = [((pages, 2, 64, 64), torch.bfloat16), ((pages, 3, 64, 128), torch.uint8),
              ((pages, 1, 64), torch.uint8), ((pages, 16), torch.uint8),
              ((pages, 5, 64, 16), torch.float32)]
    out = []
    for i in range(n):
        shape, dt = shapes[i % len(shapes)]
        size = torch.empty(0, dtype=dt).element_size()
        raw = torch.randint(0, 256, shape[:-1] + (shape[-1] * size,), generator=g, device=dev,
                            dtype=torch.uint8)
        out.append(raw.view(dt))
    return out


@pytest.mark.parametrize("n_planes", [1, 5, 64, 65, 130])
@pytest.mark.parametrize("pages,n", [(2, 1), (40, 17)])
def test_copies_every_plane(dev, n_planes, pages, n):
    ps = planes(n_planes, pages, dev)
    before = [p.clone() for p in ps]
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(n)).to(torch.int32)
    src = perm[:n].clone()
    dst = perm[pages - n:].clone() if 2 * n <= pages else perm[n:2 * n]
    src[n // 2] = src[0]  # one source may feed several pages
    bi.kv_copy_pages(ps, src.to(dev), dst.to(dev))
    for p, b in zip(ps, before):
        want = b.clone()
        want[dst.long().to(dev)] = b[src.long().to(dev)]
        assert torch.equal(p.view(torch.uint8), want.view(torch.uint8))
    assert bi.device_status() == bi.BI_OK


def test_nothing_to_do_and_bad_indices(dev):
    ps = planes(5, 9, dev)
    before = [p.clone() for p in ps]
    none = torch.empty(0, dtype=torch.int32, device=dev)
    bi.kv_copy_pages(ps, none, none)
    bi.kv_copy_pages([], none, none)
    src = torch.tensor([0, 9, -1, 3, 4], dtype=torch.int32, device=dev)
    dst = torch.tensor([5, 6, 7, -2, 8], dtype=torch.int32, device=dev)
    bi.kv_copy_pages(ps, src, dst)
    assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
    for p, b in zip(ps, before):
        want = b.clone()
        want[5], want[8] = b[0], b[4]
        assert torch.equal(p.view(torch.uint8), want.view(torch.uint8))


def test_planes_past_32_bit_offsets(dev):
    """A plane of more than 2^32 bytes: its last pages."""
    pages, page = 70000, (8, 64, 128)
    p = torch.zeros(pages, *page, dtype=torch.uint8, device=dev)
    p[pages - 2] = 7
    src = torch.tensor([pages - 2, 0], dtype=torch.int32, device=dev)
    dst = torch.tensor([1, pages - 1], dtype=torch.int32, device=dev)
    p[0] = 9
    bi.kv_copy_pages([p], src, dst)
    assert bool((p[1] == 7).all()) and bool((p[pages - 1] == 9).all())
    assert int(p.view(-1, 65536)[:, 0].to(torch.int64).sum()) == 7 * 2 + 9 * 2
    assert bi.device_status() == bi.BI_OK


def test_captured(dev):
    ps = planes(5, 8, dev)
    src = torch.tensor([0, 1], dtype=torch.int32, device=dev)
    dst = torch.tensor([4, 5], dtype=torch.int32, device=dev)
    bi.kv_copy_pages(ps, src, dst)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bi.kv_copy_pages(ps, src, dst)
    src.copy_(torch.tensor([2, 3], dtype=torch.int32))
    dst.copy_(torch.tensor([6, 7], dtype=torch.int32))
    before = [p.clone() for p in ps]
    g.replay()
    torch.cuda.synchronize()
    for p, b in zip(ps, before):
        want = b.clone()
        want[6], want[7] = b[2], b[3]
        assert torch.equal(p.view(torch.uint8), want.view(torch.uint8))
