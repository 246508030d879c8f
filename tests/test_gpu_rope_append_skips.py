"""The rotating append over a malformed block or a bad page: what is skipped stays as it was to the
byte, scales included, and every other token is served as in a good call."""
import pytest
import torch

from test_gpu_rope_append import Block

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")

LENS, QS = [70, 30, 200], [6, 5, 140]
T = sum(QS)


def places(blk, b):
    """(page, slot) of the new tokens of sequence b, by the lengths the cache was laid out for."""
    n, w = LENS[b], QS[b]
    return [(int(blk.good_table[b, p // 64]), p % 64) for p in range(n - w, n)]


def block(bits, D, hq=4, hkv=2):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    blk = Block("cuda:0", LENS, QS, hq, hkv, D, bits, seed=4)
    blk.good_table = blk.table.clone()
    blk.out = torch.full((T, hq, D), 3.0, dtype=torch.bfloat16, device="cuda:0")
    return blk


def call(blk):
    fn = bi.rope_kv_append if blk.bits == 16 else bi.rope_kv_append_q8
    fn(blk.q, blk.k, blk.v, *blk.cache, blk.table, blk.sl, blk.cu, out=blk.out)
    return bi.device_status()


def compare(blk, good, turned, appended):
    """turned: tokens whose queries are written; appended: (page, slot) whose rows are."""
    rows = torch.zeros(T, dtype=torch.bool, device="cuda:0")
    rows[turned] = True
    assert torch.equal(blk.out[rows], good.out[rows])
    assert bool((blk.out[~rows] == 3.0).all())
    pages, _, slots = blk.cache[0].shape[:3]
    touched = torch.zeros(pages, slots, dtype=torch.bool, device="cuda:0")
    for page, slot in appended:
        touched[page, slot] = True
    for plane, was, want in zip(blk.cache, blk.before, good.cache):
        mask = touched[:, None].expand(plane.shape[:3])
        assert torch.equal(plane[mask], want[mask])
        assert torch.equal(plane[~mask], was[~mask])


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [-1, -2 ** 31, 10 ** 6, 2 ** 31 - 1, "pages"])
def test_rows_without_a_page(bits, D, bad):
    good, blk = block(bits, D), block(bits, D)
    assert call(good) == bi.BI_OK
    blk.table[0, 1] = blk.table[2, 2] = blk.cache[0].shape[0] if bad == "pages" else bad
    assert call(blk) == bi.BI_ERR_DEVICE_ARG
    gone = {(0, p) for p in range(64, 70)} | {(2, p) for p in range(128, 192)}
    keep = [at for b in range(3) for p, at in zip(range(LENS[b] - QS[b], LENS[b]), places(blk, b))
            if (b, p) not in gone]
    compare(blk, good, list(range(T)), keep)


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("change,skipped", [
    (lambda b: b.sl.__setitem__(0, 5), [0]),             # a block longer than its sequence
    (lambda b: b.sl.__setitem__(1, 100000), [1]),        # ... than its row of the table
    (lambda b: b.sl.__setitem__(1, -1), [1]),
    (lambda b: b.cu.__setitem__(3, T + 1), [2]),         # past the last token
    (lambda b: b.cu.__setitem__(0, -1), [0]),
    (lambda b: b.cu.__setitem__(0, -2 ** 31), [0])])
def test_malformed_sequences(bits, D, change, skipped):
    good, blk = block(bits, D), block(bits, D)
    assert call(good) == bi.BI_OK
    change(blk)
    assert call(blk) == bi.BI_ERR_DEVICE_ARG
    served = [b for b in range(3) if b not in skipped]
    first = [0, 6, 11, T]
    compare(blk, good, [t for b in served for t in range(first[b], first[b + 1])],
            [at for b in served for at in places(blk, b)])


@pytest.mark.parametrize("bits", [16, 8])
def test_tokens_of_no_sequence(bits):
    """In front of the first offset and behind the last: left alone, and no error."""
    good, blk = block(bits, 64), block(bits, 64)
    assert call(good) == bi.BI_OK
    blk.cu[0], blk.sl[0] = 2, 70                          # four of the first sequence's six
    blk.cu[3], blk.sl[2] = T - 10, 190
    assert call(blk) == bi.BI_OK
    compare(blk, good, list(range(2, T - 10)),
            places(blk, 0)[2:] + places(blk, 1) + places(blk, 2)[:-10])
