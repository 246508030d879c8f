"""Keys and values that no query of a block sees (prefill: of a tile of 128 / G tokens) are part of
no sum, whatever they hold: attention with limits over caches with NaN and infinities in them."""
import numpy as np
import pytest
import torch

from test_gpu_shaped_scores import PAGE, Paged, alibi

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def holes(pos, every, run):
    """First keys where `run` of each `every` tokens see nothing, and the last token neither."""
    n = np.arange(len(pos))
    first = np.where(n % every < run, pos + 1 + n % 3, np.maximum(pos - pos % 40 - 20, 0))
    first[-1] = 2 ** 31 - 1
    return first


SHAPES = {
    "window": lambda p: dict(window=37),
    "documents": lambda p: dict(first_key=p.pos - p.pos % 90),
    "documents, capped": lambda p: dict(first_key=p.pos - p.pos % 90, softcap=3.0),
    "holes": lambda p: dict(first_key=holes(p.pos, 7, 3)),
    "long holes": lambda p: dict(first_key=holes(p.pos, 100, 80), slopes=alibi(p.hq)),
    "own key alone": lambda p: dict(first_key=np.where(np.arange(p.T) % 2, p.pos, p.pos + 1),
                                    softcap=3.0, slopes=alibi(p.hq)),
    "window and holes": lambda p: dict(first_key=holes(p.pos, 5, 2), window=70, softcap=3.0),
}


def seen_by(p, tokens):
    """Which keys of the tokens' (one) sequence any of them sees."""
    low = p.low()
    seen = np.zeros(p.lens[p.seq[tokens[0]]], dtype=bool)
    for t in tokens:
        seen[min(low[t], len(seen)):p.pos[t] + 1] = True
    return seen


def poison(p, unseen, value):
    """Caches of p with the keys and values of sequence b's unseen places spoilt."""
    kv = p.kv.clone()
    for b, gone in unseen.items():
        j = np.nonzero(gone)[0]
        page = p.table[b].long()[j // PAGE]
        kv[0, page, :, j % PAGE] = float("nan")
        kv[1, page, :, j % PAGE] = value
    return kv


def same(got, want, rows=slice(None)):
    return (torch.equal(got[0][rows].view(torch.int16), want[0][rows].view(torch.int16))
            and torch.equal(got[1][rows], want[1][rows]))


@pytest.mark.parametrize("value", [float("nan"), float("-inf")])
@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("form,lens,qs,hq,hkv,D", [
    ("decode", [130, 700, 64, 1], [1, 1, 1, 1], 8, 2, 64),
    ("verify", [130, 700, 66, 5], [8, 4, 3, 5], 8, 2, 128),
    ("verify", [515, 64, 70], [8, 2, 7], 4, 4, 64),
    ("prefill", [300, 70, 600], [300, 1, 90], 8, 2, 64),
    ("prefill", [700, 40], [260, 40], 2, 2, 128)])
def test_what_a_block_does_not_see(dev, form, lens, qs, hq, hkv, D, name, value):
    p = Paged(dev, lens, qs, hq, hkv, D, seed=21)
    p.shape = SHAPES[name](p)
    want = p.run(form)
    p.check(*want)
    unseen = {b: ~seen_by(p, np.nonzero(p.seq == b)[0]) for b in range(len(lens))}
    kv = poison(p, unseen, value)
    p.k, p.v = kv[0].to(dev), kv[1].to(dev)
    assert same(p.run(form), want)
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("hq,hkv,D,long", [(8, 2, 64, False), (2, 2, 128, False), (32, 2, 64, False),
                                           (8, 2, 64, True)])
def test_what_a_tile_does_not_see(dev, hq, hkv, D, long, name):
    """A tile's outputs do not depend on what lies behind its last token, either; long: blocks
    whose first keys are found in a launch of their own."""
    lens, qs = ([1900, 300], [1640, 33]) if long else ([620, 300], [333, 33])
    p = Paged(dev, lens, qs, hq, hkv, D, seed=22)
    p.shape = SHAPES[name](p)
    want = p.run("prefill")
    assert bi.device_status() == bi.BI_OK
    size = 128 // (hq // hkv)
    tiles = [(t0, min(t0 + size, qs[0])) for t0 in range(0, qs[0], size)]
    for t0, t1 in tiles[:3] + tiles[-2:]:
        kv = poison(p, {0: ~seen_by(p, np.arange(t0, t1))}, float("nan"))
        p.k, p.v = kv[0].to(dev), kv[1].to(dev)
        assert same(p.run("prefill"), want, slice(t0, t1)), (t0, t1)
    assert bi.device_status() == bi.BI_OK
