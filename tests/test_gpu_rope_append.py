"""The rotating append on the GPU, against the rotation in 64 bits and the appends that the
library already has: queries, cache rows, and what has to stay as it was."""
import math

import numpy as np
import pytest
import torch

import q8_reference as ref

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")

THETA = 500000.0


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Block:
    """A ragged block of new tokens and a bf16 or 8-bit cache that holds a pattern."""

    def __init__(self, dev, lens, qs, hq, hkv, D, bits=16, seed=0, front=0, behind=0, fused=True):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.qs, self.hq, self.hkv, self.D, self.bits = lens, qs, hq, hkv, D, bits
        self.front, T = front, front + sum(qs) + behind
        qkv = (torch.randn(T, hq + 2 * hkv, D, generator=g)
               * torch.exp2(torch.randn(T, hq + 2 * hkv, 1, generator=g))).to(torch.bfloat16).to(dev)
        self.q, self.k, self.v = qkv.split([hq, hkv, hkv], 1)
        if not fused:
            self.q, self.k, self.v = (x.contiguous() for x in (self.q, self.k, self.v))
        need = [-(-n // 64) for n in lens]
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = perm[at:at + n]
            at += n
        self.table, self.sl = table.to(dev), i32(lens, dev)
        self.cu = i32(np.concatenate([[0], np.cumsum(qs)]) + front, dev)
        shape = (pages, hkv, 64, D)
        if bits == 16:
            self.cache = [torch.randn(shape, generator=g).to(torch.bfloat16).to(dev)
                          for _ in range(2)]
        else:
            self.cache = [torch.randint(0, 120, shape[:4 - i], generator=g,
                                        dtype=torch.uint8).to(dev) for i in (0, 0, 1, 1)]
        self.before = [c.clone() for c in self.cache]

    def run(self, **kw):
        fn = bi.rope_kv_append if self.bits == 16 else bi.rope_kv_append_q8
        kw = dict(theta=THETA) | kw
        q = fn(self.q, self.k, self.v, *self.cache, self.table, self.sl, self.cu, **kw)
        assert bi.device_status() == bi.BI_OK
        return q

    def tokens(self):
        """(token, sequence, position) of every token of a sequence."""
        t = self.front
        for b, (n, w) in enumerate(zip(self.lens, self.qs)):
            for j in range(w):
                yield t, b, n - w + j
                t += 1

    def place(self, b, pos):
        return int(self.table[b, pos // 64]), pos % 64


def turned(x, pos, R, freq):
    """Rows x [H, D] (float64) turned by pos[i] * freq[i], and how far fp32 may be off: the angle
    is off by 2^-51 of itself (the frequency's rounding, twice), its fraction of a turn is
    rounded to fp32 (2^-24 of at most pi), sincospi is within 2 ulp of at most 1 (2^-22), and the
    products and their sum are rounded (2^-24 each)."""
    a = np.asarray(pos, dtype=np.float64) * freq
    y, off = x.copy(), np.zeros_like(x)
    lo, hi = x[:, :R // 2], x[:, R // 2:R]
    c, s = np.cos(a), np.sin(a)
    y[:, :R // 2] = lo * c - hi * s
    y[:, R // 2:R] = hi * c + lo * s
    each = np.abs(a) * 2.0 ** -51 + math.pi * 2.0 ** -24 + 2.0 ** -22 + 3 * 2.0 ** -24
    off[:, :R // 2] = off[:, R // 2:R] = (np.abs(lo) + np.abs(hi)) * each
    return y, off


def check(got, want, off, what):
    """bf16 rounding on top: half a step, 2^-8 of the value."""
    g = got.detach().cpu().double().numpy()
    bad = np.abs(g - want) > 2.0 ** -8 * (np.abs(want) + off) + off + 2.0 ** -133
    assert not bad.any(), (what, np.argwhere(bad)[:3], g[bad][:3], want[bad][:3])


def frequencies(R, theta=THETA):
    return theta ** (-2.0 * np.arange(R // 2) / R)


def check_block(blk, q, R=None, freq=None, positions=None, axis=None):
    R = R or blk.D
    freq = frequencies(R) if freq is None else freq
    qr, kr = blk.q.cpu().double().numpy(), blk.k.cpu().double().numpy()
    touched = torch.zeros(blk.cache[0].shape[:3], dtype=torch.bool)
    for t, b, pos in blk.tokens():
        at = pos if positions is None else positions[axis, t]
        check(q[t], *turned(qr[t], at, R, freq), f"q of token {t}")
        page, slot = blk.place(b, pos)
        touched[page, :, slot] = True
        y, off = turned(kr[t], at, R, freq)
        if blk.bits == 16:
            check(blk.cache[0][page, :, slot], y, off, f"k of token {t}")
            assert torch.equal(blk.cache[1][page, :, slot], blk.v[t])
        else:
            vals, scale = ref.quantise_rows(blk.v[t].cpu().double().numpy())
            assert np.array_equal(ref.code_values(blk.cache[1][page, :, slot]), vals)
            assert np.array_equal(blk.cache[3][page, :, slot].cpu().numpy(), scale)
            got = ref.cache_values(blk.cache[0][page, :, slot], blk.cache[2][page, :, slot])
            # e4m3 of the bf16 row: half a step, 2^-4, or 2^-10 of the scale below the normal
            # range (a scale is at most 2^-8 of the row's largest value, over 1.75)
            top = np.abs(y).max(-1, keepdims=True)
            assert np.all(np.abs(got - y) <= 2.0 ** -4 * np.abs(y) + top * 2.0 ** -17
                          + 1.1 * (2.0 ** -8 * np.abs(y) + 2 * off))
    for c, was in zip(blk.cache, blk.before):
        assert torch.equal(c.cpu()[~touched], was.cpu()[~touched]), "another slot was written"


CASES = [  # lens, qs, hq, hkv
    ([1], [1], 4, 1), ([64, 1, 65], [1, 1, 65], 8, 2), ([700, 128, 3], [129, 64, 3], 3, 3),
    ([1000, 40, 66, 64], [1, 7, 2, 1], 32, 8)]


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,qs,hq,hkv", CASES)
def test_against_64_bits(dev, lens, qs, hq, hkv, D, bits):
    blk = Block(dev, lens, qs, hq, hkv, D, bits)
    check_block(blk, blk.run())


@pytest.mark.parametrize("bits", [16, 8])
def test_tokens_of_no_sequence_stay(dev, bits):
    blk = Block(dev, [70, 9], [5, 9], 4, 2, 64, bits, front=3, behind=6)
    out = torch.full((23, 4, 64), 7.0, dtype=torch.bfloat16, device=dev)
    q = blk.run(out=out)
    assert q is out
    check_block(blk, q)
    assert bool((out[:3] == 7).all()) and bool((out[17:] == 7).all())
    same = blk.q.clone()
    back = blk.q[17:].clone()
    blk.run(out=blk.q)      # in place, tokens strided
    assert torch.equal(blk.q[3:17], out[3:17]) and torch.equal(blk.q[17:], back)
    assert torch.equal(blk.q[:3], same[:3])


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("D,sections", [(64, [16, 8, 8]), (128, [16, 24, 24]), (128, [64, 0]),
                                        (64, [1] * 32), (128, [5, 59])])
def test_several_axes(dev, D, sections, bits):
    blk = Block(dev, [90, 40], [33, 40], 4, 2, D, bits, behind=2)
    g = torch.Generator().manual_seed(5)
    positions = torch.randint(-3000, 100000, (len(sections), 75), generator=g, dtype=torch.int32)
    axis = np.repeat(np.arange(len(sections)), sections)
    q = blk.run(positions=positions.to(dev), sections=sections)
    check_block(blk, q, positions=positions.numpy(), axis=axis)


def test_axes_of_equal_positions_are_one(dev):
    blk = Block(dev, [90, 40], [33, 40], 4, 2, 128)
    q = blk.run()
    cache = [c.clone() for c in blk.cache]
    pos = i32([p for _, _, p in blk.tokens()], dev).expand(3, 73).contiguous()
    assert torch.equal(blk.run(positions=pos, sections=(16, 24, 24)), q)
    assert all(torch.equal(a, b) for a, b in zip(cache, blk.cache))


@pytest.mark.parametrize("at", [131071, 1 << 24, 2147483647, -2147483648, 0])
def test_far_positions(dev, at):
    blk = Block(dev, [9], [9], 8, 2, 128)
    positions = torch.tensor([[at] * 9], dtype=torch.int32)
    q = blk.run(positions=positions.to(dev), sections=[64])
    check_block(blk, q, positions=positions.numpy(), axis=np.zeros(64, dtype=int))


@pytest.mark.parametrize("bits", [16, 8])
@pytest.mark.parametrize("D,R", [(128, 64), (128, 16), (64, 48), (128, 112)])
def test_part_of_a_head(dev, D, R, bits):
    blk = Block(dev, [200, 70], [30, 70], 8, 2, D, bits)
    check_block(blk, blk.run(rotary_dim=R), R=R)


def test_frequencies_of_the_callers(dev):
    freq = np.concatenate([frequencies(64)[:16] / 8, frequencies(64)[16:], -frequencies(64) * 3])
    blk = Block(dev, [3000], [40], 8, 2, 128)
    check_block(blk, blk.run(inv_freq=torch.tensor(freq, dtype=torch.float64), theta=-1.0),
                freq=freq)


def test_8_bit_rows_are_the_append_of_the_turned_rows(dev):
    """The same bytes as turning into a bf16 cache and quantising what it holds."""
    a, b = (Block(dev, [300, 65], [77, 65], 8, 4, 128, bits) for bits in (16, 8))
    qa, qb = a.run(), b.run()
    assert torch.equal(qa, qb)
    k = torch.stack([a.cache[0][p, :, s] for p, s in (a.place(*x[1:]) for x in a.tokens())])
    want = [c.clone() for c in b.before]
    bi.kv_append_q8(k, b.v.contiguous(), *want, b.table, b.sl, b.cu)
    assert all(torch.equal(x, y) for x, y in zip(want, b.cache))


def test_rows_with_nan_and_infinities(dev):
    blk = Block(dev, [80], [4], 2, 2, 64, 8)
    blk.k[1, 0, 5] = float("nan")
    blk.k[2, 1, 40] = float("inf")
    blk.v[3, 1, 2] = float("-inf")
    blk.q[0, 1, 3] = float("nan")
    q = blk.run()
    assert bool(q[0, 1].isnan().any()) and not bool(q[0, 0].isnan().any())
    rows = [(0, 1, 0), (0, 2, 1), (1, 3, 1)]
    for which, t, h in rows:
        page, slot = blk.place(0, 76 + t)
        assert int(blk.cache[2 + which][page, h, slot]) == 255
        assert bool((blk.cache[which][page, h, slot] == 0).all())
    bad = sum(int((blk.cache[2 + w][blk.place(0, 76 + t)[0], h, blk.place(0, 76 + t)[1]] == 255))
              for w in (0, 1) for t in range(4) for h in range(2))
    assert bad == 3


@pytest.mark.parametrize("bits", [16, 8])
def test_bits_of_a_token_do_not_depend_on_the_block(dev, bits):
    """A large block (heads share a thread's angles) and its tokens one at a time."""
    blk = Block(dev, [5000], [5000], 8, 2, 128, bits)
    q = blk.run()
    for pos in (0, 1, 63, 64, 4097, 4999):
        one = Block(dev, [5000], [5000], 8, 2, 128, bits)
        one.q, one.k, one.v = (x[pos:pos + 1] for x in (blk.q, blk.k, blk.v))
        one.sl, one.cu = i32([pos + 1], dev), i32([0, 1], dev)
        assert torch.equal(one.run(), q[pos:pos + 1])
        page, slot = blk.place(0, pos)
        assert all(torch.equal(a[page, :, slot], b[page, :, slot])
                   for a, b in zip(one.cache, blk.cache))


@pytest.mark.parametrize("bits", [16, 8])
def test_bad_device_arguments_are_skipped(dev, bits):
    def latched(change):
        blk = Block(dev, [70, 30], [6, 5], 4, 2, 64, bits)
        change(blk)
        out = torch.zeros(11, 4, 64, dtype=torch.bfloat16, device=dev)
        fn = bi.rope_kv_append if bits == 16 else bi.rope_kv_append_q8
        fn(blk.q, blk.k, blk.v, *blk.cache, blk.table, blk.sl, blk.cu, out=out)
        assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
        return blk, out

    blk, out = latched(lambda b: b.table.__setitem__((0, 1), 10 ** 6))
    # positions 64..69 have no page: not appended, their queries turned all the same
    assert all(torch.equal(c, w) or i in (0, 1, 2, 3) for i, (c, w) in
               enumerate(zip(blk.cache, blk.before)))
    assert bool((out[:6] != 0).any())
    for change in (lambda b: b.sl.__setitem__(0, 5), lambda b: b.sl.__setitem__(0, 100000),
                   lambda b: b.cu.__setitem__(2, 12), lambda b: b.cu.__setitem__(0, -1)):
        blk, out = latched(change)
    # a block longer than its sequence: the other sequence is served
    blk, out = latched(lambda b: b.sl.__setitem__(0, 5))
    assert not bool(out[:6].any()) and bool(out[6:].any())


def test_captured_and_replayed(dev):
    blk = Block(dev, [200, 70], [3, 2], 8, 2, 128)
    out = torch.empty(5, 8, 128, dtype=torch.bfloat16, device=dev)
    blk.run(out=out)
    want, cache = out.clone(), [c.clone() for c in blk.cache]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        bi.rope_kv_append(blk.q, blk.k, blk.v, *blk.cache, blk.table, blk.sl, blk.cu,
                          theta=THETA, out=out)
    out.zero_()
    for c, w in zip(blk.cache, blk.before):
        c.copy_(w)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(cache, blk.cache))


def test_refused_tensors(dev):
    blk = Block(dev, [70], [6], 4, 2, 64)
    args = (blk.q, blk.k, blk.v, *blk.cache, blk.table, blk.sl, blk.cu)
    with pytest.raises(ValueError, match="contiguous heads"):
        bi.rope_kv_append(blk.q[:, ::2], *args[1:])
    with pytest.raises(ValueError, match="number of tokens"):
        bi.rope_kv_append(blk.q[:5], *args[1:])
    with pytest.raises(TypeError):
        bi.rope_kv_append(blk.q.float(), *args[1:])
    with pytest.raises(ValueError, match="go together"):
        bi.rope_kv_append(*args, sections=[32])
    with pytest.raises(ValueError, match="one section per axis"):
        bi.rope_kv_append(*args, sections=[32], positions=i32([[0] * 6] * 2, dev))
    with pytest.raises(ValueError, match="inv_freq"):
        bi.rope_kv_append(*args, inv_freq=[1.0] * 31)
    with pytest.raises(bi.BIError, match="sum to"):
        bi.rope_kv_append(*args, sections=[31], positions=i32([[0] * 6], dev))
    with pytest.raises(ValueError, match="cu_q"):
        bi.rope_kv_append(*args[:-1], blk.cu[:1])
    with pytest.raises(ValueError, match="shape of q"):
        bi.rope_kv_append(*args, out=blk.k.clone())
    with pytest.raises(TypeError):
        bi.rope_kv_append_q8(*args[:5], None, None, *args[5:])
    empty = [x[:0] for x in args[:3]]
    assert bi.rope_kv_append(*empty, *args[3:7], i32([0, 0], dev)).shape == (0, 4, 64)
