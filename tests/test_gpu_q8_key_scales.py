"""Key rows at the ends of the scale byte's range, in the attention over the 8-bit cache."""
import numpy as np
import pytest
import torch

import q8_reference as ref
from test_gpu_kv_q8 import attend, dev, filled, rows  # noqa: F401 (dev: a fixture)
from tolerance import bits_equal

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


def signs(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 2, shape, generator=g).float() * 2 - 1


def sizes(shape, seed):  # [0.5, 1)
    g = torch.Generator().manual_seed(seed)
    return torch.rand(*shape, generator=g) * 0.5 + 0.5


def against_64_bits(c, q, out, lse, L, scale):
    Hq, Hkv = q.shape[1], c.k.shape[1]
    r = ref.attention(q.double().numpy(), *c.values(), c.table[0].tolist(), L, q.shape[0], scale,
                      Hq // Hkv)
    ref.check_attention(out, lse, r)


@pytest.mark.parametrize("D,Hq,Hkv,qs", [(128, 8, 2, 8), (64, 8, 2, 3), (128, 4, 4, 1),
                                         (64, 8, 8, 8), (128, 32, 1, 1)])
@pytest.mark.parametrize("every", [1, 3, 97])
def test_large_keys_and_small_queries(dev, D, Hq, Hkv, qs, every):  # noqa: F811
    """Keys near 2^117 (every third of them, a few, or all) under queries near 2^-112: the scores
    are ordinary numbers, although the products of the codes with either factor alone are not."""
    L, scale = 700, 2.0 ** -8 * (128 / D)
    q = (sizes((qs, Hq, D), 1) * signs((qs, Hq, D), 2) * 2.0 ** -112).bfloat16()
    k = sizes((L, Hkv, D), 3) * signs((L, Hkv, D), 4)
    k[::2] = k[::2].abs() * q[0, ::Hq // Hkv].sign().float()       # scores up to the largest
    k[1::4] *= q[-1, ::Hq // Hkv].sign().float()
    size = torch.full((L, 1, 1), 2.0 ** 30)
    size[::every] = 2.0 ** 117
    c = filled([L], Hkv, D, dev, seed=5, k=(k * size).bfloat16(), v=rows((L, Hkv, D), 6))
    out, lse = attend(c, q.to(dev), [L], [qs], scale, "verify")
    against_64_bits(c, q, out, lse, L, scale)
    assert bi.device_status() == bi.BI_OK


def test_large_keys_at_right_angles_to_large_queries(dev):  # noqa: F811
    """Products of zero stay zero, whatever the factors: queries near 2^100 and 2^120 that share
    no element with keys near 2^110, beside a few ordinary elements that carry the scores."""
    L, Hkv, D, Hq = 600, 2, 128, 8
    q, k = torch.zeros(4, Hq, D), torch.zeros(L, Hkv, D)
    q[:2, :, :40] = sizes((2, Hq, 40), 1) * 2.0 ** 100
    q[2:, :, :40] = sizes((2, Hq, 40), 2) * 2.0 ** 120
    k[::3, :, 60:] = sizes((200, Hkv, 68), 3) * 2.0 ** 110
    k[1::3, :, :40] = sizes((200, Hkv, 40), 4) * signs((200, Hkv, 40), 5) * 2.0 ** -122
    k[1::3] *= 2.0 ** 4
    c = filled([L], Hkv, D, dev, seed=7, k=k.bfloat16(), v=rows((L, Hkv, D), 8))
    out, lse = attend(c, q.bfloat16().to(dev), [L], [4], 0.5, "verify")
    against_64_bits(c, q.bfloat16(), out, lse, L, 0.5)


def test_hidden_scale_bytes_change_no_bit(dev):  # noqa: F811
    """Key scale bytes of 0 stand for 2^-127 whatever the bytes beside them are, hidden ones
    among them: large queries see the same keys, bit for bit, with NaN, huge or small rows at
    later positions of the same chunk, and the values of the definition."""
    L, Hkv, D, Hq = 300, 2, 128, 8
    c = filled([L], Hkv, D, dev, seed=9, k=(signs((L, Hkv, D), 10) * 448).bfloat16(),
               v=rows((L, Hkv, D), 11))
    page = c.table[0].long()
    for p in page.tolist():
        c.ks[p] = 0
        c.ks[p, :, 1::4] = 3
        c.vs[p] = c.vs[p].clamp(max=200)           # (unwritten slots too)
    q = (signs((4, Hq, D), 12) * sizes((4, Hq, D), 13) * 2.0 ** 117).bfloat16()
    last = (int(page[(L - 1) // 64]), slice(None), (L - 1) % 64)
    got = {}
    for byte in (0, 3, 100, 223, 224, 230, 253, 254, 255):
        c.ks[last] = byte
        out, lse = attend(c, q.to(dev), [L], [4], 0.25, "verify")
        got[byte] = out[:3].clone(), lse[:3].clone()
        if byte == 0:
            against_64_bits(c, q, out, lse, L, 0.25)
    for byte, (o, l) in got.items():
        assert bits_equal(o, got[0][0]) and bits_equal(l, got[0][1]), byte


def test_bits_beside_hidden_large_rows(dev):  # noqa: F811
    """Ordinary queries and keys beside later rows of every large scale keep their bits, and so
    do single tokens of a sequence whose keys are large."""
    L, Hkv, D, Hq = 530, 2, 128, 8
    k, v = rows((L, Hkv, D), 14), rows((L, Hkv, D), 15)
    q = rows((8, Hq, D), 16).to(dev)
    c = filled([L], Hkv, D, dev, seed=17, k=k, v=v)
    want, wlse = attend(c, q[:4].contiguous(), [L - 4], [4], D ** -0.5, "verify")
    for size in (2.0 ** 105, 2.0 ** 120, 3e38):
        new = (k[-4:].float().sign() * size).bfloat16().to(dev)
        c.append(new, v[-4:].to(dev), [L], [4])
        out, lse = attend(c, q, [L], [8], D ** -0.5, "verify")
        assert bits_equal(out[:4], want) and bits_equal(lse[:4], wlse), size
    big = filled([L], Hkv, D, dev, seed=18, k=(k.float() * 2.0 ** 112).bfloat16(), v=v)
    small = (q.float() * 2.0 ** -110).bfloat16()
    out, lse = attend(big, small, [L], [8], D ** -0.5, "verify")
    for j in (0, 3, 7):
        o, l = attend(big, small[j:j + 1].contiguous(), [L - 7 + j], [1], D ** -0.5, "decode")
        assert bits_equal(o[0], out[j]) and bits_equal(l[0], lse[j])
