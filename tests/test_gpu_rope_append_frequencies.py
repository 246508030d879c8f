"""The rotating append's own frequencies: a negative one turns as far the other way as its
magnitude, however small and however far the position."""
import numpy as np
import pytest
import torch

from test_gpu_rope_append import Block, i32

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("pos", [1, 4097, 2 ** 31 - 1, -2 ** 31])
def test_negative_and_positive_frequencies(D, pos):
    """Heads of (1, 0) pairs turn into (cos a, sin a).  Bound of sin: bf16's 2^-8, the fraction's
    rounding 2^-24 and sincospi's 2^-22, all of itself, and the 64-bit fraction's |pos| 2^-65
    turns with the product's 2^-51 of a."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    dev, half = "cuda:0", D // 2
    mags = np.concatenate([10.0 ** np.linspace(-15, -2, half - 3), [1.0, 3.0, 500.25]])
    got = []
    for sign in (1, -1):
        blk = Block(dev, [70], [2], 4, 2, D, fused=False)
        blk.q.zero_()
        blk.q[..., :half] = 1.0
        at = i32([[pos, pos]], dev)
        got.append(blk.run(inv_freq=list(sign * mags), positions=at, sections=[half])
                   .double().cpu().numpy())
    for sign, y in zip((1, -1), got):
        a = float(pos) * sign * mags
        off = 2 * np.pi * abs(pos) * 2.0 ** -65 + 2.0 ** -51 * np.abs(a)
        c, s = np.cos(a), np.sin(a)
        near = 2.0 ** -8 + 2.0 ** -21
        for want, have in ((c, y[..., :half]), (s, y[..., half:])):
            # (a fraction of a turn near 1/2 or 1/4 leaves an absolute 2^-24 pi)
            tol = near * np.abs(want) + off * 1.01 + np.where(np.abs(a) > 1, 2.0 ** -22, 0.0)
            assert (np.abs(have - want) <= tol).all(), (sign, np.abs(have - want).max())
    assert np.array_equal(got[0][..., :half], got[1][..., :half])
    assert np.array_equal(got[0][..., half:], -got[1][..., half:])
