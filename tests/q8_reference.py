"""The 8-bit cache in 64 bits on the CPU: its format from the definition, and attention over
the values it stands for."""
import math

import numpy as np
import torch

PAGE = 64


def quantise_rows(x: np.ndarray):
    """(e4m3 values, scale bytes) of float64 rows of the last axis."""
    amax = np.abs(x).max(-1)
    bad = ~np.isfinite(x).all(-1)
    e = np.full(amax.shape, -64)
    for idx in np.ndindex(amax.shape):
        if not bad[idx]:
            while amax[idx] > 448.0 * 2.0 ** e[idx]:
                e[idx] += 1
    with np.errstate(invalid="ignore"):
        y = np.where(bad[..., None], 0.0, x * 2.0 ** (-e[..., None].astype(np.float64)))
    size = np.floor(np.log2(np.maximum(np.abs(y), 2.0 ** -40)))
    size += np.abs(y) >= 2.0 ** (size + 1)      # log2 may be off by one at powers of two
    size -= np.abs(y) < 2.0 ** size
    step = 2.0 ** (np.maximum(size, -6) - 3)
    return np.round(y / step) * step, np.where(bad, 255, e + 127).astype(np.uint8)


def code_values(codes: torch.Tensor) -> np.ndarray:
    return codes.cpu().view(torch.float8_e4m3fn).double().numpy()


def cache_values(codes: torch.Tensor, scale: torch.Tensor) -> np.ndarray:
    s = scale.cpu().numpy().astype(np.int64)
    f = np.where(s == 255, np.nan, 2.0 ** (s - 127).astype(np.float64))
    return code_values(codes) * f[..., None]


def scale_values(scale: torch.Tensor) -> np.ndarray:
    return 2.0 ** (scale.cpu().numpy().astype(np.float64) - 127)


def attention(q, k, v, ys, table, L, q_len, scale, G):
    """One sequence's block: q [q_len, Hq, D] (float64), k and v [pages, Hkv, 64, D] values, ys
    [pages, Hkv, 64] the value rows' scales; returns out, lse, A [q_len, Hq, D], the weighted
    mean of |v|, F [q_len, Hq, D], the largest (weight * value scale) times the sum of the
    codes' magnitudes |v| / scale, and S [q_len, Hq], the largest sum of |q k| * scale, over
    the keys seen."""
    n = -(-L // PAGE)
    pages = [int(p) for p in table[:n]]
    Hkv, D = k.shape[1], k.shape[3]
    out = np.zeros(q.shape)
    A = np.zeros(q.shape)
    F = np.zeros(q.shape)
    lse = np.zeros(q.shape[:2])
    S = np.zeros(q.shape[:2])
    for h in range(Hkv):
        kh = k[pages, h].reshape(-1, D)[:L]
        vh = v[pages, h].reshape(-1, D)[:L]
        yh = ys[pages, h].reshape(-1)[:L]
        for j in range(q_len):
            pos = L - q_len + j
            for g in range(h * G, (h + 1) * G):
                s = kh[:pos + 1] @ q[j, g] * scale
                m = s.max()
                p = np.exp(s - m)
                w = p / p.sum()
                a = np.abs(vh[:pos + 1])
                out[j, g], A[j, g] = w @ vh[:pos + 1], w @ a
                F[j, g] = (w * yh[:pos + 1]).max() * (a / yh[:pos + 1, None]).sum(0)
                lse[j, g] = m + math.log(p.sum())
                S[j, g] = (np.abs(kh[:pos + 1]) @ np.abs(q[j, g])).max() * abs(scale)
    return out, lse, A, F, S


def check_attention(out, lse, ref, what=""):
    """Against the 64-bit values, element by element.
    out: rounding to bf16 moves a value by at most 2^-8 of itself.  A weight times its value
    scale, p, is held as two e4m3 pieces of four bits each: off by at most 2^-9 of itself,
    which moves out by at most 2^-9 A, or, where the second piece is below e4m3's normal range
    (steps of 2^-9, in units of 1/32), by at most 2^-10 / 32 = 2^-15 where the chunk's
    largest p is 2^8: 2^-23 of the largest p per unit of a code, at most 2^-23 F in all.  The fp32
    parts (scores off by 2^-17 S, exp2, sums) stay below 2^-10 A for S up to 2^6.
    lse: fp32 scores off by at most 2^-17 of the largest sum of |q k|, and a few fp32
    roundings of a number of lse's size."""
    o, l, A, F, S = ref
    g = out.double().cpu().numpy()
    bound = 2.0 ** -8 * np.abs(o) + (2.0 ** -9 + 2.0 ** -10) * A + 2.0 ** -23 * F
    err = np.abs(g - o)
    assert np.isfinite(g).all(), f"{what}: non-finite output"
    worst = np.unravel_index(np.argmax(err - bound), err.shape)
    assert (err <= bound).all(), (f"{what}: at {worst} {g[worst]} for {o[worst]}, "
                                  f"bound {bound[worst]}")
    if lse is not None:
        d = np.abs(lse.double().cpu().numpy() - l)
        b = 2.0 ** -17 * S + 2.0 ** -20 * np.abs(l) + 2e-6
        assert (d <= b).all(), f"{what}: lse off by {d.max()}"
