"""Attention over the 8-bit cache at the ends of its number range: scores of any finite size,
the largest and smallest key scales, against 64 bits and for the contract (a query's bits depend
on the rows at its own and earlier positions alone)."""
import numpy as np
import pytest
import torch

import q8_reference as ref
from test_gpu_kv_q8 import Cache, attend, dev, filled, i32, rows  # noqa: F401 (dev: a fixture)
from tolerance import bits_equal

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


def same_scale(v):
    """Rows with one largest magnitude, 4, so that all have one scale byte."""
    v = v.float().clamp(-4, 4)
    v[..., 0] = 4.0
    return v.bfloat16()


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 8, 2), (64, 4, 4), (64, 32, 1)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("L,qs", [(1, 1), (5, 1), (512, 1), (700, 1), (9, 4), (515, 8), (600, 40)])
def test_scores_of_any_size(dev, D, Hq, Hkv, sign, L, qs):  # noqa: F811
    """All scores equal and near +-2^120: every query is the mean of the values it sees, exactly
    weighted (equal scores in fp32 too), whichever sign they have.  The value rows have one scale,
    so nothing but the rounding of the mean to bf16 and that of its sum is left: 2^-8 of the
    result, and 2^-12 of the mean magnitude for sums of up to 2^11 terms."""
    if qs * Hq // Hkv > 32 and qs <= 8:
        qs = max(1, 32 * Hkv // Hq)
    k = torch.full((L, Hkv, D), 2.0 ** 60).bfloat16()
    c = filled([L], Hkv, D, dev, seed=1, k=k, v=same_scale(rows((L, Hkv, D), 2, 0.0)))
    q = torch.full((qs, Hq, D), sign * 2.0 ** 60).bfloat16().to(dev)
    form = "prefill" if qs > 8 else "verify"
    out, lse = attend(c, q, [L], [qs], D ** -0.5, form)
    _, v, _ = c.values()
    v = v[c.table[0].tolist()].transpose(0, 2, 1, 3).reshape(-1, Hkv, D)[:L]
    for j in range(qs):
        n = L - qs + j + 1
        for h in range(Hq):
            seen = v[:n, h * Hkv // Hq]
            err = np.abs(out[j, h].double().cpu().numpy() - seen.mean(0))
            assert (err <= 2.0 ** -8 * np.abs(seen.mean(0))
                    + 2.0 ** -12 * np.abs(seen).mean(0)).all(), (j, h)
    want = sign * 2.0 ** 120 * D ** 0.5
    assert bool((lse.double() / want - 1).abs().le(2.0 ** -20).all())
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_later_rows_do_not_reach_queries_with_large_scores(dev, sign):  # noqa: F811
    """Verify blocks and single tokens at the same positions, and blocks whose later rows differ:
    the same bits, with scores of one size and of many."""
    L, Hkv, D, Hq = 530, 2, 128, 8
    k = torch.full((L, Hkv, D), 2.0 ** 60).bfloat16()
    v = rows((L, Hkv, D), 3)
    c = filled([L], Hkv, D, dev, seed=4, k=k, v=v)
    for q in (torch.full((8, Hq, D), sign * 2.0 ** 60).bfloat16(),
              (rows((8, Hq, D), 5).float() * 2.0 ** 60).bfloat16()):
        q = q.to(dev)
        out, lse = attend(c, q, [L], [8], D ** -0.5, "verify")
        assert bool(torch.isfinite(out).all() and torch.isfinite(lse).all())
        for j in range(8):
            n = L - 7 + j
            o, l = attend(c, q[j:j + 1].contiguous(), [n], [1], D ** -0.5, "decode")
            assert bits_equal(o[0], out[j]) and bits_equal(l[0], lse[j]), j
