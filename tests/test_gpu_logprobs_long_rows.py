"""Token log-probabilities of rows far longer than a vocabulary: the sums keep their accuracy."""
import math

import pytest
import torch

from tolerance import bits_equal

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [524288, 524289, 2000003, 1 << 24, (1 << 27) + 5])
def test_equal_entries_below_the_largest(dev, dtype, n):
    """Every 61st entry 0 and the rest -1.7 (rounded to the type): every partial sum grows by
    equal steps, whose roundings go one way.  A thread's running sums take up to 264 additions
    each, every one off by at most 2^-24 of the sum so far: 132 * 2^-24 of the last one.  Some 34
    folds follow (13 of a thread's groups, 8 of a lane's threads, 5 of lanes, 8 of parts) of two
    roundings each: 34 * 2^-23; all maxima are 0, so they rescale nothing.  The exponentials are
    off by 2^-21.  Together 1.25e-5, below 2^-16, of s and of the entropy's sum.  (At 2^24 and
    beyond running sums all along the row were off by 4e-5 and 8e-4.)"""
    x = torch.full((1, n), -1.7, dtype=dtype, device=dev)
    low = float(x[0, 0])
    x[0, 7::61] = 0
    zeros = len(range(7, n, 61))
    tok = torch.tensor([3], dtype=torch.int32, device=dev)
    s = zeros + (n - zeros) * math.exp(low)
    w = (n - zeros) * math.exp(low) * low
    r = bi.token_logprobs(x, tok, top=3)
    ls = math.log(s)
    rounding = 2.0 ** -23 * ls
    assert abs(float(r.lse[0]) - ls) <= 2.0 ** -16 + rounding
    assert abs(float(r.logprobs[0]) - (low - ls)) <= 2.0 ** -16 + rounding + 2.0 ** -23 * abs(low)
    assert abs(float(r.entropy[0]) - (ls - w / s)) <= 2.0 ** -15 * (1 + abs(w / s)) + 2 * rounding
    assert r.top_ids.tolist() == [[7, 68, 129]]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,off", [(1500007, 0), (1500007, 1), (4194304, 0)])
def test_random_rising_and_special_rows(dev, dtype, n, off):
    """Random entries, a row whose maximum rises all along it, -inf entries, NaN and +inf, aligned
    rows and rows off their boundary, alone and in a call of many: 64 bits, and the same bits."""
    g = torch.Generator(device=dev).manual_seed(n)
    buf = torch.empty(6 * (n + off) + 8, dtype=dtype, device=dev)
    x = buf[off:off + 6 * (n + off)].view(6, n + off)[:, :n]
    x.copy_(torch.randn(6, n, generator=g, device=dev) * 2.5)
    x[1] = torch.linspace(-12, 6, n, device=dev).to(dtype)
    x[2, ::3] = -math.inf
    x[2, n // 7:n // 2] = -math.inf
    x[3] = -math.inf
    x[3, n - 2:] = 1.0
    x[4, n // 3] = math.nan
    x[5, n - 1] = math.inf
    tok = torch.tensor([5, n - 1, 1, n - 1, 2, 3], dtype=torch.int32, device=dev)
    r = bi.token_logprobs(x, tok, top=4)
    for row in range(4):
        y = x[row].double()
        logp = torch.log_softmax(y, -1)
        H = -torch.where(logp > -math.inf, logp.exp() * logp, 0 * logp.exp()).sum()
        big = float(y[torch.isfinite(y)].abs().max() + torch.logsumexp(y, -1).abs())
        bound = 2.0 ** -15 + 2.0 ** -22 * big
        assert abs(float(r.lse[row]) - float(torch.logsumexp(y, -1))) <= bound, row
        assert abs(float(r.logprobs[row]) - float(logp[int(tok[row])])) <= bound, row
        assert abs(float(r.entropy[row]) - float(H)) <= 2.0 ** -14 * (1 + float(H) + math.log(n))
        order = torch.sort(y, descending=True, stable=True)
        assert torch.equal(r.top_ids[row].long(), order.indices[:4]), row
    for t in (r.logprobs, r.entropy, r.lse):
        assert bool(torch.isnan(t[4:]).all())
    for row in range(6):
        one = bi.token_logprobs(x[row:row + 1].clone(), tok[row:row + 1], top=4)
        for a, b in zip(one[:4], r[:4]):
            assert bits_equal(a[0], b[row]), row
        assert torch.equal(one.top_ids[0], r.top_ids[row])
    many = x[:1].repeat(330, 1)
    got = bi.token_logprobs(many, tok[:1].repeat(330), top=4)
    for a, b in zip(got[:4], r[:4]):
        assert bits_equal(a[0], b[0]) and bits_equal(a[329], b[0])
    assert bi.device_status() == bi.BI_OK
