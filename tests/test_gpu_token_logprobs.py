"""bi_token_logprobs and its gradient on the GPU, against 64 bits."""
import numpy as np
import pytest
import torch

from tolerance import bits_equal

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")

TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def logits(rows, n, dtype, seed, std=2.5, pad=0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, n + pad, generator=g) * std).to(dtype)[:, :n]


def tokens_of(rows, n, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, n, (rows,), generator=g, dtype=torch.int32)


def reference(x, tok):
    x = x.double()
    logp = torch.log_softmax(x, -1)
    p = torch.exp(logp)
    H = -torch.where(p > 0, p * logp, torch.zeros_like(p)).sum(-1)
    at = tok.long().clamp(min=0)
    lp = torch.where(tok >= 0, logp.gather(1, at.unsqueeze(1))[:, 0],
                     torch.zeros(len(tok)).double())
    return lp, H, torch.logsumexp(x, -1), logp


def ranked(x, k):
    """Indices by value descending, then index ascending; NaN last."""
    v = x.double().numpy()
    v = np.where(np.isnan(v), -np.inf, v)
    nan = np.isnan(x.double().numpy())
    out = []
    for r in range(len(v)):
        order = sorted(range(v.shape[1]), key=lambda i: (nan[r, i], -v[r, i] if v[r, i] > -np.inf
                                                         else np.inf, i))
        out.append(order[:k])
    return np.array(out)


def check(r, x, tok, k=0):
    """fp32 arithmetic: x - m exact up to a rounding, exp and log correct to a few units of
    2^-24, sums of up to n terms over a tree (depth ~ n / 1024 in a thread, then 15): the
    relative error of s and of the entropy's sum is below 2^-17 for n up to 2^18, so logp and
    lse are off by at most 2^-17 plus 2^-22 of the numbers subtracted, the entropy by 2^-17 of
    sum p |x - m| <= entropy + |log s| and as much again."""
    lp, H, lse, logp = reference(x, tok)
    big = x.double().abs().amax(-1) + lse.abs()
    assert (r.logprobs.cpu().double() - lp).abs().le(2.0 ** -17 + 2.0 ** -22 * big).all()
    assert (r.lse.cpu().double() - lse).abs().le(2.0 ** -17 + 2.0 ** -22 * big).all()
    assert (r.entropy.cpu().double() - H).abs().le(2.0 ** -16 * (1 + H + np.log(x.shape[1]))).all()
    if k:
        ids = r.top_ids.cpu().long()
        assert np.array_equal(ids.numpy(), ranked(x, k))
        want = logp.gather(1, ids)
        fin = torch.isfinite(want)
        assert torch.equal(torch.isneginf(want), torch.isneginf(r.top_logprobs.cpu().double()))
        d = (r.top_logprobs.cpu().double() - want).abs()
        assert d[fin].le((2.0 ** -17 + 2.0 ** -22 * big).unsqueeze(1).expand_as(d)[fin]).all()
    else:
        assert r.top_ids is None and r.top_logprobs is None


SIZES = [(1, 1), (3, 2), (5, 31), (2, 127), (4, 1000), (3, 4097), (2, 50001), (1, 128256),
         (2, 131073), (1, 262144), (1, 300001)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n", SIZES)
def test_against_64_bits(dev, dtype, rows, n):
    x, tok = logits(rows, n, dtype, n), tokens_of(rows, n, n + 1)
    for k in sorted({0, 1, min(8, n), min(32, n)}):
        check(bi.token_logprobs(x.to(dev), tok.to(dev), top=k), x, tok, k)
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("dtype", TYPES)
def test_bits_do_not_depend_on_rows_stride_or_alignment(dev, dtype):
    rows, n = 7, 5003
    x, tok = logits(rows, n, dtype, 1).to(dev), tokens_of(rows, n, 2).to(dev)
    want = bi.token_logprobs(x, tok, top=5)
    for pad, off in ((0, 0), (1, 0), (1, 1), (13, 3)):
        buf = torch.full((rows * (n + pad) + off,), NAN, dtype=dtype, device=dev)
        y = buf[off:].view(rows, n + pad)[:, :n]
        y.copy_(x)
        got = bi.token_logprobs(y, tok, top=5)
        for a, b in zip(got[:4], want[:4]):
            assert bits_equal(a, b), (pad, off)
        assert torch.equal(got.top_ids, want.top_ids)
        g = torch.ones(rows, device=dev)
        d = bi.token_logprobs_backward(x, tok, want.lse, want.entropy, g, g)
        assert bits_equal(bi.token_logprobs_backward(y, tok, got.lse, got.entropy, g, g), d)
    for r in range(rows):
        one = bi.token_logprobs(x[r:r + 1], tok[r:r + 1].contiguous(), top=0)
        for a, b in zip(one[:3], want[:3]):
            assert bits_equal(a, b[r:r + 1])


@pytest.mark.parametrize("n", [9, 1000, 40000, 270000])
def test_ties_and_special_rows(dev, n):
    """Equal entries (all of a row, and pairs), signed zeros, -inf entries, rows of nothing but
    -inf, NaN and +inf."""
    x = logits(9, n, torch.float32, 3)
    x[0] = 1.5
    x[1] = (torch.arange(n) % 3).float()
    x[2] = 0.0
    x[2, 1::2] = -0.0
    x[3, 2:] = -INF
    x[4, ::2] = -INF
    x[5] = -INF
    x[6, n // 2] = NAN
    x[7, n - 1] = INF
    x[8, n - 1] = 60.0          # one entry holds all the weight
    tok = torch.tensor([0, 2, 1, 5, 0, 3, 1, n - 1, n - 1], dtype=torch.int32)
    tok[4] = 2                  # a token of probability zero
    k = 8
    r = bi.token_logprobs(x.to(dev), tok.to(dev), top=k)
    ok = torch.tensor([0, 1, 2, 4, 8])
    lp, H, lse, logp = reference(x, tok)
    assert np.array_equal(r.top_ids.cpu().numpy(), ranked(x, k))
    fin = torch.isfinite(lp[ok])
    assert torch.equal(torch.isneginf(lp[ok]), torch.isneginf(r.logprobs.cpu()[ok]))
    assert (r.logprobs.cpu()[ok].double() - lp[ok])[fin].abs().max() < 1e-5
    assert (r.entropy.cpu()[[0, 1, 2, 3, 4, 8]].double()
            - H[[0, 1, 2, 3, 4, 8]]).abs().max() < 2.0 ** -16 * (2 + 2 * np.log(n))
    assert torch.isneginf(r.logprobs[3]) and torch.isfinite(r.entropy[3])
    for row in (5, 6, 7):
        for t in (r.logprobs, r.entropy, r.lse, r.top_logprobs):
            assert bool(torch.isnan(t[row]).all()), row
    g = torch.full((9,), 2.0, device=dev)
    d = bi.token_logprobs_backward(x.to(dev), tok.to(dev), r.lse, r.entropy, g, g).cpu()
    assert bool(torch.isfinite(d[ok]).all()) and bool(torch.isfinite(d[3]).all())
    assert bool((d[4, 4::2] == 0).all()) and d[4, 2] == 2.0 and bool(torch.isnan(d[6]).all())
    assert bi.device_status() == bi.BI_OK


def test_no_token_and_bad_tokens(dev):
    x = logits(4, 500, torch.bfloat16, 4)
    tok = torch.tensor([-1, 7, 500, -2], dtype=torch.int32)
    r = bi.token_logprobs(x.to(dev), tok.to(dev), top=2)
    assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
    lp, H, lse, _ = reference(x, torch.tensor([-1, 7, 0, 0]))
    assert float(r.logprobs[0]) == 0 and abs(float(r.logprobs[1]) - float(lp[1])) < 1e-5
    assert bool(torch.isnan(r.logprobs[2:]).all())
    assert (r.entropy.cpu().double() - H).abs().max() < 1e-4
    ones = torch.ones(4, device=dev)
    d = bi.token_logprobs_backward(x.to(dev), tok.to(dev), r.lse, r.entropy, ones)
    assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
    assert bool((d[[0, 2, 3]] == 0).all()) and bool((d[1] != 0).any())
    tok[2:] = -1
    bi.token_logprobs(x.to(dev), tok.to(dev))
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,n", [(1, 1), (5, 33), (3, 1000), (2, 50001), (1, 300001)])
@pytest.mark.parametrize("terms", ["logp", "entropy", "both"])
def test_gradient_against_64_bits(dev, dtype, rows, n, terms):
    """dx = g (onehot - p) - h p (log p + H), rounded once: half a step of the type; the fp32
    factors err by at most 2^-16 of themselves (p: exp of a number that is off by 2^-17; log p +
    H by 2^-17 of |log p| + H)."""
    x, tok = logits(rows, n, dtype, 5), tokens_of(rows, n, 6)
    tok[0] = -1 if rows > 1 else tok[0]
    g = torch.randn(rows, generator=torch.Generator().manual_seed(7))
    h = torch.randn(rows, generator=torch.Generator().manual_seed(8))
    r = bi.token_logprobs(x.to(dev), tok.to(dev))
    gl = g.to(dev) if terms != "entropy" else None
    gh = h.to(dev) if terms != "logp" else None
    d = bi.token_logprobs_backward(x.to(dev), tok.to(dev), r.lse,
                                   r.entropy if gh is not None else None, gl, gh)
    assert d.dtype == dtype
    lp, H, _, logp = reference(x, tok)
    p = torch.exp(logp)
    one = torch.zeros_like(p)
    one[torch.arange(rows), tok.long().clamp(min=0)] = (tok >= 0).double()
    G = (g.double() * (tok >= 0)).unsqueeze(1) if gl is not None else torch.zeros(rows, 1).double()
    E = h.double().unsqueeze(1) if gh is not None else torch.zeros(rows, 1).double()
    want = G * (one - p) - E * p * (logp + H.unsqueeze(1))
    size = G.abs() * (one + p) + E.abs() * p * (logp.abs() + H.unsqueeze(1))
    least = torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps  # subnormal step
    bound = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -15 * size + least
    assert (d.cpu().double() - want).abs().le(bound).all()


def test_gradient_against_differences(dev):
    """Central differences of the forward in 64 bits agree with the fp32 gradient."""
    rows, n, eps = 2, 40, 1e-5
    x, tok = logits(rows, n, torch.float32, 9), tokens_of(rows, n, 10)
    g, h = torch.tensor([0.7, -1.3]), torch.tensor([0.2, 0.9])
    r = bi.token_logprobs(x.to(dev), tok.to(dev))
    d = bi.token_logprobs_backward(x.to(dev), tok.to(dev), r.lse, r.entropy, g.to(dev), h.to(dev))

    def f(y):
        lp, H, _, _ = reference(y, tok)
        return (g.double() * lp + h.double() * H).sum()
    for i in range(rows):
        for j in range(n):
            up, down = x.double().clone(), x.double().clone()
            up[i, j] += eps
            down[i, j] -= eps
            assert abs(float(f(up) - f(down)) / (2 * eps) - float(d[i, j])) < 2e-5


def test_gradient_in_place_and_strided(dev):
    x, tok = logits(6, 777, torch.bfloat16, 11).to(dev), tokens_of(6, 777, 12).to(dev)
    r = bi.token_logprobs(x, tok)
    g = torch.randn(6, device=dev)
    want = bi.token_logprobs_backward(x, tok, r.lse, r.entropy, g, g)
    buf = torch.full((8, 800), 3.0, dtype=torch.bfloat16, device=dev)
    bi.token_logprobs_backward(x, tok, r.lse, r.entropy, g, g, out=buf[1:7, 5:782])
    assert bits_equal(buf[1:7, 5:782], want)
    buf[1:7, 5:782] = 3.0
    assert bool((buf == 3).all())
    y = x.clone()
    bi.token_logprobs_backward(y, tok, r.lse, r.entropy, g, g, out=y)
    assert bits_equal(y, want)


def test_empty_captured_and_streams(dev):
    none = bi.token_logprobs(torch.empty(0, 10, device=dev),
                             torch.empty(0, dtype=torch.int32, device=dev), top=3)
    assert none.logprobs.shape == (0,) and none.top_ids.shape == (0, 3)
    x, tok = logits(3, 9000, torch.float32, 13).to(dev), tokens_of(3, 9000, 14).to(dev)
    ones = torch.ones(3, device=dev)

    def both():
        r = bi.token_logprobs(x, tok, top=4)
        return r, bi.token_logprobs_backward(x, tok, r.lse, r.entropy, ones, ones)
    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r, d = both()
    x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    wr, wd = both()
    assert all(bits_equal(a, b) for a, b in zip(r[:4], wr[:4]))
    assert torch.equal(r.top_ids, wr.top_ids)
    assert bits_equal(d, wd)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    sr = bi.token_logprobs(x, tok, top=4, stream=s)
    sd = bi.token_logprobs_backward(x, tok, sr.lse, sr.entropy, ones, ones, stream=s)
    s.synchronize()
    assert bits_equal(sd, wd) and bits_equal(sr.top_logprobs, wr.top_logprobs)


def test_many_rows(dev):
    """More rows than a grid dimension of 65,535 holds."""
    rows, n = 70001, 24
    x, tok = logits(rows, n, torch.float32, 15), tokens_of(rows, n, 16)
    r = bi.token_logprobs(x.to(dev), tok.to(dev), top=2)
    check(bi.TokenLogprobs(*(t[-50:] for t in r)), x[-50:], tok[-50:], 2)
    d = bi.token_logprobs_backward(x.to(dev), tok.to(dev), r.lse, None,
                                   torch.ones(rows, device=dev)).cpu().double()
    p = torch.softmax(x.double(), -1)
    p[torch.arange(rows), tok.long()] -= 1
    assert (d + p).abs().max() < 2e-5


def test_refusals(dev):
    x, tok = logits(4, 40, torch.float32, 17).to(dev), tokens_of(4, 40, 18).to(dev)
    one = torch.ones(4, device=dev)
    for bad in (dict(logits=x.t()), dict(logits=x[0]), dict(logits=x.double()),
                dict(logits=x[:1].expand(4, 40)), dict(tokens=tok.long()), dict(tokens=tok[:3]),
                dict(tokens=tok.cpu()), dict(top=41), dict(top=-1)):
        with pytest.raises((ValueError, TypeError, bi.BIError)):
            bi.token_logprobs(**{**dict(logits=x, tokens=tok), **bad})
    r = bi.token_logprobs(x, tok)
    good = dict(logits=x, tokens=tok, lse=r.lse, entropy=r.entropy, grad_logprobs=one,
                grad_entropy=one)
    for bad in (dict(lse=r.lse[:3]), dict(lse=None), dict(entropy=None), dict(lse=r.lse.double()),
                dict(grad_logprobs=None, grad_entropy=None), dict(out=x.half()),
                dict(grad_logprobs=torch.ones(8, device=dev)[::2]), dict(out=x[:, :39]),
                dict(out=x[:1].expand(4, 40)), dict(out=x.cpu())):
        with pytest.raises((ValueError, TypeError, bi.BIError)):
            bi.token_logprobs_backward(**{**good, **bad})
    assert bi.device_status() == 0
