"""Verification of drafted tokens on the GPU, against the definition in 64 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


class Batch:
    """Logits, drafts that a fair share of them would have chosen, and uniforms, on the CPU."""

    def __init__(self, widths, n, dtype="fp32", draft="logits", seed=0, temps=None, std=2.5,
                 behind=0):
        g = torch.Generator().manual_seed(seed)
        self.widths, self.n, self.dtype = list(widths), n, TYPES[dtype]
        B, T = len(widths), sum(widths)
        self.cu = np.concatenate([[0], np.cumsum(widths)])
        self.temps = ([float(t) for t in torch.rand(B, generator=g) * 1.5 + 0.25]
                      if temps is None else list(temps))
        self.temps = [float(np.float32(t)) for t in self.temps]
        self.logits = (torch.randn(T + behind, n, generator=g) * std).to(self.dtype)
        self.u = torch.rand(T + behind, generator=g)
        rows = [self.cu[b] + j for b, w in enumerate(widths) for j in range(w - 1)]
        near = self.logits[rows].float()
        near = (near + torch.randn(near.shape, generator=g) * 0.6).to(self.dtype)
        hot = torch.tensor([self.temps[b] or 1.0 for b, w in enumerate(widths)
                            for _ in range(w - 1)]).unsqueeze(1)
        noise = -torch.log(-torch.log(torch.rand(near.shape, generator=g).clamp(1e-30, 1 - 1e-7)))
        if draft == "tokens":
            noise = noise * (torch.rand(len(rows), 1, generator=g) > 0.7)
        self.drafts = ((near.float() / hot + noise).argmax(-1).to(torch.int32) if rows else
                       torch.zeros(0, dtype=torch.int32))
        self.near = near if draft == "logits" else None

    def run(self, dev, temps=None, **kw):
        t = torch.tensor(self.temps, dtype=torch.float32, device=dev) if temps is None else temps
        kw = dict(max_q=max(self.widths)) | kw
        near = None if self.near is None else self.near.to(dev)
        r = bi.verify_drafts(self.logits.to(dev), self.drafts.to(dev), self.u.to(dev),
                             torch.tensor(self.cu, dtype=torch.int32, device=dev),
                             draft_logits=near, temperature=t, **kw)
        return r


def softmax(x, t):
    with np.errstate(over="ignore"):
        y = (x - x.max()) / t
    e = np.exp(y)
    return e / e.sum(), y - np.log(e.sum())


def check(batch, r, which=None):
    """Every sequence, in 64 bits.  A decision may fall the other way only where u q and p agree to
    2^-20 (fp32 sums of at most 2^20 entries, pairwise below 2^6 terms: 70 roundings of 2^-24), a
    drawn token may be another only where the share lies within the weights' 2^-29, for p and q,
    of an entry's border."""
    tokens, accepted, logps = (x.cpu().numpy() for x in (r.tokens, r.accepted, r.logprobs))
    W = tokens.shape[1]
    for b, w in enumerate(batch.widths):
        if which is not None and b not in which:
            continue
        t0, d0, T = int(batch.cu[b]), int(batch.cu[b]) - b, batch.temps[b]
        got = int(accepted[b])
        j = 0
        while True:
            x = batch.logits[t0 + j].double().numpy()
            p, logp = softmax(x, T or 1.0)
            if j == w - 1:
                q = None
                break
            tok, u = int(batch.drafts[d0 + j]), float(batch.u[t0 + j])
            if T == 0:
                q, keep, close = None, int(np.argmax(x)) == tok, False
            else:
                q = (softmax(batch.near[d0 + j].double().numpy(), T)[0]
                     if batch.near is not None else np.eye(1, batch.n, tok)[0])
                keep = u * q[tok] < p[tok]
                close = abs(u * q[tok] - p[tok]) <= 2.0 ** -20 * p[tok]
            if close:
                keep = got > j
            if not keep:
                break
            assert got > j, (b, j, "a draft that is kept was refused")
            assert tokens[b, j] == tok
            assert abs(logps[b, j] - logp[tok]) <= 2e-6 * max(1.0, abs(logp[tok]))
            j += 1
        assert got == j, (b, got, j)
        last = int(tokens[b, j])
        if T == 0:
            assert last == int(np.argmax(x))
        else:
            d = p if q is None else np.maximum(p - q, 0)
            if d.sum() == 0:
                d = p
            cum = np.cumsum(d)
            u = float(batch.u[t0 + w - 1])
            want = int(np.searchsorted(cum, u * cum[-1], side="right"))
            slack = 2.0 ** -28 + 1e-12
            low = cum[last] - d[last]
            assert want == last or (d[last] > 0 and low - slack <= u * cum[-1] <= cum[last] + slack)
        assert abs(logps[b, j] - logp[last]) <= 2e-6 * max(1.0, abs(logp[last]))
        assert (tokens[b, j + 1:] == -1).all() and (logps[b, j + 1:] == 0).all()
        assert W >= w
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("draft", ["logits", "tokens"])
@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("n", [1, 2, 17, 512, 999, 4097, 8192, 33000])
def test_against_64_bits(dev, n, dtype, draft):
    b = Batch([1, 4, 2, 8, 3, 1, 6], n, dtype, draft, seed=n)
    check(b, b.run(dev))


@pytest.mark.parametrize("dtype,n", [("fp32", 128256), ("bf16", 128256), ("fp32", 150001),
                                     ("fp16", 65535), ("fp32", 1 << 20)])
def test_long_rows(dev, dtype, n):
    b = Batch([3, 1, 4], n, dtype, "logits", seed=1)
    check(b, b.run(dev))
    b = Batch([1, 2], n, dtype, "tokens", seed=2, std=0.05)     # near equal entries
    check(b, b.run(dev))


def test_wide_blocks_and_many_sequences(dev):
    b = Batch([40, 33, 1], 300, seed=3, std=0.3)
    check(b, b.run(dev, max_q=64))
    b = Batch([1 + i % 5 for i in range(300)], 700, "bf16", seed=4)
    check(b, b.run(dev))


@pytest.mark.parametrize("draft", ["logits", "tokens"])
def test_temperatures(dev, draft):
    temps = [0.0, 1e-3, 0.05, 1.0, 30.0, 1e4, 0.0, 2.0 ** -60, 1e30]
    b = Batch([4] * 9, 5000, "fp32", draft, seed=5, temps=temps)
    check(b, b.run(dev), which=range(7))
    b = Batch([4] * 9, 5000, "fp32", draft, seed=5, temps=[0.7] * 9)
    one = b.run(dev, temps=0.7)
    many = b.run(dev)
    # (0.7 is rounded to fp32 either way)
    assert all(torch.equal(x, y) for x, y in zip(one, many))
    b.temps = [0.0] * 9
    assert all(torch.equal(x, y) for x, y in zip(b.run(dev, temps=0.0), b.run(dev)))
    check(b, b.run(dev))


def test_emitted_tokens_are_distributed_as_the_target(dev):
    """One row of a small vocabulary, drafts in the proportions of q, uniforms on a grid: the
    counts of the first emitted token are p's, to the grid's steps."""
    n, K = 6, 64
    g = torch.Generator().manual_seed(7)
    x, y = torch.randn(n, generator=g) * 1.2, torch.randn(n, generator=g) * 1.2
    p, q = torch.softmax(x.double(), 0).numpy(), torch.softmax(y.double(), 0).numpy()
    u1, u2 = np.meshgrid((np.arange(K) + 0.5) / K, (np.arange(K) + 0.5) / K)
    freq = np.zeros(n)
    for tok in range(n):
        B = K * K
        u = torch.tensor(np.stack([u1.ravel(), u2.ravel()], 1).ravel(), dtype=torch.float32)
        r = bi.verify_drafts(x.expand(2 * B, n).to(dev), torch.full((B,), tok, dtype=torch.int32,
                                                                    device=dev), u.to(dev),
                             (torch.arange(B + 1, dtype=torch.int32) * 2).to(dev), max_q=2,
                             draft_logits=y.expand(B, n).to(dev), temperature=1.0)
        first = r.tokens[:, 0].cpu().numpy()
        freq += q[tok] * np.bincount(first, minlength=n) / B
    # acceptance is off by at most 1/2K of each draft's q, a drawn token by n borders of 1/2K
    assert np.abs(freq - p).max() <= (n + 1) / (2 * K)
    assert abs(freq.sum() - 1) < 1e-12


def test_masked_entries_and_rows_without_a_distribution(dev):
    inf = float("inf")
    n = 1200
    b = Batch([3] * 8, n, seed=8, temps=[1.0] * 8)
    b.logits[:, ::3] = -inf                      # a grammar's mask
    b.near[:, ::3] = -inf
    b.drafts = torch.where(b.drafts % 3 == 0, b.drafts + 1, b.drafts)
    b.drafts[0] = 3                              # a draft that the target cannot say
    check(b, b.run(dev))
    assert int(b.run(dev).accepted[0]) == 0
    # q(token) = 0: kept wherever p is not
    b.near[2, int(b.drafts[2])] = -inf
    check(b, b.run(dev))
    assert int(b.run(dev).accepted[1]) >= 1
    for bad in (float("nan"), inf):
        c = Batch([3] * 4, n, seed=9, temps=[1.0, 1.0, 1.0, 0.0])
        c.u[:] = 0.0
        c.logits[0, 7] = bad                     # decides sequence 0's first draft
        c.logits[5, 11] = bad                    # sequence 1's last row
        c.near[4, 2] = bad                       # sequence 2's first draft row
        r = c.run(dev)
        assert r.accepted.tolist()[:3] == [0, 2, 0]
        assert r.tokens[0].tolist() == [-1, -1, -1] and int(r.tokens[1, 2]) == -1
        assert r.tokens[2].tolist() == [-1, -1, -1]
        assert bool(r.logprobs[0, 0].isnan()) and float(r.logprobs[0, 1]) == 0
        check(c, r, which=[3])
    c = Batch([2], n, seed=9, temps=[1.0])
    c.logits[0] = -inf
    r = c.run(dev)
    assert r.accepted.tolist() == [0] and r.tokens.tolist() == [[-1, -1]]
    # an entry of -inf everywhere but one
    c.logits[:] = -inf
    c.logits[:, 77] = -3.0
    c.drafts[:] = 77
    assert c.run(dev).tokens.tolist() == [[77, 77]]


def test_uniforms_at_their_ends(dev):
    b = Batch([3] * 5, 600, seed=10, temps=[1.0] * 5)
    for value in (0.0, 1 - 2.0 ** -24):
        b.u[:] = value
        check(b, b.run(dev))
    # outside [0, 1): the draw takes the nearest inside
    b.u[:] = 0.5
    last = [2, 5, 8]
    for value, same in ((1.0, 1 - 2.0 ** -24), (7.0, 1 - 2.0 ** -24), (-1.0, 0.0),
                        (float("nan"), 0.0)):
        b.u[last] = value
        got = b.run(dev)
        b.u[last] = same
        assert all(torch.equal(x, y) for x, y in zip(got, b.run(dev)))


@pytest.mark.parametrize("n", [5, 3000, 40000])
def test_equal_distributions(dev, n):
    """p = q: every draft is kept; a uniform of 1 refuses it, and nothing is left of p - q."""
    b = Batch([4] * 3, n, seed=11, temps=[0.8] * 3)
    b.near = b.logits[[0, 1, 2, 4, 5, 6, 8, 9, 10]].clone()
    r = b.run(dev)
    assert r.accepted.tolist() == [3, 3, 3]
    b.u[0] = 1.0
    r = b.run(dev)
    assert r.accepted.tolist() == [0, 3, 3]
    p = softmax(b.logits[0].double().numpy(), b.temps[0])[0]
    cum = np.cumsum(p)
    assert int(r.tokens[0, 0]) == int(np.searchsorted(cum, float(b.u[3]) * cum[-1], side="right"))


def test_missing_drafts(dev):
    b = Batch([4, 4, 4], 900, seed=12, temps=[1.0, 0.0, 1.0])
    b.u[:8] = 0.0
    b.drafts[3:6] = torch.tensor([int(b.logits[4 + j].argmax()) for j in range(3)])
    b.drafts[1] = -1
    b.drafts[4] = -1
    r = b.run(dev)
    assert bi.device_status() == bi.BI_OK
    assert r.accepted.tolist()[:2] == [1, 1]
    p = softmax(b.logits[1].double().numpy(), 1.0)[0]       # from p itself
    cum = np.cumsum(p)
    assert int(r.tokens[0, 1]) == int(np.searchsorted(cum, float(b.u[3]) * cum[-1], side="right"))
    assert int(r.tokens[1, 1]) == int(b.logits[5].argmax())
    check(b, r, which=[])
    for bad in (900, -2, 2 ** 31 - 1):
        b.drafts[1] = bad
        again = b.run(dev)
        assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
        assert all(torch.equal(x, y) for x, y in zip(r, again))


@pytest.mark.parametrize("dtype,n", [("fp32", 40003), ("bf16", 40003), ("fp16", 5)])
@pytest.mark.parametrize("draft", ["logits", "tokens"])
def test_a_sequence_alone_in_a_batch_and_unaligned(dev, dtype, n, draft):
    """The same bits whatever surrounds a sequence, at any alignment and stride."""
    b = Batch([3, 5, 1, 4], n, dtype, draft, seed=13, behind=3)
    whole = b.run(dev)
    check(b, whole)
    wide = b.run(dev, max_q=9)
    assert torch.equal(wide.tokens[:, :5], whole.tokens)
    assert bool((wide.tokens[:, 5:] == -1).all())
    for s, w in enumerate(b.widths):
        one = Batch([w], n, dtype, draft)
        t0, d0 = int(b.cu[s]), int(b.cu[s]) - s
        one.logits, one.u = b.logits[t0:t0 + w], b.u[t0:t0 + w]
        one.drafts, one.temps = b.drafts[d0:d0 + w - 1], [b.temps[s]]
        one.near = None if b.near is None else b.near[d0:d0 + w - 1]
        r = one.run(dev)
        assert torch.equal(r.tokens[0], whole.tokens[s, :w])
        assert torch.equal(r.logprobs[0], whole.logprobs[s, :w])
    for shift in (1, 2, 3):
        def off(x):
            y = torch.full((x.shape[0], n + 8), float("nan"), dtype=x.dtype, device=dev)
            y[:, shift:shift + n] = x.to(dev)
            return y[:, shift:shift + n]
        r = bi.verify_drafts(off(b.logits), b.drafts.to(dev), b.u.to(dev),
                             torch.tensor(b.cu, dtype=torch.int32, device=dev), max_q=5,
                             draft_logits=None if b.near is None else off(b.near),
                             temperature=torch.tensor(b.temps, dtype=torch.float32, device=dev))
        assert all(torch.equal(x, y) for x, y in zip(r, whole))


@pytest.mark.parametrize("batch", [40, 60, 65, 100, 240, 285, 300])
def test_first_sequences_of_batches_of_any_size(dev, batch):
    """However many multiprocessors a sequence gets: the outputs that it has in a batch of five."""
    b = Batch([2] * batch, 33000, dtype="bf16", seed=batch)
    whole = b.run(dev)
    some = bi.verify_drafts(b.logits[:10].to(dev), b.drafts[:5].to(dev), b.u[:10].to(dev),
                            torch.tensor(b.cu[:6], dtype=torch.int32, device=dev), max_q=2,
                            draft_logits=b.near[:5].to(dev),
                            temperature=torch.tensor(b.temps[:5], device=dev))
    assert bi.device_status() == bi.BI_OK
    for x, y in zip(whole, some):
        assert torch.equal(x[:5], y)


def test_malformed_batches_emit_nothing(dev):
    b = Batch([3, 2, 4], 500, seed=14)

    def run(cu, temps=None, max_q=4):
        r = bi.verify_drafts(b.logits.to(dev), b.drafts.to(dev), b.u.to(dev),
                             torch.tensor(cu, dtype=torch.int32, device=dev), max_q=max_q,
                             draft_logits=b.near.to(dev), temperature=torch.tensor(
                                 temps or b.temps, dtype=torch.float32, device=dev))
        return r, bi.device_status()

    for cu in ([1, 3, 5, 9], [0, 3, 3, 9], [0, 3, 5, 10], [0, 5, 3, 9], [0, -3, 5, 9],
               [0, 3, 2 ** 31 - 1, 9], [-2 ** 31, 3, 5, 2 ** 31 - 1], [0, 3, 4, 9]):
        r, status = run(cu)
        assert status == bi.BI_ERR_DEVICE_ARG, cu
        assert bool((r.tokens == -1).all()) and not bool(r.accepted.any())
        assert not bool(r.logprobs.any())
    r, status = run([0, 3, 5, 9], max_q=3)
    assert status == bi.BI_ERR_DEVICE_ARG and bool((r.tokens == -1).all())
    good, status = run([0, 3, 5, 9])
    assert status == bi.BI_OK
    for bad in (-1.0, float("nan"), float("inf"), float("-inf")):
        r, status = run([0, 3, 5, 9], [b.temps[0], bad, b.temps[2]])
        assert status == bi.BI_ERR_DEVICE_ARG
        assert bool((r.tokens[1] == -1).all()) and int(r.accepted[1]) == 0
        assert torch.equal(r.tokens[::2], good.tokens[::2])


def test_captured_beside_an_eager_call_and_on_another_stream(dev):
    a, b = Batch([3, 4], 20000, seed=15), Batch([4, 2], 20000, seed=16)
    wa, wb = a.run(dev), b.run(dev)
    lg, dr, u, nr = (x.to(dev) for x in (a.logits, a.drafts, a.u, a.near))
    cu = torch.tensor(a.cu, dtype=torch.int32, device=dev)
    temps = torch.tensor(a.temps, dtype=torch.float32, device=dev)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r = bi.verify_drafts(lg, dr, u, cu, 4, nr, temps)
    torch.cuda.synchronize()
    graph.replay()
    got = b.run(dev)
    other = bi.verify_drafts(lg, dr, u, cu, 4, nr, temps, stream=side)
    torch.cuda.synchronize()
    for x, y, z, v, w in zip(r, wa, got, wb, other):
        assert torch.equal(x, y) and torch.equal(z, v) and torch.equal(w, y)


def test_workspace_of_the_callers(dev):
    b = Batch([3, 4], 20000, "bf16", seed=17)
    size = bi.verify_drafts_workspace_size(7, 5, 20000)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=dev)
    want = b.run(dev)
    assert all(torch.equal(x, y) for x, y in zip(b.run(dev, workspace=ws), want))
    with pytest.raises(bi.BIError, match="workspace too small"):
        b.run(dev, workspace=ws[:size // 2])
    with pytest.raises(ValueError, match="one row of n entries"):
        b.near = b.near[1:]
        b.run(dev)


def test_refused_tensors(dev):
    b = Batch([3], 100, seed=18)
    b.temps = b.temps * 2
    with pytest.raises(ValueError, match="one entry per sequence"):
        b.run(dev)
    b = Batch([3], 100, seed=18)
    b.u = b.u[:2]
    with pytest.raises(ValueError, match="uniforms"):
        b.run(dev)
    b = Batch([3], 100, seed=18)
    b.drafts = b.drafts.long()
    with pytest.raises(TypeError):
        b.run(dev)
    b = Batch([3], 100, seed=18)
    b.logits = b.logits.double()
    with pytest.raises(ValueError):
        b.run(dev)
    b = Batch([3], 100, seed=18)
    b.near = b.near.to(torch.bfloat16)
    with pytest.raises(TypeError):
        b.run(dev)
    empty = bi.verify_drafts(torch.zeros(0, 10, device=dev), torch.zeros(0, dtype=torch.int32,
                                                                         device=dev),
                             torch.zeros(0, device=dev), torch.zeros(1, dtype=torch.int32,
                                                                     device=dev), 3)
    assert empty.tokens.shape == (0, 3)
