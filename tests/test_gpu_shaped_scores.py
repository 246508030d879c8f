"""Attention with capped scores, a bias of distance, windows and first keys on the GPU: decode,
verify and prefill against 64 bits and against one another."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")

PAGE = 64


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


class Paged:
    """Sequences of given lengths in a bf16 cache of shuffled pages, whose slots past the ends hold
    NaN, and a block of queries at their ends."""

    def __init__(self, dev, lens, qs, hq, hkv, D, seed=0, size=1.0, **shape):
        g = torch.Generator().manual_seed(seed)
        self.dev, self.lens, self.qs, self.hq, self.hkv, self.D = dev, lens, qs, hq, hkv, D
        need = [-(-n // PAGE) for n in lens]
        pages = sum(need) + 2
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
        at = 0
        kv = torch.randn(2, pages, hkv, PAGE, D, generator=g).to(torch.bfloat16)
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
            if lens[b] % PAGE:
                kv[:, self.table[b, n - 1].long(), :, lens[b] % PAGE:] = float("nan")
        kv[:, perm[at:].long()] = float("nan")
        self.kv = kv
        self.k, self.v = kv[0].to(dev), kv[1].to(dev)
        self.T = sum(qs)
        self.q = (torch.randn(self.T, hq, D, generator=g) * size).to(torch.bfloat16).to(dev)
        self.cu = np.concatenate([[0], np.cumsum(qs)])
        self.pos = np.concatenate([np.arange(n - w, n) for n, w in zip(lens, qs)])
        self.seq = np.repeat(np.arange(len(qs)), qs)
        self.scale = D ** -0.5
        self.shape = shape

    def slopes(self):
        s = self.shape.get("slopes")
        return None if s is None else torch.tensor(s, dtype=torch.float32, device=self.dev)

    def first(self):
        f = self.shape.get("first_key")
        return None if f is None else i32(f, self.dev)

    def run(self, form, **kw):
        args = (self.q, self.k, self.v, self.table.to(self.dev), i32(self.lens, self.dev))
        kw = dict(max_seq_len=max(self.lens), scale=self.scale, slopes=self.slopes(),
                  first_key=self.first(), softcap=self.shape.get("softcap", 0.0),
                  window=self.shape.get("window", 0)) | kw
        if form == "decode":
            r = bi.decode_attn(*args, **kw)
        else:
            fn = bi.verify_block if form == "verify" else bi.prefill_attn
            r = fn(*args, i32(self.cu, self.dev), max_q=max(self.qs), **kw)
        return r

    def low(self):
        w, f = self.shape.get("window", 0), self.shape.get("first_key")
        low = self.pos - w + 1 if w else np.zeros(self.T, dtype=np.int64)
        if f is not None:
            low = np.maximum(low, f)
        return np.maximum(low, 0)

    def check(self, out, lse):
        """With A the weighted mean of |v| and S the largest sum of |q k| scale: scores are off by
        d <= D 2^-24 S (their sums) + 2^-21 |x| (scaling, cap and bias, each a few roundings), a
        weight by d + 2^-22 of itself (its power of two) and, in the product with V, by bf16's
        2^-8; the mean by twice the former and once the latter, and its own rounding 2^-8."""
        assert bi.device_status() == bi.BI_OK
        out, lse = out.double().cpu().numpy(), lse.double().cpu().numpy()
        low, G = self.low(), self.hq // self.hkv
        cap, slopes = self.shape.get("softcap", 0.0), self.shape.get("slopes")
        q = self.q.double().cpu().numpy()
        kv = self.kv.double().numpy()
        for t in range(self.T):
            b, pos = self.seq[t], self.pos[t]
            j = np.arange(low[t], pos + 1)
            if not len(j):
                assert (out[t] == 0).all() and np.isneginf(lse[t]).all()
                continue
            page = self.table[b].numpy()[j // PAGE]
            for h in range(self.hq):
                k, v = kv[0][page, h // G, j % PAGE], kv[1][page, h // G, j % PAGE]
                x = k @ q[t, h] * self.scale
                S = (np.abs(k) @ np.abs(q[t, h])).max() * self.scale
                if cap:
                    x = cap * np.tanh(x / cap)
                big = np.abs(x)
                if slopes is not None:
                    bias = float(np.float32(slopes[h])) * (j - pos)
                    x, big = x + bias, big + np.abs(bias)
                m = x.max()
                e = np.exp(x - m)
                p = e / e.sum()
                d = self.D * 2.0 ** -24 * S + 2.0 ** -21 * float((p * big).sum() + big[np.argmax(x)])
                A = p @ np.abs(v)
                want = p @ v
                tol = (2 * d + 2.0 ** -20 + 2.0 ** -8) * A + 2.0 ** -8 * np.abs(want) * 1.01
                assert (np.abs(out[t, h] - want) <= tol).all(), (t, h, np.abs(out[t, h] - want).max())
                ref = m + np.log(e.sum())
                assert abs(lse[t, h] - ref) <= d + 2.0 ** -20 * (1 + abs(ref)), (t, h, lse[t, h], ref)


def alibi(hq):
    return [float(2.0 ** (-8.0 * (i + 1) / hq)) for i in range(hq)]


SHAPES = {
    "window": lambda hq, T, pos: dict(window=100),
    "window 1": lambda hq, T, pos: dict(window=1),
    "cap": lambda hq, T, pos: dict(softcap=20.0),
    "small cap": lambda hq, T, pos: dict(softcap=0.5),
    "large cap": lambda hq, T, pos: dict(softcap=1000.0),
    "bias": lambda hq, T, pos: dict(slopes=alibi(hq)),
    "rising bias": lambda hq, T, pos: dict(slopes=[-0.02] * hq),
    "steep bias": lambda hq, T, pos: dict(slopes=[30.0] * hq),
    "first": lambda hq, T, pos: dict(first_key=np.maximum(pos - pos % 150 - 70, -5)),
    "some see nothing": lambda hq, T, pos: dict(
        first_key=np.where(np.arange(T) % 3 == 0, pos + 1 + np.arange(T), pos - 10)),
    "none sees anything": lambda hq, T, pos: dict(first_key=pos + 1),
    "all": lambda hq, T, pos: dict(softcap=15.0, slopes=alibi(hq), window=300,
                                   first_key=pos - pos % 170),
    "cap window": lambda hq, T, pos: dict(softcap=5.0, window=513),
}
SIZES = {"cap": 4.0, "large cap": 4.0, "all": 4.0}


def make(dev, name, lens, qs, hq, hkv, D, seed=0):
    p = Paged(dev, lens, qs, hq, hkv, D, seed, SIZES.get(name, 1.0))
    p.shape = SHAPES[name](hq, p.T, p.pos)
    return p


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("lens,hq,hkv,D", [
    ([1, 64, 700, 130], 4, 1, 64), ([1100, 3, 512, 513], 8, 2, 128), ([2000], 32, 32, 128)])
def test_decode(dev, name, lens, hq, hkv, D):
    p = make(dev, name, lens, [1] * len(lens), hq, hkv, D)
    p.check(*p.run("decode"))


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("lens,qs,hq,hkv,D", [
    ([8, 64, 700, 130], [8, 1, 5, 3], 8, 2, 64), ([1100, 3, 512, 515], [4, 3, 2, 4], 16, 2, 128)])
def test_verify(dev, name, lens, qs, hq, hkv, D):
    p = make(dev, name, lens, qs, hq, hkv, D)
    p.check(*p.run("verify"))


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("lens,qs,hq,hkv,D", [
    ([40, 700, 130], [40, 200, 3], 4, 1, 64), ([1300, 3, 515], [90, 3, 200], 8, 2, 128),
    ([620], [620], 2, 2, 128)])
def test_prefill(dev, name, lens, qs, hq, hkv, D):
    p = make(dev, name, lens, qs, hq, hkv, D)
    p.check(*p.run("prefill"))


@pytest.mark.parametrize("name", SHAPES)
@pytest.mark.parametrize("hq,hkv,D", [(8, 2, 128), (4, 1, 64)])
def test_one_query_s_bits_are_the_same_everywhere(dev, name, hq, hkv, D):
    """A long block by prefill, in verify blocks, token by token, and a part of it alone."""
    lens, qs = [900, 70], [300, 64]
    p = make(dev, name, lens, qs, hq, hkv, D, seed=3)
    out, lse = p.run("prefill")
    first = p.shape.get("first_key")
    for t in list(range(0, 300, 37)) + [299, 300, 363]:
        b, pos = int(p.seq[t]), int(p.pos[t])
        t0 = max(int(p.cu[b]), t - 6)
        n = t - t0 + 1
        q = p.q[t0:t + 1].contiguous()
        shape = dict(slopes=p.slopes(), softcap=p.shape.get("softcap", 0.0),
                     window=p.shape.get("window", 0),
                     first_key=None if first is None else i32(first[t0:t + 1], dev))
        common = (p.k, p.v, p.table[b:b + 1].to(dev), i32([pos + 1], dev))
        o, l = bi.verify_block(q, *common, i32([0, n], dev), max_q=8, max_seq_len=lens[b],
                               scale=p.scale, **shape)
        assert torch.equal(o.view(torch.int16), out[t0:t + 1].view(torch.int16))
        assert torch.equal(l, lse[t0:t + 1])
        if first is not None:
            shape["first_key"] = shape["first_key"][-1:]
        o, l = bi.decode_attn(q[-1:], *common, max_seq_len=lens[b] + 40 if lens[b] == 900 else 128,
                              scale=p.scale, **shape)
        assert torch.equal(o.view(torch.int16), out[t:t + 1].view(torch.int16))
        assert torch.equal(l, lse[t:t + 1])
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("form", ["decode", "verify", "prefill"])
@pytest.mark.parametrize("D", [64, 128])
def test_limits_that_hide_nothing_give_the_plain_bits(dev, form, D):
    qs = {"decode": [1, 1], "verify": [4, 2], "prefill": [150, 31]}[form]
    p = Paged(dev, [1200, 200], qs, 8, 2, D, seed=4)
    out, lse = p.run(form)
    for kw in (dict(window=1199), dict(window=10 ** 6), dict(first_key=i32([-7] * p.T, dev)),
               dict(window=1200, first_key=i32([0] * p.T, dev))):
        if kw.get("window") == 1199 and form == "decode":
            kw["window"] = 1200
        o, l = p.run(form, **kw)
        if kw.get("window") == 1199:  # the last token of the first sequence sees one key less
            o, l, ro, rl = (x[qs[0]:] for x in (o, l, out, lse))
        else:
            ro, rl = out, lse
        assert torch.equal(o.view(torch.int16), ro.view(torch.int16)) and torch.equal(l, rl)


@pytest.mark.parametrize("form", ["decode", "verify", "prefill"])
@pytest.mark.parametrize("by", ["window", "first"])
def test_pages_out_of_sight_may_be_gone(dev, form, by):
    """Pages in front of every token's keys are neither read nor looked up; what lies in front of
    the first key in its page may be NaN."""
    qs = {"decode": [1, 1], "verify": [4, 3], "prefill": [70, 3]}[form]
    p = Paged(dev, [1500, 300], qs, 8, 2, 128, seed=5)
    p.shape = dict(window=200) if by == "window" else dict(
        first_key=np.where(p.seq == 0, 1500 - 260, 33))
    out, lse = p.run(form)
    low = p.low()
    for b in range(2):
        first = int(low[p.seq == b].min())
        gone = first // PAGE
        p.table[b, :gone] = torch.tensor([-1, 10 ** 6, -2 ** 31] * gone, dtype=torch.int32)[:gone]
        page = int(p.table[b, gone])
        p.kv[:, page, :, :first % PAGE] = float("nan")
    p.k, p.v = p.kv[0].to(dev), p.kv[1].to(dev)
    o, l = p.run(form)
    assert torch.equal(o.view(torch.int16), out.view(torch.int16)) and torch.equal(l, lse)
    p.check(o, l)
    p.table[0, int(low[0]) // PAGE + 1] = -1           # one that is seen
    p.run(form)
    assert bi.device_status() == bi.BI_ERR_DEVICE_ARG


@pytest.mark.parametrize("name", ["window", "cap", "bias", "all", "some see nothing"])
def test_outside_the_limit(dev, name):
    """Chosen chunk lengths: other bits, the same values."""
    bi.set_batch_invariant_limit(0)
    for lens, qs, form in (([3000], [1], "decode"), ([900, 2000, 64], [4, 8, 1], "verify")):
        p = make(dev, name, lens, qs, 8, 2, 128, seed=6)
        p.check(*p.run(form))
        big = torch.empty(8 * bi.attn_workspace_size(p.T, 8, 128, max(lens)), dtype=torch.uint8,
                          device=dev)
        p.check(*p.run(form, workspace=big))


@pytest.mark.parametrize("form", ["decode", "prefill"])
def test_a_large_batch(dev, form):
    """Rows enough for the merge of a warp per row, and more sequences than multiprocessors."""
    B = 200 if form == "decode" else 12
    g = np.random.default_rng(7)
    lens = [int(x) for x in g.integers(30, 1400, B)]
    qs = [1] * B if form == "decode" else [int(min(n, w)) for n, w in zip(lens, g.integers(1, 60, B))]
    p = Paged(dev, lens, qs, 8, 2, 64, seed=8)
    p.shape = dict(window=77, slopes=alibi(8))
    p.check(*p.run(form))


def test_captured_and_replayed_beside_another_call(dev):
    a = make(dev, "all", [900, 300], [150, 20], 8, 2, 128, seed=9)
    b = make(dev, "cap", [700, 80], [4, 2], 8, 2, 128, seed=10)
    want, other = a.run("prefill"), b.run("verify")
    args = (a.q, a.k, a.v, a.table.to(dev), i32(a.lens, dev), i32(a.cu, dev))
    slopes, first = a.slopes(), a.first()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r = bi.prefill_attn(*args, max_q=150, max_seq_len=900, scale=a.scale, softcap=15.0,
                            slopes=slopes, window=300, first_key=first)
    torch.cuda.synchronize()
    graph.replay()
    again = b.run("verify")
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(r, want))
    assert all(torch.equal(x, y) for x, y in zip(again, other))


def test_refused_arguments(dev):
    p = Paged(dev, [100], [3], 8, 2, 64)
    for kw in (dict(window=-1), dict(softcap=-1.0), dict(softcap=float("nan")),
               dict(softcap=float("inf")), dict(softcap=1e-9), dict(softcap=1e9),
               dict(softcap=5.0, scale=0.0), dict(window=3, scale=-1.0)):
        for form in ("verify", "prefill"):
            with pytest.raises(bi.BIError):
                p.run(form, **kw)
    with pytest.raises(ValueError, match="slopes"):
        p.run("verify", slopes=torch.zeros(4, device=dev))
    with pytest.raises(ValueError, match="first_key"):
        p.run("verify", first_key=i32([0] * 4, dev))
    with pytest.raises(TypeError):
        p.run("prefill", first_key=torch.zeros(3, device=dev))
    with pytest.raises(ValueError, match="CUDA"):
        p.run("prefill", slopes=torch.zeros(8))


@pytest.mark.parametrize("name", ["cap", "all", "some see nothing"])
@pytest.mark.parametrize("hq,hkv", [(32, 1), (64, 1), (3, 3)])
def test_wide_and_single_groups(dev, name, hq, hkv):
    """32 and 64 query heads of one KV head (tiles of four and two tokens), and as many KV heads."""
    p = make(dev, name, [300, 70, 9], [40, 70, 1], hq, hkv, 64, seed=12)
    p.check(*p.run("prefill"))
    if hq // hkv <= 32:
        p = make(dev, name, [300, 70, 9], [1, 1, 1], hq, hkv, 64, seed=13)
        p.check(*p.run("decode"))


def test_mismatched_tensors_are_refused(dev):
    p = Paged(dev, [100, 70], [3, 2], 8, 2, 64)
    p.shape = dict(window=10)
    p.table = p.table[:1]
    with pytest.raises(ValueError, match="block_table"):
        p.run("verify")
    p = Paged(dev, [100, 70], [3, 2], 8, 2, 64)
    p.shape = dict(window=10)
    p.q = p.q.repeat(1, 1, 2)
    with pytest.raises(ValueError, match="cache's D"):
        p.run("prefill")
    p = Paged(dev, [100, 70], [1, 1], 8, 2, 64)
    p.q = p.q[:1]
    with pytest.raises(ValueError, match="a token per sequence"):
        p.run("decode", window=10)


@pytest.mark.parametrize("total,fill", [(100, 0x7f), (100, 0xff), (1700, 0x7f), (1700, 0xff)])
def test_offsets_that_fall_in_a_long_block(dev, total, fill):
    """Token offsets that fall: that sequence is skipped and reported, the one behind it shares
    tokens with the one in front, and the sequences apart from these are as they should be."""
    lens, cu = [300, 200, 64, 5000], [0, 20, 90, 50, total]
    p = Paged(dev, lens, [20, 70, 1, total - 50], 8, 2, 64, seed=9)
    first = torch.randint(0, 250, (p.T,), dtype=torch.int32).tolist()
    args = (p.k, p.v, p.table.to(dev), i32(lens, dev))
    kw = dict(max_seq_len=5000, scale=p.scale, max_q=total)
    ws = torch.full((bi.attn_workspace_size(p.T, 8, 64, 5000),), fill, dtype=torch.uint8,
                    device=dev)
    want, lse = bi.prefill_attn(p.q[:20], *(x[:1] if x.dim() < 3 else x for x in args),
                                i32([0, 20], dev), first_key=i32(first[:20], dev), **kw)
    assert bi.device_status() == bi.BI_OK
    got = bi.prefill_attn(p.q, *args, i32(cu, dev), first_key=i32(first, dev), workspace=ws, **kw)
    assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
    assert torch.equal(got[0][:20].view(torch.int16), want.view(torch.int16))
    assert torch.equal(got[1][:20], lse)
