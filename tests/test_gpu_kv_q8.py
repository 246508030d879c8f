"""The 8-bit paged KV cache on the GPU: the quantising append against the format's definition,
decode, verify and prefill attention against 64 bits, and the library's contract for them: a
token's bytes and a query's bits do not depend on the batch, on how a sequence was cut into
calls, or on anything at later positions."""
import numpy as np
import pytest
import torch

import q8_reference as ref
from tolerance import bits_equal, check_rows_rel_l2

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")

POISON = 0x7F  # e4m3's NaN


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


def i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class Cache:
    """An 8-bit cache whose unwritten slots hold NaN codes, with a shuffled block table."""

    def __init__(self, lens, Hkv, D, dev, seed=0, spare=2):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // 64) for n in lens]
        pages = sum(need) + spare
        perm = torch.randperm(pages, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = perm[at:at + n]
            at += n
        self.table = self.table.to(dev)
        self.lens = list(lens)
        self.k, self.v = (torch.full((pages, Hkv, 64, D), POISON, dtype=torch.uint8, device=dev)
                          for _ in range(2))
        self.ks, self.vs = (torch.full((pages, Hkv, 64), 254, dtype=torch.uint8, device=dev)
                            for _ in range(2))

    def parts(self):
        return self.k, self.v, self.ks, self.vs

    def append(self, k, v, lens, qs, rows=None):
        """New rows of each sequence (lens include them)."""
        dev = k.device
        cu = np.concatenate([[0], np.cumsum(qs)])
        table = self.table if rows is None else self.table[rows].contiguous()
        bi.kv_append_q8(k.contiguous(), v.contiguous(), *self.parts(), table, i32(lens, dev),
                        i32(cu, dev))

    def values(self):
        return (ref.cache_values(self.k, self.ks), ref.cache_values(self.v, self.vs),
                ref.scale_values(self.vs))


def rows(shape, seed, spread=1.0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * std
    return (x * torch.exp2(torch.randn(*shape[:-1], 1, generator=g) * spread)).to(torch.bfloat16)


def filled(lens, Hkv, D, dev, seed=0, spread=1.0, std=1.0, k=None, v=None):
    c = Cache(lens, Hkv, D, dev, seed)
    T = sum(lens)
    c.k_rows = rows((T, Hkv, D), seed + 1, spread, std) if k is None else k
    c.v_rows = rows((T, Hkv, D), seed + 2, spread, std) if v is None else v
    c.append(c.k_rows.to(dev), c.v_rows.to(dev), lens, lens)
    return c


def attend(c, q, lens, qs, scale, form, sel=None, **kw):
    dev = q.device
    table = c.table if sel is None else c.table[sel].contiguous()
    common = dict(max_seq_len=max(lens), scale=scale, **kw)
    if form == "decode":
        return bi.decode_attn_q8(q, *c.parts(), table, i32(lens, dev), **common)
    cu = i32(np.concatenate([[0], np.cumsum(qs)]), dev)
    fn = bi.verify_block_q8 if form == "verify" else bi.prefill_attn_q8
    return fn(q, *c.parts(), table, i32(lens, dev), cu, max_q=max(qs), **common)


# ------------------------------------------------------------------------------- append

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv", [1, 3, 8])
@pytest.mark.parametrize("lens,qs", [([1], [1]), ([64, 65, 200], [64, 1, 130]),
                                     ([700, 5, 129, 1], [3, 5, 129, 1])])
def test_append_matches_the_definition(dev, D, Hkv, lens, qs):
    c = Cache(lens, Hkv, D, dev, seed=3)
    T = sum(qs)
    kn, vn = rows((T, Hkv, D), 10, 3.0), rows((T, Hkv, D), 11, 3.0)
    before = [t.clone() for t in c.parts()]
    c.append(kn.to(dev), vn.to(dev), lens, qs)
    want = [t.cpu().clone() for t in before]
    t = 0
    for b, (L, w) in enumerate(zip(lens, qs)):
        for j in range(w):
            pos = L - w + j
            page = int(c.table[b, pos // 64])
            for x, src in ((0, kn), (1, vn)):
                y, s = ref.quantise_rows(src[t + j].double().numpy())
                assert np.array_equal(ref.code_values(c.parts()[x][page, :, pos % 64]), y)
                want[x][page, :, pos % 64] = c.parts()[x][page, :, pos % 64].cpu()
                want[2 + x][page, :, pos % 64] = torch.from_numpy(s)
        t += w
    for got, w in zip(c.parts(), want):  # the rows' bytes, and every other byte as it was
        assert torch.equal(got.cpu(), w)
    assert bi.device_status() == bi.BI_OK


def test_append_of_special_rows(dev):
    """Zeros, the border amax = 448 * 2^e and its neighbours, ties between codes, subnormal and
    huge bf16 values, and rows with an infinity or NaN."""
    D = 64
    special = torch.zeros(14, 1, D, dtype=torch.float32)
    special[1, 0, 3] = 448.0
    special[2, 0, 3] = 450.0                       # bf16 just above 448: the next scale
    special[3, 0, :2] = torch.tensor([-448.0 * 2.0 ** 20, 1.0])
    special[4, 0] = torch.arange(D) / 16 + 2.0     # ties of the three-bit mantissa
    special[5, 0] = 2.0 ** -126                    # smallest normal bf16
    special[6, 0, 0] = 2.0 ** -133                 # bf16 subnormal: below the scale's floor
    special[7, 0, 5] = 3.3e38
    special[8, 0, 0], special[8, 0, 1] = float("inf"), 1.0
    special[9, 0, 63] = float("nan")
    special[10, 0, 1] = float("-inf")
    special[11, 0, 0], special[11, 0, 1:] = 448.0, 2.0 ** -10   # half of e4m3's least value
    special[12, 0, 0], special[12, 0, 1:] = 448.0, 3 * 2.0 ** -10  # a tie: to even
    special[13, 0] = -0.0
    x = special.to(torch.bfloat16)
    n = x.shape[0]
    c = Cache([n], 1, D, dev)
    c.append(x.to(dev), x.flip(0).to(dev), [n], [n])
    page = int(c.table[0, 0])
    for parts, src in (((c.k, c.ks), x), ((c.v, c.vs), x.flip(0))):
        y, s = ref.quantise_rows(src[:, 0].double().numpy())
        assert np.array_equal(ref.code_values(parts[0][page, 0, :n]), y)
        assert np.array_equal(parts[1][page, 0, :n].cpu().numpy(), s)


def test_append_does_not_depend_on_how_the_tokens_come(dev):
    """One block, blocks of assorted widths, single tokens, and a rejected draft written over:
    the same bytes."""
    L, Hkv, D = 150, 2, 128
    k, v = rows((L, Hkv, D), 1).to(dev), rows((L, Hkv, D), 2).to(dev)
    whole = Cache([L], Hkv, D, dev)
    whole.append(k, v, [L], [L])
    for cuts in ([0, 1, 9, 64, 100, 150], list(range(L + 1))):
        c = Cache([L], Hkv, D, dev)
        for a, b in zip(cuts[:-1], cuts[1:]):
            if b < L:  # a draft that is rejected: larger values at the next positions
                c.append(k[a:b + 1] * 64, v[a:b + 1] * 64, [b + 1], [b + 1 - a])
            c.append(k[a:b], v[a:b], [b], [b - a])
        for x, y in zip(c.parts(), whole.parts()):
            pages = c.table[0].long()
            assert torch.equal(x[pages].transpose(1, 2).flatten(0, 1)[:L],
                               y[pages].transpose(1, 2).flatten(0, 1)[:L])


def test_append_ignores_padding_and_latches_bad_pages(dev):
    """Token rows behind the last sequence are not read into the cache; a page index out of
    range is skipped and reported, the other sequence is written."""
    Hkv, D = 2, 64
    c = Cache([70, 70], Hkv, D, dev)
    k, v = rows((9, Hkv, D), 1).to(dev), rows((9, Hkv, D), 2).to(dev)
    bad = c.table.clone()
    bad[0, 1] = c.k.shape[0]
    bi.kv_append_q8(k, v, *c.parts(), bad, i32([70, 70], dev), i32([0, 2, 5], dev))
    assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
    changed = (c.ks != 254).nonzero().cpu().tolist()
    page = int(c.table[1, 1])
    assert sorted(changed) == sorted([page, h, s] for h in range(Hkv) for s in (3, 4, 5))
    # lengths that do not hold their block
    bi.kv_append_q8(k, v, *c.parts(), c.table, i32([1, 70], dev), i32([0, 2, 5], dev))
    assert bi.device_status() == bi.BI_ERR_DEVICE_ARG


# ---------------------------------------------------------------------------- attention

CASES = [
    # (lens, block widths, Hq, Hkv, D)
    ([1], [1], 4, 4, 64),
    ([1, 2, 63, 64, 65], [1, 1, 1, 1, 1], 8, 2, 128),
    ([127, 128, 129, 191, 193], [1, 2, 3, 8, 1], 8, 2, 64),
    ([511, 512, 513, 1025], [8, 1, 8, 5], 32, 8, 128),
    ([300, 5], [4, 4], 24, 8, 128),          # groups of 3
    ([640, 1100], [6, 2], 10, 2, 64),         # groups of 5
    ([130, 900], [1, 1], 32, 1, 128),         # groups of 32
    ([1500], [8], 4, 4, 128),                 # groups of 1
    ([300, 77, 1], [300, 70, 1], 8, 2, 128),  # prompts
    ([900, 40], [200, 40], 32, 1, 64),        # one token a tile
    ([1300], [37], 24, 8, 64),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_against_64_bits(dev, case):
    lens, qs, Hq, Hkv, D = CASES[case]
    c = filled(lens, Hkv, D, dev, seed=20 + case)
    T = sum(qs)
    q = rows((T, Hq, D), 90 + case, 0.5)
    forms = (["prefill"] + (["verify"] if max(qs) * Hq // Hkv <= 32 and max(qs) <= 8 else [])
             + (["decode"] if max(qs) == 1 else []))
    kv = c.values()
    outs = []
    for form in forms:
        # rows in front of and behind the block stay as they are
        obuf = torch.full((T + 2, Hq, D), 3.0, dtype=torch.bfloat16, device=dev)
        lbuf = torch.full((T + 2, Hq), 5.0, dtype=torch.float32, device=dev)
        attend(c, q.to(dev), lens, qs, D ** -0.5, form, out=obuf[1:T + 1], lse=lbuf[1:T + 1])
        assert bool((obuf[0] == 3).all() and (obuf[-1] == 3).all())
        assert bool((lbuf[0] == 5).all() and (lbuf[-1] == 5).all())
        t = 0
        for b, (L, w) in enumerate(zip(lens, qs)):
            r = ref.attention(q[t:t + w].double().numpy(), *kv, c.table[b].tolist(), L, w,
                              D ** -0.5, Hq // Hkv)
            ref.check_attention(obuf[1 + t:1 + t + w], lbuf[1 + t:1 + t + w], r,
                                f"{form} sequence {b}")
            check_rows_rel_l2(obuf[1 + t:1 + t + w], r[0], what=f"{form} sequence {b}")
            t += w
        outs.append((obuf, lbuf))
    for o, l in outs[1:]:
        assert bits_equal(o, outs[0][0]) and bits_equal(l, outs[0][1])
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 32, 8), (64, 8, 2), (128, 24, 8)])
def test_every_way_to_a_query_gives_its_bits(dev, D, Hq, Hkv):
    """A prompt in one call, cut into chunks, verify blocks, single tokens, and inside a batch
    of other sequences."""
    L = 1100
    c = filled([L, 700, 40], Hkv, D, dev, seed=5)
    q = rows((L, Hq, D), 6).to(dev)
    sc = D ** -0.5
    full, flse = attend(c, q, [L], [L], sc, "prefill", sel=[0])

    def same(o, l, a, b, what):
        assert bits_equal(o, full[a:b]) and bits_equal(l, flse[a:b]), what
    for a, b in ((0, 100), (100, 433), (433, 640), (640, 1100)):
        same(*attend(c, q[a:b].contiguous(), [b], [b - a], sc, "prefill", sel=[0]), a, b,
             f"chunk {a}:{b}")
    w = min(8, 32 * Hkv // Hq)
    for a in (0, 60, 504, 508, 1020, 1090):
        same(*attend(c, q[a:a + w].contiguous(), [a + w], [w], sc, "verify", sel=[0]), a, a + w,
             f"verify {a}")
    other = rows((8, Hq, D), 7).to(dev)
    for t in (0, 1, 63, 64, 127, 128, 511, 512, 513, 1023, 1024, 1099):
        o, l = attend(c, q[t:t + 1].contiguous(), [t + 1], [1], sc, "decode", sel=[0])
        same(o, l, t, t + 1, f"decode {t}")
        qq = torch.cat([other[:1], q[t:t + 1], other[1:2]]).contiguous()
        o, l = attend(c, qq, [700, t + 1, 40], [1, 1, 1], sc, "decode", sel=[1, 0, 2])
        same(o[1:2], l[1:2], t, t + 1, f"decode {t} in a batch")
        qq = torch.cat([other[:3], q[t:t + 1], other[3:4]]).contiguous()
        o, l = attend(c, qq, [700, t + 1, 40], [3, 1, 1], sc, "verify", sel=[1, 0, 2])
        same(o[3:4], l[3:4], t, t + 1, f"decode {t} beside a block")


def test_later_and_unwritten_keys_do_not_reach_a_query(dev):
    """NaN, infinite and huge rows behind a query's position (later drafts of its block, and
    slots past the sequence's end) leave its bits alone; the queries that see them are NaN."""
    L, Hkv, D, Hq = 200, 2, 128, 8
    clean = filled([L], Hkv, D, dev, seed=30)
    q = rows((8, Hq, D), 31).to(dev)
    want, wlse = attend(clean, q[:3].contiguous(), [L - 5], [3], D ** -0.5, "verify")
    for which in "kv":
        for bad in (float("nan"), float("inf"), 3e38):
            c = filled([L], Hkv, D, dev, seed=30, k=clean.k_rows.clone(), v=clean.v_rows.clone())
            kr, vr = clean.k_rows[-5:].clone(), clean.v_rows[-5:].clone()
            (kr if which == "k" else vr)[0, :, 7] = bad
            c.append(kr.to(dev), vr.to(dev), [L], [5])
            o, l = attend(c, q, [L], [8], D ** -0.5, "verify")
            assert bits_equal(o[:3], want) and bits_equal(l[:3], wlse), (which, bad)
            if bad != 3e38:
                assert bool(torch.isnan(o[3:]).all())
    assert bi.device_status() == bi.BI_OK


@pytest.mark.parametrize("kind", ["zero values", "spread", "peaked", "tiny", "large", "equal",
                                  "rising"])
def test_attention_of_hard_rows(dev, kind):
    L, Hkv, D, Hq = 1300, 2, 128, 8
    k, v = rows((L, Hkv, D), 40), rows((L, Hkv, D), 41)
    q = rows((4, Hq, D), 42)
    if kind == "zero values":      # rows of zeros (scale floor) among ordinary ones
        v[::3] = 0
        v[:256] = 0                # and a first chunk that starts with nothing else
        k[5::7] = 0
    elif kind == "spread":         # token sizes over 2^+-24
        v = (v.float() * torch.exp2((torch.arange(L) % 49 - 24.0).view(-1, 1, 1))).bfloat16()
    elif kind == "peaked":         # one key far above the others
        k = (k.float() * 0.1).bfloat16()
        k[700] = q[0, ::4].sign() * 4
    elif kind == "tiny":
        v = (v.float() * 2.0 ** -40).bfloat16()
        k = (k.float() * 2.0 ** -40).bfloat16()
    elif kind == "large":
        v = (v.float() * 2.0 ** 40).bfloat16()
    elif kind == "equal":
        k[:] = k[:1]
        v[:] = v[:1]
    elif kind == "rising":         # each key scores above the one before it: the maximum rises
        k = (q[0, ::4].float() * torch.linspace(-1, 1, L).view(-1, 1, 1)).bfloat16()
    c = filled([L], Hkv, D, dev, seed=43, k=k, v=v)
    out, lse = attend(c, q.to(dev), [L], [4], D ** -0.5, "verify")
    kv = c.values()
    r = ref.attention(q.double().numpy(), *kv, c.table[0].tolist(), L, 4, D ** -0.5, Hq // Hkv)
    ref.check_attention(out, lse, r, kind)


def test_caches_written_by_others(dev):
    """Any codes and scale bytes the format allows, not only what the append writes: K scales of 0
    and 1 (scores of nothing), the largest ones, V scales far from each other; rows of NaN (byte
    255) whose codes are not zero reach the queries that see them and no others."""
    L, Hkv, D, Hq = 700, 2, 128, 8
    c = filled([L], Hkv, D, dev, seed=52)
    g = torch.Generator().manual_seed(53)
    codes = torch.randint(0, 256, c.k.shape, generator=g, dtype=torch.int32)
    codes = torch.where((codes & 0x7F) == 0x7F, codes - 1, codes).to(torch.uint8)
    c.k.copy_(codes.flip(0))
    c.v.copy_(codes)
    c.ks.copy_(torch.randint(112, 119, c.ks.shape, generator=g))
    c.vs.copy_(torch.randint(100, 140, c.vs.shape, generator=g))
    page = c.table[0].long()
    c.ks[page[0], :, ::5] = 0
    c.ks[page[3], 1, 3::7] = 1
    q = rows((8, Hq, D), 54)
    out, lse = attend(c, q.to(dev), [L], [8], D ** -0.5, "verify")
    r = ref.attention(q.double().numpy(), *c.values(), c.table[0].tolist(), L, 8, D ** -0.5, 4)
    ref.check_attention(out, lse, r)
    at = (int(page[(L - 3) // 64]), 1, (L - 3) % 64)   # seen by the last three tokens, head 1
    for scale in (c.ks, c.vs):
        kept = int(scale[at])
        scale[at] = 255
        o, l = attend(c, q.to(dev), [L], [8], D ** -0.5, "verify")
        assert bool(torch.isnan(o[5:, 4:]).all())
        assert bits_equal(o[:5], out[:5]) and bits_equal(o[5:, :4].contiguous(),
                                                         out[5:, :4].contiguous())
        scale[at] = kept
    c.vs.fill_(254)
    c.v.copy_(torch.where(codes.to(dev) < 128, 1, 129))  # +-2^-9 * 2^127 = +-2^118
    out, lse = attend(c, q.to(dev), [L], [8], D ** -0.5, "verify")
    r = ref.attention(q.double().numpy(), *c.values(), c.table[0].tolist(), L, 8, D ** -0.5, 4)
    ref.check_attention(out, lse, r)


def test_query_sizes(dev):
    """Queries of zeros, and with elements 2^30 apart."""
    L, Hkv, D, Hq = 100, 1, 64, 4
    c = filled([L], Hkv, D, dev, seed=50)
    q = rows((3, Hq, D), 51)
    q[0] = 0
    q[1] = (q[1].float() * torch.exp2(-(torch.arange(D) % 31).float())).bfloat16()
    q[2] = (q[2].float() * 2.0 ** -60).bfloat16()
    out, lse = attend(c, q.to(dev), [L], [3], D ** -0.5, "verify")
    r = ref.attention(q.double().numpy(), *c.values(), c.table[0].tolist(), L, 3, D ** -0.5, 4)
    ref.check_attention(out, lse, r)


@pytest.mark.parametrize("L,qs", [(65540, 8), (16388, 1)])
def test_long_contexts(dev, L, qs):
    Hq, Hkv, D = 8, 2, 128
    c = filled([L], Hkv, D, dev, seed=60)
    q = rows((qs, Hq, D), 61)
    out, lse = attend(c, q.to(dev), [L], [qs], D ** -0.5, "verify")
    r = ref.attention(q.double().numpy(), *c.values(), c.table[0].tolist(), L, qs, D ** -0.5, 4)
    ref.check_attention(out, lse, r)
    check_rows_rel_l2(out, r[0])


@pytest.mark.parametrize("D,Hq,Hkv,qs", [(128, 32, 8, 1), (128, 32, 8, 8), (64, 8, 8, 3),
                                         (128, 16, 4, 4), (64, 8, 8, 1), (128, 8, 8, 7)])
def test_more_work_items_than_multiprocessors(dev, D, Hq, Hkv, qs):
    """Batches whose chunks give every multiprocessor many items in turn (the hand-offs between
    the kernel's warps wrap around many times), with short and long sequences: each sequence's
    bits alone, and two of them against 64 bits."""
    g = torch.Generator().manual_seed(qs)
    B = 96
    lens = [int(x) for x in torch.randint(qs, 2600, (B,), generator=g)]
    lens[5], lens[50] = 2561, qs
    widths = [min(qs, 1 + int(x)) for x in torch.randint(0, 8, (B,), generator=g)]
    widths[0] = qs
    c = filled(lens, Hkv, D, dev, seed=65)
    q = rows((sum(widths), Hq, D), 66).to(dev)
    forms = ["verify", "prefill"] + (["decode"] if qs == 1 else [])
    out, lse = attend(c, q, lens, widths, D ** -0.5, forms[0])
    for form in forms[1:]:
        o, l = attend(c, q, lens, widths, D ** -0.5, form)
        assert bits_equal(o, out) and bits_equal(l, lse), form
    cu = np.concatenate([[0], np.cumsum(widths)])
    kv = c.values()
    for b in (0, 5, 50, 95):
        a, e = int(cu[b]), int(cu[b + 1])
        o, l = attend(c, q[a:e].contiguous(), [lens[b]], [widths[b]], D ** -0.5, "verify", sel=[b])
        assert bits_equal(o, out[a:e]) and bits_equal(l, lse[a:e]), b
    for b in (5, 50):
        a, e = int(cu[b]), int(cu[b + 1])
        r = ref.attention(q[a:e].double().cpu().numpy(), *kv, c.table[b].tolist(), lens[b],
                          widths[b], D ** -0.5, Hq // Hkv)
        ref.check_attention(out[a:e], lse[a:e], r)
    assert bi.device_status() == bi.BI_OK


def test_malformed_sequences_are_skipped(dev):
    """A bad page, a block wider than max_q and a length over max_seq_len are reported; the
    other sequences' rows are right and the offenders' rows of out are not written past."""
    lens, Hq, Hkv, D = [300, 300, 300], 8, 2, 128
    c = filled(lens, Hkv, D, dev, seed=70)
    q = rows((3, Hq, D), 71).to(dev)
    good, _ = attend(c, q, lens, [1, 1, 1], 0.1, "decode")
    bad = Cache.__new__(Cache)
    bad.__dict__ = dict(c.__dict__)
    bad.table = c.table.clone()
    bad.table[1, 2] = -7
    o, _ = attend(bad, q, lens, [1, 1, 1], 0.1, "decode")
    assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
    assert bits_equal(o[0], good[0]) and bits_equal(o[2], good[2])
    o, _ = bi.decode_attn_q8(q, *c.parts(), c.table, i32([300, 320, 300], dev), max_seq_len=300,
                             scale=0.1)
    assert bi.device_status() == bi.BI_ERR_DEVICE_ARG
    assert bits_equal(o[0], good[0]) and bits_equal(o[2], good[2])
    assert bi.device_status() == bi.BI_OK


def test_rows_behind_the_last_sequence_stay(dev):
    """total_q beyond cu_q[batch] (a padded batch): the rows past it are not written."""
    Hq, Hkv, D = 8, 2, 64
    c = filled([100, 90], Hkv, D, dev, seed=80)
    q = rows((9, Hq, D), 81).to(dev)
    out = torch.full((9, Hq, D), 7.0, dtype=torch.bfloat16, device=dev)
    bi.prefill_attn_q8(q, *c.parts(), c.table, i32([100, 90], dev), i32([0, 4, 6], dev), max_q=5,
                       max_seq_len=100, scale=0.2, out=out)
    want, _ = attend(c, q[:6].contiguous(), [100, 90], [4, 2], 0.2, "prefill")
    assert bits_equal(out[:6], want) and bool((out[6:] == 7).all())
    assert bi.device_status() == bi.BI_OK


def test_the_largest_batch(dev):
    """1,024 sequences (the limit) of 1 to 130 tokens: sampled ones equal themselves alone."""
    g = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(1, 131, (1024,), generator=g)]
    c = filled(lens, 2, 64, dev, seed=84)
    q = rows((1024, 8, 64), 85).to(dev)
    out, lse = attend(c, q, lens, [1] * 1024, 0.125, "decode")
    for b in (0, 1, 511, 1022, 1023):
        o, l = attend(c, q[b:b + 1].contiguous(), [lens[b]], [1], 0.125, "decode", sel=[b])
        assert bits_equal(o[0], out[b]) and bits_equal(l[0], lse[b])
    assert bi.device_status() == bi.BI_OK


def test_caches_past_32_bit_offsets(dev):
    """K and V caches of more than 2^32 bytes each: a sequence in their last pages gives the bits
    it gives in small ones."""
    Hkv, D, L, pages = 8, 128, 300, 70000
    small = filled([L], Hkv, D, dev, seed=86)
    big = Cache.__new__(Cache)
    big.k, big.v = (torch.full((pages, Hkv, 64, D), POISON, dtype=torch.uint8, device=dev)
                    for _ in range(2))
    big.ks, big.vs = (torch.full((pages, Hkv, 64), 254, dtype=torch.uint8, device=dev)
                      for _ in range(2))
    big.table = i32([[pages - 1, pages - 3, pages - 2, 65536, pages - 4]], dev)
    big.append(small.k_rows.to(dev), small.v_rows.to(dev), [L], [L])
    q = rows((8, 32, D), 87).to(dev)
    want, wlse = attend(small, q, [L], [8], 0.1, "verify")
    for form in ("verify", "prefill"):
        o, l = attend(big, q, [L], [8], 0.1, form)
        assert bits_equal(o, want) and bits_equal(l, wlse)
    assert bi.device_status() == bi.BI_OK


def test_bounded_waits_run_out_and_leave_the_gpu_usable(dev):
    """With a wait budget far below the call's runtime the kernel's waits run out: the timeout is
    reported, and the next call with the default budget gives the right bits."""
    L = 16388
    c = filled([L], 8, 128, dev, seed=88)
    q = rows((8, 32, 128), 89).to(dev)
    want, _ = attend(c, q, [L], [8], 0.1, "verify")
    assert bi.device_status() == bi.BI_OK
    bi.selftest_set_wait_budget(1000)
    try:
        attend(c, q, [L], [8], 0.1, "verify")
        assert bi.device_status() == bi.BI_ERR_TIMEOUT
        attend(c, q, [L], [8], 0.1, "prefill")
        assert bi.device_status() in (bi.BI_OK, bi.BI_ERR_TIMEOUT)
    finally:
        bi.selftest_set_wait_budget(0)
    for form in ("verify", "prefill"):
        out, _ = attend(c, q, [L], [8], 0.1, form)
        assert bits_equal(out, want)
    assert bi.device_status() == bi.BI_OK


def test_empty_batch_and_zero_scale(dev):
    c = filled([70], 2, 64, dev, seed=82)
    q = torch.empty(0, 8, 64, dtype=torch.bfloat16, device=dev)
    none = torch.empty(0, 2, dtype=torch.int32, device=dev)
    o, l = bi.decode_attn_q8(q, *c.parts(), none, i32([], dev), max_seq_len=70, scale=1.0)
    assert o.shape == (0, 8, 64) and l.shape == (0, 8)
    q = rows((1, 8, 64), 83)
    out, lse = attend(c, q.to(dev), [70], [1], 0.0, "decode")
    r = ref.attention(q.double().numpy(), *c.values(), c.table[0].tolist(), 70, 1, 0.0, 4)
    ref.check_attention(out, lse, r, "scale 0")
    out, lse = attend(c, q.to(dev), [70], [1], -0.3, "decode")
    r = ref.attention(q.double().numpy(), *c.values(), c.table[0].tolist(), 70, 1, -0.3, 4)
    ref.check_attention(out, lse, r, "negative scale")


def test_captured_and_on_another_stream(dev):
    """A step (append, then attention) captured into a graph and replayed on new inputs and
    lengths, twice at once from two graphs on two streams, gives the eager bits."""
    Hq, Hkv, D, L = 8, 2, 128, 900
    steps = 4
    outs, eager = {}, {}
    jobs = []
    for n in range(2):
        c = filled([L + steps], Hkv, D, dev, seed=90 + n)
        k, v = rows((steps, Hkv, D), 91 + n, 1.0).to(dev), rows((steps, Hkv, D), 95 + n).to(dev)
        q = rows((steps, Hq, D), 99 + n).to(dev)
        st = dict(k=k[:1].clone(), v=v[:1].clone(), q=q[:1].clone(), sl=i32([L + 1], dev),
                  cu=i32([0, 1], dev))

        def step(c=c, st=st):
            bi.kv_append_q8(st["k"], st["v"], *c.parts(), c.table, st["sl"], st["cu"])
            return bi.decode_attn_q8(st["q"], *c.parts(), c.table, st["sl"],
                                     max_seq_len=L + steps, scale=0.1)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = step()
        jobs.append((c, k, v, q, st, step, s, g, out))
    for i in range(steps):
        for n, (c, k, v, q, st, step, s, g, out) in enumerate(jobs):
            with torch.cuda.stream(s):
                for name, src in (("k", k), ("v", v), ("q", q)):
                    st[name].copy_(src[i:i + 1])
                st["sl"].fill_(L + 1 + i)
                g.replay()
                outs[n, i] = [x.clone() for x in out]
    torch.cuda.synchronize()
    for n, (c, k, v, q, st, step, s, g, out) in enumerate(jobs):
        for i in range(steps):
            for name, src in (("k", k), ("v", v), ("q", q)):
                st[name].copy_(src[i:i + 1])
            st["sl"].fill_(L + 1 + i)
            want = step()
            for x, y in zip(outs[n, i], want):
                assert bits_equal(x, y), (n, i)
    # a stream given to the call: outputs and workspace are made for it
    c, k, v, q, st, step, s, g, out = jobs[0]
    torch.cuda.synchronize()
    want = step()
    torch.cuda.synchronize()
    for given in (s, s.cuda_stream):
        o, l = bi.decode_attn_q8(st["q"], *c.parts(), c.table, st["sl"], max_seq_len=L + steps,
                                 scale=0.1, stream=given)
        s.synchronize()
        assert bits_equal(o, want[0]) and bits_equal(l, want[1])
    assert bi.device_status() == bi.BI_OK


def test_repeats_are_identical(dev):
    c = filled([3000, 10], 8, 128, dev, seed=110)
    q = rows((12, 32, 128), 111).to(dev)
    seen = set()
    for _ in range(10):
        o, l = attend(c, q, [3000, 10], [8, 4], 0.1, "verify")
        seen.add(bytes(o.view(torch.int16).cpu().numpy()) + bytes(l.cpu().numpy()))
    assert len(seen) == 1


def test_refusals(dev):
    """Arguments that the binding turns away before anything is launched."""
    c = filled([70, 3], 2, 64, dev)
    k, v, ks, vs = c.parts()
    q = rows((2, 4, 64), 90).to(dev)
    good = dict(q=q, k_cache=k, v_cache=v, k_scale=ks, v_scale=vs, block_table=c.table,
                seq_lens=i32([70, 3], dev), max_seq_len=70, scale=0.125)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=dev)
    bi.decode_attn_q8(**good, workspace=ws)
    for bad in (dict(q=q.float()), dict(q=q[:1]), dict(q=q[:, :, :32]), dict(q=q.cpu()),
                dict(k_cache=k[:1]), dict(k_cache=k.float()), dict(k_scale=ks[:, :, :32]),
                dict(v_scale=vs.transpose(1, 2)), dict(v_cache=v.transpose(0, 1)),
                dict(block_table=c.table.long()), dict(block_table=c.table[:1]),
                dict(seq_lens=i32([70, 3, 1], dev)), dict(out=torch.empty_like(q).float()),
                dict(out=torch.empty(2, 4, 128, dtype=q.dtype, device=dev)[:, :, :64]),
                dict(lse=torch.empty(2, 3, device=dev)), dict(workspace=ws[::2]),
                dict(workspace=ws[:1].expand(1 << 20)), dict(workspace=ws[:64]),
                dict(max_seq_len=1 << 20), dict(scale=float("nan"))):
        with pytest.raises((ValueError, TypeError, bi.BIError)):
            bi.decode_attn_q8(**{**good, **bad})
    cu = i32([0, 1, 2], dev)
    new = rows((2, 2, 64), 91).to(dev)
    for bad in ((new.float(), new, cu), (new, new[:1], cu), (new[:, :1], new[:, :1], cu),
                (new, new, cu[:2]), (new, new, cu.long()), (new.cpu(), new, cu)):
        with pytest.raises((ValueError, TypeError, bi.BIError)):
            bi.kv_append_q8(bad[0], bad[1], k, v, ks, vs, c.table, i32([70, 3], dev), bad[2])
    src = i32([0], dev)
    for bad in (([k], src, src[:0]), ([k], src.long(), src.long()), ([k.cpu()], src, src),
                ([k, v[:1]], src, src), ([k.transpose(0, 1)], src, src)):
        with pytest.raises((ValueError, TypeError, bi.BIError)):
            bi.kv_copy_pages(*bad)
    assert bi.device_status() == 0
