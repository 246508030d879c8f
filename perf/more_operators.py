"""What is measured of the rotating cache append, the attention with shaped scores and the
verification of drafted tokens: the cases, their inputs, and each operator in a plain form.

Where ``own`` is false, ``run`` computes an operator from elementary torch operations in
fp32 (angles, probabilities and their sums in 64 bits); where it is true it makes the calls a
user of the library makes.  ``exact`` gives the same outputs from the definitions in 64 bits,
computed sequence by sequence.

Definitions
  append     pair i of a head joins elements i and i + D/2 and turns by the angle
             pos * theta^(-2i/D): every query and new key row is turned, and the keys and
             the values are written to their slots of the paged cache.  pos is the token's
             place in its sequence, or, with several axes, the position on the axis whose
             section holds pair i.  The turned rows are bf16; an 8-bit cache holds
             x ~ c * 2^e of each key and value row: e the smallest integer >= -64 with
             max|x| <= 448 * 2^e, stored as the byte e + 127, and c = e4m3(x * 2^-e).
  attention  x = scale * q[t, h] . k_j;  x := softcap * tanh(x / softcap) with a softcap;
             x := x + slope[h] * (j - pos(t)) with slopes;  out[t, h] = softmax_j(x) v_j over
             the keys max(first[t], pos(t) - window + 1, 0) <= j <= pos(t) of the token's own
             sequence (zeros where there is none), lse[t, h] the logarithm of the sum.
  verify     p = softmax(logits / temperature), one row per token of a block (its last input
             and the drafted tokens); q likewise from the draft's logits, or 1 at the drafted
             token.  Draft j is accepted while u_j q_j(x_j) < p_j(x_j); the first that is not
             is replaced by the first token whose cumulative sum of max(p - q, 0) exceeds the
             last uniform number's share of the whole, and after a block that is accepted in
             full one more token is drawn from p in the same way.  Temperature 0 accepts and
             draws the largest entry.  tokens and their log p (at temperature 1 where it is 0).
"""
import math

import torch

own = False

PAGE = 64
DEV = "cuda"
THETA = 500000.0
TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token for each of 32 sequences of a serving batch (latency of one launch)
        dict(name="append decode B32", op="append", B=32, q=1, L=1028, ragged=True, hq=32, hkv=8,
             D=128, bits=16, axes=1),
        # a prompt's block of a chunked prefill, far into a long 8-bit cache
        dict(name="append prompt 8192 q8", op="append", B=1, q=8192, L=65540, ragged=False, hq=32,
             hkv=8, D=128, bits=8, axes=1),
        # prompts with pictures: positions of time, height and width, a small-headed model
        dict(name="append axes B3 q600", op="append", B=3, q=600, L=1100, ragged=True, hq=8,
             hkv=2, D=64, bits=16, axes=3),
        # a serving batch of long conversations, a model that looks back 4,096 keys
        dict(name="decode window B64", op="attn", B=64, q=1, L=16388, ragged=True, hq=32, hkv=8,
             D=128, softcap=0.0, slopes=False, window=4096, documents=0),
        # a speculative block of 8 over one long context, capped scores
        dict(name="verify cap B1 q8 L65540", op="attn", B=1, q=8, L=65540, ragged=False, hq=32,
             hkv=8, D=128, softcap=30.0, slopes=False, window=0, documents=0),
        # short conversations with a bias that grows with distance, as many KV as query heads
        dict(name="decode bias B8 L2048", op="attn", B=8, q=1, L=2048, ragged=True, hq=32, hkv=32,
             D=128, softcap=0.0, slopes=True, window=0, documents=0),
        # a prompt in one block, capped scores
        dict(name="prefill cap 8192", op="attn", B=1, q=8192, L=8192, ragged=False, hq=32, hkv=8,
             D=128, softcap=50.0, slopes=False, window=0, documents=0),
        # packed documents that do not see one another, a small-headed model
        dict(name="prefill documents B3 D64", op="attn", B=3, q=600, L=1100, ragged=True, hq=8,
             hkv=2, D=64, softcap=0.0, slopes=False, window=0, documents=150),
        # one conversation's drafts, looked up in its own text
        dict(name="verify drafts B1 w4", op="verify", B=1, q=4, n=128256, type="fp32",
             draft="tokens", ragged=False, greedy=0.0),
        # a serving batch with a draft model, some clients at temperature 0
        dict(name="verify drafts B32 w5", op="verify", B=32, q=5, n=128256, type="fp32",
             draft="logits", ragged=True, greedy=0.25),
        # a large batch, 16-bit logits
        dict(name="verify drafts B128 w8 bf16", op="verify", B=128, q=8, n=128256, type="bf16",
             draft="logits", ragged=False, greedy=0.0),
        # a small vocabulary, odd sizes
        dict(name="verify drafts B7 n999", op="verify", B=7, q=6, n=999, type="fp16",
             draft="logits", ragged=True, greedy=0.2),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "verify", "verify"])
    if op == "append":
        B = _log(rng, 1, 64)
        q = _log(rng, 1, 8192 // B)
        hq, hkv = rng.choice([(32, 8), (8, 8), (8, 2), (24, 8), (10, 2), (3, 1)])
        return dict(op=op, B=B, q=q, L=q + rng.randint(0, 3000), ragged=rng.random() < 0.6,
                    hq=hq, hkv=hkv, D=rng.choice([64, 128]), bits=rng.choice([8, 16]),
                    axes=rng.choice([1, 1, 2, 3]))
    if op == "attn":
        hq, hkv = rng.choice([(32, 8), (32, 8), (8, 8), (8, 2), (16, 2), (32, 1)])
        shape = dict(op=op, hq=hq, hkv=hkv, D=rng.choice([64, 128, 128]), ragged=rng.random() < 0.7,
                     softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), slopes=rng.random() < 0.3,
                     window=rng.choice([0, 1, 2]), documents=rng.choice([0, 0, 100, 2000]))
        form = rng.choice(["decode", "decode", "verify", "prefill"])
        if form == "decode":
            L = _log(rng, 1, 65540)
            B, q = _log(rng, 1, max(1, min(64, 500000 // L))), 1
        elif form == "verify":
            L = _log(rng, 8, 65540)
            B = _log(rng, 1, max(1, min(32, 200000 // L)))
            q = rng.randint(1, max(1, min(8, 32 * hkv // hq)))
        else:
            B, q = rng.randint(1, 3), _log(rng, 9, 1500)
            L = q + _log(rng, 1, 3000)
        window = _log(rng, 1, L) if shape["window"] else 0
        return shape | dict(B=B, q=q, L=L, window=window)
    n = _log(rng, 17, 150000)
    q = rng.randint(1, 8)
    B = _log(rng, 1, max(1, min(128, 100000000 // (n * q))))
    return dict(op=op, B=B, q=q, n=n, type=rng.choice(["fp32", "bf16", "fp16"]),
                draft=rng.choice(["tokens", "logits"]), ragged=rng.random() < 0.6,
                greedy=rng.choice([0.0, 0.0, 0.3]))


# ------------------------------------------------------------------------------ inputs

def _lengths(case):
    """Lengths of the sequences and of their new blocks (the last ones of each): the case's
    own, the same for every seed, so that every state of a case has the same work."""
    B, q, L = case["B"], case["q"], case.get("L", case["q"])
    if not case["ragged"]:
        return [L] * B, [q] * B
    r = torch.rand(2, B, generator=torch.Generator().manual_seed(1)).tolist()
    qs = [max(1, min(q, round(q * (0.3 + 0.7 * v)))) for v in r[1]]
    qs[0] = q
    lens = [max(w, round(L * (0.3 + 0.7 * v))) for v, w in zip(r[0], qs)]
    lens[0] = L
    return lens, qs


def _block(case):
    """Offsets of the new blocks, and each token's sequence, place in its block and position."""
    lens, qs = _lengths(case)
    cu = torch.tensor([0] + qs).cumsum(0)
    tok_seq = torch.repeat_interleave(torch.arange(len(qs)), torch.tensor(qs))
    tok_j = torch.arange(int(cu[-1])) - cu[tok_seq]
    tok_pos = torch.tensor(lens)[tok_seq] - torch.tensor(qs)[tok_seq] + tok_j
    return dict(lens=lens, qs=qs, T=int(cu[-1]), max_q=max(qs), max_len=max(lens),
                cu_q=cu.to(torch.int32).to(DEV), tok_seq=tok_seq.to(DEV), tok_j=tok_j.to(DEV),
                tok_pos=tok_pos.to(DEV))


def _paged(case, g):
    """Block table: pages in random order, unused entries -1."""
    lens, _ = _lengths(case)
    need = [-(-n // PAGE) for n in lens]
    pages = sum(need) + 1
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return dict(pages=pages, table=table.to(DEV),
                seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV))


def _quantise(x):
    """e4m3 codes (as bytes) and scale bytes of rows of the last axis."""
    amax = x.float().abs().amax(-1)
    m, e = torch.frexp(amax)                    # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax == 0, -64, e).clamp(min=-64)
    codes = torch.ldexp(x.float(), -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _rows(shape, gc):
    """K or V rows: normal, with the spread of sizes between tokens that real caches have."""
    x = torch.randn(shape, generator=gc, device=DEV)
    return x * torch.exp2(torch.randn(shape[:-1], generator=gc, device=DEV) * 0.7).unsqueeze(-1)


def _sections(case):
    """How many pairs each axis turns: two equal shares and the rest for the first axis."""
    half, axes = case["D"] // 2, case["axes"]
    rest = 3 * half // 8 // max(1, axes - 1)
    return [half - (axes - 1) * rest] + [rest] * (axes - 1)


def _first_keys(s, case, g):
    """Where each token's document starts; tokens of padding see nothing."""
    first = torch.zeros(s["T"], dtype=torch.int64)
    pos, seq = s["tok_pos"].cpu(), s["tok_seq"].cpu()
    for b, n in enumerate(s["lens"]):
        cuts = torch.randint(0, n, (n // case["documents"] + 1,), generator=g).sort().values
        cuts = torch.cat([torch.zeros(1, dtype=torch.int64), cuts])
        mine = (seq == b).nonzero()[:, 0]
        first[mine] = cuts[torch.searchsorted(cuts, pos[mine], right=True) - 1]
    none = torch.rand(s["T"], generator=g) < 0.02
    return torch.where(none, pos + 1, first).to(torch.int32).to(DEV)


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gc = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case) | _block(case)
    op = case["op"]
    bf16 = torch.bfloat16
    if op == "verify":
        return s | _drafts(s, case, g, gc)
    s |= _paged(case, g)
    shape = (s["pages"], case["hkv"], PAGE, case["D"])
    T, hq, hkv, D = s["T"], case["hq"], case["hkv"], case["D"]
    if op == "attn":
        for x in "kv":
            s[x + "_cache"] = _rows(shape, gc).to(bf16)
        size = 4.0 if case["softcap"] else 1.0
        s["q"] = (torch.randn(T, hq, D, generator=gc, device=DEV) * size).to(bf16)
        s["scale"] = D ** -0.5
        s["first"] = _first_keys(s, case, g) if case["documents"] else None
        s["slope"] = (torch.exp2(-8.0 * torch.arange(1, hq + 1, device=DEV) / hq)
                      if case["slopes"] else None)
        return s
    # one projection's output: a token's query, key and value rows beside one another
    qkv = _rows((T, hq + 2 * hkv, D), gc).to(bf16)
    s["q"], s["k_new"], s["v_new"] = qkv.split([hq, hkv, hkv], 1)
    for x in "kv":
        if case["bits"] == 8:
            s[x + "_cache"], s[x + "_scale"] = _quantise(_rows(shape, gc))
        else:
            s[x + "_cache"] = _rows(shape, gc).to(bf16)
    s["sections"], s["positions"] = None, None
    if case["axes"] > 1:
        # text advances on all axes at once; pictures of 16 x 12 patches in between
        s["sections"] = _sections(case)
        i = s["tok_pos"] % 192
        picture = (s["tok_pos"] // 192 + s["tok_seq"]) % 2 == 1
        at = torch.stack([s["tok_pos"] - i, s["tok_pos"] - i + i // 16, s["tok_pos"] - i + i % 16])
        s["positions"] = torch.where(picture, at, s["tok_pos"])[:case["axes"]].to(torch.int32)
    return s


def _drafts(s, case, g, gc):
    """Logits, and drafts that a fair share of them would have chosen."""
    T, B, n = s["T"], case["B"], case["n"]
    rand = lambda *shape: torch.rand(shape, generator=gc, device=DEV)  # noqa: E731
    temperature = torch.rand(B, generator=g) * 0.8 + 0.4
    temperature[torch.rand(B, generator=g) < case["greedy"]] = 0.0
    logits = (torch.randn(T, n, generator=gc, device=DEV) * 2.5).to(TYPES[case["type"]])
    drafted = s["tok_j"] > 0                    # row t - 1 is the one that drafted token t
    near = logits[:-1][drafted[1:]].float()
    near = (near + torch.randn(near.shape, generator=gc, device=DEV) * 0.6).to(logits.dtype)
    hot = temperature.to(DEV)[s["tok_seq"][drafted]].unsqueeze(1)
    noise = torch.where(hot > 0, -torch.log(-torch.log(rand(*near.shape).clamp(1e-30, 1 - 1e-7))), 0)
    if case["draft"] == "tokens":
        noise = torch.where(rand(near.shape[0], 1) < 0.8, 0, noise)
    tokens = (near.float() / torch.where(hot > 0, hot, 1) + noise).argmax(-1).to(torch.int32)
    return dict(logits=logits, draft_tokens=tokens, uniforms=rand(T), temperature=temperature.to(DEV),
                draft_logits=near if case["draft"] == "logits" else None)


# ----------------------------------------------------------------------- the plain forms

def _append(s):
    D, half = s["D"], s["D"] // 2
    freq = THETA ** (-2.0 * torch.arange(half, device=DEV, dtype=torch.float64) / D)
    pos = s["tok_pos"].unsqueeze(1)
    if s["positions"] is not None:
        axis = torch.repeat_interleave(torch.arange(s["axes"], device=DEV),
                                       torch.tensor(s["sections"], device=DEV))
        pos = s["positions"][axis].T
    angle = (pos.double() * freq).unsqueeze(1)
    c, sn = torch.cos(angle).float(), torch.sin(angle).float()

    def turn(x):
        lo, hi = x[..., :half].float(), x[..., half:].float()
        return torch.cat([lo * c - hi * sn, hi * c + lo * sn], -1).to(torch.bfloat16)

    page = s["table"][s["tok_seq"], s["tok_pos"] // PAGE].long()
    slot = s["tok_pos"] % PAGE
    for x, rows in (("k", turn(s["k_new"])), ("v", s["v_new"])):
        if s["bits"] == 8:
            s[x + "_cache"][page, :, slot], s[x + "_scale"][page, :, slot] = _quantise(rows)
        else:
            s[x + "_cache"][page, :, slot] = rows
    return dict(q=turn(s["q"])) | _caches(s)


def _caches(s):
    if s["bits"] == 16:
        return dict(k=s["k_cache"], v=s["v_cache"])
    return dict(k=s["k_cache"].view(torch.float8_e4m3fn), v=s["v_cache"].view(torch.float8_e4m3fn),
                k_scale=s["k_scale"], v_scale=s["v_scale"])


def _attention(s):
    B, hq, hkv, D = s["B"], s["hq"], s["hkv"], s["D"]
    G, mq = hq // hkv, s["max_q"]
    table = s["table"].clamp(min=0).long()
    k, v = (s[x + "_cache"][table].float()                               # [B, P, hkv, 64, D]
            .transpose(1, 2).reshape(B, hkv, -1, D) for x in "kv")
    at = s["tok_seq"], s["tok_j"]
    q = torch.zeros(B, mq, hq, D, device=DEV)
    q[at] = s["q"].float()
    pos = torch.full((B, mq), s["max_len"], device=DEV, dtype=torch.int64)
    pos[at] = s["tok_pos"]
    first = torch.zeros_like(pos)
    if s["first"] is not None:
        first[at] = s["first"].long()
    if s["window"]:
        first = torch.maximum(first, pos - s["window"] + 1)
    first, pos = (x.repeat_interleave(G, 1).unsqueeze(-1) for x in (first, pos))
    q = q.view(B, mq, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, mq * G, D)
    x = q @ k.transpose(2, 3) * s["scale"]
    if s["softcap"]:
        x = s["softcap"] * torch.tanh(x / s["softcap"])
    j = torch.arange(k.shape[2], device=DEV)
    if s["slope"] is not None:
        slope = s["slope"].view(1, hkv, 1, G).expand(1, hkv, mq, G).reshape(1, hkv, mq * G, 1)
        x = x + slope * (j - pos).float().unsqueeze(1)
    hidden = (j > pos) | (j < first)
    x = x.masked_fill_(hidden.unsqueeze(1), -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m.clamp(min=-1e30))
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, p @ v / total, 0)
    out = out.view(B, hkv, mq, G, D).permute(0, 2, 1, 3, 4).reshape(B, mq, hq, D)
    lse = (m + torch.log(total)).view(B, hkv, mq, G).permute(0, 2, 1, 3).reshape(B, mq, hq)
    return dict(out=out[at].to(torch.bfloat16), lse=lse[at])


def _verify(s):
    B, T, W, n = s["B"], s["T"], s["max_q"], s["n"]
    hot = s["temperature"].double()
    greedy = hot == 0
    hot = torch.where(greedy, 1.0, hot)[s["tok_seq"]]
    x = s["logits"].double() / hot.unsqueeze(1)
    best = x.argmax(-1)
    x -= x.amax(-1, keepdim=True)
    p = torch.exp(x)
    total = p.sum(-1, keepdim=True)
    p /= total
    drafted = s["tok_j"] > 0
    row = drafted.nonzero()[:, 0] - 1                   # the row that decides each draft
    token = s["draft_tokens"].long()
    px = p[row, token]
    if s["draft_logits"] is None:
        qx = torch.ones_like(px)
    else:
        y = s["draft_logits"].double() / hot[row].unsqueeze(1)
        q = torch.exp(y - y.amax(-1, keepdim=True))
        q /= q.sum(-1, keepdim=True)
        qx = q.gather(1, token.unsqueeze(1))[:, 0]
    seq = s["tok_seq"][row]
    good = torch.where(greedy[seq], best[row] == token, s["uniforms"][row].double() * qx < px)
    kept = torch.zeros(B, W, device=DEV, dtype=torch.bool)
    kept[seq, s["tok_j"][row]] = good
    accepted = kept.long().cumprod(1).sum(1)
    # the row that gives each sequence's last token, and the draft refused there
    cu = s["cu_q"].long()
    last = cu[:-1] + accepted
    refused = accepted < cu[1:] - cu[:-1] - 1
    d = p[last]
    if row.numel():
        at = (last - torch.arange(B, device=DEV)).clamp(max=row.numel() - 1)
        if s["draft_logits"] is None:
            less = torch.zeros_like(d).scatter_(1, token[at].unsqueeze(1), 2.0)
        else:
            less = q[at]
        rest = (d - less).clamp(min=0)
        d = torch.where((refused & (rest.sum(-1) > 0)).unsqueeze(1), rest, d)
    cum = d.cumsum(-1)
    share = s["uniforms"][cu[1:] - 1].double() * cum[:, -1]
    drawn = (cum <= share.unsqueeze(1)).sum(-1)
    final = torch.where(greedy, best[last], drawn)
    # drafts accepted, then the drawn token, -1 behind it
    j = torch.arange(W, device=DEV)
    tokens = torch.full((B, W), -1, device=DEV, dtype=torch.int64)
    tokens[seq, s["tok_j"][row]] = token
    tokens = torch.where(j < accepted.unsqueeze(1), tokens, -1)
    tokens.scatter_(1, accepted.unsqueeze(1), final.unsqueeze(1))
    rows = (cu[:-1].unsqueeze(1) + j).clamp(max=T - 1)
    logp = x[rows, tokens.clamp(min=0)] - torch.log(total[rows, 0])
    return dict(tokens=tokens.to(torch.int32), accepted=accepted.to(torch.int32),
                logprobs=torch.where(tokens >= 0, logp, 0).float())


# ------------------------------------------------------------------------------- a pass

def run(state):
    s = state
    op = s["op"]
    if not own:
        return {"append": _append, "attn": _attention, "verify": _verify}[op](s)
    import invariant_bi_matmul_gb300 as bi
    if op == "append":
        cache = s["k_cache"], s["v_cache"]
        rest = dict(theta=THETA, positions=s["positions"], sections=s["sections"])
        if s["bits"] == 8:
            q = bi.rope_kv_append_q8(s["q"], s["k_new"], s["v_new"], *cache, s["k_scale"],
                                     s["v_scale"], s["table"], s["seq_lens"], s["cu_q"], **rest)
        else:
            q = bi.rope_kv_append(s["q"], s["k_new"], s["v_new"], *cache, s["table"],
                                  s["seq_lens"], s["cu_q"], **rest)
        return dict(q=q) | _caches(s)
    if op == "attn":
        cache = s["k_cache"], s["v_cache"], s["table"], s["seq_lens"]
        rest = dict(max_seq_len=s["max_len"], scale=s["scale"], softcap=s["softcap"],
                    slopes=s["slope"], window=s["window"], first_key=s["first"])
        if s["max_q"] == 1:
            out, lse = bi.decode_attn(s["q"], *cache, **rest)
        elif s["max_q"] <= bi.ATTN_MAX_Q:
            out, lse = bi.verify_block(s["q"], *cache, s["cu_q"], max_q=s["max_q"], **rest)
        else:
            out, lse = bi.prefill_attn(s["q"], *cache, s["cu_q"], max_q=s["max_q"], **rest)
        return dict(out=out, lse=lse)
    r = bi.verify_drafts(s["logits"], s["draft_tokens"], s["uniforms"], s["cu_q"],
                         max_q=s["max_q"], draft_logits=s["draft_logits"],
                         temperature=s["temperature"])
    return dict(tokens=r.tokens, accepted=r.accepted, logprobs=r.logprobs)


def _seen(case):
    """(query, key) pairs that are visible, and keys read, without the documents' masks (which
    are drawn with the inputs)."""
    lens, qs = _lengths(case)
    w = case["window"] or max(lens)
    pairs = keys = 0
    for n, c in zip(lens, qs):
        pairs += sum(min(w, p + 1) for p in range(n - c, n))
        keys += n - max(0, n - c - w + 1)
    if case["documents"]:
        pairs = min(pairs, sum(qs) * case["documents"])
        keys = min(keys, sum(min(n, c + case["documents"]) for n, c in zip(lens, qs)))
    return pairs, keys


def work(case):
    op = case["op"]
    lens, qs = _lengths(case)
    T = sum(qs)
    if op == "append":
        size = 2 if case["bits"] == 16 else 1 + 1 / case["D"]
        return dict(bytes=T * case["D"] * (4 * case["hq"] + 2 * case["hkv"] * (2 + size)),
                    flops=T * case["D"] * 3 * (case["hq"] + case["hkv"]))
    if op == "attn":
        pairs, keys = _seen(case)
        return dict(bytes=keys * case["hkv"] * 4 * case["D"] + T * case["hq"] * (4 * case["D"] + 4),
                    flops=4 * pairs * case["hq"] * case["D"])
    rows = T + (T - case["B"] if case["draft"] == "logits" else 0)
    size = torch.finfo(TYPES[case["type"]]).bits // 8
    return dict(bytes=rows * case["n"] * size + T * 16, flops=4 * rows * case["n"])


# ----------------------------------------------------------------------- in 64 bits

def _exact_codes(x):
    """The e4m3 values and scale bytes of rows, from the definition."""
    x = x.double()
    amax = x.abs().amax(-1, keepdim=True)
    e = torch.full_like(amax, -64)
    for _ in range(200):
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, e)
    y = x * torch.exp2(-e)
    size = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -60))).clamp(min=-6)
    size = torch.where(torch.exp2(size) > y.abs().clamp(min=2.0 ** -6), size - 1, size)
    size = torch.where(torch.exp2(size + 1) <= y.abs(), size + 1, size)
    step = torch.exp2(size - 3)
    return torch.round(y / step) * step, (e[..., 0] + 127).to(torch.uint8)


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _exact_append, "attn": _exact_attention, "verify": _exact_verify}[case["op"]](
        s, case)


def _exact_append(s, case):
    D = case["D"]
    q8 = case["bits"] == 8
    r = dict(q=torch.empty(s["q"].shape, dtype=torch.float64, device=DEV))
    for x in "kv":
        r[x] = (s[x + "_cache"].view(torch.float8_e4m3fn) if q8 else s[x + "_cache"]).double()
        if q8:
            r[x + "_scale"] = s[x + "_scale"].clone()
    t = 0
    for b, (n, w) in enumerate(zip(s["lens"], s["qs"])):
        place = torch.arange(n - w, n, device=DEV)
        page, slot = s["table"][b].long()[place // PAGE], place % PAGE
        turned = {x: s[y][t:t + w].double() for x, y in (("q", "q"), ("k", "k_new"))}
        for y in turned.values():
            i0 = 0
            for axis, count in enumerate(s["sections"] or [D // 2]):
                at = place if s["positions"] is None else s["positions"][axis, t:t + w]
                for i in range(i0, i0 + count):
                    a = (at.double() / math.pow(THETA, 2 * i / D)).unsqueeze(1)
                    lo, hi = y[..., i].clone(), y[..., i + D // 2].clone()
                    y[..., i] = lo * torch.cos(a) - hi * torch.sin(a)
                    y[..., i + D // 2] = hi * torch.cos(a) + lo * torch.sin(a)
                i0 += count
        r["q"][t:t + w] = turned["q"]
        for x, rows in (("k", turned["k"]), ("v", s["v_new"][t:t + w].double())):
            if q8:
                r[x][page, :, slot], r[x + "_scale"][page, :, slot] = _exact_codes(
                    rows.to(torch.bfloat16))
            else:
                r[x][page, :, slot] = rows
        t += w
    return r


def _exact_attention(s, case):
    out = torch.zeros(s["T"], case["hq"], case["D"], dtype=torch.float64, device=DEV)
    lse = torch.empty(s["T"], case["hq"], dtype=torch.float64, device=DEV)
    G, t = case["hq"] // case["hkv"], 0
    for b, (n, w) in enumerate(zip(s["lens"], s["qs"])):
        page = s["table"][b, :-(-n // PAGE)].long()
        j = torch.arange(n, device=DEV)
        pos = torch.arange(n - w, n, device=DEV).unsqueeze(1)
        seen = j <= pos
        if s["first"] is not None:
            seen &= j >= s["first"][t:t + w].unsqueeze(1)
        if case["window"]:
            seen &= pos - j < case["window"]
        for h in range(case["hkv"]):
            k, v = (s[x + "_cache"][page, h].double().reshape(-1, case["D"])[:n] for x in "kv")
            for i in range(h * G, h * G + G):
                x = s["q"][t:t + w, i].double() @ k.T * s["scale"]
                if case["softcap"]:
                    x = torch.tanh(x / case["softcap"]) * case["softcap"]
                if s["slope"] is not None:
                    x = x - s["slope"][i].double() * (pos - j)
                x = torch.where(seen, x, torch.full_like(x, -math.inf))
                sums = torch.logsumexp(x, -1)
                lse[t:t + w, i] = sums
                p = torch.where(seen, torch.exp(x - sums.unsqueeze(1)), torch.zeros_like(x))
                out[t:t + w, i] = p @ v
        t += w
    return dict(out=out, lse=lse)


def _exact_verify(s, case):
    B, W = case["B"], s["max_q"]
    tokens = torch.full((B, W), -1, dtype=torch.int32)
    accepted = torch.zeros(B, dtype=torch.int32)
    logprobs = torch.zeros(B, W, dtype=torch.float64)
    u, drafts, hots = (s[x].tolist() for x in ("uniforms", "draft_tokens", "temperature"))
    t = d = 0
    for b, w in enumerate(s["qs"]):
        hot = hots[b]
        for j in range(w):
            row = s["logits"][t + j].double() / (hot or 1.0)
            logp = torch.log_softmax(row, -1)
            if j < w - 1:
                x = drafts[d + j]
                if hot == 0:
                    take = int(row.argmax()) == x
                elif s["draft_logits"] is None:
                    take, q = u[t + j] < float(logp[x].exp()), None
                else:
                    q = torch.softmax(s["draft_logits"][d + j].double() / hot, -1)
                    take = u[t + j] * float(q[x]) < float(logp[x].exp())
                if take:
                    tokens[b, j], logprobs[b, j] = x, logp[x]
                    continue
            p = logp.exp()
            if hot == 0:
                y = int(row.argmax())
            else:
                if j < w - 1:
                    if q is None:
                        p[x] = 0
                    else:
                        p = (p - q).clamp(min=0)
                sums = torch.cumsum(p, 0)
                y = int(torch.searchsorted(sums, sums[-1] * u[t + w - 1], right=True))
            tokens[b, j], logprobs[b, j], accepted[b] = y, logp[y], j
            break
        t += w
        d += w - 1
    return dict(tokens=tokens, accepted=accepted, logprobs=logprobs)
