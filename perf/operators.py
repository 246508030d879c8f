"""What is measured of the 8-bit paged KV cache, its attention, the page copies and the
token log-probabilities: the cases, their inputs, and each operator in a plain form.

Where ``own`` is false, ``run`` computes an operator from elementary torch operations in
fp32 (angles, long sums and ties in 64 bits or whole numbers); where it is true it makes
the calls a user of the library makes.  ``exact`` gives the same outputs from the
definitions in 64 bits, computed sequence by sequence.

Definitions
  append     each new token's K (and V) row x of D values and KV head is held as
             x ~ c * 2^e: e the smallest integer >= -64 with max|x| <= 448 * 2^e, stored as
             the byte e + 127, and c = e4m3(x * 2^-e), round to nearest even.
  attention  out[t, h] = softmax_i(scale * q[t, h] . k_i) v_i over the keys 0..pos(t) of the
             token's own sequence, k_i and v_i being the values the cache stands for;
             lse[t, h] the logarithm of the sum.
  copy       page dst[i] of every plane becomes a copy of page src[i].
  logprobs   logp = x[token] - lse, entropy = -sum p log p, and the largest entries of a row
             in descending order (ties: the lowest index first).
  gradient   dx = g_logp * (onehot - p) - g_entropy * p * (log p + entropy).
"""
import math

import torch

own = False

PAGE = 64
DEV = "cuda"


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # one new token for each of 32 sequences of a serving batch (latency of one launch)
        dict(name="append decode B32", op="append", B=32, q=1, L=1028, ragged=True, hkv=8, D=128),
        # a prompt's K and V written in one block of a chunked prefill
        dict(name="append prompt 8192", op="append", B=1, q=8192, L=8192, ragged=False, hkv=8,
             D=128),
        # a single short conversation, one token at a time
        dict(name="decode B1 L1028", op="attn", B=1, q=1, L=1028, ragged=False, hq=32, hkv=8,
             D=128),
        # a speculative block of 8 over one long context
        dict(name="verify B1 q8 L65540", op="attn", B=1, q=8, L=65540, ragged=False, hq=32,
             hkv=8, D=128),
        # a serving batch of long conversations of unlike lengths
        dict(name="decode B64 L16388", op="attn", B=64, q=1, L=16388, ragged=True, hq=32, hkv=8,
             D=128),
        # a small-headed model's ragged batch: prompts' next blocks of unlike widths
        dict(name="prefill B3 q600 D64", op="attn", B=3, q=600, L=1100, ragged=True, hq=8, hkv=2,
             D=64),
        # one sequence forked: its open page copied in the caches of eight layers
        dict(name="copy fork 1 page", op="copy", layers=8, pages=64, n=1, hkv=8, D=128, bits=16),
        # a pool compacted: many pages of the 8-bit caches moved at once
        dict(name="copy compact 1021", op="copy", layers=8, pages=2600, n=1021, hkv=8, D=128,
             bits=8),
        # the chosen tokens of a decode batch with the alternatives a client asks for
        dict(name="logprobs 32 top8", op="logprobs", rows=32, n=128256, top=8, type="fp32"),
        # a trainer scoring sampled sequences
        dict(name="logprobs 2048 bf16", op="logprobs", rows=2048, n=128256, top=0, type="bf16"),
        # the gradient of a small vocabulary's head, odd sizes
        dict(name="gradient 333", op="gradient", rows=333, n=1000, type="bf16"),
        # the gradient of a trainer's batch
        dict(name="gradient 2048 fp32", op="gradient", rows=2048, n=128256, type="fp32"),
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread evenly over its logarithm."""
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49))))))


def draw(rng):
    op = rng.choice(["append", "attn", "attn", "attn", "copy", "logprobs", "gradient"])
    if op == "append":
        B = _log(rng, 1, 64)
        q = _log(rng, 1, 8192 // B)
        return dict(op=op, B=B, q=q, L=q + rng.randint(0, 1500), ragged=rng.random() < 0.6,
                    hkv=rng.choice([1, 2, 3, 8]), D=rng.choice([64, 128]))
    if op == "attn":
        hq, hkv = rng.choice([(32, 8), (32, 8), (8, 8), (8, 2), (16, 2), (24, 8), (10, 2), (32, 1)])
        D = rng.choice([64, 128, 128])
        form = rng.choice(["decode", "decode", "verify", "prefill"])
        if form == "decode":
            L = _log(rng, 1, 65540)
            B = _log(rng, 1, max(1, min(64, 500000 // L)))
            return dict(op=op, B=B, q=1, L=L, ragged=rng.random() < 0.7, hq=hq, hkv=hkv, D=D)
        if form == "verify":
            L = _log(rng, 8, 65540)
            B = _log(rng, 1, max(1, min(32, 200000 // L)))
            q = rng.randint(1, max(1, min(8, 32 * hkv // hq)))
            return dict(op=op, B=B, q=q, L=L, ragged=rng.random() < 0.7, hq=hq, hkv=hkv, D=D)
        q = _log(rng, 9, 1500)
        return dict(op=op, B=rng.randint(1, 3), q=q, L=q + _log(rng, 1, 3000),
                    ragged=rng.random() < 0.7, hq=hq, hkv=hkv, D=D)
    if op == "copy":
        pages = _log(rng, 4, 2000)
        return dict(op=op, layers=rng.randint(1, 8), pages=pages, n=_log(rng, 1, pages // 2),
                    hkv=rng.choice([1, 2, 8]), D=rng.choice([64, 128]), bits=rng.choice([8, 16]))
    n = _log(rng, 17, 150000)
    rows = _log(rng, 1, max(1, min(3000, 200000000 // n)))
    if op == "logprobs":
        return dict(op=op, rows=rows, n=n, top=rng.choice([0, 0, 1, 5, 16]),
                    type=rng.choice(["fp32", "bf16", "fp16"]))
    return dict(op=op, rows=rows, n=n, type=rng.choice(["fp32", "bf16", "fp16"]))


# ------------------------------------------------------------------------------ inputs

TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def _lengths(case):
    """Lengths of the sequences and of their new blocks (the last ones of each): the case's
    own, the same for every seed, so that every state of a case has the same work."""
    B, q, L = case["B"], case["q"], case["L"]
    if not case["ragged"]:
        return [L] * B, [q] * B
    r = torch.rand(2, B, generator=torch.Generator().manual_seed(1)).tolist()
    qs = [max(1, min(q, round(q * (0.3 + 0.7 * v)))) for v in r[1]]
    qs[0] = q
    lens = [max(w, round(L * (0.3 + 0.7 * v))) for v, w in zip(r[0], qs)]
    lens[0] = L
    return lens, qs


def _paged(case, g, scratch_pages=1):
    """Block table (pages in random order, unused entries -1), lengths and offsets."""
    lens, qs = _lengths(case)
    need = [-(-n // PAGE) for n in lens]
    pages = sum(need) + scratch_pages
    perm = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    cu = torch.tensor([0] + qs).cumsum(0)
    tok_seq = torch.repeat_interleave(torch.arange(len(qs)), torch.tensor(qs))
    tok_j = torch.arange(int(cu[-1])) - cu[tok_seq]
    tok_pos = torch.tensor(lens)[tok_seq] - torch.tensor(qs)[tok_seq] + tok_j
    return dict(pages=pages, lens=lens, qs=qs, T=int(cu[-1]), max_q=max(qs), max_len=max(lens),
                table=table.to(DEV), seq_lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                cu_q=cu.to(torch.int32).to(DEV), tok_seq=tok_seq.to(DEV), tok_j=tok_j.to(DEV),
                tok_pos=tok_pos.to(DEV))


def _quantise(x):
    """e4m3 codes (as bytes) and scale bytes of rows of the last axis."""
    amax = x.float().abs().amax(-1)
    m, e = torch.frexp(amax)                    # amax = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax == 0, -64, e).clamp(min=-64)
    codes = torch.ldexp(x.float(), -e.unsqueeze(-1)).to(torch.float8_e4m3fn)
    return codes.view(torch.uint8), (e + 127).to(torch.uint8)


def _values(codes, scale):
    """What codes and scale bytes stand for, in fp32."""
    return torch.ldexp(codes.view(torch.float8_e4m3fn).float(), (scale.int() - 127).unsqueeze(-1))


def _rows(shape, gc):
    """K or V rows: normal, with the spread of sizes between tokens that real caches have."""
    x = torch.randn(shape, generator=gc, device=DEV)
    return x * torch.exp2(torch.randn(shape[:-1], generator=gc, device=DEV) * 0.7).unsqueeze(-1)


def prepare(case, seed):
    g = torch.Generator().manual_seed(seed)
    gc = torch.Generator(device=DEV).manual_seed(seed)
    s = dict(case)
    op = case["op"]
    if op in ("append", "attn"):
        s |= _paged(case, g)
        shape = (s["pages"], case["hkv"], PAGE, case["D"])
        if op == "append":
            for x in "kv":
                s[x + "_new"] = _rows((s["T"], case["hkv"], case["D"]), gc).to(torch.bfloat16)
                s[x + "_cache"], s[x + "_scale"] = _quantise(_rows(shape, gc))
        else:
            for x in "kv":
                s[x + "_cache"], s[x + "_scale"] = _quantise(_rows(shape, gc).to(torch.bfloat16))
            s["q"] = torch.randn(s["T"], case["hq"], case["D"], generator=gc, device=DEV).to(
                torch.bfloat16)
            s["scale"] = case["D"] ** -0.5
    elif op == "copy":
        shape = (2 * case["layers"], case["pages"], case["hkv"], PAGE)
        if case["bits"] == 16:
            s["planes"] = [torch.randn(shape + (case["D"],), generator=gc, device=DEV,
                                       dtype=torch.bfloat16)]
        else:
            s["planes"] = [torch.randint(0, 120, shape + (case["D"],), generator=gc, device=DEV,
                                         dtype=torch.uint8),
                           torch.randint(100, 150, shape, generator=gc, device=DEV,
                                         dtype=torch.uint8)]
        perm = torch.randperm(case["pages"], generator=g).to(torch.int32)
        s["src"], s["dst"] = perm[:case["n"]].to(DEV), perm[case["n"]:2 * case["n"]].to(DEV)
    else:
        rows, n = case["rows"], case["n"]
        x = torch.randn(rows, n, generator=gc, device=DEV) * 2.5
        s["logits"] = x.to(TYPES[case["type"]])
        s["tokens"] = torch.randint(0, n, (rows,), generator=gc, device=DEV, dtype=torch.int32)
        if op == "gradient":
            s["lse"], s["entropy"] = _lse_entropy(s["logits"].float())
            s["g_logp"] = torch.randn(rows, generator=gc, device=DEV)
            s["g_entropy"] = torch.randn(rows, generator=gc, device=DEV) * 0.1
    return s


# ----------------------------------------------------------------------- the plain forms

def _append(s):
    page = s["table"][s["tok_seq"], s["tok_pos"] // PAGE].long()
    slot = s["tok_pos"] % PAGE
    for x in "kv":
        codes, scale = _quantise(s[x + "_new"])
        s[x + "_cache"][page, :, slot] = codes
        s[x + "_scale"][page, :, slot] = scale
    return _caches(s)


def _caches(s):
    return dict(k=s["k_cache"].view(torch.float8_e4m3fn), v=s["v_cache"].view(torch.float8_e4m3fn),
                k_scale=s["k_scale"], v_scale=s["v_scale"])


def _attention(s):
    B, hq, hkv, D = s["B"], s["hq"], s["hkv"], s["D"]
    G, mq = hq // hkv, s["max_q"]
    table = s["table"].clamp(min=0).long()
    k, v = (_values(s[x + "_cache"][table], s[x + "_scale"][table])      # [B, P, hkv, 64, D]
            .transpose(1, 2).reshape(B, hkv, -1, D) for x in "kv")
    q = torch.zeros(B, mq, hq, D, device=DEV)
    q[s["tok_seq"], s["tok_j"]] = s["q"].float()
    pos = torch.full((B, mq), s["max_len"], device=DEV, dtype=torch.int64)
    pos[s["tok_seq"], s["tok_j"]] = s["tok_pos"]
    q = q.view(B, mq, hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, hkv, mq * G, D)
    x = q @ k.transpose(2, 3) * s["scale"]
    hidden = torch.arange(k.shape[2], device=DEV) > pos.repeat_interleave(G, 1).unsqueeze(-1)
    x = x.masked_fill_(hidden.unsqueeze(1), -math.inf)
    m = x.amax(-1, keepdim=True)
    p = torch.exp(x - m)
    total = p.sum(-1, keepdim=True)
    out = (p @ v / total).view(B, hkv, mq, G, D).permute(0, 2, 1, 3, 4).reshape(B, mq, hq, D)
    lse = (m + torch.log(total)).view(B, hkv, mq, G).permute(0, 2, 1, 3).reshape(B, mq, hq)
    at = s["tok_seq"], s["tok_j"]
    return dict(out=out[at].to(torch.bfloat16), lse=lse[at])


def _copy(s):
    src, dst = s["src"].long(), s["dst"].long()
    for p in s["planes"]:
        p[:, dst] = p[:, src]
    return _planes(s)


def _planes(s):
    p = s["planes"]
    return dict(cache=p[0] if s["bits"] == 16 else p[0].view(torch.float8_e4m3fn), scale=p[1:])


def _lse_entropy(x):
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(-1)
    return m[:, 0] + torch.log(total), torch.log(total) - (e * (x - m)).sum(-1) / total


def _logprobs(s):
    x = s["logits"].float()
    lse, entropy = _lse_entropy(x)
    r = dict(logp=x.gather(1, s["tokens"].long().unsqueeze(1))[:, 0] - lse, entropy=entropy)
    if s["top"]:
        # whole-number keys in the order (value descending, index ascending)
        b = (x + 0.0).view(torch.int32)
        b = (b ^ ((b >> 31) & 0x7fffffff)).long()
        key = (b << 32) + (0x7fffffff - torch.arange(s["n"], device=DEV))
        at = key.topk(min(s["top"], s["n"]), -1).indices
        r |= dict(top=x.gather(1, at) - lse.unsqueeze(1), ids=at.to(torch.int32))
    return r


def _gradient(s):
    logp = s["logits"].float() - s["lse"].unsqueeze(1)
    p = torch.exp(logp)
    d = -p * (s["g_logp"].unsqueeze(1) + s["g_entropy"].unsqueeze(1) * (logp + s["entropy"].unsqueeze(1)))
    d.scatter_add_(1, s["tokens"].long().unsqueeze(1), s["g_logp"].unsqueeze(1))
    return d.to(s["logits"].dtype)


# ------------------------------------------------------------------------------- a pass

def run(state):
    s = state
    op = s["op"]
    if not own:
        return {"append": _append, "attn": _attention, "copy": _copy, "logprobs": _logprobs,
                "gradient": _gradient}[op](s)
    import invariant_bi_matmul_gb300 as bi
    if op == "append":
        bi.kv_append_q8(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["k_scale"],
                        s["v_scale"], s["table"], s["seq_lens"], s["cu_q"])
        return _caches(s)
    if op == "attn":
        cache = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"], s["seq_lens"]
        if s["max_q"] == 1:
            out, lse = bi.decode_attn_q8(s["q"], *cache, max_seq_len=s["max_len"], scale=s["scale"])
        elif s["max_q"] <= bi.ATTN_MAX_Q:
            out, lse = bi.verify_block_q8(s["q"], *cache, s["cu_q"], max_q=s["max_q"],
                                          max_seq_len=s["max_len"], scale=s["scale"])
        else:
            out, lse = bi.prefill_attn_q8(s["q"], *cache, s["cu_q"], max_q=s["max_q"],
                                          max_seq_len=s["max_len"], scale=s["scale"])
        return dict(out=out, lse=lse)
    if op == "copy":
        bi.kv_copy_pages([x for p in s["planes"] for x in p.unbind(0)], s["src"], s["dst"])
        return _planes(s)
    if op == "logprobs":
        r = bi.token_logprobs(s["logits"], s["tokens"], top=min(s["top"], s["n"]))
        got = dict(logp=r.logprobs, entropy=r.entropy)
        return got | dict(top=r.top_logprobs, ids=r.top_ids) if s["top"] else got
    return bi.token_logprobs_backward(s["logits"], s["tokens"], s["lse"], s["entropy"],
                                      s["g_logp"], s["g_entropy"])


def work(case):
    op = case["op"]
    if op in ("append", "attn"):
        lens, qs = _lengths(case)
        T, D, hkv = sum(qs), case["D"], case["hkv"]
        if op == "append":
            return dict(bytes=T * hkv * 2 * (2 * D + D + 1), flops=T * hkv * 2 * D * 2)
        seen = sum(w * n - w * (w - 1) // 2 for n, w in zip(lens, qs))   # (query, key) pairs
        return dict(bytes=sum(lens) * hkv * 2 * (D + 1) + T * case["hq"] * (4 * D + 4),
                    flops=4 * seen * case["hq"] * D)
    if op == "copy":
        page = case["hkv"] * PAGE * (2 * case["D"] if case["bits"] == 16 else case["D"] + 1)
        return dict(bytes=2 * 2 * case["layers"] * case["n"] * page, flops=0)
    size = torch.finfo(TYPES[case["type"]]).bits // 8
    values = case["rows"] * case["n"]
    if op == "logprobs":
        return dict(bytes=values * size + case["rows"] * (12 + 8 * case["top"]), flops=5 * values)
    return dict(bytes=2 * values * size + case["rows"] * 20, flops=6 * values)


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
    op = case["op"]
    if op == "append":
        r = dict(k=s["k_cache"].view(torch.float8_e4m3fn).double(),
                 v=s["v_cache"].view(torch.float8_e4m3fn).double(),
                 k_scale=s["k_scale"], v_scale=s["v_scale"])
        for x in "kv":
            y, e = _exact_codes(s[x + "_new"])
            t = 0
            for b, (n, w) in enumerate(zip(s["lens"], s["qs"])):
                at = torch.arange(n - w, n, device=DEV)
                page = s["table"][b].long()[at // PAGE]
                r[x][page, :, at % PAGE] = y[t:t + w]
                r[x + "_scale"][page, :, at % PAGE] = e[t:t + w]
                t += w
        return r
    if op == "attn":
        out = torch.empty(s["T"], case["hq"], case["D"], dtype=torch.float64, device=DEV)
        lse = torch.empty(s["T"], case["hq"], dtype=torch.float64, device=DEV)
        G, t = case["hq"] // case["hkv"], 0
        for b, (n, w) in enumerate(zip(s["lens"], s["qs"])):
            page = s["table"][b, :-(-n // PAGE)].long()
            seen = torch.arange(n, device=DEV) <= torch.arange(n - w, n, device=DEV).unsqueeze(1)
            for h in range(case["hkv"]):
                k, v = ((s[x + "_cache"][page, h].view(torch.float8_e4m3fn).double()
                         * torch.exp2(s[x + "_scale"][page, h].double() - 127).unsqueeze(-1)
                         ).reshape(-1, case["D"])[:n] for x in "kv")
                for i in range(h * G, h * G + G):
                    x = s["q"][t:t + w, i].double() @ k.T * s["scale"]
                    x = torch.where(seen, x, torch.full_like(x, -math.inf))
                    lse[t:t + w, i] = torch.logsumexp(x, -1)
                    out[t:t + w, i] = torch.exp(x - lse[t:t + w, i].unsqueeze(1)) @ v
            t += w
        return dict(out=out, lse=lse)
    if op == "copy":
        return None        # no value is computed
    x = s["logits"].double()
    logp = torch.log_softmax(x, -1)
    at = s["tokens"].long()
    every = torch.arange(case["rows"], device=DEV)
    entropy = -(torch.exp(logp) * logp).sum(-1)
    if op == "logprobs":
        r = dict(logp=logp[every, at], entropy=entropy)
        if case["top"]:
            r |= dict(top=torch.sort(logp, -1, descending=True).values[:, :case["top"]], ids=None)
        return r
    p = torch.exp(logp)
    onehot = torch.zeros_like(p)
    onehot[every, at] = 1
    return (s["g_logp"].double().unsqueeze(1) * (onehot - p)
            - s["g_entropy"].double().unsqueeze(1) * p * (logp + entropy.unsqueeze(1)))
