"""Refusals of the 8-bit cache, page-copy and token-logprob entry points, without a GPU: bad
arguments are returned before anything is launched or read."""
import ctypes

import pytest
import torch

import invariant_bi_matmul_gb300 as bi

P = 1 << 20  # a fake, 16-byte aligned address: nothing may touch it
INVALID, UNSUPPORTED, OK = bi.BI_ERR_INVALID_ARG, bi.BI_ERR_UNSUPPORTED, bi.BI_OK


@pytest.fixture(scope="module")
def L():
    return bi.lib()


def append(L, **kw):
    a = dict(kn=P, vn=P, k=P, v=P, ks=P, vs=P, pages=4, bt=P, max_pages=4, sl=P, cu=P, batch=1,
             total=2, hkv=8, D=128, page=64)
    a.update(kw)
    return L.bi_kv_append_q8(a["kn"], a["vn"], a["k"], a["v"], a["ks"], a["vs"], a["pages"],
                             a["bt"], a["max_pages"], a["sl"], a["cu"], a["batch"], a["total"],
                             a["hkv"], a["D"], a["page"], None)


@pytest.mark.parametrize("change,want", [
    (dict(batch=-1), INVALID), (dict(total=-1), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(page=32), UNSUPPORTED), (dict(hkv=0), INVALID), (dict(pages=0), INVALID),
    (dict(max_pages=0), INVALID), (dict(ks=None), INVALID), (dict(cu=None), INVALID),
    (dict(kn=P + 8), UNSUPPORTED), (dict(vs=P + 4), UNSUPPORTED), (dict(sl=P + 2), UNSUPPORTED),
    (dict(total=1 << 31, hkv=1), UNSUPPORTED), (dict(pages=1 << 31), UNSUPPORTED),
    (dict(batch=0, kn=None), OK), (dict(total=0, k=None), OK)])
def test_append_refusals(L, change, want):
    assert append(L, **change) == want
    if want != OK:
        assert L.bi_last_error_message().decode().startswith("bi_kv_append_q8")


def attend(L, form, **kw):
    a = dict(q=P, k=P, v=P, ks=P, vs=P, num_pages=4, bt=P, max_pages=4, sl=P, cu=P, batch=1,
             total_q=2, max_q=2, max_seq_len=200, hq=32, hkv=8, D=128, page=64, scale=0.1, out=P,
             lse=None, ws=P, ws_bytes=1 << 30)
    a.update(kw)
    head = [a[x] for x in ("q", "k", "v", "ks", "vs", "num_pages", "bt", "max_pages", "sl")]
    mid = ([a["batch"]] if form == "decode"
           else [a["cu"], a["batch"], a["total_q"], a["max_q"]])
    tail = [a["max_seq_len"], a["hq"], a["hkv"], a["D"], a["page"], ctypes.c_float(a["scale"]),
            a["out"], a["lse"], a["ws"], a["ws_bytes"], None]
    fn = {"decode": L.bi_decode_attn_q8, "verify": L.bi_verify_block_q8,
          "prefill": L.bi_prefill_attn_q8}[form]
    return fn(*head, *mid, *tail)


@pytest.mark.parametrize("form", ["decode", "verify", "prefill"])
@pytest.mark.parametrize("change,want", [
    (dict(D=96), UNSUPPORTED), (dict(page=32), UNSUPPORTED), (dict(hq=30), INVALID),
    (dict(max_seq_len=257), INVALID), (dict(max_seq_len=0), INVALID), (dict(ws_bytes=16), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q=P + 2), UNSUPPORTED), (dict(ks=None), INVALID),
    (dict(vs=P + 8), UNSUPPORTED), (dict(ws=P + 8), UNSUPPORTED), (dict(out=None), INVALID),
    (dict(lse=P + 2), UNSUPPORTED), (dict(k=P + 8), UNSUPPORTED),
    (dict(batch=1025, total_q=1025), UNSUPPORTED),
    (dict(hq=264, hkv=8), UNSUPPORTED), (dict(batch=-1), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_pages=1 << 23), UNSUPPORTED), (dict(batch=0, total_q=0, q=None), OK)])
def test_attention_refusals(L, form, change, want):
    assert attend(L, form, **change) == want


def test_attention_widths(L):
    assert attend(L, "verify", max_q=9, total_q=9, hq=8) == UNSUPPORTED
    assert attend(L, "verify", max_q=8, total_q=8, hq=64) == UNSUPPORTED       # 64 rows
    assert attend(L, "verify", cu=None) == INVALID
    assert attend(L, "prefill", cu=None) == INVALID
    assert attend(L, "verify", total_q=3) == INVALID
    assert attend(L, "prefill", total_q=3) == INVALID
    assert attend(L, "prefill", max_q=0) == INVALID
    assert attend(L, "prefill", max_q=1 << 33, total_q=1 << 32) == INVALID
    assert "bi_prefill_attn_q8" in L.bi_last_error_message().decode()


def copy(L, **kw):
    a = dict(planes=[P, P], sizes=[64, 128], pages=4, src=P, dst=P, n=2)
    a.update(kw)
    m = len(a["planes"])
    planes = (ctypes.c_void_p * m)(*a["planes"])
    sizes = (ctypes.c_int64 * m)(*a["sizes"])
    return L.bi_kv_copy_pages(planes, sizes, m, a["pages"], a["src"], a["dst"], a["n"], None)


@pytest.mark.parametrize("change,want", [
    (dict(pages=0), INVALID), (dict(n=-1), INVALID), (dict(src=None), INVALID),
    (dict(planes=[P, None]), INVALID), (dict(planes=[P, P + 8]), UNSUPPORTED),
    (dict(sizes=[64, 24]), UNSUPPORTED), (dict(sizes=[64, 0]), INVALID),
    (dict(sizes=[1 << 36, 64]), UNSUPPORTED), (dict(dst=P + 1), INVALID),
    (dict(n=1 << 31), UNSUPPORTED), (dict(n=0, src=None), OK), (dict(planes=[], sizes=[]), OK)])
def test_copy_refusals(L, change, want):
    assert copy(L, **change) == want


def logprobs(L, **kw):
    a = dict(x=P, ldx=100, dt=bi.BI_F32, tok=P, rows=2, n=100, logp=P, ent=P, lse=P, top=0,
             tl=None, ti=None)
    a.update(kw)
    return L.bi_token_logprobs(a["x"], a["ldx"], a["dt"], a["tok"], a["rows"], a["n"], a["logp"],
                               a["ent"], a["lse"], a["top"], a["tl"], a["ti"], None)


@pytest.mark.parametrize("change,want", [
    (dict(dt=7), INVALID), (dict(n=0), INVALID), (dict(rows=-1), INVALID), (dict(ldx=99), INVALID),
    (dict(top=-1), INVALID), (dict(top=33), INVALID), (dict(n=3, top=4, tl=P, ti=P), INVALID),
    (dict(top=1), INVALID), (dict(x=None), INVALID), (dict(tok=None), INVALID),
    (dict(x=P + 2), INVALID), (dict(ti=P + 2, tl=P, top=1), INVALID),
    (dict(n=1 << 31, ldx=1 << 31), INVALID), (dict(rows=1 << 31), UNSUPPORTED),
    (dict(n=(1 << 31) - (1 << 14) + 1, ldx=1 << 31), INVALID),
    (dict(rows=0, x=None), OK)])
def test_logprobs_refusals(L, change, want):
    assert logprobs(L, **change) == want


def backward(L, **kw):
    a = dict(x=P, ldx=100, dt=bi.BI_BF16, tok=P, rows=2, n=100, lse=P, ent=P, gl=P, gh=P,
             dx=P + 4096, lddx=100)
    a.update(kw)
    return L.bi_token_logprobs_backward(a["x"], a["ldx"], a["dt"], a["tok"], a["rows"], a["n"],
                                        a["lse"], a["ent"], a["gl"], a["gh"], a["dx"], a["lddx"],
                                        None)


@pytest.mark.parametrize("change,want", [
    (dict(dt=3), INVALID), (dict(lddx=99), INVALID), (dict(gl=None, gh=None), INVALID),
    (dict(ent=None), INVALID), (dict(dx=P, lddx=104), INVALID), (dict(dx=P + 1), INVALID),
    (dict(lse=None), INVALID), (dict(rows=0, x=None), OK),
    (dict(n=(1 << 31) - (1 << 14) + 1, ldx=1 << 31, lddx=1 << 31), INVALID)])
def test_backward_refusals(L, change, want):
    assert backward(L, **change) == want


def test_binding_refuses_cpu_tensors():
    u8 = torch.zeros(2, 1, 64, 64, dtype=torch.uint8)
    sc = torch.zeros(2, 1, 64, dtype=torch.uint8)
    i = torch.zeros(1, dtype=torch.int32)
    x = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        bi.kv_append_q8(x, x, u8, u8, sc, sc, i.view(1, 1), i, i)
    with pytest.raises(ValueError, match="CUDA"):
        bi.decode_attn_q8(x, u8, u8, sc, sc, i.view(1, 1), i, max_seq_len=1, scale=1.0)
    with pytest.raises(ValueError, match="CUDA"):
        bi.kv_copy_pages([u8], i, i)
    with pytest.raises(ValueError, match="CUDA"):
        bi.token_logprobs(torch.zeros(1, 4), i)
    with pytest.raises(ValueError, match="CUDA"):
        bi.token_logprobs_backward(torch.zeros(1, 4), i, torch.zeros(1), None, torch.zeros(1))
