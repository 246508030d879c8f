"""Refusals of the attention calls with shaped scores without a GPU: bad arguments are returned
before anything is launched or read."""
import ctypes

import pytest

import invariant_bi_matmul_gb300 as bi

P = 1 << 20  # a fake, 16-byte aligned address: nothing may touch it
INVALID, UNSUPPORTED, OK = bi.BI_ERR_INVALID_ARG, bi.BI_ERR_UNSUPPORTED, bi.BI_OK


def attend(form, **kw):
    a = dict(q=P, k=P, v=P, num_pages=4, bt=P, max_pages=4, sl=P, cu=P, batch=1, total_q=2,
             max_q=2, max_seq_len=200, hq=32, hkv=8, D=128, page=64, scale=0.1, softcap=30.0,
             slopes=P, window=7, first=P, out=P, lse=None, ws=P, ws_bytes=1 << 30)
    a.update(kw)
    f32 = ctypes.c_float
    head = [a[x] for x in ("q", "k", "v", "num_pages", "bt", "max_pages", "sl")]
    mid = ([a["batch"]] if form == "decode"
           else [a["cu"], a["batch"], a["total_q"], a["max_q"]])
    tail = [a["max_seq_len"], a["hq"], a["hkv"], a["D"], a["page"], f32(a["scale"]),
            f32(a["softcap"]), a["slopes"], a["window"], a["first"], a["out"], a["lse"], a["ws"],
            a["ws_bytes"], None]
    L = bi.lib()
    fn = {"decode": L.bi_decode_attn_ex, "verify": L.bi_verify_block_ex,
          "prefill": L.bi_prefill_attn_ex}[form]
    return fn(*head, *mid, *tail)


@pytest.mark.parametrize("form", ["decode", "verify", "prefill"])
@pytest.mark.parametrize("change,want", [
    (dict(window=-1), INVALID), (dict(softcap=-0.5), INVALID),
    (dict(softcap=float("nan")), INVALID), (dict(softcap=float("inf")), INVALID),
    (dict(softcap=2.0 ** -21), UNSUPPORTED), (dict(softcap=2.0 ** 21), UNSUPPORTED),
    (dict(scale=0.0), UNSUPPORTED), (dict(scale=-0.1), UNSUPPORTED),
    (dict(scale=2.0 ** 21), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
    (dict(softcap=0.0, slopes=None, window=0, scale=-1.0), UNSUPPORTED),
    (dict(slopes=P + 2), UNSUPPORTED), (dict(first=P + 1), UNSUPPORTED), (dict(D=96), UNSUPPORTED),
    (dict(hq=30), INVALID), (dict(max_seq_len=257), INVALID), (dict(ws_bytes=16), INVALID),
    (dict(q=None), INVALID), (dict(ws=P + 8), UNSUPPORTED),
    (dict(batch=0, total_q=0, q=None, out=None), OK)])
def test_refusals(form, change, want):
    assert attend(form, **change) == want
    if want != OK:
        message = bi.lib().bi_last_error_message().decode()
        assert message.startswith({"decode": "bi_decode_attn_ex", "verify": "bi_verify_block_ex",
                                   "prefill": "bi_prefill_attn_ex"}[form])


@pytest.mark.parametrize("form", ["verify", "prefill"])
def test_offsets_are_required(form):
    assert attend(form, cu=None) == INVALID
