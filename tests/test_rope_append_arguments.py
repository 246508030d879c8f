"""Refusals of the rotating append without a GPU: bad arguments are returned before anything is
launched or read."""
import array

import pytest
import torch

import invariant_bi_matmul_gb300 as bi

P = 1 << 20  # a fake, 16-byte aligned address: nothing may touch it
INVALID, UNSUPPORTED, OK = bi.BI_ERR_INVALID_ARG, bi.BI_ERR_UNSUPPORTED, bi.BI_OK


@pytest.fixture(scope="module")
def L():
    return bi.lib()


def append(L, q8, **kw):
    a = dict(q=P, ldq=4096, k=P, ldk=1024, v=P, ldv=1024, out=P * 2, ldo=4096, kc=P, vc=P, ks=P,
             vs=P, pages=4, bt=P, max_pages=4, sl=P, cu=P, batch=1, total=2, hq=32, hkv=8, D=128,
             page=64, theta=1e4, freq=None, rd=128, pos=None, ldp=0, axes=0, sections=None)
    a.update(kw)
    hold = [None if a[x] is None else array.array(t, a[x]) for x, t in (("freq", "d"),
                                                                       ("sections", "q"))]
    freq, sections = (None if h is None else h.buffer_info()[0] for h in hold)
    head = [a[x] for x in ("q", "ldq", "k", "ldk", "v", "ldv", "out", "ldo", "kc", "vc")]
    tail = [a[x] for x in ("pages", "bt", "max_pages", "sl", "cu", "batch", "total", "hq", "hkv",
                           "D", "page", "theta")]
    tail += [freq, a["rd"], a["pos"], a["ldp"], a["axes"], sections, None]
    if q8:
        return L.bi_rope_kv_append_q8(*head, a["ks"], a["vs"], *tail)
    return L.bi_rope_kv_append(*head, *tail)


@pytest.mark.parametrize("q8", [False, True])
@pytest.mark.parametrize("change,want", [
    (dict(batch=-1), INVALID), (dict(total=-1), INVALID), (dict(D=96), UNSUPPORTED),
    (dict(page=32), UNSUPPORTED), (dict(hkv=0), INVALID), (dict(hq=0), INVALID),
    (dict(pages=0), INVALID), (dict(max_pages=0), INVALID), (dict(cu=None), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(vc=None), INVALID),
    (dict(q=P + 8), UNSUPPORTED), (dict(kc=P + 4), UNSUPPORTED), (dict(sl=P + 2), UNSUPPORTED),
    (dict(ldq=4095), INVALID), (dict(ldk=1016), INVALID), (dict(ldv=1020), INVALID),
    (dict(ldq=4100), UNSUPPORTED), (dict(ldo=4100), UNSUPPORTED),
    (dict(out=P, ldo=8192), INVALID),
    (dict(rd=0), UNSUPPORTED), (dict(rd=24), UNSUPPORTED), (dict(rd=144), UNSUPPORTED),
    (dict(theta=0.0), INVALID), (dict(theta=float("inf")), INVALID),
    (dict(theta=float("nan")), INVALID), (dict(theta=5e-324), INVALID), (dict(freq=[float("nan")] * 64), INVALID),
    (dict(axes=-1), INVALID), (dict(axes=2), INVALID),
    (dict(axes=2, sections=[32, 31], pos=P, ldp=2), INVALID),
    (dict(axes=2, sections=[32, 33], pos=P, ldp=2), INVALID),
    (dict(axes=2, sections=[65, -1], pos=P, ldp=2), INVALID),
    (dict(axes=2, sections=[32, 32], pos=P, ldp=1), INVALID),
    (dict(axes=2, sections=[32, 32], pos=None, ldp=2), INVALID),
    (dict(axes=65, sections=[1] * 64 + [0], pos=P, ldp=2), INVALID),
    (dict(pages=1 << 31), UNSUPPORTED), (dict(total=1 << 31), UNSUPPORTED),
    (dict(hq=1 << 30, ldq=1 << 40, ldo=1 << 40), UNSUPPORTED),
    (dict(batch=0, q=None), OK), (dict(total=0, k=None), OK)])
def test_refusals(L, q8, change, want):
    assert append(L, q8, **change) == want
    if want != OK:
        assert L.bi_last_error_message().decode().startswith(
            "bi_rope_kv_append_q8" if q8 else "bi_rope_kv_append:")


@pytest.mark.parametrize("change,want", [(dict(ks=None), INVALID), (dict(vs=None), INVALID)])
def test_refusals_of_the_8_bit_form(L, change, want):
    assert append(L, True, **change) == want


def test_cpu_tensors_are_refused():
    q, k = torch.zeros(2, 8, 64, dtype=torch.bfloat16), torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(4, 2, 64, 64, dtype=torch.bfloat16)
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        bi.rope_kv_append(q, k, k, cache, cache, torch.zeros(1, 4, **i32), torch.zeros(1, **i32),
                          torch.zeros(2, **i32))
    with pytest.raises(TypeError):
        bi.rope_kv_append_q8(q, k, k, cache, cache, None, None, torch.zeros(1, 4, **i32),
                             torch.zeros(1, **i32), torch.zeros(2, **i32))
