"""Refusals of the verification of drafted tokens without a GPU: bad arguments are returned before
anything is launched or read."""
import ctypes

import pytest
import torch

import invariant_bi_matmul_gb300 as bi

P = 1 << 20  # a fake, 16-byte aligned address: nothing may touch it
INVALID, UNSUPPORTED, OK = bi.BI_ERR_INVALID_ARG, bi.BI_ERR_UNSUPPORTED, bi.BI_OK


@pytest.fixture(scope="module")
def L():
    return bi.lib()


def verify(L, **kw):
    a = dict(x=P, ldl=1000, y=P, ldd=1000, dtype=bi.BI_F32, drafts=P, num=6, u=P, temps=P,
             temp=1.0, cu=P, batch=2, total=8, max_q=4, n=1000, tokens=P, accepted=P, logps=P,
             ws=P, ws_bytes=1 << 20)
    a.update(kw)
    order = ("x", "ldl", "y", "ldd", "dtype", "drafts", "num", "u", "temps")
    rest = ("cu", "batch", "total", "max_q", "n", "tokens", "accepted", "logps", "ws", "ws_bytes")
    return L.bi_verify_drafts(*[a[k] for k in order], ctypes.c_float(a["temp"]),
                              *[a[k] for k in rest], None)


@pytest.mark.parametrize("change,want", [
    (dict(dtype=7), INVALID), (dict(batch=-1), INVALID), (dict(total=-1), INVALID),
    (dict(num=-1), INVALID), (dict(max_q=0), INVALID), (dict(n=0), INVALID),
    (dict(n=(1 << 20) + 1, ldl=1 << 21, ldd=1 << 21), UNSUPPORTED), (dict(ldl=999), INVALID),
    (dict(ldd=999), INVALID), (dict(total=1), INVALID), (dict(x=None), INVALID),
    (dict(u=None), INVALID), (dict(cu=None), INVALID), (dict(tokens=None), INVALID),
    (dict(accepted=None), INVALID), (dict(ws=None), INVALID), (dict(drafts=None), INVALID),
    (dict(x=P + 2), INVALID), (dict(y=P + 1), INVALID), (dict(u=P + 2), INVALID),
    (dict(logps=P + 2), INVALID), (dict(ws=P + 8), UNSUPPORTED), (dict(ws_bytes=100), INVALID),
    (dict(temps=None, temp=-1.0), INVALID), (dict(temps=None, temp=float("nan")), INVALID),
    (dict(temps=None, temp=float("inf")), INVALID), (dict(total=1 << 31), UNSUPPORTED),
    (dict(num=1 << 31), UNSUPPORTED), (dict(batch=1 << 30, total=1 << 30), UNSUPPORTED),
    (dict(max_q=1 << 31), UNSUPPORTED), (dict(max_q=1 << 30), UNSUPPORTED), (dict(batch=0, x=None, tokens=None), OK)])
def test_refusals(L, change, want):
    assert verify(L, **change) == want
    if want != OK:
        assert L.bi_last_error_message().decode().startswith("bi_verify_drafts")


def test_workspace_size():
    size = bi.verify_drafts_workspace_size
    assert size(0, 0, 10) == 0 and size(4, 0, 1) == 4 * 16
    assert size(4, 3, 8193) == 7 * size(1, 0, 8193) > 7 * size(1, 0, 1)
    for bad in ((-1, 0, 10), (1, -1, 10), (1, 1, 0), (1, 1, (1 << 20) + 1), (1 << 31, 0, 10)):
        assert size(*bad) == 0


def test_cpu_tensors_are_refused():
    i32 = dict(dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA tensor"):
        bi.verify_drafts(torch.zeros(2, 10), torch.zeros(1, **i32), torch.zeros(2),
                         torch.tensor([0, 2], **i32), 2)
