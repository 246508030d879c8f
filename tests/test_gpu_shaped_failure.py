"""The bounded waits of the attention kernels with shaped scores: a budget shorter than the call
makes them run out, the call reports it and returns, and the next one gives the same bits."""
import pytest
import torch

from invariant_bi_matmul_gb300 import inputs

pytestmark = pytest.mark.gpu

bi = pytest.importorskip("invariant_bi_matmul_gb300")

SHORT_NS = 1000  # 1 us: far shorter than any of the calls below


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch.device("cuda:0")


@pytest.mark.parametrize("shape", ["cap", "bias", "cap and bias", "window"])
@pytest.mark.parametrize("L,q", [(65540, 4), (2048, 2048)])
def test_waits_run_out_and_the_next_call_matches(dev, L, q, shape):
    p = inputs.paged_inputs([L], [q], Hq=32, Hkv=8, D=128, seed=5, device=dev)
    d = [getattr(p, k).to(dev) for k in ("q", "k_cache", "v_cache", "block_table", "seq_lens",
                                         "cu_q")]
    kw = dict(softcap=20.0) if "cap" in shape else {}
    if "bias" in shape:
        kw["slopes"] = torch.linspace(0.01, 0.5, 32, device=dev)
    if shape == "window":
        kw["window"] = L - 1
    fn = bi.verify_block if q <= bi.ATTN_MAX_Q else bi.prefill_attn

    def call():
        return fn(*d, max_q=q, max_seq_len=L, scale=128 ** -0.5, **kw)

    want = [x.clone() for x in call()]
    assert bi.device_status() == bi.BI_OK
    try:
        bi.selftest_set_wait_budget(SHORT_NS)
        call()
        status = bi.device_status()
    finally:
        bi.selftest_set_wait_budget(0)
    assert status == bi.BI_ERR_TIMEOUT
    again = call()
    assert bi.device_status() == bi.BI_OK
    assert torch.equal(again[0].view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(again[1], want[1]) and bool(again[1].isfinite().all())
