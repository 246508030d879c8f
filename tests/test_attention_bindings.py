"""What the bf16 attention bindings hand to the library, without a GPU: tensors that call
themselves CUDA tensors, and a library that records its calls in place of making them."""
import pytest
import torch

import invariant_bi_matmul_gb300 as bi

HQ, HKV, D, PAGES, MAX_PAGES = 4, 2, 64, 4, 3


class OnDevice(torch.Tensor):
    """A host tensor that says it is on CUDA device 0."""
    is_cuda = property(lambda self: True)

    def get_device(self):
        return 0


def tensor(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(OnDevice)


class Recorder:
    def __init__(self):
        self.calls = []

    def bi_attn_workspace_size(self, *args):
        return 64

    def __getattr__(self, name):
        return lambda *args: self.calls.append((name, args)) or bi.BI_OK


@pytest.fixture
def library(monkeypatch):
    recorder = Recorder()
    monkeypatch.setattr(bi, "lib", lambda: recorder)
    monkeypatch.setattr(bi, "_device_of", lambda t: 0)
    monkeypatch.setattr(bi, "_on_current_device", lambda **tensors: None)
    monkeypatch.setattr(bi, "_stream_on", lambda stream, dev: 0)
    return recorder


def call(form, rows=2, seqs=2, table_rows=None, offsets=None, d=D, **shape):
    i32 = torch.int32
    q = tensor(rows, HQ, d)
    given = dict(out=tensor(rows, HQ, d), lse=tensor(rows, HQ, dtype=torch.float32),
                 workspace=tensor(1 << 16, dtype=torch.uint8), **shape)
    cache = tensor(PAGES, HKV, 64, D), tensor(PAGES, HKV, 64, D)
    tables = (tensor(seqs if table_rows is None else table_rows, MAX_PAGES, dtype=i32),
              tensor(seqs, dtype=i32))
    if form == "decode":
        bi.decode_attn(q, *cache, *tables, max_seq_len=100, scale=0.125, **given)
    else:
        cu_q = tensor(seqs + 1 if offsets is None else offsets, dtype=i32)
        attend = bi.verify_block if form == "verify" else bi.prefill_attn
        attend(q, *cache, *tables, cu_q, max_q=4, max_seq_len=100, scale=0.125, **given)


def batch_of(args, form):
    return args[7] if form == "decode" else args[8]


@pytest.mark.parametrize("seqs,table_rows", [(2, 2), (6, 6), (6, 2), (2, 6)])
def test_decode_serves_the_rows_of_q(library, seqs, table_rows):
    """Buffers of a fixed capacity with fewer queries: the queries say how many sequences."""
    call("decode", rows=2, seqs=seqs, table_rows=table_rows)
    (name, args), = library.calls
    assert name == "bi_decode_attn"
    assert batch_of(args, "decode") == 2


@pytest.mark.parametrize("form", ["verify", "prefill"])
@pytest.mark.parametrize("table_rows,offsets", [(2, 3), (5, 3), (2, 9)])
def test_blocks_serve_the_sequences(library, form, table_rows, offsets):
    call(form, rows=5, seqs=2, table_rows=table_rows, offsets=offsets)
    (name, args), = library.calls
    assert name == ("bi_verify_block" if form == "verify" else "bi_prefill_attn")
    assert args[8:10] == (2, 5)  # batch and total_q


@pytest.mark.parametrize("shape", [{}, {"window": 7}])
@pytest.mark.parametrize("form,change", [
    ("decode", dict(rows=3, seqs=2)), ("decode", dict(rows=3, seqs=2, table_rows=3)),
    ("decode", dict(rows=3, seqs=3, table_rows=2)), ("decode", dict(d=128)),
    ("verify", dict(table_rows=1)), ("verify", dict(offsets=2)), ("verify", dict(d=128)),
    ("prefill", dict(table_rows=1)), ("prefill", dict(offsets=2)), ("prefill", dict(d=32))])
def test_tensors_that_fall_short_are_refused(library, form, change, shape):
    """Fewer sequences, table rows or offsets than the call would read, or another head size."""
    with pytest.raises(ValueError):
        call(form, **change, **shape)
    assert not library.calls


@pytest.mark.parametrize("form", ["decode", "verify", "prefill"])
def test_shaped_calls_go_to_the_shaped_entry_points(library, form):
    call(form, window=7)
    (name, args), = library.calls
    assert name.endswith("_ex") and batch_of(args, form) == 2
