"""The condition under which a sequence's block is taken (seq_ok in attn_common.cuh), evaluated in
32 bits on the CPU for offsets whose sums and differences pass 2^31: whatever the offsets, a block
that is taken lies within the call's rows."""
import os
import re

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "invariant_bi_matmul_gb300", "csrc")


def seq_ok(L, t0, t1, max_q, max_seq_len, total_q):
    """The source's own expression, on int32 values that wrap."""
    text = open(os.path.join(CSRC, "attn_common.cuh")).read()
    body = re.search(r"bool seq_ok\(.*?\{(.*?)\}", text, re.S).group(1)
    expr = re.search(r"return (.*?);", body, re.S).group(1)
    expr = " ".join(expr.replace("s.", "").replace("&&", "and").split())
    with np.errstate(over="ignore"):
        v = {k: np.int32(x) for k, x in dict(L=L, t0=t0, max_q=max_q, max_seq_len=max_seq_len,
                                             total_q=total_q).items()}
        v["qb"] = np.int32(t1) - v["t0"]
        return bool(eval(expr, {}, v))  # noqa: S307


ENDS = [-2 ** 31, -2 ** 31 + 1, -2 ** 30, -7, -1, 0, 1, 2, 3, 8, 9, 2 ** 30, 2 ** 31 - 9,
        2 ** 31 - 2, 2 ** 31 - 1]


@pytest.mark.parametrize("total_q", [1, 2, 8, 9, 2 ** 31 - 1])
@pytest.mark.parametrize("max_q", [1, 8, 2 ** 31 - 1])
def test_a_block_that_is_taken_lies_within_the_rows(max_q, total_q):
    for t0 in ENDS:
        for t1 in ENDS:
            for L in (1, 8, 2 ** 31 - 1):
                sound = 0 <= t0 and 1 <= t1 - t0 <= min(max_q, L) and t1 <= total_q
                assert seq_ok(L, t0, t1, max_q, 2 ** 31 - 1, total_q) == sound, (t0, t1, L)
