"""The 8-bit paged KV cache at the edges of its contract, on the GPU: lengths
and boundaries that contradict each other, rows that must stay as they were,
calls without work, values near the ends of their types, and waits that give up."""

import math

import numpy as np
import pytest
import torch

import attention_forward_09_gb300 as gb
import oracle
from _helpers import dev, status_word, to_np
from test_fp8_cache_gpu import DTYPES, HEAD_SIZES, Ctx, bf16, check_decode, ints, raw, run_decode

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_09_gb300 import _build

    _build.build()
    gb.load_library()


# ---------------------------------------------------------------- boundaries of the read-back
def readable(cu, s, total, max_tokens):
    return 0 <= cu[s] <= cu[s + 1] <= total and cu[s + 1] - cu[s] <= max_tokens


@pytest.mark.parametrize("cu", [
    [0, 50, 20],                 # rows 20 to 49 are the first sequence's, past the last boundary
    [0, 300, 200],
    [0, 300, 200, 400],          # two sequences claim rows 200 to 299
    [0, 100, 1000],              # past total_tokens
    [0, 600, 700],               # nothing of the second in range
    [0, 100, 100 + 3 * 128 + 1],  # more blocks than the table has
    [0, 385, 400],               # of the first, while the second is in order
    [-5, 10, 20],
    [7, 10, 20],                 # does not begin at 0
    [0, 500, 100, 90, 560, 300, 300],
    [600, 500, 400, 300, 200, 100, 0],
    [0] + [384, 0] * 40,         # decreases beyond the first 32 sequences too
])
def test_read_reports_every_bad_boundary_and_reads_the_other_sequences(cu):
    S, total, bs, hkv, D = len(cu) - 1, 600, 128, 1, 64
    c = Ctx([384] * S, hkv, D, seed=5)
    table = c.table[:, :3].contiguous()
    k = torch.full((total, hkv, D), 7.0, dtype=torch.bfloat16, device=dev())
    v = torch.full((total, hkv, D), -7.0, dtype=torch.bfloat16, device=dev())
    cache, scales, _ = c.on_gpu()
    status = status_word()
    gb.attn_kv_cache_read_fp8(cache, scales, table.to(dev()), ints(cu), total, k=k, v=v, dev_status=status)
    assert int(status) == gb.DEV_BAD_SEQLEN
    ks, vs = oracle.paged_gather(c.values(), c.table, c.lens)
    owners = [[s for s in range(S) if readable(cu, s, total, 3 * bs) and cu[s] <= t < cu[s + 1]] for t in range(total)]
    for got, ctx, fill in ((to_np(k), ks, 7.0), (to_np(v), vs, -7.0)):
        for t in range(total):
            if not owners[t]:
                assert (got[t] == fill).all(), t
            else:
                assert any(np.array_equal(got[t], ctx[s][t - cu[s]]) for s in owners[t]), (t, owners[t])


def test_read_with_boundaries_in_order_reports_nothing():
    """Empty sequences, rows behind the last, and a table that is exactly long enough."""
    c = Ctx([0, 384, 0, 1, 0], 2, 64, seed=6)
    cache, scales, _ = c.on_gpu()
    cu = [0, 0, 384, 384, 385, 385]
    status = status_word()
    k, v = gb.attn_kv_cache_read_fp8(cache, scales, c.table[:, :3].contiguous().to(dev()), ints(cu), 385, dev_status=status)
    want = torch.from_numpy(np.concatenate(oracle.paged_gather(c.values(), c.table, c.lens)[1])).to(torch.bfloat16)
    assert int(status) == 0 and torch.equal(v.cpu(), want)
    gb.attn_kv_cache_read_fp8(cache, scales, c.table.to(dev()), ints([0] * 6), 0, dev_status=status)
    assert int(status) == 0
    gb.attn_kv_cache_read_fp8(cache, scales, c.table.to(dev()), ints([0, 0, 0, 0, 0, 3]), 0, dev_status=status)  # no rows for these
    assert int(status) == gb.DEV_BAD_SEQLEN
