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


# ---------------------------------------------------------------- several new tokens a sequence
def poison_free_memory(rows, hkv, d):
    """NaN into memory that the allocator will hand out for the contexts."""
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    held = [torch.full((rows, hkv, d), float("nan"), dtype=torch.bfloat16, device=dev()) for _ in range(8)]
    del held


@pytest.mark.parametrize("cu_k,skipped", [
    ([0, 300, 700, 850], [1]),      # 400 tokens, and a table of three blocks
    ([0, 300, 250, 400], [1]),      # decreasing; the third is [250, 400), whose first rows the first claims too
    ([0, 300, 300, 2000], [2]),     # past total_tokens
    ([0, 300, 600, 750], []),
])
def test_prefill_skips_the_sequences_that_the_read_back_refuses(cu_k, skipped):
    hq, hkv, D, T = 4, 2, 64, 1000
    c = Ctx([512] * 3, hkv, D, seed=23)
    cache, scales, table = c.on_gpu()
    q_lens = [20, 0 if cu_k[2] == cu_k[1] else 30, 25]
    cu_q = np.cumsum([0] + q_lens)
    q = bf16(int(cu_q[-1]), hq, D, seed=24)
    out = torch.full((int(cu_q[-1]), hq, D), 77.0, device=dev())
    lse = torch.full((hq, int(cu_q[-1])), 77.0, device=dev())
    status = status_word()
    poison_free_memory(T, hkv, D)
    gb.attn_fwd_paged_prefill_fp8(q.to(dev()), cache, scales, table[:, :3].contiguous(), ints(cu_q), ints(cu_k), T, 30, 900,
                                  out=out, lse=lse, dev_status=status)
    assert int(status) == (gb.DEV_BAD_SEQLEN if skipped else 0)
    for s in range(3):
        rows = slice(int(cu_q[s]), int(cu_q[s + 1]))
        if s in skipped:
            assert (out[rows] == 77).all() and (lse[:, rows] == 77).all()
        elif cu_k[1:3] != [300, 250]:  # (there the rows that two sequences claim hold either's)
            n = cu_k[s + 1] - cu_k[s]
            ref, ref_lse = oracle.attention_paged_prefill(q[rows], c.values(), c.table[s:s + 1], [n], [0, q_lens[s]], 1 / math.sqrt(D), True)
            assert np.abs(to_np(out[rows]) - ref).max(initial=0) <= 1e-2  # the prefill kernels' bounds
            assert np.abs(to_np(lse[:, rows]) - ref_lse).max(initial=0) <= 1e-3
        assert torch.isfinite(out[rows]).all()


# ---------------------------------------------------------------- decode: values near the ends of fp32
def written(key, value, d, kind="e4m3"):
    """One sequence's keys and values [n, 1, d], written into a cache of its own blocks in order."""
    n = key.shape[0]
    nb = -(-n // 128)
    cache = torch.zeros(2, nb, 128, 1, d, device=dev()).to(DTYPES[kind])
    scales = torch.ones(2, nb, 1, 128, dtype=torch.uint8, device=dev())
    gb.attn_kv_cache_write_fp8(key.to(torch.bfloat16).to(dev()), value.to(torch.bfloat16).to(dev()), ints(range(n)), cache, scales)
    c = Ctx([1], 1, d, kind)
    c.lens, c.codes, c.scales = [n], cache.view(torch.uint8).cpu(), scales.cpu()
    c.table = torch.arange(nb, dtype=torch.int32).view(1, nb)
    return c


@pytest.mark.parametrize("byte", [1, 9, 20, 27, 40])
@pytest.mark.parametrize("n,max_len", [(517, 517), (4096, 1 << 20), (131072, 1 << 20)])
def test_decode_of_values_near_the_bottom_of_fp32(n, max_len, byte):
    """Value rows whose exponent bytes are the least: fp32 and bf16 hold the
    results (of 2^-126 and a little below), and so do the outputs."""
    c = Ctx([n], 1, 64, seed=byte, exps=(119, 123), vexps=(byte, byte + 2), extra=0)
    q = bf16(1, 2, 64, seed=n)
    for out_dtype in (torch.float32, torch.bfloat16):
        out, lse = run_decode(c, q, max_len=max_len, out_dtype=out_dtype)
        check_decode(c, q, out, lse)
        # relative to what an average of n values of one sign or the other comes to
        assert float(out.double().norm()) > 0.1 / math.sqrt(n) * 8 * float(np.nanstd(c.values()[1, c.table[0, 0], :, 0]))


@pytest.mark.parametrize("n,max_len", [(900, 900), (4096, 4096), (900, 1 << 20), (100000, 1 << 20)])
def test_decode_of_small_values_under_rising_scores(n, max_len):
    """As above, with scores that rise from block to block by e^27, less than a
    reference is moved for."""
    g = torch.Generator().manual_seed(n)
    key = torch.randn(n, 1, 64, generator=g)
    key[:, 0, 0] = 8 * 27.0 * (torch.arange(n) // 128 % 7)
    value = torch.randn(n, 1, 64, generator=g) * 2.0 ** -112
    c = written(key, value, 64)
    q = torch.zeros(1, 2, 64, dtype=torch.bfloat16)
    q[:, :, 0] = torch.tensor([1.0, 0.5])
    q[0, 1, 1:] = 0.5
    for out_dtype in (torch.float32, torch.bfloat16):
        out, lse = run_decode(c, q, max_len=max_len, out_dtype=out_dtype)
        check_decode(c, q, out, lse)


@pytest.mark.parametrize("D,n,max_len", [(64, 4096, 4096), (128, 4096, 4096), (64, 200000, 200000), (256, 150000, 1 << 20)])
def test_decode_joins_of_large_values_under_rising_scores(D, n, max_len):
    """Scores of the last block e^27 above all others, less than a reference is
    moved for, so that the last part's softmax sum is 2^40 and more, and values
    of 2^110: the joined result is finite, and so is every product on the way."""
    g = torch.Generator().manual_seed(n)
    key = torch.randn(n, 1, D, generator=g)
    key[:, 0, 0] = math.sqrt(D) * 27.0 * (torch.arange(n) // 128 == (n - 1) // 128)
    value = torch.randn(n, 1, D, generator=g) * 2.0 ** 108
    c = written(key, value, D)
    q = torch.zeros(1, 2, D, dtype=torch.bfloat16)
    q[:, :, 0] = torch.tensor([1.0, 0.5])
    for out_dtype in (torch.float32, torch.bfloat16):
        out, lse = run_decode(c, q, max_len=max_len, out_dtype=out_dtype)
        check_decode(c, q, out, lse)


@pytest.mark.parametrize("D,hq", [(64, 2), (128, 4), (64, 8)])
def test_decode_of_large_queries_beside_large_keys_they_do_not_meet(D, hq):
    """Queries and keys of 2^100 in columns of their own: the factor of a score
    overflows, the score is 0 or moderate all the same."""
    n = 200
    key = torch.zeros(n, 1, D)
    key[::3, 0, 1] = 2.0 ** 100            # meets zeros of q
    key[1::3, 0, 0] = 2.0 ** -98           # scores of 4 / sqrt(D)
    key[1::3, 0, 2] = torch.randn(n // 3 + 1, generator=torch.Generator().manual_seed(1))[: len(key[1::3])] * 2.0 ** -98
    value = torch.randn(n, 1, D, generator=torch.Generator().manual_seed(2))
    c = written(key, value, D)
    q = torch.zeros(1, hq, D, dtype=torch.bfloat16)
    q[:, :, 0] = 2.0 ** 100
    q[:, 0, 2] = 2.0 ** 99
    for max_len in (n, 1 << 20):
        out, lse = run_decode(c, q, max_len=max_len)
        check_decode(c, q, out, lse)


# ---------------------------------------------------------------- decode: the weights' bits, column by column
def check_columns(c, q, out, scale=None):
    """Every column of the result against its own bound: w_t = p_t 2^(b_t - 127)
    is off by up to 2^-16 w_t + 2^-30 max(w of the block), four pieces of four
    bits, and by 4 ds + 2^-18 of itself as in check_decode (scores, ex2, fp32
    sums); a result by that times |code|, summed over the tokens."""
    S, hq, D = q.shape
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    values = c.values()
    ks, vs = oracle.paged_gather(values, c.table, c.lens)
    powers = np.exp2(c.scales[1].double().numpy() - 127.0)  # [nb, Hkv, bs]
    got, g = to_np(out), hq // values.shape[3]
    qd = q.double().numpy()
    for s in range(S):
        n = c.lens[s]
        blocks = [np.arange(b, min(b + 128, n)) for b in range(0, n, 128)]
        for h in range(hq):
            k, v = ks[s][:, h // g], vs[s][:, h // g]
            size = np.concatenate([powers[int(c.table[s, i]), h // g, :len(b)] for i, b in enumerate(blocks)])
            x = scale * (k @ qd[s, h])
            p = np.exp(x - x.max())
            p /= p.sum()
            w = p * size
            ds = (D / 32 + 12) * 2.0 ** -23 * scale * float((np.abs(k) @ np.abs(qd[s, h])).max())
            off = (2.0 ** -16 + 2.0 ** -18 + 4 * ds) * w
            for b in blocks:
                off[b] += 2.0 ** -30 * w[b].max()
            want, tol = p @ v, (off / size) @ np.abs(v)
            if out.dtype == torch.bfloat16:
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want)
            err = np.abs(got[s, h] - want)
            assert (err <= tol).all(), (s, h, float((err / tol).max()))


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,hq,hkv", [(64, 8, 1), (64, 2, 2), (128, 4, 1), (192, 8, 2), (256, 6, 1)])
def test_decode_columns_beside_one_far_larger_value(D, hq, hkv, out_dtype):
    """A value row in each block with one column 2^6 to 2^24 above everything,
    its other codes zero: the other columns keep what its bits leave."""
    n = 900
    c = Ctx([n, 300], hkv, D, seed=D)
    for s, length in enumerate(c.lens):
        for i in range(-(-length // 128)):
            b, t = int(c.table[s, i]), (37 * i) % min(128, length - 128 * i)
            c.codes[1, b, t] = 0
            c.codes[1, b, t, :, (11 * i + s) % D] = 0x7E  # 448
            c.scales[1, b, :, t] = 121 + 6 + 3 * (i % 7)
    q = bf16(2, hq, D, seed=D + 1)
    for max_len in (n, 1 << 20):
        out, lse = run_decode(c, q, max_len=max_len, out_dtype=out_dtype)
        check_columns(c, q, out)
        check_decode(c, q, out, lse)


@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vexps,kexps", [((118, 124), (119, 123)), ((110, 130), (119, 123)), ((60, 190), (105, 124)), ((1, 30), (119, 123))])
def test_decode_columns_with_scales_of_any_size(vexps, kexps, out_dtype):
    """Value rows whose sizes differ by up to 2^130, block by block and row by row."""
    c = Ctx([400, 700, 128, 1], 2, 128, seed=9, exps=kexps, vexps=vexps)
    q = bf16(4, 6, 128, seed=10)
    for max_len in (max(c.lens), 1 << 20):
        out, lse = run_decode(c, q, max_len=max_len, out_dtype=out_dtype)
        check_columns(c, q, out)
        check_decode(c, q, out, lse)


def test_decode_to_bf16_is_the_rounding_of_the_result_to_fp32():
    """The two output types differ by one rounding, whatever the head count."""
    for D, hq, hkv, lens in ((64, 20, 4, [1, 900, 4097]), (128, 32, 8, [517]), (256, 8, 1, [9000, 20000])):
        c = Ctx(lens, hkv, D, seed=hq)
        q = bf16(len(lens), hq, D, seed=D)
        a, la = run_decode(c, q)
        b, lb = run_decode(c, q, out_dtype=torch.bfloat16)
        assert torch.equal(a.to(torch.bfloat16), b) and torch.equal(la, lb)


def test_decode_of_infinite_codes_reaches_its_own_heads_and_columns_only():
    c = Ctx([200, 200], 2, 64, "e5m2", seed=6)
    q = bf16(2, 4, 64, seed=7)
    for max_len in (200, 1 << 20):
        clean, clean_lse = run_decode(c, q, max_len=max_len)
        bad = Ctx([200, 200], 2, 64, "e5m2", seed=6)
        bad.codes[0, int(bad.table[0, 0]), 7, 1, 3] = 0x7C   # a key of sequence 0, KV head 1
        bad.codes[1, int(bad.table[1, 1]), 2, 0, 9] = 0xFC   # a value of sequence 1, KV head 0, column 9
        out, lse = run_decode(bad, q, max_len=max_len)
        free, free_lse = torch.ones(2, 4, 64, dtype=torch.bool), torch.ones(2, 4, dtype=torch.bool)
        free[0, 2:], free_lse[0, 2:], free[1, :2, 9] = False, False, False
        assert torch.equal(out.cpu()[free], clean.cpu()[free]) and torch.equal(lse.cpu()[free_lse], clean_lse.cpu()[free_lse])
        assert not torch.isfinite(out[1, :2, 9]).any()


# ---------------------------------------------------------------- calls without work
@pytest.mark.parametrize("columns", [0, 3])
def test_calls_without_sequences_or_tokens(columns):
    """Empty tensors have no address; a batch of no sequences is a batch all the same."""
    hq, hkv, D = 4, 2, 64
    c = Ctx([5], hkv, D)
    cache, scales, _ = c.on_gpu()
    before = raw(cache), scales.cpu()
    plain = torch.zeros(2, 3, 128, hkv, D, dtype=torch.bfloat16, device=dev())
    q = torch.empty(0, hq, D, dtype=torch.bfloat16, device=dev())
    kv = torch.empty(0, hkv, D, dtype=torch.bfloat16, device=dev())
    table, none = torch.empty(0, columns, dtype=torch.int32, device=dev()), ints([])
    for max_len in (0, 300, 1 << 20):
        for out, lse in (gb.attn_fwd_paged_fp8(q, cache, scales, table, none, max_len, lse=True),
                         gb.attn_fwd_paged(q, plain, table, none, max_len, lse=True),
                         gb.attn_fwd_paged_noalloc(q, plain, table, none, max_len, lse=True)):
            assert out.shape == (0, hq, D) and lse.shape == (0, hq)
    gb.attn_kv_cache_write_fp8(kv, kv, none, cache, scales)
    assert np.array_equal(raw(cache), before[0]) and torch.equal(scales.cpu(), before[1])
    k, v = gb.attn_kv_cache_read_fp8(cache, scales, table, ints([0]), 0)
    assert k.shape == v.shape == (0, hkv, D)
    k, _ = gb.attn_kv_cache_read_fp8(cache, scales, table, ints([0]), 7)
    assert k.shape == (7, hkv, D)
    out, lse = gb.attn_fwd_paged_prefill_fp8(q, cache, scales, table, ints([0]), ints([0]), 0, 0, 300, lse=True)
    assert out.shape == (0, hq, D) and lse.shape == (hq, 0)
    # sequences, but no token of any
    table = torch.full((2, max(columns, 1)), -1, dtype=torch.int32, device=dev())
    status = status_word()
    out, lse = gb.attn_fwd_paged_prefill_fp8(q, cache, scales, table, ints([0, 0, 0]), ints([0, 0, 0]), 0, 0, 300, dev_status=status)
    assert out.shape == (0, hq, D) and lse is None
    out, lse = gb.attn_fwd_paged_fp8(torch.zeros(2, hq, D, dtype=torch.bfloat16, device=dev()), cache, scales, table, ints([0, 0]), 0,
                                     lse=True, dev_status=status)
    assert not out.any() and torch.isneginf(lse).all() and int(status) == 0


@pytest.mark.parametrize("most", [10 ** 6, 700])
def test_prefill_with_a_length_bound_above_the_contexts_sum(most):
    """max_seq_len bounds the contexts; it may be the model's longest."""
    hq, hkv, D, lens = 4, 2, 64, [130, 77]
    c = Ctx(lens, hkv, D, seed=25)
    cache, scales, table = c.on_gpu()
    wide = torch.full((2, 10000), -1, dtype=torch.int32, device=dev())
    wide[:, :table.shape[1]] = table
    q_lens = [30, 77]
    q = bf16(sum(q_lens), hq, D, seed=26)
    cu_q, cu_k = ints(np.cumsum([0] + q_lens)), ints(np.cumsum([0] + lens))
    ref, ref_lse = oracle.attention_paged_prefill(q, c.values(), c.table, lens, cu_q, 1 / math.sqrt(D), True)
    status = status_word()
    out, lse = gb.attn_fwd_paged_prefill_fp8(q.to(dev()), cache, scales, wide, cu_q, cu_k, sum(lens), max(q_lens), most, lse=True,
                                             dev_status=status)
    assert int(status) == 0
    assert np.abs(to_np(out) - ref).max() <= 1e-2 and np.abs(to_np(lse) - ref_lse).max() <= 1e-3  # the prefill kernels' bounds


# ---------------------------------------------------------------- waits that give up
@pytest.mark.parametrize("max_len", [3000, 1 << 20])  # a cluster a sequence and head; chunks and a join
@pytest.mark.parametrize("D,hq,hkv", [(64, 4, 2), (128, 8, 1), (256, 4, 4)])
def test_decode_that_gives_up_reports_timeout_and_the_context_stays_usable(D, hq, hkv, max_len):
    """Loads are issued and land, no product is; nothing is left waiting."""
    c = Ctx([3000, 0, 129, 700], hkv, D, seed=27)
    q = bf16(4, hq, D, seed=28)
    prev = gb.attn_set_wait_give_up(True)
    try:
        status = status_word()
        _, lse = run_decode(c, q, max_len=max_len, status=status)
        torch.cuda.synchronize()  # the call comes back
        assert int(status) == gb.DEV_TIMEOUT
        assert torch.isneginf(lse[1]).all()  # the empty sequence waits for nothing
    finally:
        gb.attn_set_wait_give_up(prev)
    # a status word that already holds a timeout: nothing more is begun
    out, lse = torch.full((4, hq, D), 77.0, device=dev()), torch.full((4, hq), 77.0, device=dev())
    cache, scales, table = c.on_gpu()
    for _ in range(2):
        gb.attn_fwd_paged_fp8(q.to(dev()), cache, scales, table, ints(c.lens), max_len, out=out, lse=lse, dev_status=status)
        assert int(status) == gb.DEV_TIMEOUT
        assert (out[[0, 2, 3]] == 77).all() and (lse[[0, 2, 3]] == 77).all() and not out[1].any()
    status.zero_()
    out, lse = run_decode(c, q, max_len=max_len, status=status)
    assert int(status) == 0
    check_decode(c, q, out, lse)


# ---------------------------------------------------------------- bad lengths, streams, the prompt form
@pytest.mark.parametrize("max_len,clamped", [(300, 300), (30000, 384)])  # a cluster each; chunks, where the table's end is the bound
def test_decode_clamps_bad_lengths_to_what_there_is(max_len, clamped):
    lens = [1 << 30, -3, 50, 300]
    c = Ctx([384, 100, 50, 384], 2, 64, seed=8)
    c.table = c.table[:, :3].contiguous()
    q = bf16(4, 4, 64, seed=9)
    cache, scales, table = c.on_gpu()
    status = status_word()
    out, lse = gb.attn_fwd_paged_fp8(q.to(dev()), cache, scales, table, ints(lens), max_len, lse=True, dev_status=status)
    assert int(status) == gb.DEV_BAD_SEQLEN
    c.lens = [clamped, 0, 50, 300]
    check_decode(c, q, out, lse)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("D", HEAD_SIZES)
def test_prefill_head_sizes_and_formats_on_a_stream_of_its_own(D, kind):
    """The whole way on a stream that is not the current one: the write, the
    prompt form, the read-back and a decode, with nothing but that stream's order."""
    hq, hkv, lens, q_lens = 6, 2, [300, 1, 0, 140], [7, 1, 0, 140]
    S, nblk = len(lens), 3
    k, v = bf16(sum(lens), hkv, D, seed=1).to(dev()), bf16(sum(lens), hkv, D, seed=2, spread=3.0).to(dev())
    q = bf16(sum(q_lens), hq, D, seed=3)
    table = torch.randperm(S * nblk, generator=torch.Generator().manual_seed(D)).to(torch.int32).view(S, nblk)
    where = torch.cat([table[s, torch.arange(n) // 128] * 128 + torch.arange(n) % 128 for s, n in enumerate(lens)]).to(torch.int32)
    cache = torch.zeros(2, S * nblk, 128, hkv, D, device=dev()).to(DTYPES[kind])
    scales = torch.ones(2, S * nblk, hkv, 128, dtype=torch.uint8, device=dev())
    cu_q, cu_k, sl = ints(np.cumsum([0] + q_lens)), ints(np.cumsum([0] + lens)), ints(lens)
    last = torch.stack([q[max(0, sum(q_lens[:s + 1]) - 1)] for s in range(S)])
    qd, where, table_d, last_d, status = q.to(dev()), where.to(dev()), table.to(dev()), last.to(dev()), status_word()
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    gb.attn_kv_cache_write_fp8(k, v, where, cache, scales, dev_status=status, stream=stream)
    out, lse = gb.attn_fwd_paged_prefill_fp8(qd, cache, scales, table_d, cu_q, cu_k, sum(lens), max(q_lens), max(lens), lse=True,
                                             dev_status=status, stream=stream)
    rk, rv = gb.attn_kv_cache_read_fp8(cache, scales, table_d, cu_k, sum(lens), dev_status=status, stream=stream)
    one, one_lse = gb.attn_fwd_paged_fp8(last_d, cache, scales, table_d, sl, max(lens), lse=True, dev_status=status, stream=stream)
    stream.synchronize()
    assert int(status) == 0
    c = Ctx([1], hkv, D, kind)
    c.lens, c.table, c.codes, c.scales = lens, table, cache.view(torch.uint8).cpu(), scales.cpu()
    gathered = oracle.paged_gather(c.values(), table, lens)
    for got, want in zip((rk, rv), gathered):
        assert np.array_equal(to_np(got), np.concatenate(want))  # (codes of at most 4 bits: bf16 holds them)
    ref, ref_lse = oracle.attention_paged_prefill(q, c.values(), table, lens, cu_q.cpu(), 1 / math.sqrt(D), True)
    # the prefill kernels' weights are bf16, 2^-8 of themselves off at most; as much again for everything else
    tol = 2.0 ** -7 * max(float(np.abs(x).max()) for x in gathered[1] if x.size)
    assert np.abs(to_np(out) - ref).max() <= tol and np.abs(to_np(lse) - ref_lse).max() <= 1e-3
    check_decode(c, last, one, one_lse)


def test_read_and_write_in_a_graph_with_new_contents():
    """Captured once, replayed with other tokens, slots and boundaries."""
    hkv, D, T = 2, 96, 300
    key, slots, cu = bf16(T, hkv, D, seed=1).to(dev()), ints(range(T)), ints([0, 100, 300])
    cache = torch.zeros(2, 4, 128, hkv, D, device=dev()).to(torch.float8_e4m3fn)
    scales = torch.ones(2, 4, hkv, 128, dtype=torch.uint8, device=dev())
    table, status = ints([[0, 1, 2, 3], [3, 2, 1, 0]]).view(2, 4), status_word()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gb.attn_kv_cache_write_fp8(key, key, slots, cache, scales, dev_status=status)
        k, v = gb.attn_kv_cache_read_fp8(cache, scales, table, cu, T, dev_status=status)
    for seed, bounds in ((2, [0, 300, 300]), (3, [0, 17, 290])):
        key.copy_(bf16(T, hkv, D, seed=seed))
        slots.copy_(torch.randperm(512, generator=torch.Generator().manual_seed(seed))[:T])
        cu.copy_(ints(bounds))
        g.replay()
        torch.cuda.synchronize()
        want = oracle.paged_gather(oracle.stands_for(raw(cache), scales.cpu().numpy(), "e4m3"), table.cpu(),
                                   [bounds[1], bounds[2] - bounds[1]])
        assert int(status) == 0
        for got, x in zip((k, v), want):
            assert np.array_equal(to_np(got[:bounds[2]]), np.concatenate(x))


# ---------------------------------------------------------------- decode: parts of little weight and large values
@pytest.mark.parametrize("top,size", [(87.5, 40), (160.0, 110)])  # weights of e^(40 - top): 2^-68, 2^-173
@pytest.mark.parametrize("D,n,max_len", [(64, 4096, 4096), (128, 4096, 1 << 20), (64, 200000, 200000), (256, 4096, 4096)])
def test_decode_joins_of_parts_with_little_weight_and_large_values(D, n, max_len, top, size):
    """The first block takes nearly all the weight; the last one, whose scores
    lie e^40 above those before it (less than a reference is moved for), has
    values large enough to matter all the same."""
    g = torch.Generator().manual_seed(n)
    key = torch.randn(n, 1, D, generator=g)
    block = torch.arange(n) // 128
    key[:, 0, 0] = math.sqrt(D) * (top * (block == 0) + 40.0 * (block == block[-1]))
    value = torch.randn(n, 1, D, generator=g)
    value[block < block[-1]] *= 2.0 ** (-30 if size == 40 else -60)
    value[block == block[-1]] *= 2.0 ** size
    c = written(key, value, D)
    q = torch.zeros(1, 2, D, dtype=torch.bfloat16)
    q[:, :, 0], q[0, 1, 1] = 1.0, 0.25
    for out_dtype in (torch.float32, torch.bfloat16):
        out, lse = run_decode(c, q, max_len=max_len, out_dtype=out_dtype)
        check_columns(c, q, out)
        check_decode(c, q, out, lse)


# ---------------------------------------------------------------- sizes and captures
def test_many_sequences_that_share_blocks():
    """70000 sequences, empty ones among them, over four blocks that they share."""
    S, hkv, hq, D = 70000, 1, 2, 64
    g = torch.Generator().manual_seed(1)
    c = Ctx([512], hkv, D, seed=30, extra=0)
    lens = torch.randint(0, 4, (S,), generator=g, dtype=torch.int32) * torch.randint(0, 60, (S,), generator=g, dtype=torch.int32)
    c.table = torch.randint(0, 4, (S, 2), generator=g, dtype=torch.int32)
    cache, scales, table = c.on_gpu()
    q = bf16(S, hq, D, seed=31)
    status = status_word()
    out, lse = gb.attn_fwd_paged_fp8(q.to(dev()), cache, scales, table, lens.to(dev()), 177, lse=True, dev_status=status)
    cu = torch.cat([torch.zeros(1, dtype=torch.int32), lens.cumsum(0).to(torch.int32)])
    k, v = gb.attn_kv_cache_read_fp8(cache, scales, table, cu.to(dev()), int(cu[-1]), dev_status=status)
    assert int(status) == 0
    keep = sorted({0, 1, 3333, 35000, S - 1} | set(torch.randint(0, S, (40,), generator=g).tolist()))
    gathered = oracle.paged_gather(c.values(), c.table[keep], lens[keep].tolist())
    for i, s in enumerate(keep):
        rows = slice(int(cu[s]), int(cu[s + 1]))
        assert np.array_equal(to_np(k[rows]), gathered[0][i]) and np.array_equal(to_np(v[rows]), gathered[1][i])
    empty = lens == 0
    assert not out.cpu()[empty].any() and torch.isneginf(lse.cpu()[empty]).all() and torch.isfinite(lse.cpu()[~empty]).all()
    c.table, c.lens = c.table[keep], lens[keep].tolist()
    check_decode(c, q[keep], out[keep], lse[keep])


@pytest.mark.parametrize("hq,hkv", [(65535, 1), (65535, 4369)])
def test_decode_of_the_most_heads(hq, hkv):
    c = Ctx([130], hkv, 64, seed=32, extra=0)
    q = bf16(1, hq, 64, seed=33)
    for max_len in (130, 1 << 20):
        out, lse = run_decode(c, q, max_len=max_len)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        part = Ctx([130], hkv, 64, seed=32, extra=0)
        g = hq // hkv
        for h in (0, hkv // 2, hkv - 1):  # the oracle takes some KV heads
            part.codes, part.scales = c.codes[:, :, :, h:h + 1], c.scales[:, :, h:h + 1]
            rows = [h * g + i for i in sorted({0, 1, 7, 8, g // 2, g - 1})]
            check_decode(part, q[:, rows], out[:, rows], lse[:, rows])


def test_prompt_form_in_a_graph_with_new_contents():
    """Captured once; replayed with other contexts, queries and boundaries."""
    hq, hkv, D, T, Tq = 4, 2, 128, 700, 90
    c = Ctx([600, 600], hkv, D, seed=34)
    cache, scales, table = c.on_gpu()
    q, cu_q, cu_k = bf16(Tq, hq, D, seed=35).to(dev()), ints([0, 40, 90]), ints([0, 300, 700])
    status = status_word()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = gb.attn_fwd_paged_prefill_fp8(q, cache, scales, table, cu_q, cu_k, T, 90, 1000, lse=True, dev_status=status)
    for seed, lens, q_lens in ((40, [300, 400], [40, 50]), (41, [600, 5], [85, 5]), (42, [1, 0], [1, 0])):
        fresh = Ctx([600, 600], hkv, D, seed=seed)
        cache.view(torch.uint8).copy_(fresh.codes)
        scales.copy_(fresh.scales)
        table.copy_(fresh.table)
        x = bf16(Tq, hq, D, seed=seed + 10)
        q.copy_(x)
        cu_q.copy_(ints(np.cumsum([0] + q_lens)))
        cu_k.copy_(ints(np.cumsum([0] + lens)))
        out.fill_(77.0)
        graph.replay()
        torch.cuda.synchronize()
        n = sum(q_lens)
        ref, ref_lse = oracle.attention_paged_prefill(x[:n], fresh.values(), fresh.table, lens, np.cumsum([0] + q_lens), 1 / math.sqrt(D), True)
        assert int(status) == 0
        assert np.abs(to_np(out[:n]) - ref).max() <= 1e-2 and np.abs(to_np(lse[:, :n]) - ref_lse).max() <= 1e-3  # the prefill kernels' bounds
        assert (out[n:] == 77).all()
