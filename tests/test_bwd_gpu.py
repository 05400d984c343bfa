"""attn_bwd_dense / _padded / _varlen against the float64 oracle, each value
within the bound that fp32 sums and the bf16 roundings of p, ds and the result
allow (oracle/gradients.py), on what the framework's own forward calls return."""

import numpy as np
import pytest
import torch

import attention_forward_09_gb300 as gb
import oracle
import workloads
from _helpers import dev, status_word, to_np

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_09_gb300 import _build

    _build.build()
    gb.load_library()


def check(got, ref, what):
    for n, g, (r, b) in zip(("dq", "dk", "dv"), got, ref):
        g = to_np(g)
        assert g.shape == r.shape
        bad = ~(np.abs(g - r) <= b)
        assert not bad.any(), (f"{what} {n}: {bad.sum()} of {bad.size} values off, worst "
                               f"{np.nanmax(np.abs(g - r) / b):.3g} of the bound, first at {np.argwhere(bad)[0]}")


def randn(g, *shape):
    return workloads.randn_bf16(g, *shape).to(dev())


def dense_case(B, Sq, Sk, Hq, Hkv, D, causal, odt=BF16, dlse=False, seed=0, scale=None):
    g = torch.Generator().manual_seed(seed + 7 * Sq + Sk + D)
    q, k, v, do = randn(g, B, Sq, Hq, D), randn(g, B, Sk, Hkv, D), randn(g, B, Sk, Hkv, D), randn(g, B, Sq, Hq, D)
    s = D ** -0.5 if scale is None else scale
    out, lse = gb.attn_fwd_dense(q, k, v, s, causal, lse=True, out_dtype=odt)
    dl = torch.randn(lse.shape, generator=g).to(dev()) if dlse else None
    st = status_word()
    got = gb.attn_bwd_dense(q, k, v, out, lse, do, s, causal, dlse=dl, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for b in range(B):
        ref = oracle.attention_gradients(q[b], k[b], v[b], out[b], lse[b], do[b], s, causal, None if dl is None else dl[b], True)
        check([x[b] for x in got], ref, f"entry {b}")
    return q, k, v, out, lse, do, s, got


SHAPES = [  # B, Sq, Sk, Hq, Hkv
    (1, 1, 1, 1, 1), (2, 37, 91, 4, 4), (1, 128, 128, 2, 1), (1, 129, 127, 2, 2), (2, 200, 333, 4, 2), (1, 333, 200, 6, 2),
    (1, 64, 1000, 3, 3), (1, 700, 65, 2, 1), (1, 1, 300, 8, 1), (1, 300, 1, 2, 2), (3, 513, 513, 2, 1)]


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("causal", [False, True])
def test_dense(shape, D, causal):
    dense_case(*shape, D, causal, odt=BF16 if shape[1] % 2 else torch.float32, dlse=shape[2] % 3 == 0)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_large_score_a_row_and_scales(D):
    """Nearly one-hot rows (scale 1: scores of tens) and flat ones (scale 1e-3)."""
    dense_case(1, 150, 260, 2, 1, D, True, scale=1.0)
    dense_case(1, 150, 260, 2, 1, D, False, scale=1e-3)


@pytest.mark.parametrize("D", [64, 96, 128, 192, 256])
def test_many_tiles_and_a_large_group(D):
    """Streams longer than the ring, eight heads on a KV head: every slot is used again and again."""
    dense_case(1, 1500, 900, 8, 1, D, True)
    dense_case(1, 900, 1500, 2, 2, D, False)


def packed(lens_q, lens_k, Hq, Hkv, D, causal, odt=BF16, dlse=False, tail=0, poison=False, seed=1):
    g = torch.Generator().manual_seed(seed + D)
    Tq, Tk = sum(lens_q) + tail, sum(lens_k) + tail
    q, k, v, do = randn(g, Tq, Hq, D), randn(g, Tk, Hkv, D), randn(g, Tk, Hkv, D), randn(g, Tq, Hq, D)
    cq, ck = workloads.cu_from_lengths(lens_q), workloads.cu_from_lengths(lens_k)
    mq, mk, s = max(lens_q + [0]), max(lens_k + [0]), D ** -0.5
    out, lse = gb.attn_fwd_varlen(q, k, v, cq.to(dev()), ck.to(dev()), mq, mk, s, causal, lse=True, out_dtype=odt)
    if tail:
        for x in (q, k, v, do, out):
            x[-tail:] = float("nan")
        lse[:, -tail:] = float("nan")
    dl = torch.randn(lse.shape, generator=g).to(dev()) if dlse else None
    grads = [torch.full_like(x, 777.0) for x in (q, k, v)]
    st = status_word()
    got = gb.attn_bwd_varlen(q, k, v, out, lse, do, cq.to(dev()), ck.to(dev()), mq, mk, s, causal, dlse=dl, dq=grads[0],
                             dk=grads[1], dv=grads[2], dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for a, b in zip(got, grads):
        assert a is b
    for n in range(len(lens_q)):
        i, j = slice(int(cq[n]), int(cq[n + 1])), slice(int(ck[n]), int(ck[n + 1]))
        ref = oracle.attention_gradients(q[i], k[j], v[j], out[i], lse[:, i], do[i], s, causal, None if dl is None else dl[:, i],
                                         True)
        check((got[0][i], got[1][j], got[2][j]), ref, f"document {n}")
    for x in got:
        assert tail == 0 or bool((x[-tail:] == 777.0).all())


DOCS = [([37, 91], [37, 91]), ([0, 130, 1, 0, 257], [5, 130, 0, 0, 257]), ([300, 1, 64], [100, 140, 1]), ([5], [700])]


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
@pytest.mark.parametrize("docs", DOCS)
@pytest.mark.parametrize("causal", [False, True])
def test_packed_documents(docs, D, causal):
    packed(*docs, 4, 2, D, causal, odt=torch.float32 if D == 96 else BF16, dlse=D == 64)


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
@pytest.mark.parametrize("causal", [False, True])
def test_rows_of_no_document_are_left_and_never_read(D, causal):
    packed([37, 150], [70, 130], 4, 2, D, causal, tail=200)


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
@pytest.mark.parametrize("causal", [False, True])
def test_a_neighbour_full_of_nan_does_not_reach_a_document(D, causal):
    g = torch.Generator().manual_seed(D)
    lens_q, lens_k = [70, 90, 150], [150, 61, 150]
    Tq, Tk, Hq, Hkv, s = sum(lens_q), sum(lens_k), 2, 1, D ** -0.5
    q, k, v, do = randn(g, Tq, Hq, D), randn(g, Tk, Hkv, D), randn(g, Tk, Hkv, D), randn(g, Tq, Hq, D)
    cq, ck = (workloads.cu_from_lengths(x).to(dev()) for x in (lens_q, lens_k))

    def run():
        out, lse = gb.attn_fwd_varlen(q, k, v, cq, ck, 150, 150, s, causal, lse=True, out_dtype=BF16)
        return gb.attn_bwd_varlen(q, k, v, out, lse, do, cq, ck, 150, 150, s, causal)

    a = [x.clone() for x in run()]
    for x in (q, do):
        x[70:160] = float("nan")
    for x in (k, v):
        x[150:211] = float("inf")
    b = run()
    torch.cuda.synchronize()
    for x, y, lo, hi in zip(a, b, (70, 150, 150), (160, 211, 211)):
        assert torch.equal(x[:lo], y[:lo]) and torch.equal(x[hi:], y[hi:])


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("which", ["both", "keys", "queries"])
def test_padded_batch(D, causal, which):
    g = torch.Generator().manual_seed(D)
    B, Sq, Sk, Hq, Hkv, s = 4, 200, 270, 4, 2, D ** -0.5
    lq, lk = [200, 0, 129, 64], [270, 100, 0, 131]
    q, k, v, do = randn(g, B, Sq, Hq, D), randn(g, B, Sk, Hkv, D), randn(g, B, Sk, Hkv, D), randn(g, B, Sq, Hq, D)
    tq = None if which == "keys" else torch.tensor(lq, dtype=torch.int32, device=dev())
    tk = None if which == "queries" else torch.tensor(lk, dtype=torch.int32, device=dev())
    lq, lk = lq if tq is not None else [Sq] * B, lk if tk is not None else [Sk] * B
    out, lse = gb.attn_fwd_padded(q, k, v, tq, tk, s, causal, lse=True, out_dtype=torch.float32)
    dl = torch.randn(lse.shape, generator=g).to(dev())
    for b in range(B):  # the padding may hold anything
        for x in (q, do, out):
            x[b, lq[b]:] = float("nan")
        for x in (k, v):
            x[b, lk[b]:] = float("inf")
        lse[b, :, lq[b]:] = float("nan")
        dl[b, :, lq[b]:] = float("nan")
    st = status_word()
    got = gb.attn_bwd_padded(q, k, v, out, lse, do, tq, tk, s, causal, dlse=dl, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for b in range(B):
        m, n = lq[b], lk[b]
        ref = oracle.attention_gradients(q[b, :m], k[b, :n], v[b, :n], out[b, :m], lse[b, :, :m], do[b, :m], s, causal,
                                         dl[b, :, :m], True)
        check((got[0][b, :m], got[1][b, :n], got[2][b, :n]), ref, f"entry {b}")
        assert not got[0][b, m:].any() and not got[1][b, n:].any() and not got[2][b, n:].any()


def test_lengths_outside_the_batch_are_clamped_and_reported():
    g = torch.Generator().manual_seed(5)
    q, k, v, do = (randn(g, 2, 100, 2, 64) for _ in range(4))
    out, lse = gb.attn_fwd_dense(q, k, v, 0.125, lse=True, out_dtype=BF16)
    lens = torch.tensor([101, 100], dtype=torch.int32, device=dev())
    ref = gb.attn_bwd_dense(q, k, v, out, lse, do, 0.125)
    for bad in ((lens, None), (None, lens)):
        st = status_word()
        got = gb.attn_bwd_padded(q, k, v, out, lse, do, *bad, 0.125, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == gb.DEV_BAD_SEQLEN
        assert all(torch.equal(a, b) for a, b in zip(ref, got))


@pytest.mark.parametrize("cq,ck,mq,mk", [([0, 60, 50, 120], [0, 60, 90, 120], 64, 64), ([0, 60, 130, 130], [0, 50, 60, 120], 70, 64),
                                         ([0, 60, 90, 120], [0, 60, 90, 121], 64, 64), ([0, 65, 90, 120], [0, 60, 90, 120], 64, 64)])
def test_documents_with_bad_boundaries_are_reported_and_left(cq, ck, mq, mk):
    g = torch.Generator().manual_seed(6)
    T, D = 120, 128
    q, k, v, do = (randn(g, T, 2, D) for _ in range(4))
    lse = torch.zeros(2, T, device=dev())
    grads = [torch.full_like(q, 777.0) for _ in range(3)]
    st = status_word()
    a, b = (torch.tensor(x, dtype=torch.int32, device=dev()) for x in (cq, ck))
    gb.attn_bwd_varlen(q, k, v, q, lse, do, a, b, mq, mk, dq=grads[0], dk=grads[1], dv=grads[2], dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == gb.DEV_BAD_SEQLEN
    good = [0 <= cq[n] <= cq[n + 1] <= T and cq[n + 1] - cq[n] <= mq and 0 <= ck[n] <= ck[n + 1] <= T and ck[n + 1] - ck[n] <= mk
            for n in range(3)]
    assert not all(good)
    for x, c in zip(grads, (cq, ck, ck)):
        mine = torch.zeros(T, dtype=torch.bool)
        for n in range(3):
            if good[n]:
                mine[c[n]:c[n + 1]] = True
        assert bool((x.cpu()[~mine] == 777.0).all()) and not bool((x.cpu()[mine] == 777.0).all(-1).any())


def test_empty_sides():
    q, k = torch.zeros(2, 0, 2, 64, dtype=BF16, device=dev()), torch.ones(2, 9, 1, 64, dtype=BF16, device=dev())
    lse = torch.zeros(2, 2, 0, device=dev())
    dq, dk, dv = gb.attn_bwd_dense(q, k, k, q, lse, q)
    assert dq.shape == q.shape and not dk.any() and not dv.any()
    q, k = torch.ones(2, 9, 2, 64, dtype=BF16, device=dev()), torch.zeros(2, 0, 1, 64, dtype=BF16, device=dev())
    lse = torch.full((2, 2, 9), -float("inf"), device=dev())
    dq, dk, dv = gb.attn_bwd_dense(q, k, k, q, lse, q)
    assert not dq.any() and dk.shape == k.shape
    e = torch.zeros(0, 2, 64, dtype=BF16, device=dev())
    z = torch.zeros(1, dtype=torch.int32, device=dev())
    assert gb.attn_bwd_varlen(e, e, e, e, torch.zeros(2, 0, device=dev()), e, z, z, 0, 0)[0].shape == e.shape


@pytest.mark.parametrize("D", [64, 128, 192, 256])
def test_the_same_inputs_give_the_same_bits(D):
    q, k, v, out, lse, do, s, got = dense_case(1, 700, 700, 4, 1, D, True)
    for _ in range(3):
        again = gb.attn_bwd_dense(q, k, v, out, lse, do, s, True)
        assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_another_stream_and_a_captured_call():
    q, k, v, out, lse, do, s, got = dense_case(2, 300, 300, 4, 2, 128, True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = gb.attn_bwd_dense(q, k, v, out, lse, do, s, True, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, a))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = gb.attn_bwd_dense(q, k, v, out, lse, do, s, True)
    do.neg_()  # replayed on new values: the gradients are linear in dout, to the sign of every rounding
    lse0 = lse.clone()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(-x, y) for x, y in zip(got, b)) and torch.equal(lse, lse0)


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("Sk", [700, 2100])
def test_a_wait_that_gives_up_reports_it_and_the_context_stays_usable(D, Sk):
    """Items a CTA has for itself, and (the longer context) items that clusters share."""
    q, k, v, out, lse, do, s, got = dense_case(1, 128, Sk, 1, 1, D, False)
    prev = gb.attn_set_wait_give_up(True)
    try:
        st = status_word()
        gb.attn_bwd_dense(q, k, v, out, lse, do, s, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) & gb.DEV_TIMEOUT
    finally:
        gb.attn_set_wait_give_up(prev)
    again = gb.attn_bwd_dense(q, k, v, out, lse, do, s)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


def test_refusals_of_the_binding():
    q = torch.zeros(1, 8, 2, 64, dtype=BF16, device=dev())
    lse = torch.zeros(1, 2, 8, device=dev())
    ok = dict(q=q, k=q, v=q, out=q, lse=lse, dout=q)
    gb.attn_bwd_dense(**ok)
    for n, bad in (("q", q.float()), ("k", q[:, ::2]), ("v", q[:, :4]), ("out", q.half()), ("lse", lse[:, :1]),
                   ("lse", lse.double()), ("dout", q.float()), ("dout", q[:, :4]), ("dlse", lse[..., :4]),
                   ("dq", torch.empty_like(q, dtype=torch.float32)), ("dk", q[:, :4]), ("dev_status", lse),
                   ("workspace", torch.empty(64, 2, device=dev())[:, 0]), ("k", q.cpu())):
        with pytest.raises(ValueError):
            gb.attn_bwd_dense(**{**ok, n: bad})
    with pytest.raises(gb.GbattnError):
        gb.attn_bwd_dense(**ok, workspace=torch.empty(256, dtype=torch.uint8, device=dev()))
    with pytest.raises(ValueError):
        gb.attn_bwd_padded(**ok, lens_q=torch.zeros(2, dtype=torch.int32, device=dev()))


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
@pytest.mark.parametrize("causal", [False, True])
def test_more_tiles_than_a_wave(D, causal):
    """Several items a CTA, some without any work between them: every buffer, ring and barrier carries on from item to item."""
    packed([130, 0, 513, 1, 250, 300], [130, 64, 260, 300, 250, 5], 48, 24, D, causal)
    dense_case(1, 200, 200, 200, 100, D, causal)


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
@pytest.mark.parametrize("Sq,Sk", [(64, 3000), (3000, 64), (130, 2500)])
def test_items_of_one_or_two_steps_follow_one_another(D, Sq, Sk):
    """Many more items than CTAs, each over after a step or two; then other values in the same places."""
    for seed in (0, 1):
        dense_case(1, Sq, Sk, 12, 12, D, False, seed=seed)


def test_offsets_past_32_bits():
    """Element offsets beyond 2^31 in every tensor: the last documents of a pack of 82000 tokens of 208 heads of 128."""
    n, L, H, D, s = 1640, 50, 208, 128, 128 ** -0.5
    T = n * L
    assert T * H * D > 2 ** 31
    g = torch.Generator(device=dev()).manual_seed(4)
    q, k, v, do = (torch.randn(T, H, D, generator=g, device=dev(), dtype=BF16) for _ in range(4))
    cu = torch.arange(0, T + 1, L, dtype=torch.int32, device=dev())
    out, lse = gb.attn_fwd_varlen(q, k, v, cu, cu, L, L, s, True, lse=True, out_dtype=BF16)
    st = status_word()
    got = gb.attn_bwd_varlen(q, k, v, out, lse, do, cu, cu, L, L, s, True, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    for d in (0, n // 2, n - 1):
        i, h = slice(d * L, d * L + L), slice(H - 9, H)
        ref = oracle.attention_gradients(q[i, h], k[i, h], v[i, h], out[i, h], lse[h, i], do[i, h], s, True, bounds=True)
        check([x[i, h] for x in got], ref, f"document {d}")


@pytest.mark.parametrize("causal", [False, True])
def test_many_documents_under_a_long_bound(causal):
    """3000 documents, most of them empty, bounded by the longest: items are claimed in runs, and skipped."""
    g = torch.Generator().manual_seed(2)
    lens = [0] * 3000
    for i, x in ((0, 3), (700, 1100), (701, 1), (1500, 130), (2999, 257)):
        lens[i] = x
    packed(lens, lens, 4, 2, 64, causal)


@pytest.mark.parametrize("D", [64, 192, 256])
def test_a_captured_call_at_other_head_sizes_and_two_graphs(D):
    """Two graphs, each with its own workspace, replayed one after the other and on two streams at once."""
    a, b = dense_case(1, 400, 300, 4, 2, D, True), dense_case(2, 130, 520, 2, 1, D, False)
    graphs, outs = [], []
    for (q, k, v, out, lse, do, s, got), causal in ((a, True), (b, False)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(gb.attn_bwd_dense(q, k, v, out, lse, do, s, causal))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in graphs]
    for x in outs:
        for t in x:
            t.zero_()
    torch.cuda.synchronize()
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for x, c in zip(outs, (a, b)):
        assert all(torch.equal(p, r) for p, r in zip(x, c[-1]))


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
def test_calls_behind_one_another_do_not_meet(D):
    """Calls of other sizes in between, nothing waiting: the passes of one call end before the next begins."""
    a, b = dense_case(1, 500, 700, 6, 2, D, True), dense_case(3, 90, 260, 40, 40, D, False)
    for _ in range(10):
        x = gb.attn_bwd_dense(*a[:6], a[6], True)
        y = gb.attn_bwd_dense(*b[:6], b[6], False)
        z = gb.attn_bwd_dense(*a[:6], a[6], True)
    torch.cuda.synchronize()
    assert all(torch.equal(p, r) for got, c in ((x, a), (y, b), (z, a)) for p, r in zip(got, c[-1]))


def test_infinities_and_nan_behind_the_causal_diagonal_of_a_row():
    """A query row's own gradient reads only the keys it sees; rows without a key read nothing at all."""
    q, k, v, out, lse, do, s, got = dense_case(1, 300, 200, 2, 1, 128, True)  # rows 0 .. 99 see no key
    q2, do2, out2 = q.clone(), do.clone(), out.clone()
    for x in (q2, do2, out2):
        x[:, :100] = float("nan")
    again = gb.attn_bwd_dense(q2, k, v, out2, lse, do2, s, True)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
@pytest.mark.parametrize("causal", [False, True])
def test_few_items_of_many_steps(D, causal):
    """Steps shared by clusters of 2, 4 and 8 CTAs: of the keys' pass (many heads to a KV head, many queries), of the
    queries' pass (long contexts), with tails, empty shares, empty entries and rows that see nothing."""
    for shape in ((1, 700, 130, 8, 1), (2, 1100, 500, 4, 1), (1, 100, 2100, 2, 1), (1, 1500, 1030, 9, 3), (1, 3000, 1, 2, 2)):
        dense_case(*shape, D, causal, dlse=True)
    packed([0, 1300, 40], [70, 120, 3], 6, 1, D, causal, odt=torch.float32, dlse=True)
    packed([130, 20], [1500, 0], 2, 1, D, causal, tail=30)


@pytest.mark.parametrize("causal", [False, True])
def test_a_scattered_padding_mask_through_the_packing_calls(causal):
    """A training step under a padding mask that keeps any tokens: packed, attended, differentiated, unpacked, without a
    host round trip; against the oracle on each row's kept tokens."""
    g = torch.Generator().manual_seed(8)
    B, S, Hq, Hkv, D, s = 3, 210, 4, 2, 96, 96 ** -0.5
    q, k, v, do = randn(g, B, S, Hq, D), randn(g, B, S, Hkv, D), randn(g, B, S, Hkv, D), randn(g, B, S, Hq, D)
    mask = (torch.rand(B, S, generator=g) < 0.6).to(torch.uint8)
    mask[1] = 0
    cu, pos = gb.attn_mask_to_varlen(mask.to(dev()))
    pq, pk, pv, pdo = (gb.attn_pack_rows(x, pos, cu) for x in (q, k, v, do))
    pq, pk, pv, pdo = (x.view(B * S, -1, D) for x in (pq, pk, pv, pdo))
    out, lse = gb.attn_fwd_varlen(pq, pk, pv, cu, cu, S, S, s, causal, lse=True, out_dtype=BF16)
    grads = gb.attn_bwd_varlen(pq, pk, pv, out, lse, pdo, cu, cu, S, S, s, causal)
    got = [gb.attn_unpack_rows(x, pos, B, S).view(B, S, -1, D) for x in grads]
    torch.cuda.synchronize()
    c = cu.cpu().tolist()
    for b in range(B):
        kept, i = mask[b].bool(), slice(c[b], c[b + 1])
        ref = oracle.attention_gradients(q[b].cpu()[kept], k[b].cpu()[kept], v[b].cpu()[kept], out[i], lse[:, i],
                                         do[b].cpu()[kept], s, causal, bounds=True)
        check([x[b].cpu()[kept] for x in got], ref, f"row {b}")
        assert not any(x[b].cpu()[~kept].any() for x in got)


def test_outputs_next_to_one_another_and_outputs_over_inputs():
    """Gradients and workspace as neighbours in one buffer are as separate ones; over an input they are refused."""
    g = torch.Generator().manual_seed(9)
    B, S, Hq, Hkv, D, s = 2, 150, 4, 2, 64, 0.125
    q, k, v, do = randn(g, B, S, Hq, D), randn(g, B, S, Hkv, D), randn(g, B, S, Hkv, D), randn(g, B, S, Hq, D)
    out, lse = gb.attn_fwd_dense(q, k, v, s, True, lse=True, out_dtype=BF16)
    ref = gb.attn_bwd_dense(q, k, v, out, lse, do, s, True)
    nq, nk, nw = q.numel(), k.numel(), gb.attn_bwd_workspace_size(B, B * S, Hq) // 2
    flat = torch.empty(nw + nq + 2 * nk, dtype=BF16, device=dev())
    ws, dq, dk, dv = flat.split([nw, nq, nk, nk])
    got = gb.attn_bwd_dense(q, k, v, out, lse, do, s, True, dq=dq.view_as(q), dk=dk.view_as(k), dv=dv.view_as(k), workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
    for bad in (dict(dq=q), dict(dq=out), dict(dq=do), dict(dk=k), dict(dv=v), dict(dk=ref[1], dv=ref[1])):
        with pytest.raises(gb.GbattnError):
            gb.attn_bwd_dense(q, k, v, out, lse, do, s, True, **bad)
