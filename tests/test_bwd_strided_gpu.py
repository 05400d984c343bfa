"""Gradients from tensors as other code leaves them: an `out` that is transposed,
a part of a wider tensor or repeated, and dout, lse and dlse of any strides.
The values are those of the contiguous call, to the bit."""

import pytest
import torch

import attention_forward_09_gb300 as gb
import oracle
import workloads
from _helpers import dev, status_word
from test_bwd_gpu import check, randn

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_09_gb300 import _build

    _build.build()
    gb.load_library()


def transposed(x):
    """x in memory as [.., heads, rows, D]."""
    return x.transpose(-3, -2).contiguous().transpose(-3, -2)


def part(x):
    """x between other values, which are no numbers: every dimension has a stride of its own."""
    wide = torch.full([n + 2 for n in x.shape[:-1]] + [x.shape[-1] + 24], float("nan"), dtype=x.dtype, device=x.device)
    y = wide[(slice(1, -1),) * (x.dim() - 1) + (slice(8, -16),)]
    return y.copy_(x)


def apart(x):
    """The values of a row one apart: no layout that rows can be read from."""
    return torch.stack((x, x), -1)[..., 0]


def off(x):
    """Rows that do not begin on 16 bytes."""
    wide = torch.zeros(*x.shape[:-1], x.shape[-1] + 1, dtype=x.dtype, device=x.device)
    return wide[..., 1:].copy_(x)


LAYOUTS = [transposed, part, apart, off]


def case(form, Hq, Hkv, D, causal, odt, seed=0):
    """(the call, its arguments but for the four that may be strided, those four)"""
    g = torch.Generator().manual_seed(seed + D)
    s = D ** -0.5
    if form == "varlen":
        lq, lk = [37, 0, 150], [70, 5, 130]
        cq, ck = workloads.cu_from_lengths(lq).to(dev()), workloads.cu_from_lengths(lk).to(dev())
        q, k, v, do = randn(g, 187, Hq, D), randn(g, 205, Hkv, D), randn(g, 205, Hkv, D), randn(g, 187, Hq, D)
        out, lse = gb.attn_fwd_varlen(q, k, v, cq, ck, 150, 130, s, causal, lse=True, out_dtype=odt)

        def run(out, lse, do, dlse, **kw):
            return gb.attn_bwd_varlen(q, k, v, out, lse, do, cq, ck, 150, 130, s, causal, dlse=dlse, **kw)
    else:
        q, k, v, do = randn(g, 3, 150, Hq, D), randn(g, 3, 130, Hkv, D), randn(g, 3, 130, Hkv, D), randn(g, 3, 150, Hq, D)
        if form == "dense":
            out, lse = gb.attn_fwd_dense(q, k, v, s, causal, lse=True, out_dtype=odt)

            def run(out, lse, do, dlse, **kw):
                return gb.attn_bwd_dense(q, k, v, out, lse, do, s, causal, dlse=dlse, **kw)
        else:
            tq, tk = (torch.tensor(x, dtype=torch.int32, device=dev()) for x in ([150, 0, 77], [130, 9, 65]))
            out, lse = gb.attn_fwd_padded(q, k, v, tq, tk, s, causal, lse=True, out_dtype=odt)

            def run(out, lse, do, dlse, **kw):
                return gb.attn_bwd_padded(q, k, v, out, lse, do, tq, tk, s, causal, dlse=dlse, **kw)
    dlse = torch.randn(lse.shape, generator=g).to(dev())
    return run, (out, lse, do, dlse), (q, k, v)


def same(a, b):
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) and y.is_contiguous() for x, y in zip(a, b))


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
@pytest.mark.parametrize("form", ["dense", "padded", "varlen"])
@pytest.mark.parametrize("odt", [BF16, torch.float32])
def test_an_out_of_any_strides_gives_the_same_bits(form, D, odt):
    run, (out, lse, do, dlse), _ = case(form, 6, 2, D, D % 128 == 0, odt)
    ref = run(out, lse, do, dlse)
    for layout in LAYOUTS:
        o = layout(out)
        assert torch.equal(o, out) and not o.is_contiguous()
        st = status_word()
        same(ref, run(o, lse, do, dlse, dev_status=st))
        assert int(st.item()) == 0


@pytest.mark.parametrize("form", ["dense", "padded", "varlen"])
def test_gradients_and_lse_of_any_strides_give_the_same_bits(form):
    run, (out, lse, do, dlse), _ = case(form, 4, 2, 128, True, BF16)
    ref = run(out, lse, do, dlse)
    for layout in LAYOUTS:
        same(ref, run(out, lse, layout(do), dlse))
    for rows in (part, apart):
        same(ref, run(out, rows(lse), do, rows(dlse)))
    same(ref, run(transposed(out), part(lse), transposed(do), apart(dlse)))
    # as autograd hands them over from sums of out and of lse
    ones, one = torch.ones_like(do), torch.ones_like(lse)
    same(run(out, lse, ones, one), run(out, lse, ones[..., :1, :1, :1].expand_as(do), one[..., :1].expand_as(lse)))


def test_a_repeated_out_and_dimensions_of_one_index():
    """Strides of 0, and of dimensions that have a single index, whatever they say."""
    D, s = 64, 0.125
    g = torch.Generator().manual_seed(3)
    for B, Sq, H in ((1, 1, 1), (3, 1, 2), (1, 40, 1), (2, 40, 3)):
        q, k, v, do = randn(g, B, Sq, H, D), randn(g, B, 9, H, D), randn(g, B, 9, H, D), randn(g, B, Sq, H, D)
        out, lse = gb.attn_fwd_dense(q, k, v, s, lse=True, out_dtype=BF16)
        ref = gb.attn_bwd_dense(q, k, v, out, lse, do, s)
        odd = torch.empty(out.numel() * 3, dtype=BF16, device=dev()).as_strided(
            out.shape, [8 * n if m > 1 else 7 for m, n in zip(out.shape[:-1], (3 * Sq * H * D // 8, D // 8, 2 * Sq * D // 8))] + [1])
        same(ref, gb.attn_bwd_dense(q, k, v, odd.copy_(out), lse, do, s))
        for dim in range(3):
            o = out.select(dim, 0).unsqueeze(dim).expand_as(out)
            same(gb.attn_bwd_dense(q, k, v, o.contiguous(), lse, do, s), gb.attn_bwd_dense(q, k, v, o, lse, do, s))


def test_a_transposed_out_against_the_oracle():
    run, (out, lse, do, dlse), (q, k, v) = case("dense", 4, 2, 128, True, BF16, seed=5)
    got = run(transposed(out), lse, transposed(do), dlse)
    torch.cuda.synchronize()
    for b in range(q.shape[0]):
        ref = oracle.attention_gradients(q[b], k[b], v[b], out[b], lse[b], do[b], 128 ** -0.5, True, dlse[b], True)
        check([x[b] for x in got], ref, f"entry {b}")


def test_strides_past_32_bits():
    """Entries, rows and heads of `out` that lie 2^31 elements and more from the first."""
    D, s = 64, 0.125
    g = torch.Generator().manual_seed(4)
    q, k, v, do = (randn(g, 2, 3, 2, D) for _ in range(4))
    out, lse = gb.attn_fwd_dense(q, k, v, s, lse=True, out_dtype=BF16)
    ref = gb.attn_bwd_dense(q, k, v, out, lse, do, s)
    far = 2 ** 31 + 64
    room = torch.empty(2 * far + 4096, dtype=BF16, device=dev())
    for strides in ((far, 128, 64, 1), (64, far, 128, 1), (64, 128, far, 1)):
        same(ref, gb.attn_bwd_dense(q, k, v, room.as_strided(out.shape, strides).copy_(out), lse, do, s))


def test_another_stream_and_a_captured_call():
    run, (out, lse, do, dlse), _ = case("dense", 4, 2, 128, True, BF16)
    ref = run(out, lse, do, dlse)
    o, d, l = transposed(out), transposed(do), apart(dlse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a = run(o, lse, d, l, stream=side)
    side.synchronize()
    same(ref, a)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b = run(o, lse, d, l)
    d.neg_()  # replayed on new values: the copies are part of the graph
    l.neg_()
    graph.replay()
    same([-x for x in ref], b)


def test_what_stays_refused():
    run, (out, lse, do, dlse), (q, k, v) = case("dense", 4, 2, 128, True, BF16)
    for bad in ((out.half(), lse, do, dlse), (transposed(out)[:, :-1], lse, do, dlse), (out, lse, transposed(do).float(), dlse),
                (out, apart(lse)[..., :-1], do, dlse), (transposed(out).cpu(), lse, do, dlse), (out, lse, do.cpu(), dlse)):
        with pytest.raises(ValueError):
            run(*bad)
    with pytest.raises(ValueError, match="contiguous"):
        gb.attn_bwd_dense(transposed(q), k, v, out, lse, do)
    with pytest.raises(gb.GbattnError):  # a gradient within what `out` reaches over
        room = torch.empty(4 * out.numel(), dtype=BF16, device=dev())
        B, S, H, D = out.shape
        o = room.as_strided(out.shape, (2 * S * H * D, D, S * D, 1)).copy_(out)
        run(o, lse, do, dlse, dq=room[S * H * D:][:out.numel()].view(out.shape))


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
def test_fp32_rows_on_16_bytes_and_rows_of_no_document(D):
    """An fp32 `out` whose rows are D + 4 apart, packed, with rows behind the last document that are no numbers."""
    g = torch.Generator().manual_seed(D)
    lens, Hq, Hkv, s, tail = [90, 1, 140], 6, 3, D ** -0.5, 20
    T = sum(lens) + tail
    q, k, v, do = randn(g, T, Hq, D), randn(g, T, Hkv, D), randn(g, T, Hkv, D), randn(g, T, Hq, D)
    cu = workloads.cu_from_lengths(lens).to(dev())
    out, lse = gb.attn_fwd_varlen(q, k, v, cu, cu, 140, 140, s, True, lse=True, out_dtype=torch.float32)
    wide = torch.full((T, Hq, D + 4), float("nan"), device=dev())
    wide[:-tail, :, 4:] = out[:-tail]

    def run(o):
        grads = [torch.full_like(x, 777.0) for x in (q, k, v)]
        return gb.attn_bwd_varlen(q, k, v, o, lse, do, cu, cu, 140, 140, s, True, dq=grads[0], dk=grads[1], dv=grads[2])

    got = run(wide[..., 4:])
    same(run(out), got)
    assert all(bool((x[-tail:] == 777.0).all()) for x in got)
