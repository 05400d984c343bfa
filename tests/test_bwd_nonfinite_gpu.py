"""Values that are not finite, within one document or batch entry: the gradients
of the others keep their bits."""

import pytest
import torch

import attention_forward_09_gb300 as gb
import workloads
from _helpers import dev, status_word
from test_bwd_gpu import randn

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_09_gb300 import _build

    _build.build()
    gb.load_library()


@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("which", ["q", "k", "v", "dout", "out"])
def test_one_row_stays_inside_its_document(which, value, D):
    """Row 90 of the second of three documents, causal: hidden from most of its rows, and in tiles with the neighbours'."""
    g = torch.Generator().manual_seed(D)
    lens, Hq, Hkv, s = [100, 120, 90], 4, 2, D ** -0.5
    T = sum(lens)
    x = dict(q=randn(g, T, Hq, D), k=randn(g, T, Hkv, D), v=randn(g, T, Hkv, D), dout=randn(g, T, Hq, D))
    cu = workloads.cu_from_lengths(lens).to(dev())
    x["out"], lse = gb.attn_fwd_varlen(x["q"], x["k"], x["v"], cu, cu, 120, 120, s, True, lse=True, out_dtype=BF16)

    def run():
        st = status_word()
        got = gb.attn_bwd_varlen(x["q"], x["k"], x["v"], x["out"], lse, x["dout"], cu, cu, 120, 120, s, True, dev_status=st)
        torch.cuda.synchronize()
        assert int(st.item()) == 0
        return got

    ref = run()
    x[which][190] = value
    for a, b in zip(ref, run()):
        assert torch.equal(a[:100], b[:100]) and torch.equal(a[220:], b[220:])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_one_row_stays_inside_its_entry(D):
    g = torch.Generator().manual_seed(D)
    q, k, v, do = randn(g, 3, 150, 4, D), randn(g, 3, 150, 2, D), randn(g, 3, 150, 2, D), randn(g, 3, 150, 4, D)
    out, lse = gb.attn_fwd_dense(q, k, v, D ** -0.5, True, lse=True, out_dtype=BF16)
    ref = gb.attn_bwd_dense(q, k, v, out, lse, do, D ** -0.5, True)
    for t in (q, k, v, do):
        t[1, 140] = float("nan")
    for a, b in zip(ref, gb.attn_bwd_dense(q, k, v, out, lse, do, D ** -0.5, True)):
        assert torch.equal(a[::2], b[::2])
