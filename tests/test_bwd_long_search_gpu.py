"""Many short documents under a long bound: the gradients' producers look at many
empty items between two that have work, for longer than a pipeline wait may
last.  A search is not a stalled pipeline: no wait runs out, and every document
gets its gradients."""

import pytest
import torch

import attention_forward_09_gb300 as gb
import oracle
from _helpers import dev, status_word
from test_bwd_gpu import check

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_09_gb300 import _build

    _build.build()
    gb.load_library()


def many(short, long_rows, bound, D=64):
    """`short` documents of one row around one of `long_rows`, causal, one head, key tiles of a document of `bound` rows."""
    g = torch.Generator(device=dev()).manual_seed(short)
    lens = [1] * short
    at = short // 3
    lens.insert(at, long_rows)
    T = sum(lens)
    cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).to(dev())
    q, do = (torch.randn(T, 1, D, generator=g, device=dev()).to(BF16) for _ in range(2))
    k, v = (torch.randn(max(T, bound), 1, D, generator=g, device=dev()).to(BF16) for _ in range(2))
    s = D ** -0.5
    # a row alone: out = v, lse = its score; the long document by the forward call
    out, lse = v[:T].clone(), ((q.double() * k[:T].double()).sum(-1) * s).float().t().contiguous()
    i = slice(at, at + long_rows)
    o, l = gb.attn_fwd_dense(q[i][None], k[i][None], v[i][None], s, True, lse=True, out_dtype=BF16)
    out[i], lse[:, i] = o[0], l[0]
    grads = [torch.full_like(x, 777.0) for x in (q, k, v)]
    st = status_word()
    gb.attn_bwd_varlen(q, k, v, out, lse, do, cu, cu, long_rows, bound, s, True, dq=grads[0], dk=grads[1], dv=grads[2],
                       dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    # a row alone: p = 1 in bf16, so dv = dout
    short_rows = torch.ones(T, dtype=torch.bool, device=dev())
    short_rows[i] = False
    assert torch.equal(grads[2][:T][short_rows], do[short_rows])
    assert all(bool((x[T:] == 777.0).all()) for x in grads[1:])
    for j in (i, slice(0, 1), slice(T - 1, T), slice(at - 1, at), slice(at + long_rows, at + long_rows + 1)):
        ref = oracle.attention_gradients(q[j], k[j], v[j], out[j], lse[:, j], do[j], s, True, bounds=True)
        check([x[j] for x in grads], ref, f"rows {j}")


def test_a_search_of_some_thousand_items():
    """Each of 152 CTAs passes over some 27000 empty items before its first one: several rests on the way."""
    many(4000, 300, 1024 * 128)


def test_a_search_that_takes_longer_than_a_wait_may():
    """5.4e8 empty items, 3.5 million a CTA at half a microsecond each: 1.65 s before the first item."""
    many(65534, 300, 8192 * 128)
