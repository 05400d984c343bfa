"""A CTA begins nothing once an earlier one gave up a wait (GBATTN_DEV_TIMEOUT in
dev_status).  Other CTAs may set the bit while a CTA's threads look at the word,
so one thread looks and the CTA shares its answer: threads that each looked for
themselves could part, some leaving and some going on without the barriers and
the tensor memory that those were to set up."""

import glob
import os
import re

import pytest
import torch

import attention_forward_09_gb300 as gb
import workloads
from _helpers import dev

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "attention_forward_09_gb300", "csrc")


@pytest.mark.parametrize("name", sorted(os.path.basename(p) for p in glob.glob(os.path.join(CSRC, "*.cu*"))))
def test_one_thread_reads_the_word(name):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    for m in re.finditer(r"\bstatus_has_timeout\(", text):
        before = text[:m.start()].rstrip()
        assert before.endswith("threadIdx.x == 0 &&") or before.endswith("bool"), f"{name}: {text[m.start() - 60:m.end() + 30]!r}"


def test_a_kernel_shares_the_answer():
    """The kernels that may leave do so through the shared form."""
    for name, n in (("bwd.cu", 1), ("prefill.cu", 2), ("vsa.cu", 1), ("decode.cu", 1)):
        assert len(re.findall(r"\bcta_has_timeout\(p\.status, kDevTimeout\)", open(os.path.join(CSRC, name)).read())) == n, name


# ------------------------------------------------------------------ on the GPU
@pytest.fixture(scope="module")
def built():
    from attention_forward_09_gb300 import _build

    _build.build()
    gb.load_library()


def given_up():
    return torch.tensor([gb.DEV_TIMEOUT], dtype=torch.int32, device=dev())


def rows(seed, *shape):
    return workloads.randn_bf16(torch.Generator().manual_seed(seed), *shape).to(dev())


def left_alone(call, *outputs):
    """The call comes back with its outputs as they were and the word as it was; without the bit it writes them."""
    st = given_up()
    for x in outputs:
        x.fill_(777.0)
    call(st)
    torch.cuda.synchronize()
    assert int(st.item()) == gb.DEV_TIMEOUT
    assert all(bool((x == 777.0).all()) for x in outputs)
    st.zero_()
    call(st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    assert not any(bool((x == 777.0).any()) for x in outputs)


@pytest.mark.gpu
@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
def test_gradients_begin_nothing_after_a_give_up(built, D):
    q, k, v, do = (rows(i, 1, 300, 96, D) for i in range(4))
    out, lse = gb.attn_fwd_dense(q, k, v, lse=True, out_dtype=torch.bfloat16)
    grads = [torch.empty_like(q) for _ in range(3)]
    left_alone(lambda st: gb.attn_bwd_dense(q, k, v, out, lse, do, dq=grads[0], dk=grads[1], dv=grads[2], dev_status=st), *grads)


@pytest.mark.gpu
@pytest.mark.parametrize("D", workloads.HEAD_SIZES)
@pytest.mark.parametrize("S", [100, 700])
def test_prefill_begins_nothing_after_a_give_up(built, D, S):
    q, k, v = (rows(i, 2, S, 4, D) for i in range(3))
    out, lse = torch.empty(2, S, 4, D, device=dev()), torch.empty(2, 4, S, device=dev())
    left_alone(lambda st: gb.attn_fwd_dense(q, k, v, causal=True, out=out, lse=lse, dev_status=st), out, lse)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_block_sparse_begins_nothing_after_a_give_up(built, D):
    plan = gb.VsaPlan([100, 37], (5, 9, 10), device=dev())
    q, k, v = (rows(i, plan.tokens, 2, D) for i in range(3))
    qt, kt, vt = (gb.attn_gather_rows(x, plan.tile_index) for x in (q, k, v))
    pq, pk = gb.attn_vsa_pool(qt, plan.block_sizes), gb.attn_vsa_pool(kt, plan.block_sizes)
    kv_list, kv_num = gb.attn_vsa_block_map(pq, pk, plan.block_sizes, plan.num_prefix_blocks, 5, D ** -0.5)
    out = torch.empty(plan.tokens, 2, D, device=dev())
    left_alone(lambda st: gb.attn_fwd_vsa(qt, kt, vt, kv_list, kv_num, plan.num_blocks, plan.num_prefix_blocks, 5,
                                          out_index=plan.tile_index, out_rows=plan.tokens, out=out, dev_status=st), out)
