"""attn_rotary and attn_rotary_kv_cache_write against the float64 oracle, each
value within the bound of oracle/rotary.py; what is not turned has to be equal."""

import numpy as np
import pytest
import torch

import attention_forward_09_gb300 as gb
import oracle
import workloads
from _helpers import assert_close, dev, status_word, to_np

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_09_gb300 import _build

    _build.build()
    gb.load_library()


def check(got, x, pos, plan, what, transpose=False):
    r, b = oracle.rotary(x, pos.cpu().numpy(), plan.inv_freq, plan.rot_dim, plan.interleaved, plan.gain, transpose, True)
    g = to_np(got)
    assert g.shape == r.shape
    bad = ~(np.abs(g - r) <= b)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} values off, first at {np.argwhere(bad)[0]}"


def inputs(T, Hq, Hkv, D, far=4096, fused=False, seed=0):
    g = torch.Generator().manual_seed(seed + T + D)
    if fused:
        x = workloads.randn_bf16(g, T, Hq + 2 * Hkv, D).to(dev())
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    else:
        q, k, v = (workloads.randn_bf16(g, T, h, D).to(dev()) for h in (Hq, Hkv, Hkv))
    return q, k, v, torch.randint(-far, far, (T,), generator=g).to(torch.int32).to(dev())


ROTS = [(64, 64), (64, 20), (64, 2), (96, 96), (96, 48), (96, 24), (128, 128), (128, 64), (128, 126), (192, 192), (192, 12),
        (256, 256), (256, 128)]


@pytest.mark.parametrize("D,rot", ROTS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (5, 6, 2), (67, 8, 8), (700, 3, 1)])
def test_turned(D, rot, interleaved, T, Hq, Hkv):
    q, k, _, pos = inputs(T, Hq, Hkv, D)
    plan = gb.RotaryPlan(rot, interleaved=interleaved, gain=1.25)
    a, b = gb.attn_rotary(q, k, pos, plan)
    check(a, q, pos, plan, "q")
    check(b, k, pos, plan, "k")
    a, b = gb.attn_rotary(q, k, pos, plan, transpose=True)
    check(a, q, pos, plan, "q back", True)
    check(b, k, pos, plan, "k back", True)


@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True), (20, False)])
def test_far_positions(rot, interleaved):
    """Every 32-bit position, the extremes among them: an fp32 angle would be off by whole turns."""
    q, k, _, _ = inputs(300, 2, 1, 128)
    g = torch.Generator().manual_seed(1)
    pos = torch.randint(-2 ** 31, 2 ** 31 - 1, (300,), generator=g)
    pos[:4] = torch.tensor([2 ** 31 - 1, -2 ** 31, 0, 1])
    pos = pos.to(torch.int32).to(dev())
    plan = gb.RotaryPlan(rot, interleaved=interleaved)
    a, b = gb.attn_rotary(q, k, pos, plan)
    check(a, q, pos, plan, "q")
    check(b, k, pos, plan, "k")
    assert torch.equal(a[2], q[2])  # position 0 turns nothing


@pytest.mark.parametrize("scaling", [dict(kind="linear", factor=3.0), dict(kind="ntk", factor=8.0),
                                     dict(kind="by_parts", factor=8.0, low=1.0, high=4.0, length=8192),
                                     dict(kind="yarn", factor=4.0, low=1.0, high=32.0, length=8192)])
def test_scaled_for_long_contexts(scaling):
    q, k, _, pos = inputs(200, 4, 2, 128, far=1 << 20)
    plan = gb.RotaryPlan(128, base=5e5, scaling=scaling)
    a, b = gb.attn_rotary(q, k, pos, plan)
    check(a, q, pos, plan, "q")
    check(b, k, pos, plan, "k")


@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (96, 20)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strided_in_place_and_single(D, rot, interleaved):
    q, k, v, pos = inputs(130, 6, 2, D, fused=True)
    plan = gb.RotaryPlan(rot, interleaved=interleaved)
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    a, b = gb.attn_rotary(q, k, pos, plan)  # strided in, packed out
    check(a, q0, pos, plan, "q")
    check(b, k0, pos, plan, "k")
    c, d = gb.attn_rotary(q, None, pos, plan)
    assert torch.equal(c, a) and d is None
    wide = torch.full((130, 9, D), 5.0, dtype=BF16, device=dev())
    gb.attn_rotary(q, k, pos, plan, q_out=wide[:, 1:7], k_out=k)  # strided out; one of the two in place
    assert torch.equal(wide[:, 1:7], a) and torch.equal(k, b)
    assert bool((wide[:, 0] == 5).all()) and bool((wide[:, 7:] == 5).all())
    k.copy_(k0)
    c, d = gb.attn_rotary(q, k, pos, plan, q_out=q, k_out=k)  # in place, the values beside them untouched
    assert c is q and d is k and torch.equal(q, a) and torch.equal(k, b) and torch.equal(v, v0)


def test_values_that_are_not_finite_stay_in_their_pair():
    q, _, _, pos = inputs(40, 2, 1, 64)
    plan = gb.RotaryPlan(32)
    ref, _ = gb.attn_rotary(q, None, pos, plan)
    q[3, 1, 5], q[7, 0, 40], q[9, 0, 20] = float("nan"), float("inf"), float("-inf")
    got, _ = gb.attn_rotary(q, None, pos, plan)
    bad = torch.zeros(q.shape, dtype=torch.bool, device=dev())
    for t, h, i in ((3, 1, 5), (3, 1, 21), (7, 0, 40), (9, 0, 20), (9, 0, 4)):
        bad[t, h, i] = True
    assert torch.equal(got[~bad], ref[~bad]) and bool(got[7, 0, 40] == float("inf")) and bool(got[3, 1, 5].isnan())


@pytest.mark.parametrize("D,rot", [(64, 64), (96, 48), (128, 128), (128, 20), (192, 192), (256, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,bs,fused", [(1, 128, False), (67, 16, True), (900, 128, True)])
def test_stored(D, rot, interleaved, T, bs, fused):
    Hq, Hkv = 6, 2
    q, k, v, pos = inputs(T, Hq, Hkv, D, fused=fused)
    nb = -(-T // bs) + 2
    slots = torch.randperm(nb * bs, generator=torch.Generator().manual_seed(T))[:T].to(torch.int32)
    slots[::7] = -1
    slots = slots.to(dev())
    plan = gb.RotaryPlan(rot, interleaved=interleaved)
    cache = torch.full((2, nb, bs, Hkv, D), 3.0, dtype=BF16, device=dev())
    want = cache.clone()
    ref_q, ref_k = gb.attn_rotary(q, k, pos, plan)
    gb.attn_kv_cache_write(ref_k, v.contiguous(), slots, want)
    st = status_word()
    got = gb.attn_rotary_kv_cache_write(q, k, v, pos, plan, slots, cache, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0 and torch.equal(got, ref_q) and torch.equal(cache, want)
    check(ref_k, k, pos, plan, "k")
    again = gb.attn_rotary_kv_cache_write(q, k, v, pos, plan, slots, cache, q_out=q)  # in place
    assert again is q and torch.equal(q, ref_q) and torch.equal(cache, want)


def test_slots_past_the_cache_are_skipped_and_reported():
    q, k, v, pos = inputs(20, 4, 2, 128)
    plan = gb.RotaryPlan(128)
    slots = torch.arange(20, dtype=torch.int32)
    slots[5], slots[9] = 64, 2 ** 31 - 1
    cache, want = (torch.zeros(2, 4, 16, 2, 128, dtype=BF16, device=dev()) for _ in range(2))
    st = status_word()
    got = gb.attn_rotary_kv_cache_write(q, k, v, pos, plan, slots.to(dev()), cache, dev_status=st)
    ref_q, ref_k = gb.attn_rotary(q, k, pos, plan)
    slots[5] = slots[9] = -1
    gb.attn_kv_cache_write(ref_k, v, slots.to(dev()), want)
    torch.cuda.synchronize()
    assert int(st.item()) == gb.DEV_BAD_INDEX and torch.equal(got, ref_q) and torch.equal(cache, want)


def test_a_decode_step_as_it_is_used():
    """Positions turned and stored, then attended through the paged cache: equal to attention on the oracle's turned rows."""
    lens, Hq, Hkv, D = [1, 130, 300], 8, 2, 128
    T, plan = sum(lens), gb.RotaryPlan(128, scaling=dict(kind="linear", factor=2.0))
    q, k, v, _ = inputs(T, Hq, Hkv, D, fused=True)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).to(dev())
    table = torch.tensor([[4, -1, -1], [2, 0, -1], [5, 1, 3]], dtype=torch.int32)
    slots = torch.cat([table[s, torch.arange(n) // 128] * 128 + torch.arange(n) % 128 for s, n in enumerate(lens)]).to(torch.int32)
    cache = torch.zeros(2, 6, 128, Hkv, D, dtype=BF16, device=dev())
    st = status_word()
    qr = gb.attn_rotary_kv_cache_write(q, k, v, pos, plan, slots.to(dev()), cache, dev_status=st)
    last = torch.tensor(lens).cumsum(0) - 1
    out, lse = gb.attn_fwd_paged(qr[last.to(dev())].contiguous(), cache, table.to(dev()),
                                 torch.tensor(lens, dtype=torch.int32, device=dev()), max(lens), lse=True, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    at = 0
    for s, n in enumerate(lens):
        kr = oracle.rotary(k[at:at + n], pos[at:at + n].cpu().numpy(), plan.inv_freq, 128)
        qo = oracle.rotary(q[at + n - 1:at + n], [n - 1], plan.inv_freq, 128)
        r = torch.from_numpy(kr).to(BF16), torch.from_numpy(qo).to(BF16)  # rounded as they are stored
        ro, rl = oracle.attention_single(r[1], r[0], v[at:at + n].cpu(), D ** -0.5, True)
        assert_close(out[s:s + 1], None, ro, None, out_tol=2e-2, what=f"sequence {s}")
        at += n


def test_a_training_step_as_it_is_used():
    """q and k turned, attended, the gradients taken and turned back: against the oracle's chain on the same rounded steps."""
    lens, Hq, Hkv, D, s = [150, 41], 4, 2, 64, 0.125
    T, plan = sum(lens), gb.RotaryPlan(64, interleaved=True)
    q, k, v, _ = inputs(T, Hq, Hkv, D)
    do = inputs(T, Hq, Hkv, D, seed=9)[0]
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).to(dev())
    cu = workloads.cu_from_lengths(lens).to(dev())
    qr, kr = gb.attn_rotary(q, k, pos, plan)
    out, lse = gb.attn_fwd_varlen(qr, kr, v, cu, cu, max(lens), max(lens), s, True, lse=True, out_dtype=BF16)
    dq, dk, dv = gb.attn_bwd_varlen(qr, kr, v, out, lse, do, cu, cu, max(lens), max(lens), s, True)
    gq, gk = gb.attn_rotary(dq, dk, pos, plan, transpose=True)
    at = 0
    for n in lens:
        i = slice(at, at + n)
        ref = oracle.attention_gradients(qr[i], kr[i], v[i], out[i], lse[:, i], do[i], s, True, bounds=True)
        for name, x, (r, b) in (("dq", dq, ref[0]), ("dk", dk, ref[1]), ("dv", dv, ref[2])):
            assert np.all(np.abs(to_np(x[i]) - r) <= b), name
        check(gq[i], dq[i], pos[i], plan, "dq back", True)
        check(gk[i], dk[i], pos[i], plan, "dk back", True)
        at += n


def test_another_stream_a_captured_call_and_no_tokens():
    q, k, v, pos = inputs(70, 4, 2, 128)
    plan = gb.RotaryPlan(128)
    a = gb.attn_rotary(q, k, pos, plan)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = gb.attn_rotary(q, k, pos, plan, stream=side)
    side.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    graph = torch.cuda.CUDAGraph()
    cache = torch.zeros(2, 1, 128, 2, 128, dtype=BF16, device=dev())
    slots = torch.arange(70, dtype=torch.int32, device=dev())
    with torch.cuda.graph(graph):
        c = gb.attn_rotary_kv_cache_write(q, k, v, pos, plan, slots, cache)
    pos.add_(5)  # replayed for the next positions and slots
    slots.add_(3)
    graph.replay()
    a = gb.attn_rotary(q, k, pos, plan)
    torch.cuda.synchronize()
    assert torch.equal(c, a[0]) and torch.equal(cache[0].view(128, 2, 128)[3:73], a[1])
    assert torch.equal(cache[1].view(128, 2, 128)[3:73], v) and not cache[0].view(128, 2, 128)[:3].any()
    e = q[:0]
    assert gb.attn_rotary(e, k[:0], pos[:0], plan)[0].shape == e.shape


def test_refusals_of_the_binding():
    q, k, v, pos = inputs(6, 4, 2, 128)
    plan = gb.RotaryPlan(128)
    cache = torch.zeros(2, 1, 16, 2, 128, dtype=BF16, device=dev())
    slots = torch.arange(6, dtype=torch.int32, device=dev())
    for kw in (dict(q=q.float()), dict(q=q[0]), dict(q=q[:, ::2]), dict(k=k[:5]), dict(k=k[..., :64]), dict(k=k.cpu()),
               dict(positions=pos.long()), dict(positions=pos[:5]), dict(q_out=q[:5]), dict(k_out=q), dict(k=None, k_out=k),
               dict(plan=gb.RotaryPlan(128, device="cpu"))):
        with pytest.raises(ValueError):
            gb.attn_rotary(**{**dict(q=q, k=k, positions=pos, plan=plan), **kw})
    with pytest.raises(gb.GbattnError):
        gb.attn_rotary(q, k, pos, gb.RotaryPlan(256))  # wider than the head
    with pytest.raises(gb.GbattnError):
        gb.attn_rotary(q, k, pos, plan, q_out=q[:1].expand(6, 4, 128))
    for kw in (dict(value=v[:5]), dict(value=q), dict(slot_mapping=slots.long()), dict(kv_cache=cache[0]),
               dict(kv_cache=cache.float()), dict(kv_cache=cache[..., :1, :]), dict(dev_status=cache)):
        with pytest.raises(ValueError):
            gb.attn_rotary_kv_cache_write(**{**dict(q=q, key=k, value=v, positions=pos, plan=plan, slot_mapping=slots,
                                                    kv_cache=cache), **kw})


@pytest.mark.parametrize("interleaved", [False, True])
def test_offsets_past_32_bits(interleaved):
    """Element offsets beyond 2^31 in queries, outputs and the cache."""
    T, Hq, Hkv, D = 300000, 52, 52, 128
    assert T * Hq * D < 2 ** 31 < T * (Hq + 2 * Hkv) * D and 2 * T * Hkv * D > 2 ** 31
    g = torch.Generator(device=dev()).manual_seed(3)
    x = torch.empty(T, Hq + 2 * Hkv, D, device=dev(), dtype=BF16)
    for i in range(0, T, 50000):
        x[i:i + 50000].normal_(generator=g)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    pos = torch.arange(T, dtype=torch.int32, device=dev())
    slots = pos.flip(0).contiguous()
    cache = torch.zeros(2, T // 100, 100, Hkv, D, dtype=BF16, device=dev())
    plan = gb.RotaryPlan(64, interleaved=interleaved)
    a = gb.attn_rotary_kv_cache_write(q, k, v, pos, plan, slots, cache)
    torch.cuda.synchronize()
    rows = [0, 1, T // 2, T - 2, T - 1]
    check(a[rows], q[rows], pos[rows], plan, "q")
    keys, values = cache.view(2, T, Hkv, D)
    check(keys[slots[rows].long()], k[rows], pos[rows], plan, "k")
    assert torch.equal(values[slots[rows].long()], v[rows]) and torch.equal(values.flip(0), v)
    b, c = gb.attn_rotary(q, k, pos, plan, q_out=q, k_out=k)  # in place, in the strided tensor
    assert torch.equal(b, a) and torch.equal(c.flip(0), keys) and b is q


def test_outputs_over_other_inputs_are_refused_and_neighbours_are_not():
    g = torch.Generator().manual_seed(10)
    T, H, D = 33, 4, 64
    fused = torch.randn(T, 4, H, D, generator=g).to(torch.bfloat16).cuda()
    q, k, qo, ko = fused.unbind(1)
    pos, plan = torch.arange(T, dtype=torch.int32, device="cuda"), gb.RotaryPlan(D)
    ref = gb.attn_rotary(q, k, pos, plan)
    gb.attn_rotary(q, k, pos, plan, q_out=qo, k_out=ko)
    assert torch.equal(qo, ref[0]) and torch.equal(ko, ref[1])
    for q_out, k_out in ((k, q), (k, None), (None, q), (qo, qo), (q.as_strided((T, H, D), (H * D, D, 1)), None)):
        with pytest.raises(gb.GbattnError):
            gb.attn_rotary(q, k, pos, plan, q_out=q_out, k_out=k_out)
    gb.attn_rotary(q, k, pos, plan, q_out=q, k_out=k)
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1])
