"""The 8-bit paged KV cache on the CPU: the oracle's code formats and rounding
against torch's float8 types and hand-worked rows, and what the entry points
refuse before they touch a device."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import attention_forward_09_gb300 as gb
import oracle
from attention_forward_09_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
DTYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
NAMES = ["attn_fwd_paged_fp8", "attn_fwd_paged_fp8_workspace_size", "attn_kv_cache_read_fp8",
         "attn_kv_cache_write_fp8"]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gb.load_library()


# ---------------------------------------------------------------- the oracle's pins
@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_code_values_are_those_of_the_float8_types(kind):
    want = torch.arange(256, dtype=torch.uint8).view(DTYPES[kind]).float().double().numpy()
    np.testing.assert_array_equal(oracle.code_values(kind), want)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_rounding_is_that_of_the_float8_types(kind):
    """Rows whose largest value is the format's own c_max have e = 0, so their
    codes are torch's conversion; values on every edge between two codes too."""
    pos = oracle.code_values(kind)[:128]
    pos = pos[np.isfinite(pos)]
    x = np.concatenate([pos, (pos[1:] + pos[:-1]) / 2, np.random.default_rng(0).uniform(0, pos[-1], 500).astype(np.float32)])
    x = np.concatenate([x, -x])[None]
    c, b = oracle.quantise_rows(x, kind)
    assert b[0] == 127
    want = torch.from_numpy(x).float().to(DTYPES[kind]).view(torch.uint8).numpy()
    assert np.array_equal(c, want)


def test_quantise_hand_worked_rows():
    nan, inf = float("nan"), float("inf")
    x = np.array([[448.0, 1.0, 0.0, -448.0],        # e = 0
                  [448.5, 1.0, 0.0, -2.0],          # just above: e = 1
                  [0.0, -0.0, 0.0, 0.0],            # e = -126
                  [nan, 1.75, inf, -inf],           # non-finite: NaN codes, not in the maximum: 1.75 = 448 * 2^-8
                  [2.0 ** -133, 0.0, 0.0, 0.0]])    # below every row scale: e = -126
    c, b = oracle.quantise_rows(x, "e4m3")
    v = oracle.code_values("e4m3")[c]
    assert b.tolist() == [127, 128, 1, 119, 1]
    np.testing.assert_array_equal(v[0], [448.0, 1.0, 0.0, -448.0])
    np.testing.assert_array_equal(v[1], [224.0, 0.5, 0.0, -1.0])
    np.testing.assert_array_equal(v[2], 0.0)
    assert np.isnan(v[3, [0, 2, 3]]).all() and v[3, 1] == 448.0
    np.testing.assert_array_equal(v[4], [2.0 ** -7, 0, 0, 0])


# ---------------------------------------------------------------- the boundary
def test_declared_exported_and_bound(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gbattn.h")).read(), flags=re.S)
    assert sorted(set(re.findall(r"\b(attn_\w*fp8\w*)\s*\(", text))) == NAMES
    for n in NAMES:
        assert hasattr(lib, n) and n in gb.SIGNATURES


P = ctypes.c_void_p(0x10000)  # a fake aligned "device" address: every case fails, or is a no-op, before any use
ODD = ctypes.c_void_p(0x10008)


def write(lib, **kw):
    a = dict(key=P, value=P, ks=1024, vs=1024, slots=P, T=4, cache=P, scales=P, kv=0, nb=8, bs=128, Hkv=8, D=128)
    a.update(kw)
    return lib.attn_kv_cache_write_fp8(*a.values(), None, None)


def test_write_validation(lib):
    assert write(lib, D=80) == UNSUPPORTED
    assert write(lib, kv=2) == UNSUPPORTED
    assert write(lib, nb=1 << 25) == UNSUPPORTED  # 2^32 slots
    assert write(lib, Hkv=1 << 24) == UNSUPPORTED
    for bad in (dict(T=-1), dict(nb=0), dict(bs=0), dict(Hkv=0), dict(ks=1016), dict(vs=0), dict(key=None),
                dict(value=None), dict(slots=None), dict(cache=None), dict(scales=None)):
        assert write(lib, **bad) == INVALID, bad
    for bad in (dict(key=ODD), dict(value=ODD), dict(cache=ODD), dict(scales=ODD), dict(ks=1028), dict(vs=1025)):
        assert write(lib, **bad) == ALIGN, bad
    assert write(lib, T=0) == OK
    assert write(lib, T=0, key=None, value=None, slots=None) == OK


def read(lib, **kw):
    a = dict(cache=P, scales=P, kv=0, nb=8, bs=128, bt=P, maxb=4, cu=P, S=2, Tk=100, Hkv=8, D=128, k=P, v=P)
    a.update(kw)
    return lib.attn_kv_cache_read_fp8(*a.values(), None, None)


def test_read_validation(lib):
    assert read(lib, D=100) == UNSUPPORTED
    assert read(lib, kv=-1) == UNSUPPORTED
    assert read(lib, Tk=0x7FFFFFFF) == UNSUPPORTED
    for bad in (dict(S=-1), dict(Tk=-1), dict(maxb=0), dict(nb=0), dict(bs=-1), dict(Hkv=0), dict(cache=None),
                dict(scales=None), dict(bt=None), dict(cu=None), dict(k=None), dict(v=None)):
        assert read(lib, **bad) == INVALID, bad
    for bad in (dict(cache=ODD), dict(scales=ODD), dict(k=ODD), dict(v=ODD)):
        assert read(lib, **bad) == ALIGN, bad
    assert read(lib, S=0) == OK and read(lib, Tk=0) == OK


def paged(lib, **kw):
    a = dict(q=P, qs=4096, cache=P, scales=P, kv=0, nb=16, bs=128, bt=P, maxb=4, sl=P, S=2, maxlen=8192, Hq=32, Hkv=8,
             D=128, scale=0.1, causal=1, out=P, odt=1, lse=None, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.attn_fwd_paged_fp8(*a.values(), None, None)


def test_paged_validation(lib):
    for bad in (dict(bs=64), dict(D=48), dict(kv=3), dict(odt=7), dict(nb=1 << 24)):
        assert paged(lib, **bad) == UNSUPPORTED, bad
    for bad in (dict(q=None), dict(cache=None), dict(scales=None), dict(bt=None), dict(sl=None), dict(out=None),
                dict(Hq=12), dict(Hkv=0), dict(Hq=0), dict(scale=0.0), dict(scale=float("inf")), dict(maxb=0),
                dict(S=-1), dict(maxlen=-1), dict(nb=0), dict(qs=4088)):
        assert paged(lib, **bad) == INVALID, bad
    for bad in (dict(q=ODD), dict(cache=ODD), dict(scales=ODD), dict(out=ODD), dict(qs=4100)):
        assert paged(lib, **bad) == ALIGN, bad
    assert paged(lib, ws=None) == WORKSPACE
    assert paged(lib, wsb=16) == WORKSPACE
    assert paged(lib, ws=ctypes.c_void_p(0x10010)) == WORKSPACE  # must be 256-byte aligned
    assert paged(lib, S=0) == OK


def test_workspace_size_is_pure(lib):
    size = lib.attn_fwd_paged_fp8_workspace_size
    assert size(0, 8, 8, 128, 100) == 0 and size(1, 8, 3, 128, 100) == 0 and size(1, 8, 8, 100, 100) == 0
    assert size(1, 32, 8, 128, 128) == 0  # one block: nothing to join
    assert size(1, 32, 8, 128, 4096) == 0  # a cluster of CTAs joins on chip
    a = size(64, 32, 8, 128, 32768)
    assert a == size(64, 32, 8, 128, 32768) > 0
    assert size(64, 32, 8, 128, 131072) == a  # by the card's size, not the context's


def _args(T=5, Hkv=2, D=64, bs=128, nb=3, kv=torch.float8_e4m3fn):
    return dict(key=torch.zeros(T, Hkv, D, dtype=torch.bfloat16), value=torch.zeros(T, Hkv, D, dtype=torch.bfloat16),
                slots=torch.zeros(T, dtype=torch.int32), cache=torch.zeros(2, nb, bs, Hkv, D).to(kv),
                scales=torch.zeros(2, nb, Hkv, bs, dtype=torch.uint8))


@pytest.mark.parametrize("change, message", [
    (dict(cache=torch.zeros(2, 3, 128, 2, 64, dtype=torch.bfloat16)), "float8"),
    (dict(cache=torch.zeros(3, 128, 2, 64).to(torch.float8_e5m2)), "kv_cache"),
    (dict(scales=torch.zeros(2, 3, 128, 2, dtype=torch.uint8)), "kv_scales"),
    (dict(scales=torch.zeros(2, 3, 2, 128)), "kv_scales"),
    (dict(key=torch.zeros(5, 2, 64)), "key"),
    (dict(value=torch.zeros(5, 3, 64, dtype=torch.bfloat16)), "value"),
    (dict(key=torch.zeros(5, 64, 2, dtype=torch.bfloat16).transpose(1, 2)), "contiguous"),
    (dict(slots=torch.zeros(5, dtype=torch.int64)), "slot_mapping"),
    (dict(slots=torch.zeros(4, dtype=torch.int32)), "token count"),
    (dict(), "CUDA"),
])
def test_write_binding_refuses(lib, change, message):
    a = {**_args(), **change}
    with pytest.raises(ValueError, match=message):
        gb.attn_kv_cache_write_fp8(a["key"], a["value"], a["slots"], a["cache"], a["scales"])


@pytest.mark.parametrize("change, message", [
    (dict(bt=torch.zeros(1, 2, dtype=torch.int64)), "block_table"),
    (dict(bt=torch.zeros(2, 2, dtype=torch.int32)), "row"),
    (dict(cu=torch.zeros(2)), "cu_seqlens_k"),
    (dict(cu=torch.zeros(0, dtype=torch.int32)), "boundary"),
    (dict(), "CUDA"),
])
def test_read_binding_refuses(lib, change, message):
    a = {**_args(), "bt": torch.zeros(1, 2, dtype=torch.int32), "cu": torch.zeros(2, dtype=torch.int32), **change}
    with pytest.raises(ValueError, match=message):
        gb.attn_kv_cache_read_fp8(a["cache"], a["scales"], a["bt"], a["cu"], 10)


@pytest.mark.parametrize("change, message", [
    (dict(q=torch.zeros(1, 128, dtype=torch.bfloat16)), "q must be"),
    (dict(q=torch.zeros(1, 4, 96, dtype=torch.bfloat16)), "q must be"),
    (dict(q=torch.zeros(1, 4, 64)), "q must be"),
    (dict(bt=torch.zeros(1, 4, dtype=torch.int32)[:, ::2]), "block_table"),
    (dict(sl=torch.zeros(2, dtype=torch.int32)), "seq_lens"),
    (dict(status=torch.zeros(1, dtype=torch.uint8)), "dev_status"),
    (dict(), "CUDA"),
])
def test_paged_binding_refuses(lib, change, message):
    a = {**_args(), "q": torch.zeros(1, 4, 64, dtype=torch.bfloat16), "bt": torch.zeros(1, 2, dtype=torch.int32),
         "sl": torch.zeros(1, dtype=torch.int32), "status": None, **change}
    with pytest.raises(ValueError, match=message):
        gb.attn_fwd_paged_fp8(a["q"], a["cache"], a["scales"], a["bt"], a["sl"], 256, dev_status=a["status"])


@pytest.mark.parametrize("change, message", [
    (dict(q=torch.zeros(3, 4, 64)), "q must be"),
    (dict(q=torch.zeros(3, 4, 96, dtype=torch.bfloat16)), "q must be"),
    (dict(q=torch.zeros(3, 64, 4, dtype=torch.bfloat16).transpose(1, 2)), "q must be"),
    (dict(cu_q=torch.zeros(2, dtype=torch.int64)), "cu_seqlens_q"),
    (dict(cu_q=torch.zeros(3, dtype=torch.int32)), "boundaries"),
    (dict(out=torch.zeros(2, 4, 64)), "out must be"),
    (dict(lse=torch.zeros(3, 4)), "lse must be"),
    (dict(most=2 ** 31), "max_seqlen_q"),
    (dict(), "CUDA"),
])
def test_paged_prefill_binding_refuses(lib, change, message):
    a = {**_args(), "q": torch.zeros(3, 4, 64, dtype=torch.bfloat16), "bt": torch.zeros(1, 2, dtype=torch.int32),
         "cu": torch.zeros(2, dtype=torch.int32), "cu_q": torch.zeros(2, dtype=torch.int32), "out": None, "lse": None,
         "most": 3, **change}
    with pytest.raises(ValueError, match=message):
        gb.attn_fwd_paged_prefill_fp8(a["q"], a["cache"], a["scales"], a["bt"], a["cu_q"], a["cu"], 10, a["most"], 256,
                                      out=a["out"], lse=a["lse"])
