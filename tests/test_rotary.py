"""Rotary positions on the host: the oracle's pins, frequencies and scalings,
the fixed-point steps, and the refusals (no GPU call is made)."""

import ctypes
import math
import os
import re
from fractions import Fraction

import numpy as np
import pytest

import attention_forward_09_gb300 as gb
import oracle
from attention_forward_09_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIGN = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gb.load_library()


# ------------------------------------------------------------------ the oracle
def test_oracle_quarter_turns():
    x = np.arange(1.0, 7.0).reshape(1, 1, 6)
    f = [math.pi / 2, math.pi]
    y = oracle.rotary(x, [1], f, 4)[0, 0]
    assert np.allclose(y, [-3, -2, 1, -4, 5, 6], atol=1e-15)
    y = oracle.rotary(x, [1], f, 4, interleaved=True, gain=2.0)[0, 0]
    assert np.allclose(y, [-4, 2, -6, -8, 5, 6], atol=1e-15)
    y = oracle.rotary(x, [1], f, 4, transpose=True)[0, 0]
    assert np.allclose(y, [3, -2, -1, -4, 5, 6], atol=1e-15)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_products_depend_on_the_distance_alone_and_the_transpose_undoes(interleaved):
    rng = np.random.default_rng(1)
    q, k = rng.normal(size=(2, 1, 1, 16))
    f = [1.0, 0.3, 0.1, 0.02, 0.001]
    dots = [np.sum(oracle.rotary(q, [t + 11], f, 10, interleaved) * oracle.rotary(k, [t], f, 10, interleaved)) for t in (0, 5, 900)]
    assert np.allclose(dots, dots[0], rtol=0, atol=1e-12)
    y = oracle.rotary(oracle.rotary(q, [77], f, 10, interleaved), [77], f, 10, interleaved, transpose=True)
    assert np.allclose(y, q, atol=1e-14)
    # <R x, y> = <x, R^T y> with the gain: the transpose is the gradient
    a = np.sum(oracle.rotary(q, [9], f, 10, interleaved, 1.3) * k)
    b = np.sum(q * oracle.rotary(k, [9], f, 10, interleaved, 1.3, transpose=True))
    assert abs(a - b) < 1e-13


# ----------------------------------------------------------- frequencies, steps
@pytest.mark.parametrize("rot", [2, 20, 64, 128, 256])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies(lib, rot, base):
    f, gain = gb.attn_rotary_frequencies(rot, base)
    assert gain == 1.0 and len(f) == rot // 2
    want = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    assert np.allclose(f, want, rtol=1e-14)
    assert np.allclose(gb.attn_rotary_frequencies(rot, base, dict(kind="linear", factor=4.0))[0], want / 4, rtol=1e-14)
    if rot > 2:
        g, _ = gb.attn_rotary_frequencies(rot, base, dict(kind="ntk", factor=8.0))
        assert g[0] == 1.0 and math.isclose(g[-1], want[-1] / 8.0, rel_tol=1e-12)  # the slowest pair is slowed by s exactly


@pytest.mark.parametrize("kind,low,high", [("by_parts", 1.0, 4.0), ("yarn", 1.0, 32.0)])
def test_scalings_by_parts_keep_fast_pairs_and_slow_slow_ones(lib, kind, low, high):
    rot, base, length, s = 128, 10000.0, 8192, 4.0
    want = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    f, gain = gb.attn_rotary_frequencies(rot, base, dict(kind=kind, factor=s, low=low, high=high, length=length))
    f, turns = np.array(f), length * want / (2 * math.pi)
    assert np.allclose(f[turns > high * 1.2], want[turns > high * 1.2], rtol=1e-14)
    assert np.allclose(f[turns < low / 1.2], want[turns < low / 1.2] / s, rtol=1e-14)
    assert np.all(np.diff(f) < 0) and np.all(f <= want * (1 + 1e-14)) and np.all(f >= want / s * (1 - 1e-14))
    assert math.isclose(gain, 0.1 * math.log(4.0) + 1.0 if kind == "yarn" else 1.0, rel_tol=1e-15)
    mid = (turns > low) & (turns < high)
    assert mid.sum() > 5
    if kind == "by_parts":
        g = (turns[mid] - low) / (high - low)
        assert np.allclose(f[mid], want[mid] * (g + (1 - g) / s), rtol=1e-13)
    else:  # equal steps of the mixing share
        share = (f[mid] / want[mid] - 1 / s) / (1 - 1 / s)
        assert np.allclose(np.diff(share), np.diff(share)[0], atol=1e-12) and np.diff(share)[0] < 0


def test_steps_are_the_rounded_turns(lib):
    two_pi = Fraction(2 * 3141592653589793238462643383279502884197, 10 ** 39)
    f = [1.0, 0.5, 1e-3, 1e-7, 3.0, 6.0, 7.0, 100.0, 0.0, -1.0, -1e-5] + gb.attn_rotary_frequencies(128)[0]
    for x, s in zip(f, gb.attn_rotary_steps(f)):
        exact = Fraction(x) / two_pi * 2 ** 64
        off = (exact - s) % 2 ** 64
        off = min(off, 2 ** 64 - off)
        # the quotient, and 2 pi, rounded to 53 bits: 1.5 units of 2^-53 of the turns; then one rounding to an integer
        assert off <= abs(exact) * Fraction(3, 2) / 2 ** 52 + 1, x
    assert gb.attn_rotary_steps([]) == []


def test_plan_on_the_host(lib):
    p = gb.RotaryPlan(64, base=5e5, interleaved=True, scaling=dict(kind="yarn", factor=2.0, low=1.0, high=32.0, length=4096),
                      device="cpu")
    assert p.rot_dim == 64 and p.interleaved and math.isclose(p.gain, 0.1 * math.log(2.0) + 1.0)
    assert [int(x) % 2 ** 64 for x in p.steps] == gb.attn_rotary_steps(p.inv_freq)
    p = gb.RotaryPlan(4, inv_freq=[1.0, 0.25], gain=0.5, device="cpu")
    assert p.inv_freq == [1.0, 0.25] and p.gain == 0.5
    for bad in (dict(rot_dim=5), dict(rot_dim=0), dict(rot_dim=4, base=1.0), dict(rot_dim=4, base=float("nan")),
                dict(rot_dim=2, scaling=dict(kind="ntk", factor=2.0)), dict(rot_dim=4, scaling=dict(kind="linear", factor=0.5)),
                dict(rot_dim=4, scaling=dict(kind="yarn", factor=2.0, low=4.0, high=1.0, length=100)),
                dict(rot_dim=4, scaling=dict(kind="by_parts", factor=2.0, low=1.0, high=4.0, length=0)),
                dict(rot_dim=2, inv_freq=[float("inf")])):
        with pytest.raises(gb.GbattnError):
            gb.RotaryPlan(**bad, device="cpu")
    for bad in (dict(rot_dim=4, scaling=dict(kind="other", factor=2.0)), dict(rot_dim=4, scaling=dict(kind="linear")),
                dict(rot_dim=4, inv_freq=[1.0]), dict(rot_dim=2, inv_freq=[1.0], scaling=dict(kind="linear", factor=2.0))):
        with pytest.raises(ValueError):
            gb.RotaryPlan(**bad, device="cpu")


# ---------------------------------------------------------------- the boundary
def test_header_and_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gbattn_rotary.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(attn_\w+)\s*\(", text)))
    assert names == ["attn_rotary", "attn_rotary_frequencies", "attn_rotary_kv_cache_write", "attn_rotary_steps"]
    for n in names:
        assert hasattr(lib, n) and n in gb.SIGNATURES


P, OFF, NULL = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), None


def rotary(lib, **kw):
    a = dict(q=P, qs=512, k=P, ks=256, pos=P, T=4, steps=P, rot=128, il=0, tr=0, gain=1.0, Hq=4, Hkv=2, D=128, qo=P, qos=512,
             ko=P, kos=256)
    a.update(kw)
    return lib.attn_rotary(a["q"], a["qs"], a["k"], a["ks"], a["pos"], a["T"], a["steps"], a["rot"], a["il"], a["tr"],
                           a["gain"], a["Hq"], a["Hkv"], a["D"], a["qo"], a["qos"], a["ko"], a["kos"], None)


def store(lib, **kw):
    a = dict(q=P, qs=512, k=P, ks=256, v=P, vs=256, pos=P, slots=P, T=4, steps=P, rot=128, il=0, gain=1.0, qo=P, qos=512,
             cache=P, nb=4, bs=128, Hq=4, Hkv=2, D=128)
    a.update(kw)
    return lib.attn_rotary_kv_cache_write(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["pos"], a["slots"], a["T"],
                                          a["steps"], a["rot"], a["il"], a["gain"], a["qo"], a["qos"], a["cache"], a["nb"],
                                          a["bs"], a["Hq"], a["Hkv"], a["D"], None, None)


@pytest.mark.parametrize("call,outs", [(rotary, ("qo", "ko")), (store, ("qo", "cache"))])
def test_refusals(lib, call, outs):
    for n in ("q", "k", "pos", "steps") + outs:
        assert call(lib, **{n: NULL}) == INVALID, n
    for n in ("q", "k") + outs:
        assert call(lib, **{n: OFF}) == ALIGN, n
    assert call(lib, steps=ctypes.c_void_p(0x10004)) == ALIGN
    assert call(lib, T=-1) == call(lib, Hq=0) == call(lib, Hkv=-1) == call(lib, il=2) == INVALID
    assert call(lib, gain=float("nan")) == call(lib, gain=float("inf")) == INVALID
    assert call(lib, D=80) == call(lib, rot=0) == call(lib, rot=3) == call(lib, rot=130) == call(lib, T=1 << 30) == UNSUPPORTED
    assert call(lib, Hq=1 << 23, qs=1 << 30, qos=1 << 30) == UNSUPPORTED
    assert call(lib, qs=511) == call(lib, ks=255) == call(lib, qos=500) == call(lib, qs=-512) == INVALID
    assert call(lib, qs=516) == call(lib, ks=260) == call(lib, qos=513) == ALIGN
    null = {n: NULL for n in ("q", "k", "pos", "steps") + outs}
    assert call(lib, T=0, **null) == OK


def test_refusals_of_each(lib):
    assert rotary(lib, tr=2) == rotary(lib, kos=200) == INVALID
    assert rotary(lib, kos=257) == ALIGN
    assert store(lib, v=NULL) == store(lib, slots=NULL) == store(lib, Hkv=0) == store(lib, nb=0) == store(lib, bs=0) == INVALID
    assert store(lib, vs=255) == INVALID and store(lib, vs=257) == store(lib, v=OFF) == ALIGN
    assert store(lib, nb=1 << 24, bs=128) == UNSUPPORTED


def test_outputs_that_overlap_are_refused(lib):
    """4 tokens of 4 query and 2 KV heads of 128: rows of 1024 and 512 bytes."""
    def at(x):
        return ctypes.c_void_p((1 << 20) + x)

    far = {n: at(i << 20) for i, n in enumerate(("q", "k", "qo", "ko", "v", "cache"))}
    turn = {n: far[n] for n in ("q", "k", "qo", "ko")}
    for o, others in (("qo", ("k", "ko")), ("ko", ("q", "qo"))):
        for n in others:
            assert rotary(lib, **{**turn, o: far[n]}) == INVALID
    assert rotary(lib, **{**turn, "qo": at(16)}) == INVALID                 # a part of q
    assert rotary(lib, **{**turn, "qo": at(3 * 1024 + 1008)}) == INVALID    # its last bytes
    assert rotary(lib, **{**turn, "qo": far["q"], "qos": 520}) == INVALID   # q at another stride
    assert rotary(lib, **{**turn, "ko": far["k"], "kos": 512}) == INVALID
    # q, k side by side in rows of 2048 bytes: an output one unit into the other part, or past the row's end
    fused = dict(q=at(0), qs=1024, k=at(1024), ks=1024, qo=at(0), qos=1024, ko=at(1024), kos=1024)
    assert rotary(lib, **{**fused, "ko": at(1008)}) == INVALID
    assert rotary(lib, **{**fused, "ko": at(1552)}) == INVALID
    store_far = {n: far[n] for n in ("q", "k", "v", "qo", "cache")}
    for o, n in (("qo", "k"), ("qo", "v"), ("qo", "cache"), ("cache", "q"), ("cache", "k"), ("cache", "v"), ("cache", "qo")):
        assert store(lib, **{**store_far, o: far[n]}) == INVALID
    last = 2 * 4 * 128 * 512 - 16  # the cache's last unit
    assert store(lib, **{**store_far, "v": ctypes.c_void_p(far["cache"].value + last)}) == INVALID


def test_binding_refuses_host_tensors(lib):
    import torch

    q = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    plan, pos = gb.RotaryPlan(64, device="cpu"), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        gb.attn_rotary(q, q, pos, plan)
    with pytest.raises(ValueError, match="CUDA"):
        gb.attn_rotary_kv_cache_write(q, q, q, pos, plan, pos, torch.zeros(2, 1, 4, 2, 64, dtype=torch.bfloat16))
