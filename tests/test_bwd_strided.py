"""The backward calls with an `out` that is not contiguous: the boundary and its
host-side refusals (no GPU call is made)."""

import ctypes
import os
import re

import pytest

import attention_forward_09_gb300 as gb
from attention_forward_09_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4
NULL = None


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gb.load_library()


def test_header_and_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gbattn_bwd_strided.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(attn_\w+)\s*\(", text)))
    assert names == ["attn_bwd_padded_strided", "attn_bwd_varlen_strided"]
    for n in names:
        assert hasattr(lib, n) and n in gb.SIGNATURES


# a megabyte each, apart
WHERE = {n: (i + 1) << 20 for i, n in enumerate(("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "ws"))}


def call(lib, fn, strides, odt=0, B=3, S=8, Hq=4, Hkv=2, D=128, wsb=0, **at):
    """No workspace is given, so that a call whose other arguments are right ends with WORKSPACE, before any device call."""
    p = {n: ctypes.c_void_p(at.get(n, x)) for n, x in WHERE.items()}
    head = (p["q"], p["k"], p["v"], p["out"], odt, *strides, p["lse"], p["dout"], NULL)
    tail = (Hq, Hkv, D, 0.1, 0, p["dq"], p["dk"], p["dv"], p["ws"], wsb, NULL, NULL)
    if fn == "attn_bwd_varlen_strided":
        return getattr(lib, fn)(*head, p["lse"], p["lse"], B, B * S, B * S, S, S, *tail)
    return getattr(lib, fn)(*head, NULL, NULL, B, S, S, *tail)


def test_strides_are_refused_on_the_host(lib):
    """bf16 `out` (odt 0): strides in eights; fp32 (odt 1): in fours."""
    f = "attn_bwd_padded_strided"
    good = (8 * 512, 512, 128)
    assert call(lib, f, good) == call(lib, f, (128, 384, 3 * 8 * 128)) == call(lib, f, (0, 0, 0)) == WORKSPACE
    for x in range(3):
        bad = list(good)
        for value, want in ((-8, INVALID), (good[x] + 4, ALIGN), (1 << 58, UNSUPPORTED), ((1 << 63) - 8, UNSUPPORTED)):
            bad[x] = value
            assert call(lib, f, bad) == want, (x, value)
        bad[x] = good[x] + 4
        assert call(lib, f, bad, odt=1) == WORKSPACE
        bad[x] = good[x] + 2
        assert call(lib, f, bad, odt=1) == ALIGN
    # what no index uses is not looked at
    assert call(lib, f, (-1, 512, 128), B=1) == call(lib, f, (512, -1, 128), S=1) == WORKSPACE
    assert call(lib, f, (512, 512, 3), Hq=1, Hkv=1) == WORKSPACE
    g = "attn_bwd_varlen_strided"
    assert call(lib, g, (512, 128)) == call(lib, g, (128, 24 * 128)) == WORKSPACE
    assert call(lib, g, (-8, 128)) == call(lib, g, (512, -8)) == INVALID
    assert call(lib, g, (516, 128)) == call(lib, g, (512, 132)) == ALIGN
    assert call(lib, g, (512, 128), D=80) == UNSUPPORTED
    assert call(lib, g, (512, 128), out=WHERE["out"] + 8) == ALIGN


@pytest.mark.parametrize("fn", ["attn_bwd_padded_strided", "attn_bwd_varlen_strided"])
def test_outputs_within_the_reach_of_a_strided_out_are_refused(lib, fn):
    """3 x 8 rows of 4 heads of 128 in bf16, heads 2^16 elements apart: `out` reaches 3 * 2^17 + 2 * (last row) + 256 bytes."""
    strides = (8 * 128, 128, 1 << 16) if fn == "attn_bwd_padded_strided" else (128, 1 << 16)
    reach = 3 * (1 << 17) + 2 * 23 * 128 + 256
    for o in ("dq", "dk", "dv", "ws"):
        for to, want in ((WHERE["out"] + 256, INVALID), (WHERE["out"] + reach - 256, INVALID), (WHERE["out"] + reach, None)):
            got = call(lib, fn, strides, wsb=1 << 19, **{o: to})
            assert got == INVALID if want else got != INVALID, (o, to, got)
