"""The gradients' oracle against differences of the forward oracle, and the
backward calls' host-side refusals (no GPU call is made)."""

import ctypes
import os
import re

import numpy as np
import pytest

import attention_forward_09_gb300 as gb
import oracle
from attention_forward_09_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, ALIGN, WORKSPACE = 0, 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return gb.load_library()


# ------------------------------------------------------------------ the oracle
@pytest.mark.parametrize("Lq,Lk,Hq,Hkv,causal", [(5, 7, 2, 1, False), (5, 7, 4, 2, True), (7, 4, 2, 2, True),
                                                 (1, 1, 1, 1, True), (3, 1, 2, 1, False)])
def test_oracle_gradients_equal_differences_of_the_forward_oracle(Lq, Lk, Hq, Hkv, causal):
    """Every derivative of sum(out * a) + sum(lse * b) by a central difference in 64 bits: step h = 2^-17, error
    h^2 times the third derivative plus 2^-52 / h of the value, far below 1e-8 for inputs of about unit size."""
    rng = np.random.default_rng(Lq * 100 + Lk)
    D, scale = 4, 0.6
    x = {"q": rng.normal(size=(Lq, Hq, D)), "k": rng.normal(size=(Lk, Hkv, D)), "v": rng.normal(size=(Lk, Hkv, D))}
    a, b = rng.normal(size=(Lq, Hq, D)), rng.normal(size=(Hq, Lq))

    def value(x):
        out, lse = oracle.attention_single(x["q"], x["k"], x["v"], scale, causal)
        return np.sum(out * a) + np.sum(np.where(np.isfinite(lse), lse, 0.0) * b)

    out, lse = oracle.attention_single(x["q"], x["k"], x["v"], scale, causal)
    grads = dict(zip("qkv", oracle.attention_gradients(x["q"], x["k"], x["v"], out, lse, a, scale, causal, dlse=b)))
    h = 2.0 ** -17
    for n in "qkv":
        for at in np.ndindex(x[n].shape):
            up, dn = dict(x), dict(x)
            up[n], dn[n] = x[n].copy(), x[n].copy()
            up[n][at] += h
            dn[n][at] -= h
            assert abs((value(up) - value(dn)) / (2 * h) - grads[n][at]) < 1e-8, (n, at)


def test_oracle_rows_without_a_key_give_nothing_whatever_they_hold():
    rng = np.random.default_rng(3)
    q, k, v, do = (rng.normal(size=(n, 1, 4)) for n in (5, 3, 3, 5))
    out, lse = oracle.attention_single(q, k, v, 0.5, True)  # rows 0 and 1 see no key
    ref = oracle.attention_gradients(q, k, v, out, lse, do, 0.5, True)
    for x in (q, do, out):
        x[:2] = np.nan
    got = oracle.attention_gradients(q, k, v, out, lse, do, 0.5, True)
    for a, b in zip(ref, got):
        assert np.array_equal(a, b)
    assert not got[0][:2].any()


# ---------------------------------------------------------------- the boundary
def test_header_and_exports(lib):
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gbattn_bwd.h")).read(), flags=re.S)
    names = sorted(set(re.findall(r"\b(attn_\w+)\s*\(", text)))
    assert names == ["attn_bwd_dense", "attn_bwd_padded", "attn_bwd_varlen", "attn_bwd_workspace_size"]
    for n in names:
        assert hasattr(lib, n) and n in gb.SIGNATURES


def test_workspace_size(lib):
    f = lib.attn_bwd_workspace_size
    # two fp32 arrays [Hq, rows + alignment of each document + a tile], each rounded up to 256 bytes, and counters
    for n, t, h in ((1, 1, 1), (3, 1000, 7), (65535, 65535, 2), (2, 8192, 24)):
        stride = (t + 4 * n + 3) // 4 * 4 + 128
        assert f(n, t, h) == 2 * ((stride * h * 4 + 255) // 256 * 256) + 256
    assert f(1, 2 ** 31 - 1, 64) > 2 ** 39  # no 32-bit product
    assert f(-1, 1, 1) == f(1, -1, 1) == f(1, 1, 0) == f(65536, 1, 1) == 0


P, NULL = ctypes.c_void_p(0x10000), None
OFF = ctypes.c_void_p(0x10008)


def dense(lib, fn="attn_bwd_dense", **kw):
    a = dict(q=P, k=P, v=P, out=P, odt=0, lse=P, dout=P, dlse=NULL, B=1, Sq=8, Sk=8, Hq=4, Hkv=2, D=128, scale=0.1, dq=P, dk=P,
             dv=P, ws=P, wsb=1 << 30)
    a.update(kw)
    lens = (NULL, NULL) if fn == "attn_bwd_padded" else ()
    return getattr(lib, fn)(a["q"], a["k"], a["v"], a["out"], a["odt"], a["lse"], a["dout"], a["dlse"], *lens, a["B"], a["Sq"],
                            a["Sk"], a["Hq"], a["Hkv"], a["D"], a["scale"], 0, a["dq"], a["dk"], a["dv"], a["ws"], a["wsb"],
                            None, None)


@pytest.mark.parametrize("fn", ["attn_bwd_dense", "attn_bwd_padded"])
def test_batch_refusals(lib, fn):
    def d(**kw):
        return dense(lib, fn, **kw)

    for n in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv"):
        assert d(**{n: NULL}) == INVALID, n
    for n in ("q", "k", "v", "out", "dout", "dq", "dk", "dv"):
        assert d(**{n: OFF}) == ALIGN, n
    assert d(D=80) == d(D=32) == d(odt=2) == UNSUPPORTED
    assert d(Hq=6, Hkv=4) == d(Hkv=0) == d(Hq=0) == d(B=-1) == d(Sq=-1) == d(Sk=-1) == INVALID
    assert d(scale=0.0) == d(scale=-1.0) == d(scale=float("nan")) == d(scale=float("inf")) == INVALID
    assert d(B=65536) == d(B=65535, Sq=65535) == d(B=2, Sk=2 ** 30) == UNSUPPORTED
    assert d(B=1, Sq=2 ** 31 - 1, Hq=256, Hkv=1) == UNSUPPORTED  # more tiles than a grid holds
    need = lib.attn_bwd_workspace_size(1, 8, 4)
    assert d(ws=NULL) == d(wsb=need - 1) == d(ws=ctypes.c_void_p(0x10010)) == WORKSPACE
    # nothing to do: no pointer is needed
    null = {n: NULL for n in ("q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv", "ws")}
    assert d(B=0, **null) == OK and d(Sq=0, Sk=0, **null) == OK


def varlen(lib, **kw):
    a = dict(cq=P, ck=P, N=2, Tq=16, Tk=16, mq=8, mk=8, Hq=4, Hkv=4, D=64, ws=P, wsb=1 << 30)
    a.update(kw)
    return lib.attn_bwd_varlen(P, P, P, P, 1, P, P, None, a["cq"], a["ck"], a["N"], a["Tq"], a["Tk"], a["mq"], a["mk"],
                               a["Hq"], a["Hkv"], a["D"], 0.125, 1, P, P, P, a["ws"], a["wsb"], None, None)


def test_packed_refusals(lib):
    assert varlen(lib, cq=None) == varlen(lib, ck=None) == varlen(lib, N=-1) == varlen(lib, mq=-1) == INVALID
    assert varlen(lib, mq=17) == varlen(lib, mk=17) == INVALID
    assert varlen(lib, N=65536) == varlen(lib, D=48) == UNSUPPORTED
    assert varlen(lib, N=60000, Tq=2 ** 30, mq=2 ** 30) == UNSUPPORTED
    assert varlen(lib, wsb=lib.attn_bwd_workspace_size(2, 16, 4) - 1) == WORKSPACE
    assert varlen(lib, N=0) == varlen(lib, Tq=0, Tk=0, mq=0, mk=0) == OK


def test_outputs_that_overlap_are_refused(lib):
    """Of 8 rows, 4 query and 2 KV heads of 128: q, dout, dq 8192 bytes, out 16384 in fp32, k, v, dk, dv 4096, lse 128."""
    at, where = 1 << 20, {}
    for n in ("q", "k", "v", "out", "lse", "dlse", "dout", "dq", "dk", "dv", "ws"):
        where[n] = at
        at += 1 << 20
    size = dict(q=8192, dout=8192, out=16384, k=4096, v=4096, lse=128, dlse=128, dq=8192, dk=4096, dv=4096,
                ws=lib.attn_bwd_workspace_size(1, 8, 4))
    for fn in ("attn_bwd_dense", "attn_bwd_padded"):
        for o in ("dq", "dk", "dv", "ws"):
            for n in where:
                if n == o:
                    continue
                # the same place, the last bytes of the other, the other at this one's last bytes
                step = 256 if o == "ws" else 16
                for to in (where[n], where[n] + (size[n] - 1) // step * step):
                    a = {x: ctypes.c_void_p(p) for x, p in where.items()}
                    a[o] = ctypes.c_void_p(to)
                    assert dense(lib, fn, odt=1, **a) == INVALID, (o, n, to)


def test_binding_refuses_host_tensors():
    import torch

    q = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    lse = torch.zeros(1, 2, 4)
    with pytest.raises(ValueError, match="CUDA"):
        gb.attn_bwd_dense(q, q, q, q, lse, q)
    with pytest.raises(ValueError):
        gb.attn_bwd_dense(q[0], q, q, q, lse, q)
    with pytest.raises(ValueError):
        gb.attn_bwd_varlen(q, q, q, q, lse, q, torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 4, 4)
