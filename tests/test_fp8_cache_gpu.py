"""The 8-bit paged KV cache on the GPU against the float64 oracle.

Codes and exponent bytes are compared exactly, read-back values too.  The
decode's bounds follow from its arithmetic, per (sequence, head):

  A  = max over keys of scale * sum_d |q_d k_d|: the score's size before cancellation
  ds = (D / 32 + 12) * 2^-23 * A: the products are exact (8-bit pieces), the
       sums and the four factors after them fp32, one step a K-slice of 32
  V  = the largest |v| of the context (per block of 128 where weights of 0 matter)

  |lse - ref| <= 2 ds + 2^-20 (1 + |ref|): ex2 and log2 are good to 2^-21
  |out - ref| <= V (4 ds + 2^-18 + 2^-b + 128 * 2^-t): the weights relative to the
       sum, ex2, the weights' b bits (16 for fp32 output: four pieces of 4; 11
       for bf16: an fp16 number in three pieces; half a step is 2^-b of a
       weight), and for weights below the pieces' normal range half the last
       piece's smallest step, 2^-10 * 16^-(NP-1) of the 256 that the block's
       largest weight is: 2^-t, t = 14 + 4 NP (NP = 4 or 3), 128 of them a block
  and half a bf16 step of the result, 2^-8 |ref|, for bf16 output.
"""

import math

import numpy as np
import pytest
import torch

import attention_forward_09_gb300 as gb
import oracle
from _helpers import dev, status_word, to_np

pytestmark = pytest.mark.gpu

DTYPES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
HEAD_SIZES = (64, 96, 128, 192, 256)


@pytest.fixture(scope="module", autouse=True)
def built():
    from attention_forward_09_gb300 import _build

    _build.build()
    gb.load_library()


def raw(t):
    return t.view(torch.uint8).cpu().numpy()


def same_codes(got, want, kind):
    """Equal codes; any NaN code is as good as another."""
    v = oracle.code_values(kind)
    both_nan = np.isnan(v[got]) & np.isnan(v[want])
    return np.array_equal(got[~both_nan], want[~both_nan])


def bf16(*shape, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * spread).to(torch.bfloat16)


# ---------------------------------------------------------------- write
def write_case(T, nb, bs, hkv, d, kind, seed=0, pad_every=0, key=None, value=None, slots=None):
    g = torch.Generator().manual_seed(seed)
    key = bf16(T, hkv, d, seed=seed + 1) if key is None else key
    value = bf16(T, hkv, d, seed=seed + 2, spread=9.0) if value is None else value
    if slots is None:
        slots = torch.randperm(nb * bs, generator=g)[:T].to(torch.int32)
        if pad_every:
            slots[::pad_every] = -1
    codes = torch.randint(0, 126, (2, nb, bs, hkv, d), generator=g, dtype=torch.uint8)
    scales = torch.randint(1, 250, (2, nb, hkv, bs), generator=g, dtype=torch.uint8)
    status = status_word()
    cache_d, scales_d = codes.to(dev()).view(DTYPES[kind]), scales.to(dev())
    gb.attn_kv_cache_write_fp8(key.to(dev()), value.to(dev()), slots.to(dev()), cache_d, scales_d, dev_status=status)
    torch.cuda.synchronize()
    want_c, want_s = oracle.kv_cache_write_fp8(key.double().numpy(), value.double().numpy(), slots.numpy(), codes.numpy(),
                                               scales.numpy(), kind)
    assert int(status) == 0
    assert np.array_equal(scales_d.cpu().numpy(), want_s)
    assert same_codes(raw(cache_d), want_c, kind)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("D", HEAD_SIZES)
def test_write_bit_exact(D, kind):
    write_case(37, 3, 128, 3, D, kind, seed=D, pad_every=5)


@pytest.mark.parametrize("T,nb,bs,hkv", [(1, 1, 1, 1), (1, 2, 128, 40), (300, 20, 16, 8), (1000, 9, 128, 5), (513, 41, 13, 2)])
def test_write_sizes(T, nb, bs, hkv):
    write_case(T, nb, bs, hkv, 128, "e4m3", seed=T, pad_every=7 if T > 1 else 0)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
def test_write_special_values(kind):
    """Rows of zeros, NaN, infinities, subnormal and the largest bf16 numbers,
    and of values that lie on the edges between two codes."""
    D = 128
    x = bf16(16, 1, D, seed=3)
    x[0] = 0.0
    x[1, 0, 5] = float("nan")
    x[2, 0, 7], x[2, 0, 8] = float("inf"), float("-inf")
    x[3] = float("nan")
    x[4] = float("inf")
    x[5] = torch.tensor(2.0 ** -133).to(torch.bfloat16)  # the smallest bf16
    x[6] = x[6] * 2.0 ** -120
    x[7, 0, 0] = torch.finfo(torch.bfloat16).max
    x[8] = x[8] * 2.0 ** 120
    pos = oracle.code_values(kind)[:128]
    pos = pos[np.isfinite(pos)]
    edges = torch.from_numpy((pos[1:] + pos[:-1]) / 2).to(torch.bfloat16)  # one bit more than a code: exact
    x[9, 0, :126], x[9, 0, 126] = edges[:126] if edges.numel() >= 126 else torch.cat([edges, edges])[:126], float(pos[-1])
    x[10, 0, :100], x[10, 0, 100] = -edges[-100:] * 2.0 ** 30, float(pos[-1]) * 2.0 ** 30
    x[11, 0, 0] = -0.0
    write_case(16, 1, 128, 1, D, kind, key=x, value=x.flip(0), slots=torch.arange(16, dtype=torch.int32))


def test_write_strided_tokens_and_one_token_tensors():
    """Keys and values as parts of a fused projection's output."""
    T, hq, hkv, D = 50, 6, 2, 96
    qkv = bf16(T, hq + 2 * hkv, D, seed=8).to(dev())
    slots = torch.arange(T, dtype=torch.int32, device=dev()).flip(0).contiguous()
    a = torch.zeros(2, 1, 128, hkv, D, device=dev()).to(torch.float8_e4m3fn), torch.zeros(2, 1, hkv, 128, dtype=torch.uint8, device=dev())
    b = tuple(t.clone() for t in a)
    k, v = qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    gb.attn_kv_cache_write_fp8(k, v, slots, *a)
    gb.attn_kv_cache_write_fp8(k.contiguous(), v.contiguous(), slots, *b)
    assert np.array_equal(raw(a[0]), raw(b[0])) and torch.equal(a[1], b[1])
    assert int(a[1][0, 0, :, :T].min()) > 0
    # starts and strides that are multiples of 16 bytes only
    odd = torch.zeros(T * (hkv * D + 8) + 8, dtype=torch.bfloat16, device=dev())[8:].view(T, hkv * D + 8)
    odd = odd[:, :hkv * D].unflatten(1, (hkv, D))
    odd.copy_(k)
    c = tuple(torch.zeros_like(t) for t in a)
    gb.attn_kv_cache_write_fp8(odd, v, slots, *c)
    assert np.array_equal(raw(c[0]), raw(b[0])) and torch.equal(c[1], b[1])
    gb.attn_kv_cache_write_fp8(k[3:4], v[3:4], slots[:1].contiguous(), *a)  # a stride that is never used
    gb.attn_kv_cache_write_fp8(k[3:4].contiguous(), v[3:4].contiguous(), slots[:1].contiguous(), *b)
    assert np.array_equal(raw(a[0]), raw(b[0])) and torch.equal(a[1], b[1])


def test_write_slot_past_the_cache_is_skipped_and_reported():
    key = bf16(3, 1, 64).to(dev())
    cache, scales = torch.zeros(2, 1, 128, 1, 64, device=dev()).to(torch.float8_e4m3fn), torch.zeros(2, 1, 1, 128, dtype=torch.uint8, device=dev())
    status = status_word()
    gb.attn_kv_cache_write_fp8(key, key, torch.tensor([128, 3, 2 ** 31 - 1], dtype=torch.int32, device=dev()), cache, scales, dev_status=status)
    assert int(status) == gb.DEV_BAD_INDEX
    written = raw(cache).reshape(2, 128, 64).any(-1)
    assert written[:, 3].all() and written.sum() == 2 and int((scales != 0).sum()) == 2


def test_write_repeated_slot_keeps_one_of_the_tokens():
    key = torch.stack([torch.full((1, 64), 1.0), torch.full((1, 64), 1.75)]).to(torch.bfloat16).to(dev())
    cache, scales = torch.zeros(2, 1, 128, 1, 64, device=dev()).to(torch.float8_e4m3fn), torch.zeros(2, 1, 1, 128, dtype=torch.uint8, device=dev())
    gb.attn_kv_cache_write_fp8(key, key, torch.zeros(2, dtype=torch.int32, device=dev()), cache, scales)
    row = raw(cache)[:, 0, 0, 0]
    assert (row == row[:, :1]).all() and scales[:, 0, 0, 0].tolist() == [119, 119]  # both rows have e = -8


# ---------------------------------------------------------------- caches to read and attend
class Ctx:
    """A filled 8-bit cache: random codes and exponents, blocks permuted, unused
    table entries -1 and unused slots poisoned (NaN codes, exponent byte 255)."""

    def __init__(self, lens, hkv, d, kind="e4m3", bs=128, seed=0, exps=(119, 123), vexps=None, extra=2):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.kind, self.bs = list(lens), kind, bs
        nblk = [-(-n // bs) for n in lens]
        nb = sum(nblk) + extra
        top = 60.0 if kind == "e4m3" else 6000.0
        codes = (torch.randn(2, nb, bs, hkv, d, generator=g) * top).clamp(-4 * top, 4 * top).to(DTYPES[kind]).view(torch.uint8)
        scales = torch.empty(2, nb, hkv, bs, dtype=torch.uint8)
        for half, (lo, hi) in enumerate((exps, vexps or exps)):
            scales[half] = torch.randint(lo, hi, (nb, hkv, bs), generator=g, dtype=torch.uint8)
        if kind == "e5m2":
            scales -= 7
        perm = torch.randperm(nb, generator=g).to(torch.int32)
        self.table = torch.full((len(lens), max(nblk + [1]) + 1), -1, dtype=torch.int32)
        used = torch.zeros(nb, bs, dtype=torch.bool)
        at = 0
        for s, n in enumerate(lens):
            ids = perm[at:at + nblk[s]]
            self.table[s, :nblk[s]] = ids
            flat = torch.arange(n)
            used[ids[flat // bs].long(), flat % bs] = True
            at += nblk[s]
        codes[:, ~used] = 127
        scales = torch.where(used[None, :, None, :], scales, torch.tensor(255, dtype=torch.uint8))
        self.codes, self.scales = codes, scales

    def values(self):
        with np.errstate(invalid="ignore", over="ignore"):
            return oracle.stands_for(self.codes.numpy(), self.scales.numpy(), self.kind)

    def on_gpu(self):
        return (self.codes.to(dev()).view(DTYPES[self.kind]), self.scales.to(dev()), self.table.to(dev()))


def ints(x):
    return torch.tensor(list(x), dtype=torch.int32, device=dev())


def run_read(c, total=None, status=None, k=None, v=None):
    cu = [0]
    for n in c.lens:
        cu.append(cu[-1] + n)
    total = cu[-1] if total is None else total
    return gb.attn_kv_cache_read_fp8(*c.on_gpu(), ints(cu), total, k=k, v=v, dev_status=status)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("D", HEAD_SIZES)
def test_read_exact(D, kind):
    c = Ctx([130, 0, 1, 257], 3, D, kind, seed=D)
    status = status_word()
    k, v = run_read(c, status=status)
    assert int(status) == 0
    for got, half in ((k, 0), (v, 1)):
        gathered = oracle.paged_gather(c.values(), c.table, c.lens)[half]
        want = torch.from_numpy(np.concatenate(gathered)).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("bs", [1, 13, 16, 128])
def test_read_block_sizes_and_rows_behind_the_last(bs):
    c = Ctx([40, 3, 0, 0, 77], 2, 64, bs=bs, seed=bs)
    k = torch.full((130, 2, 64), 7.0, dtype=torch.bfloat16, device=dev())
    v = k.clone()
    run_read(c, total=130, k=k, v=v)
    want = torch.from_numpy(np.concatenate(oracle.paged_gather(c.values(), c.table, c.lens)[1])).to(torch.bfloat16)
    assert torch.equal(v[:120].cpu(), want)
    assert (k[120:] == 7).all() and (v[120:] == 7).all()


def test_read_special_codes_and_exponents():
    """Every code at exponents 1, 127, 247 and 254: overflow to infinity and
    values below bf16's normal range are rounded once."""
    for kind in ("e4m3", "e5m2"):
        codes = torch.arange(256, dtype=torch.uint8).repeat(2, 4, 1, 1).reshape(2, 1, 4, 1, 256)
        scales = torch.tensor([1, 127, 247, 254], dtype=torch.uint8).expand(2, 1, 1, 4).contiguous()
        k, _ = gb.attn_kv_cache_read_fp8(codes.to(dev()).view(DTYPES[kind]), scales.to(dev()), ints([0]).view(1, 1), ints([0, 4]), 4)
        want = oracle.stands_for(codes.numpy(), scales.numpy(), kind)[0, 0]
        with np.errstate(over="ignore"):
            want = torch.from_numpy(want.astype(np.float32)).to(torch.bfloat16)  # fp32 holds them but for overflow
        assert torch.equal(k.cpu().nan_to_num(nan=1.5), want.nan_to_num(nan=1.5)), kind
        assert torch.equal(k.cpu().isnan(), want.isnan())


def test_read_bad_block_and_bad_boundaries():
    c = Ctx([200, 100], 1, 64, seed=5)
    c.table[0, 1] = 99
    status = status_word()
    k, v = run_read(c, status=status)
    assert int(status) == gb.DEV_BAD_INDEX
    assert not k[128:200].any() and not v[128:200].any() and k[:128].any()
    cache, scales, table = c.on_gpu()
    for cu in ([0, 50, 20], [0, 100, 1000], [0, 100, 100 + 128 * table.shape[1] + 1], [-5, 10, 20]):
        status.zero_()
        gb.attn_kv_cache_read_fp8(cache, scales, table, ints(cu), 600, dev_status=status)
        assert int(status) & ~(gb.DEV_BAD_SEQLEN | gb.DEV_BAD_INDEX) == 0
        torch.cuda.synchronize()


# ---------------------------------------------------------------- decode
def run_decode(c, q, max_len=None, out_dtype=torch.float32, status=None, **kw):
    cache, scales, table = c.on_gpu()
    return gb.attn_fwd_paged_fp8(q.to(dev()), cache, scales, table, ints(c.lens), max(c.lens) if max_len is None else max_len,
                                 lse=True, out_dtype=out_dtype, dev_status=status, **kw)


def check_decode(c, q, out, lse, scale=None):
    S, hq, D = q.shape
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    values = c.values()
    ks, vs = oracle.paged_gather(values, c.table, c.lens)
    ref, ref_lse = oracle.attention_paged(q, values, c.table, c.lens, scale)
    got, got_lse = to_np(out), to_np(lse)
    bits, pieces = (16, 4) if out.dtype == torch.float32 else (11, 3)
    g = hq // values.shape[3]
    qa = np.abs(q.double().numpy())
    for s in range(S):
        if c.lens[s] == 0:
            assert not got[s].any() and (got_lse[s] == -np.inf).all()
            continue
        for h in range(hq):
            A = scale * float((np.abs(ks[s][:, h // g]) @ qa[s, h]).max())
            V = float(np.abs(vs[s][:, h // g]).max())
            ds = (D / 32 + 12) * 2.0 ** -23 * A
            tol_lse = 2 * ds + 2.0 ** -20 * (1 + abs(ref_lse[s, h]))
            assert abs(got_lse[s, h] - ref_lse[s, h]) <= tol_lse, (s, h, got_lse[s, h], ref_lse[s, h], tol_lse)
            tol = V * (4 * ds + 2.0 ** -18 + 2.0 ** -bits + 128 * 2.0 ** -(14 + 4 * pieces))
            if out.dtype == torch.bfloat16:
                tol = tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(ref[s, h])
            err = np.abs(got[s, h] - ref[s, h])
            assert (err <= tol).all(), (s, h, float(err.max()), tol)


@pytest.mark.parametrize("kind", ["e4m3", "e5m2"])
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", HEAD_SIZES)
def test_decode_head_sizes(D, out_dtype, kind):
    c = Ctx([1, 0, 127, 128, 129, 600], 2, D, kind, seed=D)
    q = bf16(6, 8, D, seed=D + 1)
    status = status_word()
    for max_len in (max(c.lens), 1 << 20):  # a cluster a sequence and head; chunks of all blocks
        out, lse = run_decode(c, q, max_len=max_len, out_dtype=out_dtype, status=status)
        assert int(status) == 0
        check_decode(c, q, out, lse)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (2, 1), (3, 1), (5, 1), (12, 2), (7, 1), (8, 1), (9, 1), (16, 1), (34, 2), (40, 1), (40, 40)])
def test_decode_gqa_ratios(hq, hkv):
    for out_dtype in (torch.float32, torch.bfloat16):
        c = Ctx([300, 5, 0, 1000], hkv, 64, seed=hq)
        q = bf16(4, hq, 64, seed=hq + 1)
        for max_len in (max(c.lens), 1 << 20):
            out, lse = run_decode(c, q, max_len=max_len, out_dtype=out_dtype)
            check_decode(c, q, out, lse)


@pytest.mark.parametrize("lens", [[1025], [4096, 0, 7], [5000], [20000], [1] * 700, [0] * 300 + [129] + [0] * 300, [64, 9000, 64, 0, 3000], [0, 0, 0]])
def test_decode_splits(lens):
    """One long sequence over all chunks, many short ones in a chunk, long and short."""
    c = Ctx(lens, 2, 64, seed=len(lens))
    q = bf16(len(lens), 4, 64, seed=2)
    for max_len in (max(lens), 128 * c.table.shape[1], 1 << 30):  # a loose bound gives chunks without work
        out, lse = run_decode(c, q, max_len=max_len)
        check_decode(c, q, out, lse)


@pytest.mark.parametrize("D,hq,hkv", [(64, 4, 2), (128, 4, 2), (128, 16, 2), (192, 2, 1), (256, 10, 2)])
@pytest.mark.parametrize("S", [1, 9, 14, 20, 27, 36, 48, 60, 75, 76, 80, 100, 123, 160, 200])
def test_decode_short_sequences_in_any_number(S, D, hq, hkv):
    """From a cluster of eight CTAs a sequence down to one, each with one to
    several blocks, and chunks where the sequences are too many for that."""
    longest = {1: 4096}.get(S, 1000 if S < 40 else 511)
    lens = [longest - 128 * (i % 4) - 3 * (i % 5) for i in range(S)]
    c = Ctx(lens, hkv, D, seed=S)
    q = bf16(S, hq, D, seed=S + 1)
    out, lse = run_decode(c, q, max_len=longest)
    keep = sorted({0, S // 3, S // 2, S - 2, S - 1} & set(range(S)))  # the oracle takes a few of them
    c.table, c.lens = c.table[keep], [lens[i] for i in keep]
    check_decode(c, q[keep], out[keep], lse[keep])
    assert torch.isfinite(out).all() and float(out.abs().max()) <= 60.0 * 4 * 2.0 ** -4  # an average of values


@pytest.mark.parametrize("hkv,lens", [(2000, [300, 0, 5]), (153, [200] * 6 + [1, 0, 129]), (1, [1 + i % 3 for i in range(2500)])])
def test_decode_many_heads_or_sequences(hkv, lens):
    """More heads than CTAs run at once, and more sequences than a CTA has threads."""
    c = Ctx(lens, hkv, 64, seed=hkv)
    q = bf16(len(lens), hkv, 64, seed=7)
    out, lse = run_decode(c, q)
    check_decode(c, q, out, lse)


def test_decode_scales_of_any_size():
    """Keys and values whose rows differ by many binades within a block, value
    rows of zeros, and queries of any size (scores kept moderate)."""
    c = Ctx([400, 700], 2, 128, seed=9, exps=(105, 124), vexps=(60, 190))
    c.codes[1, :, ::5] = 0
    c.scales[1, :, :, ::5] = 1
    c.scales[c.codes.view(2, -1, 128, 2, 128).eq(127).all(-1).transpose(2, 3)] = 255  # poison kept
    q = bf16(2, 6, 128, seed=10)
    q[:, 1] *= 2.0 ** -40
    q[:, 2, ::2] *= 2.0 ** -13
    q[0, 3] = 0
    for max_len in (max(c.lens), 1 << 20):
        out, lse = run_decode(c, q, max_len=max_len)
        check_decode(c, q, out, lse)


def test_decode_sink_with_a_tiny_value_row():
    """The first token takes nearly all the weight and its value row is 2^-30
    of the others': what the others contribute still counts, to relative
    accuracy (their weights lie far below the sink's in the same block)."""
    D, n = 64, 100
    key = torch.zeros(n, 1, D)
    key[0, 0, 0] = 160.0
    value = torch.randn(n, 1, D, generator=torch.Generator().manual_seed(1))
    value[0] *= 2.0 ** -30
    cache, scales = torch.zeros(2, 1, 128, 1, D, device=dev()).to(torch.float8_e4m3fn), torch.ones(2, 1, 1, 128, dtype=torch.uint8, device=dev())
    gb.attn_kv_cache_write_fp8(key.to(torch.bfloat16).to(dev()), value.to(torch.bfloat16).to(dev()), ints(range(n)), cache, scales)
    q = torch.zeros(1, 1, D, dtype=torch.bfloat16)
    q[0, 0, 0] = 1.0
    out, lse = gb.attn_fwd_paged_fp8(q.to(dev()), cache, scales, ints([0]).view(1, 1), ints([n]), n, lse=True)  # score 20: weights e^-20
    vals = oracle.stands_for(cache.view(torch.uint8).cpu().numpy(), scales.cpu().numpy(), "e4m3")
    ref, ref_lse = oracle.attention_paged(q, vals, np.zeros((1, 1), np.int64), [n], 1 / 8)
    assert np.abs(to_np(lse) - ref_lse).max() < 1e-4
    scale_of_sum = np.exp(-20.0) * np.sqrt(n)
    assert np.abs(to_np(out) - ref).max() <= 2.0 ** -14 * 4 * scale_of_sum  # 16-bit weights, values up to about 4


@pytest.mark.parametrize("max_len", [900, 1 << 20])
def test_decode_rising_scores_and_values_near_the_top_of_fp32(max_len):
    """Scores that rise from block to block by less than a reference is moved
    for, and value rows of up to 2^110: neither the sum, the references nor
    their quotient leaves fp32's range."""
    D, n = 64, 900
    g = torch.Generator().manual_seed(2)
    key = torch.randn(n, 1, D, generator=g)
    key[:, 0, 0] = 8 * 27.0 * (torch.arange(n) // 128)  # by e^27 = 2^39 a block of 128
    value = torch.randn(n, 1, D, generator=g) * 2.0 ** 108
    cache, scales = torch.zeros(2, 8, 128, 1, D, device=dev()).to(torch.float8_e4m3fn), torch.ones(2, 8, 1, 128, dtype=torch.uint8, device=dev())
    gb.attn_kv_cache_write_fp8(key.to(torch.bfloat16).to(dev()), value.to(torch.bfloat16).to(dev()), ints(range(n)), cache, scales)
    c = Ctx([n], 1, D)
    c.codes, c.scales, c.table = cache.view(torch.uint8).cpu(), scales.cpu(), torch.arange(8, dtype=torch.int32).view(1, 8)
    q = torch.zeros(1, 3, D, dtype=torch.bfloat16)
    q[:, :, 0] = torch.tensor([1.0, 0.5, 1.0])
    q[0, 2, 1:] = 0.5
    for out_dtype in (torch.float32, torch.bfloat16):
        out, lse = run_decode(c, q, max_len=max_len, out_dtype=out_dtype)
        assert torch.isfinite(out).all()
        check_decode(c, q, out, lse)


@pytest.mark.parametrize("max_len", [300, 1 << 20])
def test_decode_scores_and_scales_near_the_ends_of_fp32(max_len):
    """Equal keys, so that the result is the values' mean: scores of about
    -2^23, and keys of 2^120 under queries of 2^-110."""
    D, n = 128, 300
    value = torch.randn(n, 1, D, generator=torch.Generator().manual_seed(3))
    for qv, kv in ((2.0 ** 60, -(2.0 ** -41)), (2.0 ** -110, 2.0 ** 120)):
        cache, scales = torch.zeros(2, 3, 128, 1, D, device=dev()).to(torch.float8_e4m3fn), torch.ones(2, 3, 1, 128, dtype=torch.uint8, device=dev())
        gb.attn_kv_cache_write_fp8(torch.full((n, 1, D), kv, dtype=torch.bfloat16, device=dev()), value.to(torch.bfloat16).to(dev()),
                                   ints(range(n)), cache, scales)
        q = torch.full((1, 2, D), qv, dtype=torch.bfloat16)
        out, lse = gb.attn_fwd_paged_fp8(q.to(dev()), cache, scales, ints(range(3)).view(1, 3), ints([n]), max_len, lse=True)
        v = oracle.stands_for(cache.view(torch.uint8).cpu().numpy(), scales.cpu().numpy(), "e4m3")[1].reshape(-1, D)[:n]
        # every weight is the same number, so only the fp32 sums and the quotient round
        assert np.abs(to_np(out)[0] - v.mean(0)).max() <= 2.0 ** -16 * np.abs(v).max()
        want = qv * kv * math.sqrt(D) + math.log(n)
        assert np.abs(to_np(lse) - want).max() <= 2.0 ** -20 * (1 + abs(want))


def test_decode_exponent_byte_zero():
    """Exponent byte 0 (2^-127) under queries of 2^126: scores of some hundreds
    of either sign.  A scale that is not positive is refused."""
    D, n, scale = 64, 200, 2.0 ** -7
    codes, scales = torch.zeros(2, 2, 128, 1, D, dtype=torch.uint8), torch.zeros(2, 2, 1, 128, dtype=torch.uint8)
    codes[0] = 0x7E  # 448
    codes[0, :, ::3] |= 0x80
    codes[1] = torch.randint(0, 0x7F, codes[1].shape, generator=torch.Generator().manual_seed(6), dtype=torch.uint8)
    scales[1] = 120
    q = torch.full((1, 2, D), 2.0 ** 126, dtype=torch.bfloat16)
    vals = oracle.stands_for(codes.numpy(), scales.numpy(), "e4m3")
    table = torch.arange(2, dtype=torch.int32).view(1, 2)
    ref, ref_lse = oracle.attention_paged(q, vals, table, [n], scale)
    for max_len in (n, 1 << 20):
        out, lse = gb.attn_fwd_paged_fp8(q.to(dev()), codes.to(dev()).view(torch.float8_e4m3fn), scales.to(dev()), table.to(dev()),
                                         ints([n]), max_len, scale, lse=True)
        # scores of +-112: one number in all that count, so only the sums and the quotient round
        assert np.abs(to_np(out) - ref).max() <= 2.0 ** -15 * np.abs(vals[1]).max()
        assert np.abs(to_np(lse) - ref_lse).max() <= 2.0 ** -20 * (1 + np.abs(ref_lse).max())
    for bad in (-scale, 0.0, float("nan")):
        with pytest.raises(gb.GbattnError) as e:
            gb.attn_fwd_paged_fp8(q.to(dev()), codes.to(dev()).view(torch.float8_e4m3fn), scales.to(dev()), table.to(dev()),
                                  ints([n]), n, bad)
        assert e.value.status == 1


@pytest.mark.parametrize("max_len", [700, 1 << 20])
def test_decode_references_that_move(max_len):
    """Scores that jump up and down by thousands from block to block, a first
    block that is not there, far negative scores behind it, and values whose
    exponents differ: the last bits of the exponents still count."""
    D, n = 64, 700
    base = torch.tensor([0.0, -3e6, 2e3, -5e3, 1e7, 1e7])  # by block; the two last share the weight
    key = torch.zeros(n, 1, D)
    key[:, 0, 0] = base[torch.arange(n) // 128]
    key[:, 0, 1] = torch.randn(n, generator=torch.Generator().manual_seed(4))
    value = torch.randn(n, 1, D, generator=torch.Generator().manual_seed(5)) * torch.exp2(torch.arange(n) % 7 * 1.0).view(n, 1, 1)
    cache, scales = torch.zeros(2, 6, 128, 1, D, device=dev()).to(torch.float8_e4m3fn), torch.ones(2, 6, 1, 128, dtype=torch.uint8, device=dev())
    gb.attn_kv_cache_write_fp8(key.to(torch.bfloat16).to(dev()), value.to(torch.bfloat16).to(dev()), ints(range(n)), cache, scales)
    vals = oracle.stands_for(cache.view(torch.uint8).cpu().numpy(), scales.cpu().numpy(), "e4m3")
    k, v = vals[0].reshape(-1, D)[:n], vals[1].reshape(-1, D)[:n]
    q = torch.zeros(1, 2, D, dtype=torch.bfloat16)
    q[0, 0, 0], q[0, 1, 0], q[0, 1, 1] = 8.0, 0.125, 1.0  # head 0: scores of up to 1e7; head 1: to 2e5
    for lens, first in (([n], 0), ([n], 1), ([256], 1), ([400], 1)):
        table = ints(range(6)).view(1, 6)
        if first:
            table[0, 0] = -1
        status = status_word()
        out, lse = gb.attn_fwd_paged_fp8(q.to(dev()), cache, scales, table, ints(lens), max_len, lse=True, dev_status=status)
        assert int(status) == (gb.DEV_BAD_INDEX if first else 0)
        rows = slice(128 * first, lens[0])
        for h in range(2):
            x = k[rows] @ q[0, h].double().numpy() / 8
            w = np.exp(x - x.max())
            want, want_lse = (w / w.sum()) @ v[rows], x.max() + np.log(w.sum())
            # products with one or two columns of q: a score is off by four roundings of fp32
            ds = 2.0 ** -22 * np.abs(x[x > x.max() - 40]).max()
            same = np.ptp(x[x > x.max() - 40]) == 0  # one number in all scores that count: off by the same
            V = np.abs(v[rows]).max()
            assert np.abs(to_np(out)[0, h] - want).max() <= V * ((0 if same else 4 * ds) + 2.0 ** -15)
            assert abs(to_np(lse)[0, h] - want_lse) <= 2 * ds + 2.0 ** -20 * (1 + abs(want_lse))


def test_decode_large_logits():
    c = Ctx([129, 1000], 1, 128, seed=4, exps=(122, 126))
    q = bf16(2, 4, 128, seed=5, spread=30.0)  # scores of some thousands: one key takes all the weight
    for max_len in (max(c.lens), 1 << 20):
        out, lse = run_decode(c, q, max_len=max_len)
        check_decode(c, q, out, lse)


@pytest.mark.parametrize("max_len", [200, 1 << 20])
def test_decode_nan_stays_in_its_sequence_and_head(max_len):
    c = Ctx([200, 200, 200], 2, 64, seed=6)
    q = bf16(3, 4, 64, seed=7)
    clean, clean_lse = run_decode(c, q, max_len=max_len)
    b = int(c.table[1, 0])
    c.codes[0, b, 7, 1, 3] = 127     # a key of sequence 1, KV head 1
    c.codes[1, int(c.table[2, 1]), 2, 0, 9] = 127  # a value of sequence 2, KV head 0, column 9
    q[0, 2, 5] = float("inf")
    out, lse = run_decode(c, q, max_len=max_len)
    nan, nan_lse = torch.isnan(out).cpu(), torch.isnan(lse).cpu()
    want, want_lse = torch.zeros(3, 4, 64, dtype=torch.bool), torch.zeros(3, 4, dtype=torch.bool)
    want[1, 2:], want_lse[1, 2:] = True, True
    want[2, :2, 9] = True
    want[0, 2], want_lse[0, 2] = True, True
    assert torch.equal(nan, want) and torch.equal(nan_lse, want_lse)
    assert torch.equal(out.cpu()[~want], clean.cpu()[~want]) and torch.equal(lse.cpu()[~want_lse], clean_lse.cpu()[~want_lse])


@pytest.mark.parametrize("max_len", [300, 1 << 20])
def test_decode_bad_block_is_skipped_and_reported(max_len):
    c = Ctx([300, 100], 1, 64, seed=8)
    q = bf16(2, 2, 64, seed=9)
    kept = Ctx([300, 100], 1, 64, seed=8)
    c.table[0, 1] = 1 << 20
    status = status_word()
    out, lse = run_decode(c, q, max_len=max_len, status=status)
    assert int(status) == gb.DEV_BAD_INDEX
    # the same as without those 128 tokens: blocks 0 and 2 of the sequence
    kept.table[0, 1] = kept.table[0, 2]
    kept.lens = [300 - 128, 100]
    check_decode(kept, q, out, lse)
    c.table[0, :3] = -7  # no block left: an empty row
    out, lse = run_decode(c, q, max_len=max_len)
    assert not out[0].any() and torch.isinf(lse[0]).all()


def test_decode_bad_lengths_are_clamped_and_reported():
    c = Ctx([300, 100, 50], 1, 64, seed=8)
    q = bf16(3, 2, 64, seed=9)
    cache, scales, table = c.on_gpu()
    status = status_word()
    out, lse = gb.attn_fwd_paged_fp8(q.to(dev()), cache, scales, table, ints([400, -3, 50]), 300, lse=True, dev_status=status)
    assert int(status) == gb.DEV_BAD_SEQLEN
    c.lens = [300, 0, 50]
    check_decode(c, q, out, lse)
    many = 100  # past 300 * many the bound is the table's: chunks
    status.zero_()
    out, lse = gb.attn_fwd_paged_fp8(q.to(dev()), cache, scales, table[:, :3].contiguous(), ints([1 << 30, -3, 50]), 300 * many, lse=True, dev_status=status)
    assert int(status) & gb.DEV_BAD_SEQLEN
    c.lens = [384, 0, 50]
    assert torch.isfinite(lse[2]).all() and torch.isinf(lse[1]).all()


def test_decode_strided_queries_given_outputs_and_workspace():
    c = Ctx([400, 20, 1300], 2, 96, seed=3)
    qkv = bf16(3, 4 + 4, 96, seed=4).to(dev())
    q = qkv[:, :4]
    cache, scales, table = c.on_gpu()
    need = gb.attn_fwd_paged_fp8_workspace_size(3, 4, 2, 96, 13000)
    assert need > 0
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device=dev())
    out, lse = torch.empty(3, 4, 96, dtype=torch.bfloat16, device=dev()), torch.empty(3, 4, device=dev())
    got = gb.attn_fwd_paged_fp8(q, cache, scales, table, ints(c.lens), 13000, out=out, lse=lse, workspace=ws[:need])
    assert got[0] is out and got[1] is lse
    check_decode(c, q.cpu(), out, lse)
    assert (ws[need:] == 255).all()  # nothing behind the stated size
    with pytest.raises(gb.GbattnError) as e:
        gb.attn_fwd_paged_fp8(q, cache, scales, table, ints(c.lens), 13000, workspace=ws[:need - 256])
    assert e.value.status == 4
    for bad in (dict(out=torch.empty(3, 4, 64, device=dev())), dict(lse=torch.empty(4, 3, device=dev())), dict(out=out.transpose(0, 1))):
        with pytest.raises(ValueError):
            gb.attn_fwd_paged_fp8(q, cache, scales, table, ints(c.lens), 1300, **bad)


@pytest.mark.parametrize("max_len", [3000, 30000])
def test_decode_repeats_bit_for_bit(max_len):
    c = Ctx([3000, 50, 700], 2, 128, seed=12)
    q = bf16(3, 8, 128, seed=13).to(dev())
    cache, scales, table = c.on_gpu()
    sl = ints(c.lens)
    a = gb.attn_fwd_paged_fp8(q, cache, scales, table, sl, max_len, lse=True)
    for _ in range(20):
        b = gb.attn_fwd_paged_fp8(q, cache, scales, table, sl, max_len, lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("max_len", [2000, 20000])
def test_decode_on_two_streams_at_once_and_in_graphs(max_len):
    """Two streams with a workspace each; a captured graph replayed with new
    lengths, queries and cache contents, beside eager calls."""
    c = Ctx([2000, 900, 0, 128], 2, 128, seed=14)
    c.lens = [1000, 900, 0, 5]
    q = bf16(4, 8, 128, seed=15)
    cache, scales, table = c.on_gpu()
    qd, sl = q.to(dev()), ints(c.lens)
    want = gb.attn_fwd_paged_fp8(qd, cache, scales, table, sl, max_len, lse=True)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            outs[i].append(gb.attn_fwd_paged_fp8(qd, cache, scales, table, sl, max_len, lse=True, stream=s))
    torch.cuda.synchronize()
    for o in outs[0] + outs[1]:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
    graphs = []
    given = torch.empty(4, 8, 128, device=dev())
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            lens = sl
            if i == 1:  # behind a copy and a memset in the graph
                lens = torch.empty_like(sl)
                lens.copy_(sl)
                given.zero_()
            graphs.append((g, gb.attn_fwd_paged_fp8(qd, cache, scales, table, lens, max_len, lse=True, out=given if i else None)))
    c.lens = [2000, 1, 0, 128]
    sl.copy_(ints(c.lens))
    q = bf16(4, 8, 128, seed=16)
    qd.copy_(q)
    for g, _ in graphs:
        g.replay()
    eager = gb.attn_fwd_paged_fp8(qd, cache, scales, table, sl, max_len, lse=True)
    torch.cuda.synchronize()
    for o in [x for _, x in graphs] + [eager]:
        check_decode(c, q, *o)


def test_first_call_inside_a_capture():
    """A process whose first call of each kind is captured into a graph."""
    import os
    import subprocess
    import sys

    code = """
import torch, attention_forward_09_gb300 as gb
d = torch.device("cuda:0")
k = torch.randn(300, 2, 192, device=d).to(torch.bfloat16)
q = torch.randn(1, 10, 192, device=d).to(torch.bfloat16)
ints = lambda x: torch.tensor(x, dtype=torch.int32, device=d)
cache, scales = torch.zeros(2, 3, 128, 2, 192, device=d).to(torch.float8_e5m2), torch.ones(2, 3, 2, 128, dtype=torch.uint8, device=d)
slots, table, lens, cu = ints(list(range(300))), ints([[0, 1, 2]]), ints([300]), ints([0, 300])
torch.cuda.synchronize()
def go():
    gb.attn_kv_cache_write_fp8(k, k, slots, cache, scales)
    kv = gb.attn_kv_cache_read_fp8(cache, scales, table, cu, 300)
    return kv + tuple(x for n in (300, 1 << 20) for x in gb.attn_fwd_paged_fp8(q, cache, scales, table, lens, n, lse=True))
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    got = go()
cache.view(torch.uint8).zero_()
g.replay()
want = go()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want)) and bool(got[2].any())
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_streams_and_host_ints_that_cannot_be_meant():
    c = Ctx([5], 1, 64)
    cache, scales, table = c.on_gpu()
    q = bf16(1, 1, 64).to(dev())
    for call in (lambda: gb.attn_fwd_paged_fp8(q, cache, scales, table, ints([5]), 2 ** 32 + 5),
                 lambda: gb.attn_kv_cache_read_fp8(cache, scales, table, ints([0, 5]), 2 ** 32),
                 lambda: gb.attn_fwd_paged_fp8_workspace_size(1, 1, 1, 64, 2 ** 31)):
        with pytest.raises(ValueError, match="2\\*\\*31"):
            call()
    for call in (lambda: gb.attn_fwd_paged_fp8(q, cache, scales, table, ints([5]), -1),
                 lambda: gb.attn_kv_cache_read_fp8(cache, scales, table[:, :0].contiguous(), ints([0, 5]), 5)):
        with pytest.raises(gb.GbattnError) as e:
            call()
        assert e.value.status == 1


def test_decode_offsets_past_32_bits():
    """A cache of 5 GB whose last blocks hold the context."""
    hkv, D = 16, 256
    nb = 5 * 2 ** 30 // (2 * 128 * hkv * D)
    small = Ctx([300], hkv, D, seed=17, extra=0)
    cache = torch.zeros(2, nb, 128, hkv, D, dtype=torch.uint8, device=dev())
    scales = torch.ones(2, nb, hkv, 128, dtype=torch.uint8, device=dev())
    table = small.table.clone()
    for b in range(3):
        src = int(small.table[0, b])
        cache[:, nb - 1 - b], scales[:, nb - 1 - b] = small.codes[:, src].to(dev()), small.scales[:, src].to(dev())
        table[0, b] = nb - 1 - b
    cache = cache.view(torch.float8_e4m3fn)
    q = bf16(1, 2 * hkv, D, seed=18)
    out, lse = gb.attn_fwd_paged_fp8(q.to(dev()), cache, scales, table.to(dev()), ints([300]), 300, lse=True)
    check_decode(small, q, out, lse)
    k, v = gb.attn_kv_cache_read_fp8(cache, scales, table.to(dev()), ints([0, 300]), 300)
    want = torch.from_numpy(np.concatenate(oracle.paged_gather(small.values(), small.table, [300])[1])).to(torch.bfloat16)
    assert torch.equal(v.cpu(), want)
    before = raw(cache[:, nb - 1])
    slot = ints([(nb - 1) * 128 + 127])
    gb.attn_kv_cache_write_fp8(k[:1].contiguous(), v[:1].contiguous(), slot, cache, scales)
    after = raw(cache[:, nb - 1])
    assert np.array_equal(before[:, :127], after[:, :127]) and not np.array_equal(before[:, 127], after[:, 127])


# ---------------------------------------------------------------- together
def test_a_prefill_then_decode_steps():
    """Chunks written and attended through the read-back, then single tokens
    written and attended, against the oracle over the quantised values."""
    hq, hkv, D, S = 8, 2, 128, 3
    lens, nblk = [300, 1, 140], 4
    table = torch.randperm(S * nblk, generator=torch.Generator().manual_seed(0)).to(torch.int32).view(S, nblk)
    cache = torch.zeros(2, S * nblk, 128, hkv, D, device=dev()).to(torch.float8_e4m3fn)
    scales = torch.ones(2, S * nblk, hkv, 128, dtype=torch.uint8, device=dev())
    status = status_word()

    def slots(s, a, b):
        t = torch.arange(a, b)
        return (table[s, t // 128] * 128 + t % 128).to(torch.int32)

    def values():
        return oracle.stands_for(raw(cache), scales.cpu().numpy(), "e4m3")

    T = sum(lens)
    k, v = bf16(T, hkv, D, seed=1).to(dev()), bf16(T, hkv, D, seed=2).to(dev())
    where = torch.cat([slots(s, 0, n) for s, n in enumerate(lens)]).to(dev())
    gb.attn_kv_cache_write_fp8(k, v, where, cache, scales, dev_status=status)
    q_lens = [100, 1, 140]
    q = bf16(sum(q_lens), hq, D, seed=3)
    cu_q, cu_k = ints(np.cumsum([0] + q_lens)), ints(np.cumsum([0] + lens))
    out, lse = gb.attn_fwd_paged_prefill_fp8(q.to(dev()), cache, scales, table.to(dev()), cu_q, cu_k, T, max(q_lens), max(lens),
                                             lse=True, dev_status=status)
    ref, ref_lse = oracle.attention_paged_prefill(q, values(), table, lens, cu_q, 1 / math.sqrt(D), True)
    assert np.abs(to_np(out) - ref).max() <= 1e-2 and np.abs(to_np(lse) - ref_lse).max() <= 1e-3  # the prefill kernels' bounds
    for step in range(3):
        qkv = bf16(S, hq + 2 * hkv, D, seed=10 + step).to(dev())
        where = torch.cat([slots(s, n, n + 1) for s, n in enumerate(lens)]).to(dev())
        gb.attn_kv_cache_write_fp8(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], where, cache, scales, dev_status=status)
        lens = [n + 1 for n in lens]
        out, lse = gb.attn_fwd_paged_fp8(qkv[:, :hq], cache, scales, table.to(dev()), ints(lens), 128 * nblk, lse=True, dev_status=status)
        ref, ref_lse = oracle.attention_paged(qkv[:, :hq].cpu(), values(), table, lens, 1 / math.sqrt(D))
        assert np.abs(to_np(out) - ref).max() <= 2.0 ** -12 and np.abs(to_np(lse) - ref_lse).max() <= 2.0 ** -16
    assert int(status) == 0


def test_prefill_with_rows_behind_the_contexts():
    """total_tokens above the contexts' sum: the rows behind them are whatever
    the allocator's memory held, here NaN, and no result feels them."""
    hq, hkv, D, lens = 4, 2, 64, [130, 77]
    c = Ctx(lens, hkv, D, seed=21)
    cache, scales, table = c.on_gpu()
    q_lens, T = [130, 20], 1000
    q = bf16(sum(q_lens), hq, D, seed=22)
    cu_q, cu_k = ints(np.cumsum([0] + q_lens)), ints(np.cumsum([0] + lens))
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    poison = [torch.full((T, hkv, D), float("nan"), dtype=torch.bfloat16, device=dev()) for _ in range(8)]
    del poison
    status = status_word()
    out, lse = gb.attn_fwd_paged_prefill_fp8(q.to(dev()), cache, scales, table, cu_q, cu_k, T, max(q_lens), max(lens), lse=True,
                                             dev_status=status)
    ref, ref_lse = oracle.attention_paged_prefill(q, c.values(), c.table, lens, cu_q, 1 / math.sqrt(D), True)
    assert int(status) == 0
    assert np.abs(to_np(out) - ref).max() <= 1e-2 and np.abs(to_np(lse) - ref_lse).max() <= 1e-3  # the prefill kernels' bounds
    with pytest.raises(ValueError, match="q must be on"):
        gb.attn_fwd_paged_prefill_fp8(q, cache, scales, table, cu_q, cu_k, T, max(q_lens), max(lens))


def test_decode_of_a_quantised_cache_is_near_the_bf16_decode():
    """Against attn_fwd_paged over the unquantised cache: the difference is that
    of the codes, at most half a step (2^-4) of each key and value."""
    hq, hkv, D, n = 8, 2, 128, 500
    k, v = bf16(n, hkv, D, seed=1).to(dev()), bf16(n, hkv, D, seed=2).to(dev())
    plain = torch.zeros(2, 4, 128, hkv, D, dtype=torch.bfloat16, device=dev())
    cache, scales = torch.zeros(2, 4, 128, hkv, D, device=dev()).to(torch.float8_e4m3fn), torch.ones(2, 4, hkv, 128, dtype=torch.uint8, device=dev())
    where, table = ints(range(n)), ints(range(4)).view(1, 4)
    gb.attn_kv_cache_write(k, v, where, plain)
    gb.attn_kv_cache_write_fp8(k, v, where, cache, scales)
    q = bf16(1, hq, D, seed=3).to(dev())
    a, la = gb.attn_fwd_paged(q, plain, table, ints([n]), n, lse=True)
    b, lb = gb.attn_fwd_paged_fp8(q, cache, scales, table, ints([n]), n, lse=True)
    # scores move by at most 2^-4 A, so weights by a factor e^(2^-3 A); A from the inputs
    A = float((q.float().abs().view(hkv, -1, D) @ k.float().abs().permute(1, 2, 0)).max()) / math.sqrt(D)
    V = float(v.float().abs().max())
    move = 2.0 ** -4 * A
    assert float((la - lb).abs().max()) <= move
    assert float((a - b).abs().max()) <= V * (math.expm1(2 * move) + 2.0 ** -4)
    assert float((a - b).norm() / a.norm()) < 0.1  # and typically a few per cent
