"""The operators of the 8-bit paged key-value cache, as cases that can be timed and checked.

Three operators, each through the package's own entry point where ``own`` is
true and in elementary torch operations where it is false:

  write   attn_kv_cache_write_fp8: new tokens' keys and values quantised into the paged cache
  read    attn_kv_cache_read_fp8:  the contexts of several sequences read back, packed, in bf16
  decode  attn_fwd_paged_fp8:      one new token a sequence attends its context in the 8-bit cache

A row of D values of one (token, KV head, key or value) is held as D codes c
(float8 e4m3fn or e5m2) and one exponent byte b, and stands for c * 2^(b - 127).
The exponent is the least e >= -126 with max |x| <= c_max * 2^e over the row's
finite values (c_max: 448 or 57344; a row without a non-zero finite value has
e = -126); codes are x / 2^e rounded to nearest, ties to even, and NaN where x
is NaN or infinite.  Cache [2, blocks, 128, Hkv, D], exponents [2, blocks, Hkv, 128].
"""

import math

import torch

own = False

BLOCK = 128
HEAD_SIZES = (64, 96, 128, 192, 256)
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # a chat of a few hundred tokens on its own: what one answer's next token waits for
        dict(name="decode one short chat", op="decode", S=1, lo=517, hi=517, Hq=32, Hkv=8, D=128, kv="e4m3", out="bf16"),
        # the framework's paged decode workload (64 sequences, contexts 1024 to 32768) over the 8-bit cache
        dict(name="decode batch of 64", op="decode", S=64, lo=1024, hi=32768, Hq=32, Hkv=8, D=128, kv="e4m3", out="bf16"),
        # two long documents, one KV head for eight query heads: few rows, so the length has to be split
        dict(name="decode two long documents", op="decode", S=2, lo=120011, hi=131071, Hq=8, Hkv=1, D=256, kv="e4m3", out="bf16"),
        # a slot table with empty and short sequences, a KV head for each query head, fp32 results
        dict(name="decode ragged D=96 e5m2", op="decode", S=48, lo=0, hi=2999, Hq=16, Hkv=16, D=96, kv="e5m2", out="fp32"),
        # many medium contexts with an odd number of query heads to a KV head
        dict(name="decode 128 seqs D=64", op="decode", S=128, lo=1, hi=4097, Hq=20, Hkv=4, D=64, kv="e4m3", out="bf16"),
        # the keys and values of one decode step of 64 sequences, some slots padding
        dict(name="write one step", op="write", T=64, pad=5, Hkv=8, D=128, kv="e4m3", fused=False),
        # the framework's cache write workload: a packed prefill of 27654 tokens
        dict(name="write a prefill", op="write", T=27654, pad=0, Hkv=8, D=128, kv="e4m3", fused=False),
        # a chunk taken straight out of a fused projection's output: rows with a stride
        dict(name="write a fused chunk D=96", op="write", T=4099, pad=3, Hkv=16, D=96, kv="e5m2", fused=True),
        # one short context read back before its next chunk
        dict(name="read one context", op="read", S=1, lo=701, hi=701, Hkv=8, D=128, kv="e4m3"),
        # the contexts of the framework's chunked prefill workload (16 sequences, 2048 to 32768)
        dict(name="read 16 contexts", op="read", S=16, lo=2048, hi=32768, Hkv=8, D=128, kv="e4m3"),
        # ragged contexts, empty ones among them
        dict(name="read ragged D=64 e5m2", op="read", S=33, lo=0, hi=1501, Hkv=4, D=64, kv="e5m2"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("decode", "decode", "write", "read"))
    D, kv, Hkv = rng.choice(HEAD_SIZES), rng.choice(("e4m3", "e5m2")), rng.choice((1, 2, 3, 4, 5, 8, 10, 16))
    if op == "write":
        T = min(_log_int(rng, 1, 30000), 27654 * 8 * 128 // (Hkv * D))
        return dict(op=op, T=T, pad=rng.choice((0, 2, 7)), Hkv=Hkv, D=D, kv=kv, fused=rng.random() < 0.4)
    S = _log_int(rng, 1, 160)
    most = (64 * 32768 if op == "decode" else 16 * 32768) * 8 * 128  # of the listed largest, padded to the longest
    hi = max(1, min(_log_int(rng, 1, 131072), most // (S * Hkv * D)))
    lo = rng.choice((0, 1, hi // 3, hi))
    if op == "read":
        return dict(op=op, S=S, lo=lo, hi=hi, Hkv=Hkv, D=D, kv=kv)
    group = rng.choice((1, 2, 3, 4, 5, 7, 8, 12, 16))
    return dict(op=op, S=S, lo=lo, hi=hi, Hq=Hkv * group, Hkv=Hkv, D=D, kv=kv, out=rng.choice(("bf16", "bf16", "fp32")))


def _lengths(case):
    """Context lengths spread evenly from lo to hi; prepare() shuffles them."""
    S, lo, hi = case["S"], case["lo"], case["hi"]
    return [hi] if S == 1 else [lo + (hi - lo) * i // (S - 1) for i in range(S)]


def _blocks(n):
    return -(-n // BLOCK)


def work(case):
    Hkv, D = case["Hkv"], case["D"]
    if case["op"] == "write":
        kept = case["T"] - (case["T"] // case["pad"] if case["pad"] else 0)
        return {"bytes": kept * Hkv * 2 * (2 * D + D + 1) + 4 * case["T"], "flops": 0}
    lens = _lengths(case)
    tokens, tables = sum(lens), 4 * sum(map(_blocks, lens)) + 4 * case["S"]
    held = tokens * Hkv * 2 * (D + 1)  # codes and exponents
    if case["op"] == "read":
        return {"bytes": held + tokens * Hkv * 2 * 2 * D + tables + 4, "flops": 0}
    rows = case["S"] * case["Hq"]
    return {"bytes": held + tables + rows * (2 * D + (2 if case["out"] == "bf16" else 4) * D + 4),
            "flops": 4 * D * case["Hq"] * tokens}


# ---------------------------------------------------------------- inputs
def _cache(case, lens, g, dev):
    """A cache in use: codes and exponents of rows of about unit size, the sequences' blocks in random order."""
    nb = max(1, sum(map(_blocks, lens)))
    dt = CODES[case["kv"]]
    top = 100.0 if case["kv"] == "e4m3" else 12800.0
    cache = torch.empty(2, nb, BLOCK, case["Hkv"], case["D"], dtype=dt, device=dev)
    step = max(1, (1 << 27) // (BLOCK * case["Hkv"] * case["D"]))
    for half in range(2):
        for a in range(0, nb, step):
            b = min(nb, a + step)
            x = torch.randn(b - a, BLOCK, case["Hkv"], case["D"], generator=g, device=dev, dtype=torch.float32)
            cache[half, a:b] = (x * top).clamp_(-4.0 * top, 4.0 * top).to(dt)
    middle = 127 - int(math.log2(top))
    scales = torch.randint(middle - 1, middle + 2, (2, nb, case["Hkv"], BLOCK), generator=g, device=dev, dtype=torch.uint8)
    perm = torch.randperm(nb, generator=g, device=dev).to(torch.int32).cpu()
    table = torch.full((len(lens), max([_blocks(n) for n in lens] + [1])), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(lens):
        table[s, :_blocks(n)] = perm[at:at + _blocks(n)]
        at += _blocks(n)
    return cache, scales, table.to(dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    Hkv, D = case["Hkv"], case["D"]
    st = dict(case=case)
    if case["op"] == "write":
        T = case["T"]
        gain = torch.exp(0.7 * torch.randn(1, Hkv, D, generator=g, device=dev))  # channels of unequal size, as keys have
        if case["fused"]:  # queries, keys and values of a token side by side
            x = torch.randn(T, 4 * Hkv, D, generator=g, device=dev)
            x[:, 2 * Hkv:3 * Hkv] *= gain
            x = x.to(torch.bfloat16)
            st["key"], st["value"] = x[:, 2 * Hkv:3 * Hkv], x[:, 3 * Hkv:]
        else:
            st["key"] = (torch.randn(T, Hkv, D, generator=g, device=dev) * gain).to(torch.bfloat16)
            st["value"] = torch.randn(T, Hkv, D, generator=g, device=dev).to(torch.bfloat16)
        nb = _blocks(T) + 1
        slots = torch.randperm(nb, generator=g, device=dev)[:, None] * BLOCK + torch.arange(BLOCK, device=dev)
        slots = slots.reshape(-1)[:T].to(torch.int32)
        if case["pad"]:
            slots[case["pad"] - 1::case["pad"]] = -1
        st["slots"] = slots.contiguous()
        st["cache"] = torch.zeros(2, nb, BLOCK, Hkv, D, device=dev).to(CODES[case["kv"]])
        st["scales"] = torch.full((2, nb, Hkv, BLOCK), 1, dtype=torch.uint8, device=dev)
        return st
    lens = _lengths(case)
    order = torch.randperm(len(lens), generator=g, device=dev).tolist()
    lens = [lens[i] for i in order]
    st["lens"] = lens
    st["cache"], st["scales"], st["table"] = _cache(case, lens, g, dev)
    st["most"] = max(lens)
    if case["op"] == "read":
        cu = [0]
        for n in lens:
            cu.append(cu[-1] + n)
        st["cu"], st["total"] = torch.tensor(cu, dtype=torch.int32, device=dev), cu[-1]
    else:
        st["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        st["q"] = torch.randn(len(lens), case["Hq"], D, generator=g, device=dev).to(torch.bfloat16)
        st["scale"] = 1.0 / math.sqrt(D)
        st["out_dtype"] = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    op = st["case"]["op"]
    if own:
        import attention_forward_09_gb300 as gb

        if op == "write":
            gb.attn_kv_cache_write_fp8(st["key"], st["value"], st["slots"], st["cache"], st["scales"])
            return {"cache": st["cache"], "scales": st["scales"]}
        if op == "read":
            k, v = gb.attn_kv_cache_read_fp8(st["cache"], st["scales"], st["table"], st["cu"], st["total"])
            return {"k": k, "v": v}
        out, lse = gb.attn_fwd_paged_fp8(st["q"], st["cache"], st["scales"], st["table"], st["seq_lens"], st["most"],
                                         softmax_scale=st["scale"], lse=True, out_dtype=st["out_dtype"])
        return {"out": out, "lse": lse}
    return {"write": _write, "read": _read, "decode": _decode}[op](st)


def _power(e):
    """2^(e - 127) of exponent bytes e >= 1, exactly, in fp32."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _write(st):
    cache, scales = st["cache"], st["scales"]
    top = 9 if cache.dtype == torch.float8_e4m3fn else 16  # c_max = 0.875 * 2^top
    x = torch.stack((st["key"], st["value"])).float()  # [2, T, Hkv, D]
    fine = x.isfinite()
    most = torch.where(fine, x.abs(), 0.0).amax(-1)
    mant, ex = torch.frexp(most)  # most = mant * 2^ex, mant in [0.5, 1)
    e = (ex - top + (mant > 0.875).int()).clamp(min=-126)
    e = torch.where(most > 0, e, -126)
    codes = torch.where(fine, x * _power(127 - e)[..., None], float("nan")).to(cache.dtype)
    kept = st["slots"] >= 0
    slots = st["slots"][kept].long()
    block, at = slots // BLOCK, slots % BLOCK
    cache.view(torch.uint8)[:, block, at] = codes.view(torch.uint8)[:, kept]
    scales[0, block, :, at] = (e[0, kept] + 127).to(torch.uint8)
    scales[1, block, :, at] = (e[1, kept] + 127).to(torch.uint8)
    return {"cache": cache, "scales": scales}


def _read(st):
    t = torch.arange(st["total"], device=st["cu"].device, dtype=torch.int32)
    s = torch.searchsorted(st["cu"], t, right=True) - 1
    pos = t - st["cu"][s]
    block, at = st["table"][s, pos // BLOCK].long(), (pos % BLOCK).long()
    codes = st["cache"].view(torch.uint8)[:, block, at].view(st["cache"].dtype)  # [2, total, Hkv, D]
    e = torch.stack((st["scales"][0, block, :, at], st["scales"][1, block, :, at]))
    kv = (codes.float() * _power(e)[..., None]).to(torch.bfloat16)
    return {"k": kv[0], "v": kv[1]}


def _decode(st):
    q, cache, scales, lens = st["q"], st["cache"], st["scales"], st["seq_lens"]
    S, Hq, D = q.shape
    Hkv = cache.shape[3]
    table = st["table"].clamp(min=0).long()
    L = table.shape[1] * BLOCK
    seen = torch.arange(L, device=q.device) < lens[:, None]  # [S, L]

    def values(half):  # [S, Hkv, L, D] in fp32
        c = cache[half].view(torch.uint8)[table].view(cache.dtype).float()  # [S, blocks, 128, Hkv, D]
        e = _power(scales[half][table])  # [S, blocks, Hkv, 128]
        c = c * e.transpose(2, 3)[..., None]
        return c.reshape(S, L, Hkv, D).transpose(1, 2)

    qg = q.float().reshape(S, Hkv, Hq // Hkv, D)
    s = torch.matmul(qg, values(0).transpose(2, 3)) * st["scale"]  # [S, Hkv, group, L]
    s = torch.where(seen[:, None, None], s, float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, None, :, None], values(1), 0.0)
    o = torch.matmul(p, v) / torch.where(l > 0, l, 1.0)
    lse = m + torch.log(l)
    return {"out": o.reshape(S, Hq, D).to(st["out_dtype"]), "lse": lse.reshape(S, Hq)}


# ---------------------------------------------------------------- the definition in 64 bits
def _stands_for(kv, dev):
    """The value of each of the 256 codes, from the formats' definition."""
    exps, bias = (4, 7) if kv == "e4m3" else (5, 15)
    mants = 7 - exps
    table = []
    for c in range(256):
        e, f = (c >> mants) & ((1 << exps) - 1), c & ((1 << mants) - 1)
        v = math.ldexp(f, 1 - bias - mants) if e == 0 else math.ldexp((1 << mants) + f, e - bias - mants)
        if kv == "e4m3" and c & 127 == 127:
            v = math.nan
        elif kv == "e5m2" and e == 31:
            v = math.nan if f else math.inf
        table.append(-v if c & 128 else v)
    return torch.tensor(table, dtype=torch.float64, device=dev)


def exact(case, seed):
    st = prepare(case, seed)
    dev = st["cache"].device
    values = _stands_for(case["kv"], dev)
    raw = st["cache"].view(torch.uint8)
    if case["op"] == "write":
        # the nearest code of each value, found among all of them; ties to the even code
        pos = values[:128]
        pos = pos[pos.isfinite()]
        edges = (pos[1:] + pos[:-1]) / 2
        held = values[raw.long()]
        exps = st["scales"].clone()
        for half, x in enumerate((st["key"], st["value"])):
            x = x.double()
            fine = x.isfinite()
            most = torch.where(fine, x.abs(), 0.0).amax(-1)
            e = torch.ceil(torch.log2(most / pos[-1])).clamp(-126, 127)
            e = torch.where(most > pos[-1] * torch.exp2(e), e + 1, e)
            e = torch.where(most <= pos[-1] * torch.exp2(e - 1), e - 1, e).clamp(min=-126)
            a = (x / torch.exp2(e)[..., None]).abs()
            lo, up = torch.bucketize(a, edges), torch.bucketize(a, edges, right=True)
            code = torch.where(lo == up, lo, torch.where(lo % 2 == 0, lo, up))  # on an edge: the even of its two codes
            c = torch.where(fine, pos[code.clamp(max=pos.numel() - 1)] * torch.sign(x), math.nan)
            rows = torch.nonzero(st["slots"] >= 0).flatten()
            slots = st["slots"][rows].long()
            held[half].view(-1, case["Hkv"], case["D"]).index_copy_(0, slots, c[rows])
            by_slot = exps[half].transpose(1, 2).reshape(-1, case["Hkv"])
            by_slot.index_copy_(0, slots, (e[rows] + 127).to(torch.uint8))
            exps[half] = by_slot.view(-1, BLOCK, case["Hkv"]).transpose(1, 2)
        return {"cache": held, "scales": exps}

    def context(half, s):  # [tokens, Hkv, D]
        n = st["lens"][s]
        ids = st["table"][s, :_blocks(n)].long()
        e = st["scales"][half, ids].double() - 127.0  # [blocks, Hkv, 128]
        x = values[raw[half, ids].long()] * torch.exp2(e).permute(0, 2, 1)[..., None]
        return x.reshape(-1, case["Hkv"], case["D"])[:n]

    if case["op"] == "read":
        return {name: torch.cat([context(half, s) for s in range(case["S"])]) for half, name in enumerate("kv")}
    out = torch.zeros(case["S"], case["Hq"], case["D"], dtype=torch.float64, device=dev)
    lse = torch.full((case["S"], case["Hq"]), -math.inf, dtype=torch.float64, device=dev)
    group = case["Hq"] // case["Hkv"]
    for s, n in enumerate(st["lens"]):
        if n:
            k, v = context(0, s), context(1, s)
            q = st["q"][s].double().reshape(case["Hkv"], group, case["D"])
            scores = torch.einsum("hgd,nhd->hgn", q, k) * st["scale"]
            lse[s] = torch.logsumexp(scores, -1).reshape(-1)
            out[s] = torch.einsum("hgn,nhd->hgd", torch.softmax(scores, -1), v).reshape(case["Hq"], case["D"])
    return {"out": out, "lse": lse}
