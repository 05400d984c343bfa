"""Attention's backward pass and rotary positions, as cases that can be timed and checked.

Three operators, each through the package's own entry points where ``own`` is
true and in elementary torch operations where it is false:

  bwd     attn_bwd_dense, attn_bwd_padded, attn_bwd_varlen: the gradients of q, k and v from
          what the forward pass returned (out, lse) and the gradient of out (and of lse)
  rotate  attn_rotary: queries and keys turned by their positions, or (transpose) gradients turned back
  store   attn_rotary_kv_cache_write: queries turned; keys turned and, with the values, stored in the paged cache

bwd, with s_ij = scale * q_i.k_j over the visible pairs and out, lse as they were given:
  p_ij = exp(s_ij - lse_i),  delta_i = dout_i.out_i - dlse_i,  ds_ij = p_ij (dout_i.v_j - delta_i),
  dv_j = sum_i p_ij dout_i,  dq_i = scale sum_j ds_ij k_j,  dk_j = scale sum_i ds_ij q_i
(dk and dv summed over the query heads that share a KV head).  A row that sees no key has lse = -inf
and gives nothing; query rows and keys past a padded entry's lengths have gradient 0.

rotate, for pair i < rot / 2 of a head's first ``rot`` values at position t, a = t * f_i:
  (x, y) -> gain * (x cos a - y sin a, x sin a + y cos a)   (transpose: -a for a)
with (x, y) at i and i + rot / 2 ("half") or at 2 i and 2 i + 1 ("interleaved"); the rest of the head stays.
f_i = base^(-2 i / rot), changed for contexts longer than the trained length L by a factor s:
  linear    f / s
  ntk       base * s^(rot / (rot - 2)) in base's place
  by_parts  g f + (1 - g) f / s, g = clamp((L f / 2 pi - low) / (high - low), 0, 1)
  yarn      the same with g falling from 1 to 0 in equal steps of i, from floor(i(high)) to ceil(i(low)) where
            i(r) = rot ln(L / 2 pi r) / (2 ln base) is the pair that makes r turns over L (the ends kept within
            [0, rot - 1], 0.001 apart at least); gain = 0.1 ln s + 1
"""

import math

import torch

own = False

BLOCK = 128
HEAD_SIZES = (64, 96, 128, 192, 256)
MOST_FLOPS = 3.0e12       # of a drawn backward pass: about the largest listed one
MOST_SCORES = 1.1e9       # scores of all heads of a document (or batch) at once, in a drawn one
MOST_ROWS = 27654 * 48 * 128  # values turned or stored in a drawn case


# ---------------------------------------------------------------- cases
def listed():
    return [
        # the framework's tiny packed workload: what a short step waits for
        dict(name="backward of two short documents", op="bwd", form="varlen", N=2, lo=37, hi=91, ratio=1.0, Hq=4, Hkv=4, D=64,
             causal=False, out="fp32", dlse=False),
        # the framework's diffusion-transformer self-attention
        dict(name="backward of dit self-attention", op="bwd", form="dense", B=2, Sq=4096, Sk=4096, Hq=24, Hkv=24, D=128,
             causal=False, out="bf16", dlse=False),
        # eight packed documents, causal, four query heads to a KV head, as in the framework's packed workload
        dict(name="backward of packed causal documents", op="bwd", form="varlen", N=8, lo=512, hi=6401, ratio=1.0, Hq=32, Hkv=8,
             D=128, causal=True, out="bf16", dlse=False),
        # the framework's cross-attention: many video queries, few text keys; lse is used further on, so it has a gradient
        dict(name="backward of cross-attention", op="bwd", form="dense", B=1, Sq=16384, Sk=512, Hq=40, Hkv=40, D=128,
             causal=False, out="bf16", dlse=True),
        # a right-padded batch of odd lengths, one entry empty
        dict(name="backward of a padded batch D=96", op="bwd", form="padded", B=5, Sq=1021, Sk=1021, lo=0, hi=1021, Hq=12, Hkv=4,
             D=96, causal=True, out="fp32", dlse=False),
        # the framework's head size sweep at its ends
        dict(name="backward of self-attention D=64", op="bwd", form="dense", B=1, Sq=8192, Sk=8192, Hq=16, Hkv=16, D=64,
             causal=False, out="bf16", dlse=False),
        dict(name="backward of self-attention D=256", op="bwd", form="dense", B=1, Sq=8192, Sk=8192, Hq=16, Hkv=16, D=256,
             causal=False, out="bf16", dlse=False),
        # queries and keys of one decode step of 64 sequences
        dict(name="rotate one step", op="rotate", T=64, far=32768, Hq=32, Hkv=8, D=128, rot=128, layout="half", scaling="none",
             transpose=False, fused=False),
        # a packed prefill with positions scaled to four times the trained length
        dict(name="rotate a prefill", op="rotate", T=27654, far=32768, Hq=32, Hkv=8, D=128, rot=128, layout="half",
             scaling="yarn", transpose=False, fused=False),
        # gradients of a fused projection's queries and keys, half of each head turned
        dict(name="rotate gradients back D=96", op="rotate", T=4099, far=1 << 20, Hq=16, Hkv=16, D=96, rot=48,
             layout="interleaved", scaling="by_parts", transpose=True, fused=True),
        # one decode step of 64 sequences, some slots padding
        dict(name="rotate and store one step", op="store", T=64, far=32768, pad=5, Hq=32, Hkv=8, D=128, rot=128, layout="half",
             scaling="none", fused=True),
        # a packed prefill straight out of a fused projection
        dict(name="rotate and store a prefill", op="store", T=27654, far=32768, pad=0, Hq=32, Hkv=8, D=128, rot=128,
             layout="half", scaling="linear", fused=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("bwd", "bwd", "bwd", "rotate", "store"))
    D, Hkv = rng.choice(HEAD_SIZES), rng.choice((1, 2, 3, 4, 5, 8, 16))
    Hq = Hkv * rng.choice((1, 1, 2, 3, 4, 7, 8))
    if op != "bwd":
        T = max(1, min(_log_int(rng, 1, 27654), MOST_ROWS // ((Hq + 2 * Hkv) * D)))
        case = dict(op=op, T=T, far=rng.choice((1024, 32768, 1 << 20)), Hq=Hq, Hkv=Hkv, D=D,
                    rot=rng.choice((D, D, D // 2, 32, 20)), layout=rng.choice(("half", "interleaved")),
                    scaling=rng.choice(("none", "linear", "ntk", "by_parts", "yarn")), fused=rng.random() < 0.5)
        if op == "rotate":
            case["transpose"] = rng.random() < 0.5
        else:
            case["pad"] = rng.choice((0, 3, 5))
        return case
    Hkv = min(Hkv, 8)
    Hq = Hkv * rng.choice((1, 1, 2, 3, 4, 8))
    form = rng.choice(("dense", "padded", "varlen"))
    case = dict(op=op, form=form, Hq=Hq, Hkv=Hkv, D=D, causal=rng.random() < 0.5, out=rng.choice(("bf16", "fp32")),
                dlse=rng.random() < 0.25)
    n = _log_int(rng, 1, 12)
    Sq = _log_int(rng, 1, 9000)
    ratio = rng.choice((1.0, 1.0, 1.0, 0.25, 3.0))
    while 10 * D * Hq * n * Sq * max(1, Sq * ratio) > MOST_FLOPS or Hq * Sq * max(1, Sq * ratio) * (n if form != "varlen" else 1) > MOST_SCORES:
        Sq = Sq * 3 // 4
    Sq = max(1, Sq)
    if form == "varlen":
        case.update(N=n, lo=rng.choice((0, 1, Sq // 3, Sq)), hi=Sq, ratio=ratio)
        return case
    case.update(B=n, Sq=Sq, Sk=max(1, int(Sq * ratio)))
    if form == "padded":
        case.update(lo=rng.choice((0, 1, Sq // 2)), hi=Sq)
    return case


def _spread(lo, hi, n):
    """n lengths spread evenly from lo to hi."""
    return [hi] if n == 1 else [lo + (hi - lo) * i // (n - 1) for i in range(n)]


def _lengths(case):
    """(query rows, keys) of each document or batch entry; prepare() shuffles them."""
    if case["form"] == "dense":
        return [(case["Sq"], case["Sk"])] * case["B"]
    if case["form"] == "padded":
        return [(n, n * case["Sk"] // case["Sq"]) for n in _spread(case["lo"], case["hi"], case["B"])]
    return [(n, int(n * case["ratio"])) for n in _spread(case["lo"], case["hi"], case["N"])]


def _pairs(lq, lk, causal):
    if not causal:
        return lq * lk
    first = max(0, lq - lk)  # rows before this one see nothing
    n = lq - first
    return n * (lk - lq + first + 1) + n * (n - 1) // 2


def work(case):
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    if case["op"] == "bwd":
        lens = _lengths(case)
        rows, keys = sum(a for a, _ in lens), sum(b for _, b in lens)
        out_bytes = 2 if case["out"] == "bf16" else 4
        return {"bytes": rows * Hq * (D * (2 + 2 + 2 + out_bytes) + 4 + (4 if case["dlse"] else 0)) + keys * Hkv * D * 2 * 4,
                "flops": 10 * D * Hq * sum(_pairs(a, b, case["causal"]) for a, b in lens)}
    T, rot = case["T"], case["rot"]
    if case["op"] == "rotate":
        return {"bytes": T * ((Hq + Hkv) * D * 4 + 4), "flops": T * (Hq + Hkv) * rot * 3}
    kept = T - (T // case["pad"] if case["pad"] else 0)
    return {"bytes": T * (Hq * D * 4 + 8) + kept * Hkv * D * 8, "flops": (T * Hq + kept * Hkv) * rot * 3}


# ---------------------------------------------------------------- inputs
BASE = 10000.0


def _scaling(case):
    """The scaling's numbers, as a model's configuration holds them."""
    return {"none": None, "linear": dict(kind="linear", factor=2.0), "ntk": dict(kind="ntk", factor=8.0),
            "by_parts": dict(kind="by_parts", factor=8.0, low=1.0, high=4.0, length=8192),
            "yarn": dict(kind="yarn", factor=4.0, low=1.0, high=32.0, length=8192)}[case["scaling"]]


def _frequencies(rot, scaling):
    """(f_i of every pair, gain) in Python's floats."""
    s = scaling["factor"] if scaling else 1.0
    kind = scaling["kind"] if scaling else "none"
    base = BASE * s ** (rot / (rot - 2)) if kind == "ntk" else BASE
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        f = [x / s for x in f]
    elif kind == "by_parts":
        span = scaling["high"] - scaling["low"]
        g = [min(1.0, max(0.0, (scaling["length"] * x / (2 * math.pi) - scaling["low"]) / span)) for x in f]
        f = [a * x + (1 - a) * x / s for a, x in zip(g, f)]
    elif kind == "yarn":
        at = [rot * math.log(scaling["length"] / (2 * math.pi * r)) / (2 * math.log(base)) for r in (scaling["high"], scaling["low"])]
        lo, hi = min(max(math.floor(at[0]), 0), rot - 1), min(max(math.ceil(at[1]), 0), rot - 1)
        g = [1.0 - min(1.0, max(0.0, (i - lo) / max(hi - lo, 0.001))) for i in range(rot // 2)]
        f = [a * x + (1 - a) * x / s for a, x in zip(g, f)]
    return f, 0.1 * math.log(s) + 1.0 if kind == "yarn" else 1.0


def _visible(lq, lk, causal, dev):
    """[lq, lk]: which keys each row sees (the last row the last key)."""
    if not causal:
        return None
    return torch.arange(lk, device=dev) <= torch.arange(lq, device=dev)[:, None] + (lk - lq)


def _grouped(x, group):
    """[..., n, H, D] -> [..., H, group, n, D] in fp32, heads that share a KV head together."""
    n, H, D = x.shape[-3:]
    return x.float().reshape(*x.shape[:-2], H // group, group, D).movedim(-4, -2)


def _forward(q, k, v, scale, seen):
    """out and lse of [..., n, H, D] rows, out as it comes in fp32: [..., n, Hq, D], [..., Hq, n]."""
    group = q.shape[-2] // k.shape[-2]
    s = torch.matmul(_grouped(q, group), _grouped(k, 1).transpose(-1, -2)) * scale
    if seen is not None:
        s = torch.where(seen, s, float("-inf"))
    if s.shape[-1] == 0:
        m = torch.full(s.shape[:-1] + (1,), float("-inf"), device=s.device)
    else:
        m = s.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), 0.0, m)
    p = torch.exp(s - m0)
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _grouped(v, 1)) / torch.where(l > 0, l, 1.0)
    lse = (m0 + torch.log(l))[..., 0]
    return o.movedim(-2, -4).reshape(q.shape), lse.reshape(*q.shape[:-3], q.shape[-2], q.shape[-3])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    st = dict(case=case)

    def rows(*shape):
        return torch.randn(*shape, generator=g, device=dev).to(torch.bfloat16)

    if case["op"] != "bwd":
        T = case["T"]
        heads = Hq + 2 * Hkv
        if case["fused"]:  # queries, keys and values of a token side by side, as a fused projection leaves them
            x = rows(T, heads, D)
            st["q"], st["k"], st["v"] = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        else:
            st["q"], st["k"], st["v"] = rows(T, Hq, D), rows(T, Hkv, D), rows(T, Hkv, D)
        start = int(torch.randint(max(1, case["far"] - T), (1,), generator=g, device=dev))
        if T <= 256:  # a decode step: every token at a position of its own
            st["pos"] = torch.randint(case["far"], (T,), generator=g, device=dev).to(torch.int32)
        else:
            st["pos"] = (start + torch.arange(T, device=dev)).remainder(case["far"]).to(torch.int32)
        st["freqs"], st["gain"] = _frequencies(case["rot"], _scaling(case))
        if case["op"] == "store":
            nb = -(-T // BLOCK) + 1
            slots = torch.randperm(nb, generator=g, device=dev)[:, None] * BLOCK + torch.arange(BLOCK, device=dev)
            slots = slots.reshape(-1)[:T].to(torch.int32)
            if case["pad"]:
                slots[case["pad"] - 1::case["pad"]] = -1
            st["slots"] = slots.contiguous()
            st["cache"] = torch.zeros(2, nb, BLOCK, Hkv, D, dtype=torch.bfloat16, device=dev)
        if own:
            import attention_forward_09_gb300 as gb

            st["plan"] = gb.RotaryPlan(case["rot"], base=BASE, interleaved=case["layout"] == "interleaved",
                                       scaling=_scaling(case), device=dev)
        return st

    st["scale"] = 1.0 / math.sqrt(D)
    odt = torch.bfloat16 if case["out"] == "bf16" else torch.float32
    lens = _lengths(case)
    if case["form"] != "dense":
        order = torch.randperm(len(lens), generator=g, device=dev).tolist()
        lens = [lens[i] for i in order]
    st["lens"] = lens
    if case["form"] == "varlen":
        cq, ck = [0], [0]
        for a, b in lens:
            cq.append(cq[-1] + a)
            ck.append(ck[-1] + b)
        st["at"] = (cq, ck)
        st["q"], st["k"], st["v"], st["dout"] = rows(cq[-1], Hq, D), rows(ck[-1], Hkv, D), rows(ck[-1], Hkv, D), rows(cq[-1], Hq, D)
        st["cu_q"], st["cu_k"] = (torch.tensor(c, dtype=torch.int32, device=dev) for c in (cq, ck))
        st["out"] = torch.empty(cq[-1], Hq, D, dtype=odt, device=dev)
        st["lse"] = torch.empty(Hq, cq[-1], device=dev)
        for n, (a, b) in enumerate(lens):
            i, j = slice(cq[n], cq[n + 1]), slice(ck[n], ck[n + 1])
            o, st["lse"][:, i] = _forward(st["q"][i], st["k"][j], st["v"][j], st["scale"], _visible(a, b, case["causal"], dev))
            st["out"][i] = o.to(odt)
    else:
        B, Sq, Sk = case["B"], case["Sq"], case["Sk"]
        st["q"], st["k"], st["v"], st["dout"] = rows(B, Sq, Hq, D), rows(B, Sk, Hkv, D), rows(B, Sk, Hkv, D), rows(B, Sq, Hq, D)
        if case["form"] == "padded":
            st["lens_q"], st["lens_k"] = (torch.tensor(c, dtype=torch.int32, device=dev) for c in zip(*lens))
            st["out"] = torch.zeros(B, Sq, Hq, D, dtype=odt, device=dev)
            st["lse"] = torch.full((B, Hq, Sq), float("-inf"), device=dev)
            for n, (a, b) in enumerate(lens):
                o, st["lse"][n, :, :a] = _forward(st["q"][n, :a], st["k"][n, :b], st["v"][n, :b], st["scale"],
                                                  _visible(a, b, case["causal"], dev))
                st["out"][n, :a] = o.to(odt)
        else:
            o, st["lse"] = _forward(st["q"], st["k"], st["v"], st["scale"], _visible(Sq, Sk, case["causal"], dev))
            st["out"], st["lse"] = o.to(odt), st["lse"].contiguous()
    st["dlse"] = torch.randn(st["lse"].shape, generator=g, device=dev) if case["dlse"] else None
    return st


# ---------------------------------------------------------------- one pass
def run(st):
    case = st["case"]
    if own:
        import attention_forward_09_gb300 as gb

        if case["op"] == "rotate":
            q, k = gb.attn_rotary(st["q"], st["k"], st["pos"], st["plan"], transpose=case["transpose"])
            return {"q": q, "k": k}
        if case["op"] == "store":
            q = gb.attn_rotary_kv_cache_write(st["q"], st["k"], st["v"], st["pos"], st["plan"], st["slots"], st["cache"])
            return {"q": q, "cache": st["cache"]}
        known = (st["q"], st["k"], st["v"], st["out"], st["lse"], st["dout"])
        more = dict(softmax_scale=st["scale"], causal=case["causal"], dlse=st["dlse"])
        if case["form"] == "dense":
            dq, dk, dv = gb.attn_bwd_dense(*known, **more)
        elif case["form"] == "padded":
            dq, dk, dv = gb.attn_bwd_padded(*known, lens_q=st["lens_q"], lens_k=st["lens_k"], **more)
        else:
            dq, dk, dv = gb.attn_bwd_varlen(*known, st["cu_q"], st["cu_k"], max(a for a, _ in st["lens"]),
                                            max(b for _, b in st["lens"]), **more)
        return {"dq": dq, "dk": dk, "dv": dv}
    if case["op"] == "rotate":
        a = _angles(st, case["transpose"])
        return {"q": _turn(st["q"], a, case, st["gain"]), "k": _turn(st["k"], a, case, st["gain"])}
    if case["op"] == "store":
        a = _angles(st, False)
        kept = st["slots"] >= 0
        slots = st["slots"][kept].long()
        cache = st["cache"].view(2, -1, case["Hkv"], case["D"])
        cache[0, slots] = _turn(st["k"], a, case, st["gain"])[kept]
        cache[1, slots] = st["v"][kept]
        return {"q": _turn(st["q"], a, case, st["gain"]), "cache": st["cache"]}
    return _backward(st)


def _angles(st, transpose):
    """cos and sin [T, 1, rot / 2] in fp32, of angles in fp64."""
    a = st["pos"].double()[:, None] * torch.tensor(st["freqs"], dtype=torch.float64, device=st["pos"].device)
    a = -a if transpose else a
    return torch.cos(a).float()[:, None], torch.sin(a).float()[:, None]


def _turn(x, cos_sin, case, gain):
    c, s = cos_sin
    rot = case["rot"]
    x = x.float()
    if case["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * c - b * s, a * s + b * c), -1)
    else:
        a, b = x[..., :rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * c - b * s, a * s + b * c), -1).flatten(-2)
    return torch.cat((turned * gain, x[..., rot:]), -1).to(torch.bfloat16)


def _gradients(q, k, v, out, lse, dout, dlse, scale, seen):
    """dq, dk, dv in bf16 of [..., n, H, D] rows."""
    Hq, Hkv = q.shape[-2], k.shape[-2]
    group = Hq // Hkv
    Q, K, V, O, G = _grouped(q, group), _grouped(k, 1), _grouped(v, 1), _grouped(out, group), _grouped(dout, group)
    stat = lse.reshape(*lse.shape[:-2], Hkv, group, lse.shape[-1], 1)
    delta = (G * O).sum(-1, keepdim=True)
    if dlse is not None:
        delta = delta - dlse.reshape(stat.shape)
    empty = stat == float("-inf")
    p = torch.exp(torch.matmul(Q, K.transpose(-1, -2)) * scale - torch.where(empty, 0.0, stat))
    hidden = empty if seen is None else empty | ~seen
    p = torch.where(hidden, 0.0, p)
    dv = torch.matmul(p.transpose(-1, -2), G).sum(-3)
    ds = p * (torch.matmul(G, V.transpose(-1, -2)) - delta)
    dq = torch.matmul(ds, K) * scale
    dk = torch.matmul(ds.transpose(-1, -2), Q).sum(-3) * scale
    return (dq.movedim(-2, -4).reshape(q.shape).to(torch.bfloat16), dk.movedim(-2, -3).to(torch.bfloat16),
            dv.movedim(-2, -3).to(torch.bfloat16))


def _backward(st):
    case, dev = st["case"], st["q"].device
    causal, scale, dlse = case["causal"], st["scale"], st["dlse"]
    names = ("q", "k", "v", "out", "lse", "dout")
    if case["form"] == "dense":
        dq, dk, dv = _gradients(*(st[n] for n in names), dlse, scale, _visible(case["Sq"], case["Sk"], causal, dev))
        return {"dq": dq, "dk": dk.contiguous(), "dv": dv.contiguous()}
    dq, dk, dv = (torch.zeros_like(st[n]) for n in "qkv")
    for n, (a, b) in enumerate(st["lens"]):
        if case["form"] == "padded":
            i, j, stat = (n, slice(0, a)), (n, slice(0, b)), (n, slice(None), slice(0, a))
        else:
            cq, ck = st["at"]
            i, j = slice(cq[n], cq[n + 1]), slice(ck[n], ck[n + 1])
            stat = (slice(None), i)
        dq[i], dk[j], dv[j] = _gradients(st["q"][i], st["k"][j], st["v"][j], st["out"][i], st["lse"][stat], st["dout"][i],
                                         None if dlse is None else dlse[stat], scale, _visible(a, b, causal, dev))
    return {"dq": dq, "dk": dk, "dv": dv}


# ---------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    dev = st["q"].device
    if case["op"] == "bwd":
        dq, dk, dv = (torch.zeros(st[n].shape, dtype=torch.float64, device=dev) for n in "qkv")
        group = case["Hq"] // case["Hkv"]
        for n, (a, b) in enumerate(st["lens"]):
            for h in range(case["Hq"]):
                if case["form"] == "varlen":
                    i, j = slice(st["at"][0][n], st["at"][0][n + 1]), slice(st["at"][1][n], st["at"][1][n + 1])
                    i, j, r = (i, h), (j, h // group), (h, i)
                else:
                    i, j, r = (n, slice(0, a), h), (n, slice(0, b), h // group), (n, h, slice(0, a))
                q, k, v = st["q"][i].double(), st["k"][j].double(), st["v"][j].double()
                go, lse = st["dout"][i].double(), st["lse"][r].double()
                delta = torch.einsum("nd,nd->n", go, st["out"][i].double())
                if st["dlse"] is not None:
                    delta -= st["dlse"][r].double()
                p = torch.mm(q, k.t()).mul_(st["scale"]).sub_(lse[:, None]).exp_()
                if case["causal"]:
                    p.tril_(b - a)  # key j of row i is kept where j <= i + (b - a)
                p[lse == -math.inf] = 0.0
                dv[j] += torch.mm(p.t(), go)
                p.mul_(torch.mm(go, v.t()).sub_(delta[:, None])).mul_(st["scale"])
                dq[i] = torch.mm(p, k)
                dk[j] += torch.mm(p.t(), q)
        return {"dq": dq, "dk": dk, "dv": dv}
    rot, D = case["rot"], case["D"]
    # the frequency of each pair from the definition, one at a time
    sc, half, freqs, gain = _scaling(case) or dict(kind="none", factor=1.0), rot // 2, [], 1.0
    kind, s = sc["kind"], sc["factor"]
    for i in range(half):
        log_f = -(2.0 * i / rot) * math.log(BASE)
        if kind == "ntk":
            log_f -= (2.0 * i / (rot - 2)) * math.log(s)
        f = math.exp(log_f)
        keep = 1.0
        if kind == "linear":
            keep = 0.0
        elif kind == "by_parts":
            turns = sc["length"] * f / (2.0 * math.pi)
            keep = 0.0 if turns <= sc["low"] else 1.0 if turns >= sc["high"] else (turns - sc["low"]) / (sc["high"] - sc["low"])
        elif kind == "yarn":
            ends = [half * (math.log(sc["length"]) - math.log(2.0 * math.pi * r)) / math.log(BASE) for r in (sc["high"], sc["low"])]
            a, b = max(0, min(rot - 1, math.floor(ends[0]))), max(0, min(rot - 1, math.ceil(ends[1])))
            keep = 1.0 if i <= a else 0.0 if i >= b else 1.0 - (i - a) / (b - a)
            gain = 1.0 + math.log(s) / 10.0
        freqs.append(f * keep + f * (1.0 - keep) / s)
    turn = torch.polar(torch.full((half,), gain, dtype=torch.float64, device=dev).expand(case["T"], half).contiguous(),
                       torch.outer(st["pos"].double(), torch.tensor(freqs, dtype=torch.float64, device=dev)))
    if case.get("transpose"):
        turn = turn.conj()
    pair = torch.arange(half, device=dev)
    first, second = (pair, pair + half) if case["layout"] == "half" else (2 * pair, 2 * pair + 1)

    def turned(x):
        y = x.double().clone()
        z = torch.complex(y[..., first], y[..., second]) * turn[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        return y

    if case["op"] == "rotate":
        return {"q": turned(st["q"]), "k": turned(st["k"])}
    cache = st["cache"].double()
    by_slot = cache.view(2, -1, case["Hkv"], D)
    rows = torch.nonzero(st["slots"] >= 0).flatten()
    for half_of, x in ((0, turned(st["k"])), (1, st["v"].double())):
        by_slot[half_of].index_copy_(0, st["slots"][rows].long(), x[rows])
    return {"q": turned(st["q"]), "cache": cache}
