"""Measured cases of the serving operators on the 4-bit K/V cache.

Three operators, in the order a serving step uses them:

* ``rope``   rotary positions on queries (``mxs_rope``);
* ``cache``  new keys and values quantised into a paged 4-bit cache as they
             are written, keys rotated on the way (``mxs_kv4_append``), and
             the sequences' tokens read back (``mxs_kv4_read``);
* ``tree``   attention of drafted tokens, one or many per sequence, over that
             cache, with a mask between the drafted tokens
             (``mxs_attend_kv4_tree``).

``own`` selects the library's kernels; otherwise the operators run in their
plain form. ``exact`` evaluates the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------- cases
def listed():
    return [
        # eight drafted tokens of one user, 70B query heads: latency of a small step
        dict(name="rope_draft8", op="rope", T=8, H=64, D=128, rot=128, dtype="bf16", layout="half",
             scaling="none", factor=1.0, base=10000.0, far=30000, fused=True),
        # a prompt of 2048 tokens, queries inside the fused q/k/v rows, scaled for long contexts
        dict(name="rope_prompt2048", op="rope", T=2048, H=64, D=128, rot=128, dtype="bf16", layout="half",
             scaling="parts", factor=8.0, base=500000.0, far=120000, fused=True),
        # fp32, interleaved pairs, two thirds of an odd head dimension, odd length, positions near a million
        dict(name="rope_pairs_f32", op="rope", T=4099, H=32, D=96, rot=64, dtype="f32", layout="pairs",
             scaling="linear", factor=4.0, base=10000.0, far=1000000, fused=False),
        # eight drafted tokens written to a short sequence, which is read back
        dict(name="cache_draft8", op="cache", T=8, S=520, H=8, D=128, page=64, rot=128, dtype="bf16",
             layout="half", base=10000.0, far=520),
        # odd head count and dimension, pages of 17 tokens, fp32, interleaved pairs on part of the head
        dict(name="cache_odd_f32", op="cache", T=777, S=1901, H=3, D=96, page=17, rot=64, dtype="f32",
             layout="pairs", base=10000.0, far=1901),
        # a chunk of 2048 prompt tokens behind 8192 cached ones, read back for the chunk's attention
        dict(name="cache_chunk2048", op="cache", T=2048, S=10240, H=8, D=128, page=64, rot=128, dtype="bf16",
             layout="half", base=500000.0, far=10240),
        # a long prompt stored without rotation and read back whole
        dict(name="cache_long32768", op="cache", T=32768, S=65536, H=8, D=128, page=256, rot=0, dtype="bf16",
             layout="half", base=10000.0, far=65536),
        # one user, one token, a short fp32 context: latency of the smallest step
        dict(name="tree_single", op="tree", B=1, n=1, L=500, Hq=64, Hkv=8, D=128, page=64, dtype="f32", mask="tree",
             empty=False),
        # a batch of 32 plain decode steps over ragged contexts, 8B heads: cache bytes are what counts
        dict(name="tree_decode32", op="tree", B=32, n=1, L=16384, Hq=32, Hkv=8, D=128, page=64, dtype="bf16",
             mask="causal", empty=False),
        # eight users with drafted trees of up to 26 tokens, 70B heads
        dict(name="tree_draft26", op="tree", B=8, n=26, L=8192, Hq=64, Hkv=8, D=128, page=64, dtype="bf16",
             mask="tree", empty=False),
        # odd everything: fp32, three query heads per KV head, D = 96, pages of 16, an empty sequence, empty rows
        dict(name="tree_odd_f32", op="tree", B=5, n=13, L=1777, Hq=12, Hkv=4, D=96, page=16, dtype="f32",
             mask="holes", empty=True),
        # sixteen users with trees of 64 tokens over long contexts: arithmetic is what counts
        dict(name="tree_wide64", op="tree", B=16, n=64, L=16384, Hq=64, Hkv=8, D=128, page=64, dtype="bf16",
             mask="tree", empty=False),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "cache", "tree", "tree"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    layout = rng.choice(["half", "pairs"])
    if op == "rope":
        D = rng.choice([64, 96, 128, 128, 256])
        scaling = rng.choice(["none", "linear", "ntk", "parts"])
        return dict(op=op, T=_log_int(rng, 1, 6000), H=rng.choice([1, 7, 8, 32, 64]), D=D,
                    rot=rng.choice([D, D, D // 2]), dtype=dtype, layout=layout, scaling=scaling,
                    factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                    base=rng.choice([10000.0, 500000.0]), far=_log_int(rng, 6000, 1000000), fused=rng.random() < 0.5)
    if op == "cache":
        D = rng.choice([32, 64, 96, 128, 128, 256])
        T = _log_int(rng, 1, 16000)
        return dict(op=op, T=T, S=T + _log_int(rng, 1, 16000), H=rng.choice([1, 3, 8, 8]), D=D,
                    page=rng.choice([16, 17, 64, 256]), rot=rng.choice([0, D, D, D // 2]), dtype=dtype, layout=layout,
                    base=rng.choice([10000.0, 500000.0]), far=40000)
    Hkv, G = rng.choice([(8, 8), (8, 4), (8, 1), (4, 3), (1, 16), (2, 5)])
    return dict(op=op, B=_log_int(rng, 1, 24), n=_log_int(rng, 1, 64), L=_log_int(rng, 65, 12000), Hq=Hkv * G, Hkv=Hkv,
                D=rng.choice([64, 96, 128, 128, 128, 256]), page=rng.choice([16, 17, 64, 256]), dtype=dtype,
                mask=rng.choice(["tree", "causal", "holes"]), empty=rng.random() < 0.3)


def _batch(case):
    """Lengths and drafted counts of a tree case: ragged, fixed by the case."""
    lens, ns = [], []
    for b in range(case["B"]):
        f = (b * 0.6180339887498949) % 1.0
        n = case["n"] if b == 0 else max(1, int(round(case["n"] * (1.0 - 0.5 * f))))
        L = case["L"] if b == 0 else max(n, int(round(case["L"] * (1.0 - 0.7 * f))))
        if case["empty"] and b == case["B"] - 1:
            L = n = 0 if case["B"] > 1 else 1
        lens.append(L)
        ns.append(n)
    return lens, ns


# ---------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda")


def _channels(H, D, g):
    """Gains of an outlier-channel model: a few strong channels, more mild ones."""
    u = torch.rand(H * D, generator=g, device="cuda")
    return (1.0 + 49.0 * (u < 0.002) + 3.0 * (u > 0.99)).view(H, D)


def _freq(rot, base, scaling, factor):
    """Radians per position of each rotated pair, 64 bits (original context 8192 for 'parts')."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2))
    f = base ** (-2.0 * i / rot)
    if scaling == "linear":
        f = f / factor
    if scaling == "parts":
        turns = 8192.0 * f / (2.0 * math.pi)
        keep = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        f = keep * f + (1.0 - keep) * f / factor
    return f.cuda()


def _pow2(e):
    """2^e in 64 bits, exactly, for whole -1022 <= e <= 1023."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _quantise64(x):
    """Codes (fp64 whole numbers) and scale exponents of 32-blocks of the last axis, x fp64."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax).exponent - 1 - 2).clamp(min=-127)
    e = torch.where(amax > 0, e, torch.full_like(e, -127))
    c = torch.round(b * _pow2(-e)).clamp(-7, 7)
    return c, e


def _pack(c, e):
    """(codes uint8 [..., D/2], scale bytes uint8 [..., D/32]) of _quantise64's result."""
    n = c.to(torch.int32).reshape(*c.shape[:-2], -1) & 15
    return (n[..., 0::2] | (n[..., 1::2] << 4)).to(torch.uint8), (e.squeeze(-1) + 127).to(torch.uint8)


def _unpack(codes, scales, dtype):
    """Values of packed codes [..., D/2] with scale bytes [..., D/32]."""
    c = codes.to(torch.int32)
    n = torch.stack([c & 15, c >> 4], -1).reshape(*codes.shape[:-1], -1)
    n = n - 16 * (n > 7)
    s = _pow2(scales.to(torch.int32) - 127).to(dtype)
    return (n.reshape(*n.shape[:-1], -1, 32).to(dtype) * s.unsqueeze(-1)).reshape(n.shape)


def _cache(slots_used, pages, page, H, D, g):
    """A cache whose used slots hold quantised keys and values, made in pieces."""
    parts = []
    for _ in range(2):
        codes = torch.randint(0, 256, (pages * page, H, D // 2), generator=g, device="cuda", dtype=torch.uint8)
        scales = torch.full((pages * page, H, D // 32), 120, device="cuda", dtype=torch.uint8)
        gain = _channels(H, D, g)
        for s in slots_used.split(16384):
            codes[s], scales[s] = _pack(*_quantise64((_randn((s.numel(), H, D), g) * gain).double()))
        parts += [codes.view(pages, page, H, D // 2), scales.view(pages, page, H, D // 32)]
    return parts


def _tree_mask(n, kind, g):
    """uint8 [n, n]: row i sees drafted token j (i itself and its ancestors, or j <= i)."""
    if kind == "causal":
        return torch.ones(n, n, dtype=torch.bool).tril()
    m = torch.eye(n, dtype=torch.bool)
    for j in range(1, n):
        p = int(torch.randint(0, j, (1,), generator=g))
        m[j] |= m[p]
    if kind == "holes":
        m &= torch.rand(n, n, generator=g) < 0.5
    return m


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case=case)
    if case["op"] == "rope":
        T, H, D = case["T"], case["H"], case["D"]
        rows = _randn((T, H + (16 if case["fused"] else 0), D), g).to(DTYPES[case["dtype"]])
        st["x"] = rows[:, :H]
        st["out"] = torch.empty((T, H, D), dtype=rows.dtype, device="cuda")
        first = int(torch.randint(0, max(1, case["far"] - T), (1,), generator=torch.Generator().manual_seed(seed)))
        st["positions"] = torch.arange(first, first + T, device="cuda")
        st["freq"] = _freq(case["rot"], case["base"], case["scaling"], case["factor"])
        return st
    cpu = torch.Generator().manual_seed(int(seed) + 1)
    if case["op"] == "cache":
        T, S, H, D, page = (case[k] for k in ("T", "S", "H", "D", "page"))
        need = -(-S // page)
        pages = need + 3
        order = torch.randperm(pages, generator=cpu)[:need]
        t = torch.arange(S)
        slots = (order[t // page] * page + t % page).cuda()
        st["slots_all"], st["slots_new"] = slots, slots[S - T:].contiguous()
        kc, ks, vc, vs = _cache(slots, pages, page, H, D, g)
        dt = DTYPES[case["dtype"]]
        gk, gv = _channels(H, D, g), _channels(H, D, g)
        st["k"] = (_randn((T, H, D), g) * gk).to(dt)
        st["v"] = (_randn((T, H, D), g) * gv).to(dt)
        st["positions"] = torch.arange(S - T, S, device="cuda")
        st["freq"] = _freq(case["rot"], case["base"], "none", 1.0) if case["rot"] else None
        st["k_out"], st["v_out"] = (torch.empty((S, H, D), dtype=dt, device="cuda") for _ in range(2))
    else:
        lens, ns = _batch(case)
        B, Hq, Hkv, D, page = (case[k] for k in ("B", "Hq", "Hkv", "D", "page"))
        width = max(1, -(-max(lens) // page))
        need = [-(-L // page) for L in lens]
        pages = sum(need) + 1
        order = torch.randperm(pages, generator=cpu)
        table = torch.full((B, width), -1, dtype=torch.int32)
        used, at = [], 0
        for b in range(B):
            table[b, :need[b]] = order[at:at + need[b]].to(torch.int32)
            at += need[b]
            t = torch.arange(lens[b])
            used.append(table[b, t // page].long() * page + t % page)
        kc, ks, vc, vs = _cache(torch.cat(used).cuda(), pages, page, Hkv, D, g)
        total = sum(ns)
        words = max(1, -(-max(ns) // 64))
        bits = torch.zeros(total, words, 64, dtype=torch.bool)
        r0 = 0
        for n in ns:
            m = torch.zeros(n, words * 64, dtype=torch.bool)
            if n:
                m[:, :n] = _tree_mask(n, case["mask"], cpu)
            bits[r0:r0 + n] = m.view(n, words, 64)
            r0 += n
        weight = (torch.ones(64, dtype=torch.int64) << torch.arange(64))
        st["bits"] = bits.view(total, -1).cuda()
        st["mask"] = (bits * weight).sum(-1).cuda()
        st["table"], st["lens"] = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        st["cu"] = torch.tensor([0] + ns, dtype=torch.int32).cumsum(0).to(torch.int32).cuda()
        st["host"] = (lens, ns)
        st["q"] = (_randn((total, Hq, D), g) * 1.5).to(DTYPES[case["dtype"]])
        st["out"] = torch.empty_like(st["q"])
        st["scale"] = 1.0 / math.sqrt(D)
    st["kc"], st["ks"], st["vc"], st["vs"] = kc, ks, vc, vs
    if own:
        import bit_gemm_hdiag_amd as mx
        st["cache"] = mx.KV4Cache(kc, ks, vc, vs)
        if case["op"] == "tree":
            n = mx.mxs_attend_kv4_tree_workspace(st["q"].dtype, case["B"], total, max(ns), max(lens), Hq, Hkv, D)
            st["ws"] = torch.empty(max(1, n), dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------------ plain forms
def _rotate(x, cos, sin, rot, layout):
    """x [T, H, D] with the first rot elements of each head rotated (cos, sin [T, 1, rot / 2])."""
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if layout == "pairs" else (r[..., :rot // 2], r[..., rot // 2:])
    y = (a * cos - b * sin, b * cos + a * sin)
    y = torch.stack(y, -1).flatten(-2) if layout == "pairs" else torch.cat(y, -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_rope(st):
    c = st["case"]
    ang = st["positions"].double()[:, None, None] * st["freq"]
    y = _rotate(st["x"].float(), ang.cos().float(), ang.sin().float(), c["rot"], c["layout"])
    return y.to(st["x"].dtype)


def _plain_cache(st):
    c = st["case"]
    k, v = st["k"].double(), st["v"].double()
    if c["rot"]:
        ang = st["positions"].double()[:, None, None] * st["freq"]
        k = _rotate(k, ang.cos(), ang.sin(), c["rot"], c["layout"])
    out = []
    for x, codes, scales in ((k, st["kc"], st["ks"]), (v, st["vc"], st["vs"])):
        codes, scales = codes.flatten(0, 1), scales.flatten(0, 1)
        codes[st["slots_new"]], scales[st["slots_new"]] = _pack(*_quantise64(x))
        out.append(_unpack(codes[st["slots_all"]], scales[st["slots_all"]], torch.float32).to(st["k"].dtype))
    return out


def _plain_tree(st):
    c = st["case"]
    page, Hkv = c["page"], c["Hkv"]
    G, r0, out = c["Hq"] // Hkv, 0, []
    for b, (L, n) in enumerate(zip(*st["host"])):
        if n == 0:
            continue
        q = st["q"][r0:r0 + n].float().view(n, Hkv, G, -1).transpose(0, 1).reshape(Hkv, n * G, -1)
        used = st["table"][b, :-(-L // page)].long()
        K, V = (_unpack(x[used].flatten(0, 1)[:L], s[used].flatten(0, 1)[:L], torch.float32).transpose(0, 1)
                for x, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
        s = (q @ K.transpose(1, 2).contiguous()) * st["scale"]                    # [Hkv, n G, L]
        s = s.view(Hkv, n, G, L)
        hide = ~st["bits"][r0:r0 + n, :n]
        s[..., L - n:] = s[..., L - n:].masked_fill(hide[None, :, None, :], -math.inf)
        m = s.amax(-1, keepdim=True)
        p = torch.exp(s - torch.where(m == -math.inf, torch.zeros_like(m), m))
        total = p.sum(-1, keepdim=True)
        o = (p.view(Hkv, n * G, L) @ V.contiguous()).view(Hkv, n, G, -1)
        o = o / torch.where(total == 0, torch.ones_like(total), total)
        out.append(o.transpose(0, 1).reshape(n, Hkv * G, -1).to(st["q"].dtype))
        r0 += n
    return torch.cat(out)


# ----------------------------------------------------------------------- one pass
def run(st):
    c = st["case"]
    if not own:
        return {"rope": _plain_rope, "cache": _plain_cache, "tree": _plain_tree}[c["op"]](st)
    import bit_gemm_hdiag_amd as mx
    if c["op"] == "rope":
        return mx.mxs_rope(st["x"], st["positions"], st["freq"], layout=c["layout"], out=st["out"])
    if c["op"] == "cache":
        rot = dict(positions=st["positions"], freq=st["freq"], layout=c["layout"]) if c["rot"] else {}
        mx.mxs_kv4_append(st["cache"], st["k"], st["v"], st["slots_new"], **rot)
        return list(mx.mxs_kv4_read(st["cache"], st["slots_all"], k_out=st["k_out"], v_out=st["v_out"]))
    return mx.mxs_attend_kv4_tree(st["q"], st["cache"], st["table"], st["lens"], st["cu"], st["scale"],
                                  mask=None if c["mask"] == "causal" else st["mask"], max_q=max(st["host"][1]),
                                  max_len=max(st["host"][0]), out=st["out"], ws=st["ws"])


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    D = case["D"]
    if case["op"] == "rope":
        n = case["T"] * case["H"]
        return {"bytes": 2 * n * D * es + 8 * case["T"] + 4 * case["rot"], "flops": 3 * n * case["rot"]}
    row = D // 2 + D // 32
    if case["op"] == "cache":
        T, S, H = case["T"], case["S"], case["H"]
        new = 2 * T * H * (D * es + row) + 8 * T * (2 if case["rot"] else 1)
        back = 2 * S * H * (D * es + row) + 8 * S
        return {"bytes": new + back, "flops": T * H * (3 * case["rot"] + 4 * 2 * D) + 2 * S * H * D}
    lens, ns = _batch(case)
    nbytes = 2 * sum(ns) * case["Hq"] * D * es + 2 * sum(lens) * case["Hkv"] * row
    # every row sees the context and, of the drafted tokens, itself at least
    seen = sum(n * (L - n + 1) for L, n in zip(lens, ns))
    return {"bytes": nbytes, "flops": 4 * D * case["Hq"] * seen}


# ------------------------------------------------------------- definitions, 64 bits
def _exact_pairs(rot, layout):
    """Element indices (first, second) of every rotated pair."""
    i = torch.arange(rot // 2, device="cuda")
    return (2 * i, 2 * i + 1) if layout == "pairs" else (i, i + rot // 2)


def _exact_rotation(x, pos, freq, rot, layout):
    """Pair (a, b) as the complex number a + ib, times exp(i pos freq)."""
    y = x.double().clone()
    i, j = _exact_pairs(rot, layout)
    z = torch.complex(y[..., i], y[..., j]) * torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                                                          pos.double()[:, None] * freq)[:, None, :]
    y[..., i], y[..., j] = z.real, z.imag
    return y


def _exact_steps():
    """2^(byte - 127) of every scale byte."""
    return torch.tensor([2.0 ** (i - 127) for i in range(256)], dtype=torch.float64, device="cuda")


def _exact_block_values(x):
    """The values that 4-bit blocks of 32 stand for: step 2^(floor(log2 amax) - 2), nearest whole step, at most 7."""
    b = x.unflatten(-1, (-1, 32))
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    step = _exact_steps()[(e - 3).clamp(min=-127).long() + 127]
    return (torch.round(b / step).clamp(-7, 7) * step).flatten(-2)


def _exact_stored(codes, scales):
    table = torch.tensor([0, 1, 2, 3, 4, 5, 6, 7, -8, -7, -6, -5, -4, -3, -2, -1], dtype=torch.float64, device="cuda")
    idx = codes.long()
    v = torch.empty((*codes.shape[:-1], codes.shape[-1] * 2), dtype=torch.float64, device="cuda")
    v[..., 0::2], v[..., 1::2] = table[idx % 16], table[idx // 16]
    return v * _exact_steps()[scales.long()].repeat_interleave(32, -1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        return _exact_rotation(st["x"], st["positions"], st["freq"], case["rot"], case["layout"])
    if case["op"] == "cache":
        T, S = case["T"], case["S"]
        k = st["k"].double()
        if case["rot"]:
            k = _exact_rotation(k, st["positions"], st["freq"], case["rot"], case["layout"])
        out = []
        for new, codes, scales in ((k, st["kc"], st["ks"]), (st["v"].double(), st["vc"], st["vs"])):
            old = st["slots_all"][:S - T]
            page, off = old // case["page"], old % case["page"]
            out.append(torch.cat([_exact_stored(codes[page, off], scales[page, off]), _exact_block_values(new)]))
        return out
    lens, ns = st["host"]
    G = case["Hq"] // case["Hkv"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    r0 = 0
    for b, (L, n) in enumerate(zip(lens, ns)):
        if L == 0 or n == 0:
            r0 += n
            continue
        t = torch.arange(L, device="cuda")
        page, off = st["table"][b].long()[t // case["page"]], t % case["page"]
        seen = torch.ones(n, L, dtype=torch.bool, device="cuda")
        seen[:, L - n:] = st["bits"][r0:r0 + n, :n]
        for h in range(case["Hkv"]):
            K = _exact_stored(st["kc"][page, off, h], st["ks"][page, off, h])
            V = _exact_stored(st["vc"][page, off, h], st["vs"][page, off, h])
            for g in range(G):
                s = st["q"][r0:r0 + n, h * G + g].double() @ K.t().contiguous() * st["scale"]
                w = torch.where(seen, torch.softmax(torch.where(seen, s, s.new_full((), -1e300)), -1), s.new_zeros(()))
                out[r0:r0 + n, h * G + g] = w @ V
        r0 += n
    return out
