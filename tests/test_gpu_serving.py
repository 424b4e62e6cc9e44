"""The serving calls on the GPU (rotary positions, the paged 4-bit cache,
attention of drafted tokens over it) against plain 64-bit forms.

Tolerances, from the number of roundings (u = 2^-24, one fp32 rounding):

* Rotary positions: the reduced angle is rounded to fp32 (at most pi u
  relative to a turn's half: an absolute error of pi u in the angle), cosine
  and sine are within 2 ulp (4 u), mscale, each product and the sum round once
  (4 u together): |y - exact| <= (|a| + |b|) |mscale| (pi + 4 + 4) u, taken as
  16 u, plus the output's own rounding.
* Read, and append without rotation: bit-exact. Rotated keys are formed and
  quantised in fp64, so their codes are those of the exact values.
* Attention: the score's dot product is a D-term fp32 sum of exact products,
  eps_t = |scale| (D + 2) u sum_d |q_d K_td|; the score scale and the reference
  of the exponents are fp32 numbers, so the exponent moves by up to
  4 u max |s|; exponential, T-term sums and merges: 8 (T + D) u, all relative
  errors of the weights. bf16 queries: a weight is rounded to bf16 (2^-8 at
  most) in the product and in the sum that normalises, 2^-7 together; codes may
  enter with 8 added, taken out by further products, so the sums' terms are
  at most |q| (|K| + 16 step) and p (|V| + 16 step), step = 2^s the block's scale.
  |o - exact| <= 2 expm1(2 max eps + 8 u max |s| + 8 (T + D) u (+ 2^-7)) sum_t
  p_t |V_t|, plus the output's rounding (bf16: half of 2^-7 relative).
"""
import math

import numpy as np
import pytest
import torch

from bit_gemm_hdiag_amd import synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import bit_gemm_hdiag_amd as mx
    return mx


def gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------ 64-bit forms
def rotated64(x, pos, freq, layout, mscale=1.0):
    """x [T, H, D] float64 -> (rotated, |a| + |b| of every element's pair)."""
    half = len(freq)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if layout == "pairs" else (i, i + half)
    ang = pos.astype(np.float64)[:, None, None] * freq
    y, m = x.copy(), np.zeros_like(x)
    y[..., a] = mscale * (x[..., a] * np.cos(ang) - x[..., b] * np.sin(ang))
    y[..., b] = mscale * (x[..., b] * np.cos(ang) + x[..., a] * np.sin(ang))
    m[..., a] = m[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    return y, m * abs(mscale)


def quantised64(x):
    """(codes uint8 [..., D/2], scales uint8 [..., D/32]) of float64 values."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = np.abs(b).max(-1)
    bad = ~np.isfinite(amax)
    safe = np.where(bad | (amax == 0), 1.0, amax)
    s = np.clip(np.frexp(safe)[1] - 1 - 2, -127, 127)
    s = np.where(amax == 0, -127, s)
    with np.errstate(invalid="ignore", over="ignore"):
        c = np.clip(np.rint(np.ldexp(b, -s[..., None])), -7, 7)
    c = np.where(bad[..., None], 0, c).astype(np.int64).reshape(x.shape) & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8), np.where(bad, 255, s + 127).astype(np.uint8)


def values64(codes, scales):
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1]).astype(np.int64)
    c = np.where(c > 7, c - 16, c).astype(np.float64)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127.0))
    return c * np.repeat(s, 32, -1)


def n64(t):
    return t.detach().double().cpu().numpy()


# ----------------------------------------------------------------------- rotary
@pytest.mark.parametrize("T,H,D,rot,dtype,form", [
    (1, 1, 2, 2, F32, "plain"), (1, 64, 128, 128, BF, "plain"), (8, 64, 128, 128, BF, "fused"),
    (37, 7, 96, 64, F32, "plain"), (37, 7, 96, 64, BF, "heads"), (5, 3, 80, 20, BF, "plain"),
    (300, 5, 64, 64, F32, "fused"), (130, 1, 256, 128, BF, "inplace"), (19, 3, 66, 34, BF, "odd"),
    (2, 300, 64, 32, F32, "inplace"), (1030, 33, 128, 128, BF, "fused"), (3, 2, 4096, 4096, F32, "plain")])
@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rope(mx, T, H, D, rot, dtype, form, layout):
    g = gen(T * 31 + H * 7 + D)
    if form == "heads":                                          # [H, T, D] storage
        x = torch.randn(H, T, D, generator=g).to(dtype).to(DEV).transpose(0, 1)
    elif form == "odd":                                          # rows that no 16-byte access fits
        x = torch.randn(T, H, D + 3, generator=g).to(dtype).to(DEV)[..., 1:D + 1]
    else:
        x = torch.randn(T, H + (5 if form == "fused" else 0), D, generator=g).to(dtype).to(DEV)[:, :H]
    pos = torch.randint(-1000000, 3000000, (T,), generator=g)
    pos[0] = 0
    freq = mx.mxs_rope_frequencies(rot, 10000.0, "linear", 2.0)
    out = x if form == "inplace" else None
    x0 = n64(x)
    y = mx.mxs_rope(x, pos.to(DEV), freq, layout=layout, mscale=1.25, out=out)
    ref, mag = rotated64(x0, pos.numpy(), n64(freq), layout, 1.25)
    err = np.abs(n64(y) - ref)
    assert np.all(err <= 16 * U * mag + HALF[dtype] * (np.abs(ref) + 16 * U * mag) + 1e-45)
    assert np.array_equal(n64(y)[..., rot:], x0[..., rot:])
    if form != "inplace":
        assert np.array_equal(n64(x), x0)


@pytest.mark.parametrize("layout", ["half", "pairs"])
def test_rope_negated_positions_are_its_gradient(mx, layout):
    T, H, D = 9, 4, 64
    g = gen(3)
    x, dy, step = (torch.randn(T, H, D, generator=g).to(DEV) for _ in range(3))
    pos = torch.randint(0, 100000, (T,), generator=g).to(DEV)
    freq = mx.mxs_rope_frequencies(D)
    dx = mx.mxs_rope(dy, -pos, freq, layout=layout, mscale=0.75)
    # the formula's gradient
    ref, mag = rotated64(n64(dy), -pos.cpu().numpy(), n64(freq), layout, 0.75)
    assert np.all(np.abs(n64(dx) - ref) <= 16 * U * mag + U * np.abs(ref))
    # differences: the map is linear, so one difference of any length is exact up to the calls' errors
    f = lambda t: (n64(mx.mxs_rope(t, pos, freq, layout=layout, mscale=0.75)) * n64(dy)).sum()
    want = (n64(dx) * n64(step)).sum()
    scale = 2 * (np.abs(n64(dy)) * (np.abs(n64(x)) + np.abs(n64(step)))).sum() + np.abs(n64(dx) * n64(step)).sum()
    assert abs(f(x + step) - f(x) - want) <= 64 * U * scale
    # and back
    back = mx.mxs_rope(mx.mxs_rope(x, pos, freq, layout=layout), -pos, freq, layout=layout)
    _, mag = rotated64(n64(x), pos.cpu().numpy(), n64(freq), layout)
    assert np.all(np.abs(n64(back) - n64(x)) <= 3 * 17 * U * mag)


def test_rope_nothing_to_do(mx):
    freq = mx.mxs_rope_frequencies(64)
    x = torch.empty(0, 4, 64, device=DEV)
    assert mx.mxs_rope(x, torch.empty(0, dtype=torch.int64, device=DEV), freq).shape == (0, 4, 64)
    with pytest.raises(ValueError):
        mx.mxs_rope(torch.zeros(2, 4, 64, device=DEV), torch.zeros(3, dtype=torch.int64, device=DEV), freq)
    with pytest.raises(ValueError):
        mx.mxs_rope(torch.zeros(2, 4, 64, device=DEV), torch.zeros(2, dtype=torch.int32, device=DEV), freq)
    with pytest.raises(TypeError):
        mx.mxs_rope(torch.zeros(2, 4, 64, device=DEV, dtype=torch.float16),
                    torch.zeros(2, dtype=torch.int64, device=DEV), freq)


# ------------------------------------------------------------------------ cache
def cache_arrays(c):
    return [t.cpu().numpy().reshape(-1, *t.shape[2:]) for t in (c.kc, c.ks, c.vc, c.vs)]


def filled(mx, pages, page, H, D, seed):
    """A pool whose every byte is set, scales in a sane range."""
    c = mx.kv4_cache_alloc(pages, page, H, D)
    g = torch.Generator(device=DEV).manual_seed(seed)
    for t in (c.kc, c.vc):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    for t in (c.ks, c.vs):
        t.copy_(torch.randint(118, 126, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    return c


CACHES = [(1, 1, 32, 1, 32, "half"), (3, 2, 64, 7, 32, "pairs"), (40, 3, 96, 17, 64, "half"),
          (129, 8, 128, 64, 128, "half"), (129, 8, 128, 64, 128, "pairs"), (70, 1, 256, 16, 20, "half"),
          (33, 5, 160, 16, 34, "pairs"), (2000, 8, 128, 256, 128, "half"), (600, 40, 128, 1, 64, "pairs")]


@pytest.mark.parametrize("T,H,D,page,rot,layout", CACHES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rotate", [False, True])
def test_append_then_read(mx, T, H, D, page, rot, layout, dtype, rotate):
    pages = -(-T // page) + 2
    g = gen(T + H * 13 + D)
    c = filled(mx, pages, page, H, D, T)
    before = cache_arrays(c)
    slots = torch.randperm(pages * page, generator=g)[:T]
    if T > 2:
        slots[1], slots[T - 1] = -1, pages * page              # skipped
    fused = synth.kv(T, 2 * H, D, T + 5, dtype=dtype).to(DEV)   # k and v as slices of fused rows
    k, v = fused[:, :H], fused[:, H:]
    pos = torch.randint(0, 40000, (T,), generator=g)
    pos[0] = 0
    kw = {}
    k64 = n64(k)
    if rotate:
        freq = mx.mxs_rope_frequencies(rot, 500000.0)
        kw = dict(positions=pos.to(DEV), freq=freq, layout=layout, mscale=1.5)
        k64, _ = rotated64(k64, pos.numpy(), n64(freq), layout, 1.5)
    mx.mxs_kv4_append(c, k, v, slots.to(DEV), **kw)
    want = [a.copy() for a in before]
    ok = (slots >= 0) & (slots < pages * page)
    dst = slots[ok].numpy()
    for j, x in ((0, k64), (2, n64(v))):
        codes, scales = quantised64(x)
        want[j][dst], want[j + 1][dst] = codes[ok.numpy()], scales[ok.numpy()]
    for name, got, ref in zip(("kc", "ks", "vc", "vs"), cache_arrays(c), want):
        assert np.array_equal(got, ref), name
    if not rotate:                                              # the rule of the contiguous quantiser
        kc, ks = mx.mxs_quantize_kv(k.contiguous())
        assert np.array_equal(kc.cpu().numpy()[ok.numpy()], want[0][dst])
        assert np.array_equal(ks.cpu().numpy()[ok.numpy()], want[1][dst])

    # read back: a permutation with repeats and rows that are left alone
    rd = torch.cat([slots, torch.tensor([-5, pages * page + 3]), slots[:1], slots[:1]])
    ok = ((rd >= 0) & (rd < pages * page)).numpy()
    for od in (BF, F32):
        outs = torch.full((rd.numel(), 2 * H, D), 7.0, dtype=od, device=DEV)
        mx.mxs_kv4_read(c, rd.to(DEV), k_out=outs[:, :H], v_out=outs[:, H:])
        got = n64(outs)
        for j, o in ((0, got[:, :H]), (2, got[:, H:])):
            ref = np.full(o.shape, 7.0)
            ref[ok] = values64(want[j][rd.numpy()[ok]], want[j + 1][rd.numpy()[ok]])
            assert np.array_equal(o, ref)
    ko, vo = mx.mxs_kv4_read(c, rd.to(DEV), F32)
    assert np.array_equal(n64(ko)[ok], values64(want[0][rd.numpy()[ok]], want[1][rd.numpy()[ok]]))
    assert not n64(vo)[~ok].any()


@pytest.mark.parametrize("rotate", [False, True])
def test_cache_blocks_at_the_edges(mx, rotate):
    """Zero, tiny, huge and non-finite blocks, and values on rounding borders."""
    D, H = 64, 2
    vals = [0.0, 1e-45, 1e-38, 2.0 ** -126, 3.0e38, 2.0 ** 100, float("inf"), float("-inf"), float("nan")]
    rows = torch.zeros(len(vals) + 2, H, D)
    for i, x in enumerate(vals):
        rows[i, :, 3] = x
        rows[i, 1, 40] = 1.0
    rows[len(vals)] = torch.arange(D).float() / 8 - 4           # steps of half a code and finer
    rows[len(vals) + 1] = -torch.arange(D).float() * 1.75
    T = rows.shape[0]
    c = filled(mx, 1, T, H, D, 5)
    k = rows.to(DEV)
    kw = {}
    k64 = n64(k)
    if rotate:
        freq = mx.mxs_rope_frequencies(32)
        pos = torch.zeros(T, dtype=torch.int64, device=DEV)     # the turn by zero keeps every bit
        kw = dict(positions=pos, freq=freq)
    mx.mxs_kv4_append(c, k, k, torch.arange(T, device=DEV), **kw)
    with np.errstate(invalid="ignore"):
        ref = quantised64(k64)
    kc, ks, vc, vs = cache_arrays(c)
    assert np.array_equal(vc, ref[0]) and np.array_equal(vs, ref[1])
    if rotate:                                                  # a pair holding Inf or NaN spoils both its blocks
        fin = np.isfinite(k64).all(axis=(1, 2))
        assert np.array_equal(kc[fin], ref[0][fin]) and np.array_equal(ks[fin], ref[1][fin])
        assert (ks[~fin][:, :, 0] == 255).all() and (kc[~fin][:, :, :16] == 0).all()
    else:
        assert np.array_equal(kc, ref[0]) and np.array_equal(ks, ref[1])
    ko, _ = mx.mxs_kv4_read(c, torch.arange(T, device=DEV), F32)
    assert np.array_equal(n64(ko), values64(kc, ks), equal_nan=True)


def test_cache_shapes_are_checked(mx):
    c = filled(mx, 2, 16, 2, 64, 1)
    k = torch.zeros(3, 2, 64, device=DEV)
    s = torch.arange(3, device=DEV)
    for bad in (dict(k=k[:2]), dict(v=k.bfloat16()), dict(slots=s.int()), dict(slots=s.cpu()), dict(k=k.cpu()),
                dict(k=k[..., ::2]), dict(positions=s), dict(k=torch.zeros(3, 2, 96, device=DEV))):
        a = dict(k=k, v=k, slots=s)
        a.update(bad)
        with pytest.raises(ValueError):
            mx.mxs_kv4_append(c, **a)
    with pytest.raises(TypeError):
        mx.mxs_kv4_append(c, k.half(), k.half(), s)
    with pytest.raises(ValueError):
        mx.KV4Cache(c.kc, c.ks, c.vc, c.vs[..., :1])
    with pytest.raises(ValueError):
        mx.mxs_kv4_read(c, s, k_out=k, v_out=k[:, :1])
    mx.mxs_kv4_append(c, k[:0], k[:0], s[:0])


# -------------------------------------------------------- attention of drafted tokens
def pack_bits(m):
    """bool [rows, n] -> int64 [rows, ceil(n / 64)]"""
    n = m.shape[1]
    w = max(1, -(-n // 64))
    b = np.zeros((m.shape[0], w * 64), dtype=np.uint64)
    b[:, :n] = m
    return torch.from_numpy((b.reshape(-1, w, 64) << np.arange(64, dtype=np.uint64)).sum(-1, dtype=np.uint64)
                            .view(np.int64)).to(DEV)


class Batch:
    """Sequences of the given cached and query token counts over random pages."""

    def __init__(self, mx, lens, ns, Hq, Hkv, D, page, dtype, mask, seed, spread=1.0, spare=2):
        rng = np.random.default_rng(seed)
        self.lens, self.ns, self.Hq, self.Hkv, self.D, self.page = lens, ns, Hq, Hkv, D, page
        B = len(lens)
        width = max(1, max(-(-L // page) for L in lens)) + 1
        need = [-(-L // page) for L in lens]
        self.cache = mx.kv4_cache_alloc(sum(need) + spare, page, Hkv, D)
        pages = self.cache.kc.shape[0]
        order = rng.permutation(pages)
        self.table = np.full((B, width), -1, dtype=np.int32)
        at = 0
        for b in range(B):
            self.table[b, :need[b]] = order[at:at + need[b]]
            at += need[b]
        T = pages * page
        K, V = (synth.kv(T, Hkv, D, seed + i, dtype=torch.float32) * spread for i in range(2))
        mx.mxs_kv4_append(self.cache, K.to(DEV), V.to(DEV), torch.arange(T, device=DEV))
        total = sum(ns)
        self.cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        g = gen(seed)
        self.q = torch.randn(total, Hq, D, generator=g).to(dtype).to(DEV)
        n_max = max(max(ns), 1)
        self.seen = np.zeros((total, n_max), dtype=bool)
        for b, n in enumerate(ns):
            m = np.tril(np.ones((n, n), dtype=bool))
            if mask != "causal":
                m = np.eye(n, dtype=bool)
                for j in range(1, n):
                    m[j] |= m[rng.integers(0, j)]
            if mask == "holes":
                m &= rng.random((n, n)) < 0.5
            self.seen[self.cu[b]:self.cu[b] + n, :n] = m
        self.bits = None if mask == "causal" else pack_bits(self.seen)
        self.scale = 1.0 / math.sqrt(D)

    def dev(self, x):
        return torch.from_numpy(np.asarray(x, dtype=np.int32)).to(DEV)

    def args(self, **kw):
        a = dict(table=self.dev(self.table), lens=self.dev(self.lens), cu=self.dev(self.cu), scale=self.scale,
                 mask=self.bits, max_q=max(max(self.ns), 1), max_len=max(self.lens))
        a.update(kw)
        return a

    def run(self, mx, **kw):
        return mx.mxs_attend_kv4_tree(kw.pop("q", self.q), self.cache, **self.args(**kw))

    def reference(self, scale=None):
        """(outputs, bounds) in float64."""
        scale = self.scale if scale is None else scale
        scale = float(np.float32(scale))
        kc, ks, vc, vs = cache_arrays(self.cache)
        pages = self.cache.kc.shape[0]
        q = n64(self.q)
        D, G = self.D, self.Hq // self.Hkv
        out, tol = np.zeros(q.shape), np.zeros(q.shape)
        low = 0.0 if self.q.dtype == F32 else 2.0 ** -7
        for b, (L, n) in enumerate(zip(self.lens, self.ns)):
            t = np.arange(L)
            pg = self.table[b, t // self.page]
            valid = (pg >= 0) & (pg < pages)
            slot = np.where(valid, pg, 0).astype(np.int64) * self.page + t % self.page
            K, V = values64(kc[slot], ks[slot]), values64(vc[slot], vs[slot])
            sk, sv = (np.repeat(np.exp2(x[slot].astype(np.float64) - 127.0), 32, -1) for x in (ks, vs))
            for i in range(n):
                row = self.cu[b] + i
                see = valid.copy()
                see[L - n:] &= self.seen[row, :n]
                if not see.any():
                    continue
                for h in range(self.Hq):
                    g = h // G
                    qk = K[see, g] * q[row, h]
                    s = scale * qk.sum(1)
                    with np.errstate(invalid="ignore"):
                        p = np.exp(s - s.max())
                    p /= p.sum()
                    out[row, h] = p @ V[see, g]
                    mk, mv = np.abs(K[see, g]), np.abs(V[see, g])
                    if low:
                        mk, mv = mk + 16 * sk[see, g], mv + 16 * sv[see, g]
                    eps = abs(scale) * (D + 2) * U * (mk * np.abs(q[row, h])).sum(1).max()
                    sums = 8 * (L + D) * U
                    rel = np.expm1(2 * eps + 8 * U * np.abs(s).max() + sums + low)
                    tol[row, h] = 2 * rel * (p @ np.abs(V[see, g])) + 2 * sums * (p @ mv)
        return out, tol + HALF[self.q.dtype] * (np.abs(out) + tol) + 1e-30

    def check(self, got, scale=None):
        ref, tol = self.reference(scale)
        err = np.abs(n64(got) - ref)
        bad = ~(err <= tol) & ~(np.isnan(ref) & np.isnan(n64(got)))
        assert not bad.any(), (np.argwhere(bad)[:4], float(np.nanmax(err / tol)))


# (lens, ns, Hq, Hkv, D, page, mask)
TREES = [
    ([1], [1], 1, 1, 32, 1, "causal"),
    ([5, 64, 65, 0, 1], [1, 1, 1, 1, 1], 8, 8, 64, 16, "causal"),
    ([300, 17, 256], [3, 17, 5], 8, 1, 128, 7, "tree"),
    ([500], [8], 64, 8, 128, 64, "tree"),
    ([0, 40, 333, 70], [0, 9, 13, 70], 12, 4, 96, 16, "holes"),
    ([200, 90], [33, 2], 16, 1, 256, 64, "tree"),
    ([130, 5], [129, 5], 5, 1, 160, 16, "tree"),
    ([700, 120, 64, 63, 128], [64, 65, 64, 63, 1], 6, 2, 64, 16, "causal"),
    ([190], [190], 4, 4, 32, 17, "causal"),
    ([2100, 900], [1, 1], 8, 2, 224, 64, "causal"),
    ([5000, 257, 1], [4, 2, 1], 16, 2, 128, 256, "tree"),
    ([1500] * 3, [40, 7, 21], 32, 4, 128, 64, "tree"),
    ([400, 600], [70, 90], 24, 3, 192, 32, "holes"),
    ([17000], [1], 2, 1, 32, 64, "causal"),                      # many token ranges, few lanes a row
    ([9000, 3], [3, 3], 16, 1, 64, 64, "tree"),
]


@pytest.mark.parametrize("lens,ns,Hq,Hkv,D,page,mask", TREES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_attention(mx, lens, ns, Hq, Hkv, D, page, mask, dtype):
    b = Batch(mx, lens, ns, Hq, Hkv, D, page, dtype, mask, sum(lens) + D)
    out = torch.full_like(b.q, float("nan"))
    b.run(mx, out=out)
    again = b.run(mx)
    assert torch.equal(out, again)                               # deterministic
    b.check(out)


# batches of more than 64 sequences (the schedule reads them 64 at a time), some
# without tokens or without queries: more tiles than workgroups, long tiles that
# lie in several shares, and one very long sequence among short ones
@pytest.mark.parametrize("case", ["short", "many", "ragged", "wide"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_attention_large_batches(mx, dtype, case):
    rng = np.random.default_rng(5)
    B, L, n, Hq, Hkv, D = {"short": (200, 40, 3, 2, 1, 32), "many": (150, 700, 1, 4, 4, 64),
                           "ragged": (70, 90, 2, 4, 2, 64), "wide": (66, 130, 70, 2, 1, 32)}[case]
    lens = rng.integers(1, L + 1, B)
    ns = np.minimum(rng.integers(0, n + 1, B), lens)
    lens[3] = ns[3] = 0
    ns[5:9] = 0
    if case == "ragged":
        lens[66], ns[66] = 6000, 2
    ns[B - 1], lens[B - 1] = min(n, L), L
    b = Batch(mx, lens.tolist(), ns.tolist(), Hq, Hkv, D, 16, dtype, "tree", 90 + B)
    got = b.run(mx)
    b.check(got)
    assert torch.equal(got, b.run(mx, max_len=None if case == "short" else int(lens.max())))


# 17 to 32 query rows a KV head in batches with many KV heads, and in the same batches with few
@pytest.mark.parametrize("D,longest", [(32, 300), (64, 1200), (96, 300), (128, 1200)])
@pytest.mark.parametrize("Hkv", [1, 4])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_attention_drafts_of_large_batches(mx, dtype, Hkv, D, longest):
    rng = np.random.default_rng(D)
    lens = rng.integers(0, 80, 68)
    lens[[7, 66]] = longest, longest - 1
    ns = np.minimum(rng.integers(0, 4, 68), lens)
    ns[[7, 66]] = 3
    b = Batch(mx, lens.tolist(), ns.tolist(), 10 * Hkv, Hkv, D, 16, dtype, "tree", 300 + D)
    got = b.run(mx)
    b.check(got)
    assert torch.equal(got, b.run(mx))


@pytest.mark.parametrize("Hq,Hkv,D,n", [(128, 1, 64, 1), (8, 8, 128, 1), (12, 12, 32, 2), (6, 6, 256, 1), (64, 8, 128, 1),
                                        (64, 2, 128, 5), (64, 1, 128, 9), (32, 1, 32, 40)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_attention_head_groups(mx, dtype, Hq, Hkv, D, n):
    """Every grouping of heads: one KV head to one a query head, over tiles that several shares hold."""
    b = Batch(mx, [1300, 60], [n, n], Hq, Hkv, D, 64, dtype, "tree", Hq + D)
    b.check(b.run(mx))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_attention_long_shares(mx, dtype):
    """More work than the workgroups take in one piece of a tile each."""
    b = Batch(mx, [9000, 8500, 7000, 8999], [1, 1, 1, 1], 8, 8, 128, 64, dtype, "causal", 61)
    b.check(b.run(mx))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_attention_mask_words(mx, dtype):
    """Bits past the drafted tokens and words past the mask do not count; unaligned query rows."""
    b = Batch(mx, [150, 90], [70, 10], 4, 2, 64, 16, dtype, "tree", 33)
    ref = b.run(mx)
    wide = torch.full((80, 5), -1, dtype=torch.int64, device=DEV)
    wide[:, :2] = b.bits
    n = torch.tensor([70] * 70 + [10] * 10)
    for r in range(80):                                          # set every bit from n on
        k = int(n[r])
        wide[r, 0] |= (-1 << k) if k < 64 else 0
        wide[r, 1] |= (-1 << max(0, k - 64)) if k >= 64 else -1
    assert torch.equal(b.run(mx, mask=wide), ref)
    b.seen[:70, 64:] = False                                     # one word: tokens 64 .. 69 unseen
    b.check(b.run(mx, mask=b.bits[:, :1].contiguous()))
    rows = torch.zeros(80, 4 * 64 + 3, dtype=dtype, device=DEV)
    rows[:, 1:257] = b.q.view(80, 256)
    odd = rows[:, 1:257].unflatten(1, (4, 64))
    assert odd.data_ptr() % 16 and torch.equal(b.run(mx, q=odd), ref)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_attention_of_one_token_agrees_with_attend_kv4(mx, dtype):
    b = Batch(mx, [1000], [1], 16, 2, 128, 1000, dtype, "causal", 4, spare=0)
    out = b.run(mx)
    flat = [t[0].contiguous() for t in (b.cache.kc, b.cache.ks, b.cache.vc, b.cache.vs)]
    b.table[0, 0] = 0
    one = mx.mxs_attend_kv4(b.q[0].float().contiguous(), flat[:2], flat[2:], b.scale)
    ref, tol = b.reference()
    assert np.all(np.abs(n64(one) - ref[0]) <= tol[0])
    assert np.all(np.abs(n64(out)[0] - n64(one)) <= 2 * tol[0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
def test_tree_attention_scales(mx, dtype, scale):
    b = Batch(mx, [150, 80], [9, 4], 8, 2, 64, 16, dtype, "tree", 11)
    b.check(b.run(mx, scale=scale), scale)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("wide", [False, True])
def test_tree_attention_unseen_tokens_do_not_reach_the_output(mx, dtype, wide):
    """NaN and huge values in tokens that a row does not see, in pages past the
    length and in pages that are not there; a row that sees a NaN gets it."""
    G = 8 if wide else 1
    b = Batch(mx, [210, 100, 64], [40, 12, 3], 2 * G, 2, 128, 16, dtype, "holes", 21)
    bad = {0: 200, 1: 95}                                        # one drafted token each
    c = b.cache
    for s, t in bad.items():
        pg, off = int(b.table[s, t // 16]), t % 16
        c.vs[pg, off, 1, 2] = 255
        c.vc[pg, off, 1, 32:48] = 0
        c.ks[pg, off, 0, 0] = 255
        c.kc[pg, off, 0, :16] = 0
    last = int(b.table[1, 99 // 16])                             # rows past the length of sequence 1
    for plane in (c.ks, c.vs):
        plane[last, 100 % 16:] = 255
    b.table[2, 1] = -1                                           # pages that are not there
    b.table[2, 2] = c.kc.shape[0]
    got = b.run(mx)
    ref, tol = b.reference()
    assert np.isnan(ref).any() and not np.isnan(ref).all()
    assert np.array_equal(np.isnan(n64(got)), np.isnan(ref))
    b.check(got)


def test_tree_attention_huge_scores(mx):
    b = Batch(mx, [300], [4], 8, 2, 64, 16, F32, "tree", 5, spread=30.0)
    b.check(b.run(mx))
    b.q.mul_(50.0)
    b.check(b.run(mx))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_attention_padded_rows_and_strides(mx, dtype):
    b = Batch(mx, [90, 40], [6, 5], 8, 2, 64, 16, dtype, "tree", 31)
    ref = b.run(mx, max_q=9, max_len=100)                        # the same bounds: the same split
    b.check(ref)
    rows = torch.full((20, 8 + 4, 64), float("nan"), dtype=dtype, device=DEV)
    rows[:11, :8] = b.q
    out = torch.full((20, 10, 64), 3.0, dtype=dtype, device=DEV)
    mask = torch.full((20, 1), -1, dtype=torch.int64, device=DEV)
    mask[:11] = b.bits
    b.run(mx, q=rows[:, :8], out=out[:, :8], mask=mask, max_q=9, max_len=100)
    assert torch.equal(out[:11, :8], ref)
    assert (out[11:] == 3.0).all() and (out[:, 8:] == 3.0).all()


def test_tree_attention_reads_padded_batches_in_bounds(mx):
    """Lengths and offsets past the host's bounds are cut off at them."""
    b = Batch(mx, [64, 64], [2, 2], 4, 2, 64, 16, F32, "causal", 8)
    ref = b.run(mx)
    got = b.run(mx, cu=b.dev([0, 2, 1 << 30]), lens=b.dev([64, 64]), max_q=2)
    assert torch.equal(got, ref)
    got = b.run(mx, lens=b.dev([64, 1 << 30]))
    assert torch.equal(got[:2], ref[:2]) and torch.isfinite(got).all()
    got = b.run(mx, lens=b.dev([64, -5]), cu=b.dev([0, 2, 2]))
    assert torch.equal(got[:2], ref[:2]) and not got[2:].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [5, 70])
def test_tree_attention_fewer_cached_tokens_than_queries(mx, dtype, n):
    """Three cached tokens: rows 0 to 2 see up to themselves, later rows all three."""
    b = Batch(mx, [n], [n], 4, 2, 64, 16, dtype, "causal", 9)
    bound = dict(max_q=n, max_len=n)
    got = b.run(mx, lens=b.dev([3]), **bound)
    first = b.run(mx, q=b.q[:3].contiguous(), lens=b.dev([3]), cu=b.dev([0, 3]), **bound)
    rest = b.run(mx, q=b.q[3:].contiguous(), lens=b.dev([3] * (n - 3)), cu=b.dev(range(n - 2)),
                 table=b.dev(np.repeat(b.table, n - 3, 0)), **bound)
    assert torch.equal(got, torch.cat([first, rest]))


def test_tree_attention_arguments_are_checked(mx):
    b = Batch(mx, [64, 64], [2, 2], 4, 2, 64, 16, F32, "tree", 8)
    for bad in (dict(table=b.dev(b.table).long()), dict(lens=b.dev([64])), dict(cu=b.dev([0, 2])),
                dict(mask=b.bits[:3]), dict(mask=b.bits.int()), dict(q=b.q[..., :32]), dict(q=b.q[:, :, ::2]),
                dict(out=torch.empty(4, 4, 64, dtype=BF, device=DEV)), dict(ws=torch.empty(8))):
        with pytest.raises(ValueError):
            b.run(mx, **bad)
    with pytest.raises(mx.MxsError):
        b.run(mx, max_len=16 * b.table.shape[1] + 1)
    with pytest.raises(mx.MxsError):
        b.run(mx, q=torch.zeros(4, 3, 64, device=DEV))


# -------------------------------------------------------------------- used together
class Server:
    """One layer's serving state: a pool, a page table, and a step that rotates
    and stores new tokens and attends over everything stored."""

    def __init__(self, mx, B, Hq, Hkv, D, page, width, seed):
        self.mx, self.B, self.Hq, self.Hkv, self.D, self.page = mx, B, Hq, Hkv, D, page
        self.cache = filled(mx, B * width + 1, page, Hkv, D, seed)
        self.table = torch.randperm(B * width + 1, generator=gen(seed))[:B * width].view(B, width).to(torch.int32)
        self.freq = mx.mxs_rope_frequencies(D, 10000.0, "parts", 4.0, original_length=256)
        self.keys = [[] for _ in range(B)]
        self.vals = [[] for _ in range(B)]

    def step(self, ns, depths, seen, seed):
        """Drafted tokens: positions = stored length + depth. Returns (got, want, tol)."""
        mx, H = self.mx, self.Hq + 2 * self.Hkv
        total = sum(ns)
        rows = torch.randn(total, H, self.D, generator=gen(seed)).to(BF).to(DEV)
        q, k, v = rows[:, :self.Hq], rows[:, self.Hq:self.Hq + self.Hkv], rows[:, self.Hq + self.Hkv:]
        old = [len(x) for x in self.keys]
        pos, slots, r = [], [], 0
        for b, n in enumerate(ns):
            for j in range(n):
                t = old[b] + j
                pos.append(old[b] + depths[r + j])
                slots.append(int(self.table[b, t // self.page]) * self.page + t % self.page)
            r += n
        pos, slots = torch.tensor(pos), torch.tensor(slots)
        lens = [o + n for o, n in zip(old, ns)]
        cu = np.concatenate([[0], np.cumsum(ns)]).astype(np.int32)
        i32 = lambda x: torch.tensor(np.asarray(x, dtype=np.int32), device=DEV)
        qr = mx.mxs_rope(q, pos.to(DEV), self.freq)
        mx.mxs_kv4_append(self.cache, k, v, slots.to(DEV), pos.to(DEV), self.freq)
        got = mx.mxs_attend_kv4_tree(qr, self.cache, self.table.to(DEV), i32(lens), i32(cu), self.D ** -0.5,
                                     mask=pack_bits(seen), max_q=max(ns), max_len=max(lens))
        # 64-bit: the stored tokens, rotated and quantised by the formulas
        f = n64(self.freq)
        k64, _ = rotated64(n64(k), pos.numpy(), f, "half")
        kq, vq = values64(*quantised64(k64)), values64(*quantised64(n64(v)))
        q64 = n64(qr)
        want, tol = np.zeros(q64.shape), np.zeros(q64.shape)
        G, r = self.Hq // self.Hkv, 0
        for b, n in enumerate(ns):
            self.keys[b] += list(kq[r:r + n])
            self.vals[b] += list(vq[r:r + n])
            K, V = np.array(self.keys[b]), np.array(self.vals[b])
            for i in range(n):
                see = np.ones(len(K), dtype=bool)
                see[old[b]:] = seen[r + i, :n]
                for h in range(self.Hq):
                    qk = K[see, h // G] * q64[r + i, h]
                    s = qk.sum(1) * self.D ** -0.5
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    want[r + i, h] = p @ V[see, h // G]
                    eps = self.D ** -0.5 * (self.D + 2) * U * np.abs(qk).sum(1).max()
                    rel = np.expm1(2 * eps + 8 * U * np.abs(s).max() + 8 * (len(K) + self.D) * U + 2.0 ** -7)
                    tol[r + i, h] = 2 * rel * (p @ np.abs(V[see, h // G]))
            r += n
        tol += HALF[BF] * (np.abs(want) + tol)
        ref, mag = rotated64(n64(q), pos.numpy(), f, "half")
        assert np.all(np.abs(q64 - ref) <= 16 * U * mag + HALF[BF] * (np.abs(ref) + 16 * U * mag))
        return got, want, tol

    def keep(self, counts):
        """The first counts[b] tokens of each sequence were accepted."""
        for b, n in enumerate(counts):
            del self.keys[b][n:], self.vals[b][n:]


def test_prompt_drafts_and_decode_together(mx):
    """A prompt in chunks, a drafted tree, some of it accepted, plain decode."""
    s = Server(mx, 2, 8, 2, 64, 16, 12, 3)
    chain = lambda ns: (np.concatenate([np.arange(n) for n in ns]),
                        np.concatenate([np.pad(np.tril(np.ones((n, n), bool)), ((0, 0), (0, max(ns) - n))) for n in ns]))
    for step, ns in enumerate(([50, 33], [40, 20])):             # the prompt in two chunks
        d, seen = chain(ns)
        got, want, tol = s.step(ns, d, seen, 100 + step)
        assert np.all(np.abs(n64(got) - want) <= tol)
    # a tree: token 0, children 1 2, grandchildren 3 (of 1), 4 (of 2); the other sequence drafts three in a chain
    seen = np.zeros((8, 5), bool)
    for i, anc in enumerate(([0], [0, 1], [0, 2], [0, 1, 3], [0, 2, 4])):
        seen[i, anc] = True
    seen[5:, :3] = np.tril(np.ones((3, 3), bool))
    got, want, tol = s.step([5, 3], [0, 1, 1, 2, 2, 0, 1, 2], seen, 200)
    assert np.all(np.abs(n64(got) - want) <= tol)
    s.keep([92, 55])                                             # tokens 0 and 1; 0 and 1
    for step in range(3):
        d, seen = chain([1, 1])
        got, want, tol = s.step([1, 1], d, seen, 300 + step)
        assert np.all(np.abs(n64(got) - want) <= tol)


@pytest.mark.parametrize("long", [False, True])
def test_serving_graph_replays_serve_growing_lengths(mx, long):
    """Rotation, append and attention captured once; every replay takes the
    lengths, slots and positions that its inputs hold then."""
    B, n, Hq, Hkv, D, page, width = 3, 4, 8, 2, 64, 16, (260 if long else 20)
    c = filled(mx, B * width, page, Hkv, D, 9)
    table = torch.randperm(B * width, generator=gen(1)).view(B, width).to(torch.int32).to(DEV)
    freq = mx.mxs_rope_frequencies(D)
    rows = torch.empty(B * n, Hq + 2 * Hkv, D, dtype=BF, device=DEV)
    q, k, v = rows[:, :Hq], rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:]
    qr, out = torch.empty(B * n, Hq, D, dtype=BF, device=DEV), torch.empty(B * n, Hq, D, dtype=BF, device=DEV)
    lens = torch.zeros(B, dtype=torch.int32, device=DEV)
    cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device=DEV)
    slots, pos = (torch.zeros(B * n, dtype=torch.int64, device=DEV) for _ in range(2))
    max_len = page * width
    ws = torch.empty(max(1, mx.mxs_attend_kv4_tree_workspace(BF, B, B * n, n, max_len, Hq, Hkv, D)), dtype=torch.uint8,
                     device=DEV)

    def step(o=out):
        mx.mxs_rope(q, pos, freq, out=qr)
        mx.mxs_kv4_append(c, k, v, slots, pos, freq)
        mx.mxs_attend_kv4_tree(qr, c, table, lens, cu, 0.125, max_q=n, max_len=max_len, out=o, ws=ws)

    def inputs(start, seed):
        rows.copy_(torch.randn(rows.shape, generator=gen(seed)))
        L = np.array([start, start // 2, max(n, start // 3)])
        lens.copy_(torch.from_numpy(L.astype(np.int32)))
        t = (L[:, None] - n + np.arange(n)).reshape(-1)
        tb = np.repeat(np.arange(B), n)
        slots.copy_(torch.from_numpy(table.cpu().numpy()[tb, t // page].astype(np.int64) * page + t % page))
        pos.copy_(torch.from_numpy(t))

    inputs(40, 1)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    eager = torch.empty_like(out)
    for rep, start in enumerate((40, 44, 200, 17, max_len, 300)):
        inputs(start, rep + 50)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        step(eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), rep
        ws.fill_(255)


def test_two_streams_at_once(mx):
    """Two batches on two streams, each with its own workspace."""
    bs = [Batch(mx, [3000], [4], 8, 2, 128, 64, BF, "tree", 50 + i) for i in range(2)]
    refs = [b.run(mx) for b in bs]
    args = [b.args() for b in bs]
    outs = [torch.empty_like(b.q) for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for b, a, o, s in zip(bs, args, outs, streams):
            with torch.cuda.stream(s):
                mx.mxs_attend_kv4_tree(b.q, b.cache, out=o, **a)
    torch.cuda.synchronize()
    for o, r in zip(outs, refs):
        assert torch.equal(o, r)


def test_two_graphs_share_a_workspace(mx):
    """Two captured calls over one workspace, replayed in turn and mixed with eager ones."""
    bs = [Batch(mx, [3000, 40], [5, 3], 8, 2, 64, 64, BF, "tree", 70), Batch(mx, [700], [40], 8, 2, 64, 16, BF, "tree", 71)]
    args = [b.args() for b in bs]
    need = max(mx.mxs_attend_kv4_tree_workspace(BF, len(b.lens), b.q.shape[0], max(b.ns), max(b.lens), 8, 2, 64) for b in bs)
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(b.q) for b in bs]
    call = lambda i: mx.mxs_attend_kv4_tree(bs[i].q, bs[i].cache, out=outs[i], ws=ws, **args[i])
    refs = [call(i).clone() for i in range(2)]
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1):
        for o in outs:
            o.fill_(float("nan"))
        graphs[i].replay()
        call(1 - i)
        torch.cuda.synchronize()
        assert torch.equal(outs[0], refs[0]) and torch.equal(outs[1], refs[1])


def test_slots_past_four_gigabytes(mx):
    """Offsets that pass 32 bits: the last slots of a pool of 5.1 GB of codes."""
    H, D, page = 64, 256, 1024
    pages = 620
    c = mx.kv4_cache_alloc(pages, page, H, D)
    assert c.kc.numel() > 2 ** 32
    T = 100
    k, v = (synth.kv(T, H, D, 60 + i).to(DEV) for i in range(2))
    first = pages * page - T
    slots = torch.arange(first, first + T, device=DEV)
    mx.mxs_kv4_append(c, k, v, slots)
    kc, ks = mx.mxs_quantize_kv(k)
    assert torch.equal(c.kc[-1, -T:], kc) and torch.equal(c.ks[-1, -T:], ks)
    ko, vo = mx.mxs_kv4_read(c, slots)
    small = mx.kv4_cache_alloc(1, page, H, D)
    mx.mxs_kv4_append(small, k, v, slots - (pages - 1) * page)
    kr, vr = mx.mxs_kv4_read(small, slots - (pages - 1) * page)
    assert torch.equal(ko, kr) and torch.equal(vo, vr)
    q = torch.randn(2, H, D, generator=gen(1)).to(BF).to(DEV)
    tokens = lambda p: torch.tensor([[p]], dtype=torch.int32, device=DEV)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    for x in (small.ks, small.vs, c.ks[-1:], c.vs[-1:]):
        x[:, :page - T].fill_(120)
    small.kc[0, :page - T] = c.kc[-1, :page - T]
    small.vc[0, :page - T] = c.vc[-1, :page - T]
    far = mx.mxs_attend_kv4_tree(q, c, tokens(pages - 1), i32(page), i32(0, 2), 0.0625, max_q=2, max_len=page)
    near = mx.mxs_attend_kv4_tree(q, small, tokens(0), i32(page), i32(0, 2), 0.0625, max_q=2, max_len=page)
    assert torch.equal(far, near)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 8, 40])
def test_tree_attention_zero_values_give_zero(mx, dtype, rows):
    """Blocks of zeros (byte 0) and tiny values: no offset or scale is left over."""
    b = Batch(mx, [200], [rows], 4, 2, 64, 16, dtype, "tree", 70)
    b.cache.vc[:] = 0
    b.cache.vs[:] = 0
    assert not b.run(mx).any()
    b.cache.kc[:] = 0
    b.cache.ks[:] = 0
    b.cache.vs[:] = 130                                          # zeros at a scale of 8
    assert not b.run(mx).any()
    b.cache.vc[..., 0] = 0x21                                    # 1 and 2, times 8, in every token
    out = n64(b.run(mx))
    # constant columns: the ratio of two T-term fp32 sums over the same weights (each
    # within 8 (T + D) u of its exact value), then the output's rounding
    tol = 2 * 8 * (200 + 64) * U + (1 + 2 ** -8) * HALF[dtype]
    assert np.all(np.abs(out[..., 0] - 8.0) <= 8.0 * tol)
    assert np.all(np.abs(out[..., 1] - 16.0) <= 16.0 * tol) and not out[..., 2:].any()
