"""Attention of drafted tokens, token by token: every cached token is counted
once, wherever it lies in stages, pieces, shares and pages.

Keys are 4 times rows of a Hadamard matrix for one anchor token and for the
tokens under test, and codes of 1 or -1 for all others. The query of a row is
the sum of the anchor's key and of one tested token t's, so these two score
exactly 16 D and the other tested ones exactly 0; any other token scores at most
8 D / 2 and, for random signs, within 6 sqrt(32 D) of 0 (checked). At scale 1/8
all others together weigh less than T e^-40 of the two, so the output is
(V_t + V_a) / 2, or V_a where the row does not see t: multiples of a half, exact
in both types. A token lost or counted twice moves it by |V_t - V_a| / 6 at
least, which the test checks to be far past the bound.

Bound (u = 2^-24): one rounding of the running sum, or its half ulp, for every
32 tokens and for merging and normalising (64 more), on terms of at most
|V_t| + |V_a| + 32 (codes may enter with 8 added and be taken out again), and
the output's own rounding.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
HALF = {F32: U, BF: 2.0 ** -8}


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import bit_gemm_hdiag_amd as mx
    return mx


def packed(codes):
    """Whole numbers -8 .. 7 [..., D] -> bytes [..., D / 2]."""
    c = codes.to(torch.int32) & 15
    return (c[..., 0::2] | (c[..., 1::2] << 4)).to(torch.uint8)


def hadamard(D):
    """32 orthogonal rows of D signs."""
    h = torch.ones(1, 1)
    while h.shape[0] < 32:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    return h.repeat(1, D // 32)


class Pinned:
    """Sequences of lens cached and ns query tokens (causal); anchors[b] is seen by every row."""

    def __init__(self, mx, lens, ns, Hkv, G, D, page, dtype, seed, anchors=None):
        self.mx, self.lens, self.ns, self.Hkv, self.G, self.D, self.dtype = mx, lens, ns, Hkv, G, D, dtype
        self.anchors = anchors or [0] * len(lens)
        g = torch.Generator().manual_seed(seed)
        need = [-(-L // page) for L in lens]
        pages = sum(need) + 1
        order = torch.randperm(pages, generator=g).to(torch.int32)
        table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.slots = [(table[b, torch.arange(L) // page].long() * page + torch.arange(L) % page).to(DEV)
                      for b, L in enumerate(lens)]
        self.cache = mx.kv4_cache_alloc(pages, page, Hkv, D)
        sign = 2 * torch.randint(0, 2, (pages * page, Hkv, D), generator=g) - 1
        self.v = torch.randint(-7, 8, (pages * page, Hkv, D), generator=g).to(DEV)
        self.keys = hadamard(D).to(DEV)
        for b, a in enumerate(self.anchors):
            sign[self.slots[b][a].cpu()] = 4 * self.keys[0].cpu().long()
        self.others = packed(sign).to(DEV)
        c = self.cache
        self.kc = c.kc.view(-1, Hkv, D // 2)
        self.kc.copy_(self.others)
        c.vc.view(-1, Hkv, D // 2).copy_(packed(self.v))
        c.ks.fill_(127)
        c.vs.fill_(127)
        # no other token comes near 16 D
        q = (self.keys[0] + self.keys[1:]).double()
        far = sign.double().to(DEV).flatten(0, 1) @ q.t().contiguous() * 4
        hit = (far.abs() > 15 * D).any(1).view(pages * page, Hkv)      # the anchors
        assert int(hit.sum()) == Hkv * len(lens)
        assert float(far.abs()[~hit.flatten()].max()) <= min(6 * (32 * D) ** 0.5, 16 * D - 320)
        dev = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)
        self.table, self.dlens = table.to(DEV), dev(lens)
        self.cu = dev([0] + list(np.cumsum(ns)))
        self.total = sum(ns)
        self.ws = torch.empty(max(1, mx.mxs_attend_kv4_tree_workspace(dtype, len(lens), self.total, max(ns), max(lens),
                                                                      Hkv * G, Hkv, D)), dtype=torch.uint8, device=DEV)

    def one(self, sets):
        """Tokens sets[b] of every sequence, each the target of some row of every KV head: the worst
        excess over the bound, and the least margin of a lost or doubled token."""
        Hkv, G, D = self.Hkv, self.G, self.D
        touched, qs, refs, tols, margins = [], [], [], [], []
        for b, s in enumerate(sets):
            n, L, anchor = self.ns[b], self.lens[b], self.anchors[b]
            if n == 0:
                continue
            assert 1 <= len(s) <= min(31, n * G) and anchor not in s
            slots = self.slots[b][torch.tensor(s, device=DEV)]
            self.kc[slots] = packed(4 * self.keys[1:1 + len(s)])[:, None]
            touched.append(slots)
            r = torch.arange(n * G, device=DEV).view(n, 1, G) + 7 * torch.arange(Hkv, device=DEV).view(1, Hkv, 1)
            j = r % len(s)                                        # [n, Hkv, G]: the row's target
            qs.append(4 * (self.keys[0] + self.keys[1 + j]))
            t = torch.tensor(s, device=DEV)[j]
            see = (t < L - n) | (t - (L - n) <= torch.arange(n, device=DEV).view(n, 1, 1))
            head = torch.arange(Hkv, device=DEV).view(1, Hkv, 1).expand(n, Hkv, G)
            vt = self.v[self.slots[b][t], head].double()
            va = self.v[self.slots[b][anchor]].double().view(1, Hkv, 1, D)
            refs.append(torch.where(see[..., None], (vt + va) / 2, va.expand_as(vt)))
            tol = 2 * U * (L / 32 + 64) * (vt.abs() + va.abs() + 32) + HALF[self.dtype] * refs[-1].abs()
            tols.append(tol)
            margins.append(((vt - va).abs() / 6 - 8 * tol).amax(-1).min())
        q = torch.cat(qs).reshape(self.total, Hkv * G, D).to(self.dtype)
        out = self.mx.mxs_attend_kv4_tree(q, self.cache, self.table, self.dlens, self.cu, 0.125, max_q=max(self.ns),
                                          max_len=max(self.lens), ws=self.ws)
        for slots in touched:
            self.kc[slots] = self.others[slots]
        err = (out.double().view(self.total, Hkv, G, D) - torch.cat(refs)).abs() - torch.cat(tols)
        return torch.where(err == err, err, torch.full_like(err, 9.0)).max(), torch.stack(margins).min()

    def sweep(self, tokens=None):
        """Every token of every sequence (or those of tokens[b]), in passes."""
        todo = [[t for t in (range(L) if tokens is None else tokens[b]) if t != self.anchors[b]]
                for b, L in enumerate(self.lens)]
        per = [min(31, n * self.G) for n in self.ns]
        passes = max(-(-len(t) // p) for t, p in zip(todo, per) if p)
        worst = []
        for k in range(passes):
            # a sequence that is through starts again
            sets = []
            for t, p in zip(todo, per):
                first = (k * p) % max(1, len(t))
                sets.append((t[first:] + t)[:min(p, len(t))])
            worst.append(torch.stack(self.one(sets)))
        worst = torch.stack(worst).cpu()
        assert float(worst[:, 1].min()) > 0, "a lost token would not show"
        bad = torch.nonzero(worst[:, 0] > 0).flatten().tolist()
        assert not bad, (bad[:5], worst[bad[:5]])


def near(L, step, width=1):
    """Tokens around every multiple of step."""
    return sorted({t for m in range(0, L + step, step) for t in range(m - width, m + width + 1) if 0 <= t < L})


# One tile in 2 to 64 pieces: the join's groups of lanes take several turns, or
# only some of them have a row (few rows of a workgroup, many groups)
@pytest.mark.parametrize("D", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("L", [600, 1100, 1300, 1700, 2000, 2100, 4100, 7000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_join_takes_every_piece_once(mx, D, L, dtype):
    for n, G in ((1, 1), (3, 8)) if L < 4000 else ((1, 2),):
        p = Pinned(mx, [L], [n], 1, G, D, 64, dtype, L + D, anchors=[L // 2 + 3])
        step = 64 if L < 4000 else 256
        p.sweep([near(L, step)[::1 if n * G > 1 else 3]])


# (lens, ns, Hkv, G, D, page): every kernel, tiles whole and in pieces, pages that
# end inside stages, ragged batches (shares end anywhere), rows past the last tile
SWEEPS = {
    "rows, decode": ([1500, 333, 65], [1, 1, 1], 8, 8, 128, 64),
    "rows, one head a group": ([1100, 700], [1, 1], 1, 16, 64, 17),
    "rows, chain": ([900, 1290], [4, 2], 2, 4, 96, 16),
    "rows, D 256": ([1300], [2], 2, 8, 256, 64),
    "rows, short": ([500, 1, 257], [1, 1, 1], 4, 8, 128, 16),
    "rows, D 32": ([2100], [1], 4, 16, 32, 1),
    "tile, two waves a row group": ([1000, 203], [5, 3], 2, 8, 128, 64),
    "tile, four row groups": ([777, 130], [12, 5], 1, 8, 64, 16),
    "tile, D 224": ([700, 513], [9, 2], 1, 8, 224, 33),
    "pair": ([1030, 450, 129], [40, 17, 33], 2, 8, 128, 64),
    "pair, odd": ([640, 900], [129, 70], 3, 2, 64, 7),
    "pair, prompt from nothing": ([400], [400], 2, 4, 96, 16),
    "tile, prompt from nothing": ([200, 90], [200, 90], 2, 1, 160, 64),
}


@pytest.mark.parametrize("case", SWEEPS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_token_counts_once(mx, case, dtype):
    lens, ns, Hkv, G, D, page = SWEEPS[case]
    # a token that every row sees: any of the context, else the first
    rng = np.random.default_rng(len(case))
    anchors = [int(rng.integers(0, L - n + 1)) for L, n in zip(lens, ns)]
    if case == "rows, short":                                    # a sequence of one token has no other to pin
        lens, ns, anchors = [lens[0], lens[2]], [1, 1], [anchors[0], anchors[2]]
    Pinned(mx, lens, ns, Hkv, G, D, page, dtype, 7 * D + page, anchors).sweep()


# many sequences: more tiles than workgroups, long ones among short, and (17 to
# 32 rows a KV head) the kernel of two column tiles a wave
@pytest.mark.parametrize("n,G,Hkv,D", [(1, 4, 8, 128), (3, 8, 4, 64), (3, 8, 4, 128), (9, 4, 4, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_every_token_counts_once_in_large_batches(mx, n, G, Hkv, D, dtype):
    rng = np.random.default_rng(n * D)
    B = 70
    lens = rng.integers(n + 1, 90, B)
    lens[[5, 66]] = (1200, 641) if n > 1 else (500, 301)
    ns = rng.integers(1, n + 1, B)
    ns[[5, 66]] = n
    Pinned(mx, lens.tolist(), ns.tolist(), Hkv, G, D, 16, dtype, n + D).sweep()


@pytest.mark.parametrize("L", [17001, 33000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_tokens_at_borders_of_long_contexts(mx, L, dtype):
    p = Pinned(mx, [L, 2049], [1, 1], 2, 16, 128, 64, dtype, L, anchors=[L // 3, 5])
    p.sweep([near(L, 128), near(2049, 32)])
    p = Pinned(mx, [L], [20], 1, 8, 64, 256, dtype, L + 1, anchors=[7])
    p.sweep([near(L, 64)])
