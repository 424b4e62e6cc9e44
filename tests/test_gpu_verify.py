"""Verification of drafted tokens on the GPU against the definition in 64 bits,
one sequence and one child after the other. Paths and tokens are whole numbers
and have to be equal: they would differ only where a random number falls within
the rounding of a 64-bit sum (V 2^-53 relative, below 1e-10 for the sizes here)
of a border."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import bit_gemm_hdiag_amd as mx
    return mx


def weights(l, T):
    """e(v) of a row of float64 logits."""
    l = np.where(np.isnan(l), -np.inf, l)
    m = l.max()
    if m == -np.inf:
        return np.zeros_like(l)
    if not T > 0:
        e = np.zeros_like(l)
        e[int(np.argmax(l))] = 1.0
        return e
    if m == np.inf:
        return (l == np.inf).astype(np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        return np.where(l == -np.inf, 0.0, np.where(l == m, 1.0, np.exp((l - m) * (1.0 / T))))


def drawn(w, u):
    cum = np.cumsum(w)
    at = np.nonzero((cum > u * cum[-1]) & (w > 0))[0]
    return int(at[0]) if len(at) else (int(np.nonzero(w > 0)[0][-1]) if (w > 0).any() else -1)


def walk(logits, tokens, parents, u, T, draft, replacement, max_n):
    """(kept nodes, next token) of one sequence."""
    n, V = min(len(tokens), max_n), logits.shape[1]
    if n == 0:
        return [], -1
    greedy = not T > 0
    cur, kept = 0, [0]
    e = weights(logits[0], T)
    S, R, left, q = 0.0, e.sum(), 1.0, None
    clean = lambda d: np.where((d > 0) & np.isfinite(d), d, 0.0).astype(np.float64)
    for i in range(1, n):
        if parents[i] != cur or not 0 <= tokens[i] < V:
            continue
        x = int(tokens[i])
        if greedy:
            ok = e[x] > 0
        elif draft is None:
            ok = u[i] * R < e[x]
            if not ok:
                e[x] = 0.0
                R = e.sum()
        else:
            q = clean(draft[cur])
            ok = left > 0 and u[i] * q[x] * R < max(e[x] - S * q[x], 0.0) * left
            if not ok and left > 0:
                S += R / left
                if not replacement:
                    left -= q[x]
                R = np.maximum(e - S * q, 0.0).sum()
        if ok:
            kept.append(i)
            cur = i
            e = weights(logits[i], T)
            S, R, left = 0.0, e.sum(), 1.0
    if e.sum() == 0:
        return kept, -1
    w = np.maximum(e - S * clean(draft[cur]), 0.0) if draft is not None and S > 0 else e
    if not w.sum() > 0:
        w = weights(logits[cur], T)
    return kept, drawn(w, u[0])


class Case:
    def __init__(self, ns, V, dtype, draft, seed, kind="tree", temps=None, ld=0, tail=0, sharp=3.0, alike=0.7):
        g = np.random.default_rng(seed)
        self.cu = np.concatenate([[0], np.cumsum(ns)])
        total = int(self.cu[-1]) + tail
        self.ns, self.V, self.total = ns, V, total
        base = g.standard_normal((total, V)) * sharp
        self.t_logits = torch.zeros((total, V + ld), dtype=dtype, device=DEV)[:, :V]
        self.t_logits.copy_(torch.from_numpy(base))
        self.draft = None
        q = np.exp(base + alike * g.standard_normal((total, V)))
        q /= q.sum(1, keepdims=True)
        q = q.astype(np.float32)
        if draft:
            self.t_draft = torch.zeros((total, V + ld), dtype=F32, device=DEV)[:, :V]
            self.t_draft.copy_(torch.from_numpy(q))
            self.draft = q
        self.tokens, self.parents = np.zeros(total, np.int64), np.full(total, -1, np.int32)
        for b, n in enumerate(ns):
            kids = {}
            for i in range(1, n):
                p = i - 1 if kind == "chain" else int(g.integers(max(0, (i - 1) // 3), i))
                r = self.cu[b] + i
                self.parents[r] = p
                left = q[self.cu[b] + p].astype(np.float64).copy()
                if kind != "again":
                    left[kids.get(p, [])] = 0.0
                x = int(g.choice(V, p=left / left.sum())) if left.sum() > 0 else int(g.integers(V))
                self.tokens[r] = x
                kids.setdefault(p, []).append(x)
        self.u = g.random(total)
        self.temps = temps
        self.replacement = kind == "again"
        self.max_n = max(list(ns) + [1])

    def run(self, mx, **kw):
        d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
        args = dict(parents=d(self.parents), draft=None if self.draft is None else self.t_draft,
                    replacement=self.replacement, max_n=self.max_n,
                    temperature=None if self.temps is None else d(np.array(self.temps, np.float32)))
        args.update(kw)
        return mx.mxs_verify_tree(self.t_logits, d(self.tokens), d(self.cu.astype(np.int32)), d(self.u), **args)

    def check(self, got, rows=None):
        path, count, nxt = (x.cpu().numpy() for x in got)
        l = self.t_logits.double().cpu().numpy()
        seen = [0, 0]
        for b, n in enumerate(self.ns):
            s = slice(self.cu[b], self.cu[b + 1])
            T = 1.0 if self.temps is None else float(np.float32(self.temps[b]))
            kept, token = walk(l[s], self.tokens[s], self.parents[s], self.u[s], T,
                               None if self.draft is None else self.draft[s], self.replacement, self.max_n)
            assert count[b] == len(kept) and nxt[b] == token, (b, n, kept, token, path[s], count[b], nxt[b])
            assert path[s].tolist() == kept + [-1] * (n - len(kept)), b
            seen[0] += len(kept) > 1
            seen[1] += len(kept) < min(n, self.max_n)
        return seen


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("ns,V,kind,ld", [
    ([5], 32000, "chain", 0), ([1], 1, "chain", 0), ([2, 2], 2, "tree", 0), ([8] * 6, 1000, "chain", 0),
    ([13, 0, 9, 1, 12], 1025, "tree", 0), ([26, 20, 15], 5003, "tree", 1), ([64, 40], 2048, "tree", 0),
    ([9, 7], 1023, "again", 2), ([30, 30], 50, "again", 0), ([20] * 70, 37, "tree", 3), ([3, 4], 131072, "tree", 0)])
def test_against_the_definition(mx, ns, V, kind, ld, draft, dtype):
    temps = [0.4 + 0.3 * (b % 5) if b % 4 != 3 else 0.0 for b in range(len(ns))]
    c = Case(ns, V, dtype, draft, V + len(ns), kind, temps, ld, tail=2 if ld else 0)
    out = torch.full((c.total,), 77, dtype=torch.int32, device=DEV)
    got = c.run(mx, path=out)
    c.check(got)
    assert (out[int(c.cu[-1]):] == 77).all()                     # rows of no sequence
    c.temps = None
    c.check(c.run(mx))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("ns,V,kind", [([3, 5, 1], 262145, "tree"), ([4, 3], 270001, "tree"), ([2], 1 << 20, "chain"),
                                       ([8] * 300, 5003, "tree"), ([2] * 2100, 4097, "chain"),
                                       ([64] + [1] * 200, 700, "tree"), ([64] + [1] * 4100, 600, "chain"),
                                       ([40] + [2] * 1100, 9000, "tree")])
def test_sizes_that_take_other_kernels(mx, ns, V, kind, draft, dtype):
    """Vocabularies past 2^18, batches that fill the chip with a wave a chunk, one long tree among short ones."""
    if draft and V * sum(ns) > 1 << 24:
        ns = ns[:3] + ns[-100:]
    temps = [0.5 + 0.2 * (b % 4) if b % 5 != 2 else 0.0 for b in range(len(ns))]
    c = Case(ns, V, dtype, draft, V % 1000, kind, temps)
    c.check(c.run(mx))
    c.max_n = min(1024, max(ns) + 30)                             # a loose bound
    c.check(c.run(mx))


@pytest.mark.parametrize("draft", [True, False])
def test_draws_follow_both_outcomes(mx, draft):
    """Many small trees: nodes accepted and rejected, siblings tried after a rejection."""
    for seed in range(4):
        c = Case([12] * 64, 11, F32, draft, seed, "tree" if seed < 3 else "again", None, sharp=1.5, alike=1.5)
        seen = c.check(c.run(mx))
        assert seen[0] > 0 and seen[1] > 0                        # both outcomes occur


@pytest.mark.parametrize("form", ["draft", "again", "none"])
def test_tokens_are_distributed_as_the_targets(mx, form):
    """The first token after the root, over 60000 sequences with one row of logits: every frequency within five
    standard deviations of the target's probability, and so for the second token where the first was kept."""
    B, V, k = 60000, 9, 4
    g = np.random.default_rng(5)
    l = g.standard_normal(V) * 1.2
    q = np.exp(l + g.standard_normal(V))
    q = (q / q.sum()).astype(np.float32)
    p = np.exp(l) / np.exp(l).sum()
    n = k + 1
    keys = g.random((B, V)) if form == "none" else g.exponential(size=(B, V)) / q
    tok = np.zeros((B, n), np.int64)
    tok[:, 1:] = g.choice(V, size=(B, k), p=q.astype(np.float64) / q.sum(dtype=np.float64)) if form == "again" \
        else np.argsort(keys, 1)[:, :k]
    d = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to(t).to(DEV)
    logits = d(np.tile(l, (B * n, 1)), F32)
    pars = np.zeros((B, n), np.int32)
    pars[:, 0] = -1
    path, count, nxt = mx.mxs_verify_tree(
        logits, d(tok.reshape(-1), torch.int64), d(np.arange(B + 1) * n, torch.int32),
        d(g.random(B * n), torch.float64), parents=d(pars.reshape(-1), torch.int32),
        draft=None if form == "none" else d(np.tile(q, (B * n, 1)), F32), replacement=form == "again", max_n=n)
    count, nxt = count.cpu().numpy(), nxt.cpu().numpy()
    kept = path.cpu().numpy().reshape(B, n)[:, 1]
    first = np.where(count > 1, np.take_along_axis(tok, np.maximum(kept, 0)[:, None], 1)[:, 0], nxt)
    for sample in (first, nxt[count > 1]):
        f = np.bincount(sample, minlength=V) / len(sample)
        assert (np.abs(f - p) <= 5 * np.sqrt(p * (1 - p) / len(sample))).all(), (f, p)
    assert 0.2 < (count > 1).mean() < 0.999


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_masks_infinities_and_nan(mx, dtype, draft):
    V = 1500
    c = Case([6] * 12, V, dtype, draft, 3, "tree", [0.0, 0.7, 1.0] * 4, alike=0.2)
    l = c.t_logits.view(12, 6, V)
    low = torch.finfo(dtype).min
    l[0:3] = -math.inf                                            # nothing to draw from
    l[3:6, :, 100:] = low                                         # masked by the lowest value
    l[3:6, :, :7] = -math.inf
    l[6] = low                                                    # all masked by it: even chances
    l[7] = low
    l[8, :, 5] = math.inf                                         # certain
    l[8, :, 1400] = math.inf
    l[9:11, :, ::3] = math.nan
    l[11] = math.nan
    if draft:
        t = c.t_draft.view(12, 6, V)
        t[9, :, 1::3] = math.nan
        t[10, :, 1::3] = -1.0
        t[10, :, 2::3] = math.inf
        t[7] = 0.0
        c.draft = c.t_draft.cpu().numpy()
    c.check(c.run(mx))
    c.temps = [math.inf, math.nan, 1e-38, 1e30] * 3
    c.check(c.run(mx))


def test_greedy_ties_go_to_the_lowest_index(mx):
    V = 40000
    c = Case([3] * 4, V, BF, False, 1, "chain", [0.0] * 4)
    l = c.t_logits.view(4, 3, V)
    l.zero_()
    l[1, :, 39999] = 1.0
    l[2, :, [7, 2049, 2050]] = 1.0
    l[3, :, [1024, 1023, 5000]] = 1.0
    c.tokens[:] = np.repeat([0, 39999, 7, 1023], 3)
    path, count, nxt = c.run(mx)
    assert count.tolist() == [3] * 4 and nxt.tolist() == [0, 39999, 7, 1023]
    c.check((path, count, nxt))
    c.tokens[:] = np.repeat([1, 39998, 2049, 1024], 3)
    got = c.run(mx)
    assert got[1].tolist() == [1] * 4 and got[2].tolist() == [0, 39999, 7, 1023]


@pytest.mark.parametrize("draft", [True, False])
def test_ends_of_the_random_numbers(mx, draft):
    """0 draws the first token of any weight and accepts what has some; the largest below 1 draws the last."""
    c = Case([4] * 6, 5000, F32, draft, 8, "tree", [0.8] * 6)
    c.t_logits[:, :2100] = -math.inf
    c.t_logits[:, 4000:] = -math.inf
    for u in (0.0, 1.0 - 2.0 ** -53):
        c.u[:] = u
        got = c.run(mx)
        c.check(got)
    c = Case([1] * 3, 5000, F32, draft, 9, "chain", [1.0] * 3)
    c.t_logits[:, :2100] = -math.inf
    c.t_logits[:, 4000:] = -math.inf
    c.u[:] = 0.0
    assert c.run(mx)[2].tolist() == [2100] * 3
    c.u[:] = 1.0 - 2.0 ** -53
    assert c.run(mx)[2].tolist() == [3999] * 3


@pytest.mark.parametrize("kind", ["tree", "again", "none"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V,first", [(9000, 5000), (2600, 1500), (30011, 20500), (270001, 70000)])
def test_remainders_behind_masked_tokens(mx, V, first, dtype, kind):
    """The draw from a remainder whose first chunks hold masked tokens alone: 0 draws the first token that has any left."""
    B = 40 if V < 20000 else 6
    c = Case([5] * B, V, dtype, kind != "none", V, "again" if kind == "again" else "tree", sharp=1.0)
    g = np.random.default_rng(1)
    c.t_logits[:, :first] = -math.inf
    c.parents = np.tile(np.array([-1, 0, 0, 0, 0], np.int32), B)
    if c.draft is not None:
        q = c.draft.copy()
        q[:, :first] = 0
        q[:, first:first + 3] *= 30                               # these are used up by a rejection
        q = (q / q.sum(1, keepdims=True)).astype(np.float32)
        c.draft = q
        c.t_draft.copy_(torch.from_numpy(q))
    c.tokens = g.choice(first + np.arange(40), c.total).astype(np.int64)
    c.u[:] = 1 - 2.0 ** -53
    c.u[::5] = 0.0
    assert c.check(c.run(mx))[1] > 0


@pytest.mark.parametrize("V", [3 * 4096, 40000, 300000])
@pytest.mark.parametrize("kids", [2, 3, 5])
def test_chunks_of_taken_tokens_alone(mx, V, kids):
    """Without a draft's distribution: rejected tokens are all that the first chunk had. None of them is drawn."""
    B = 64 if V < 100000 else 16
    c = Case([kids + 1] * B, V, F32, False, kids, "tree", sharp=1.0)
    g = np.random.default_rng(2)
    c.parents = np.tile(np.array([-1] + [0] * kids, np.int32), B)
    l = c.t_logits.view(B, kids + 1, V)
    l[:, :, :16384 if V > 1 << 18 else 4096] = -math.inf
    tok = np.zeros((B, kids + 1), np.int64)
    for b in range(B):
        at = g.choice(4096, kids, replace=False)
        tok[b, 1:] = at
        l[b, 0, torch.from_numpy(at).to(DEV)] = torch.from_numpy(g.standard_normal(kids)).float().to(DEV)
    c.tokens = tok.reshape(-1)
    for u in (0.0, 1e-17, 0.5):
        c.u[:] = 1 - 2.0 ** -53
        c.u[::kids + 1] = u
        c.check(c.run(mx))


def border(e, at, side):
    """The random number just on one side of where the draw passes from token at - 1 to `at`, from extended precision.

    The kernel's two sums that decide are off, relative to theirs, by no more than (in units of 2^-53, with (m - l) / T
    <= 2): 7 each for the weights, and the roundings of 7 sums and products and of the number: 22. It lies 32 off."""
    cum = np.cumsum(e, axis=1)
    return (cum[:, at - 1] / cum[:, -1] * (1 + side * np.longdouble(2.0) ** -48)).astype(np.float64)


@pytest.mark.parametrize("T", [1.0, 0.37])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("B,V,places", [(4000, 2, (0, 1)), (300, 3 * 4096, (0, 4096, 5120, 5127)),
                                        (40, 300000, (7, 16384, 17500, 17501)), (900, 2000, (0, 1023, 1024, 1999))])
def test_borders_of_the_draw(mx, B, V, places, dtype, T):
    """Random numbers next to a border: the weights have the bits that 64-bit sums need, in one wave, over the waves of
    a chunk and over chunks."""
    g = np.random.default_rng(V + B)
    few = torch.zeros(B, len(places), dtype=dtype)
    few[:, 1:] = torch.from_numpy(-2 * float(np.float32(T)) * np.sort(g.random((B, len(places) - 1)), axis=1)).to(dtype)
    l = torch.full((B, V), -math.inf, dtype=dtype, device=DEV)
    l[:, torch.tensor(places, device=DEV)] = few.to(DEV)
    e = np.exp(few.double().numpy().astype(np.longdouble) / np.longdouble(np.float32(T)))
    d = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to(t).to(DEV)
    for at in range(1, len(places)):
        for side in (-1, 1):
            nxt = mx.mxs_verify_tree(l, torch.zeros(B, dtype=torch.int64, device=DEV), d(np.arange(B + 1), torch.int32),
                                     d(border(e, at, side), torch.float64), max_n=1,
                                     temperature=torch.full((B,), T, device=DEV))[2]
            want = places[at - 1 if side < 0 else at]
            assert bool((nxt == want).all()), (at, side, int((nxt != want).sum()))


@pytest.mark.parametrize("offset", [-300.0, 1024.0, 70000.0])
def test_borders_of_the_draw_far_from_zero(mx, offset):
    """As test_borders_of_the_draw, logits (fp32, of which the weights are taken) far from 0."""
    g = np.random.default_rng(7)
    B = 2000
    l = torch.full((B, 2), offset, dtype=F32)
    l[:, 1] -= torch.from_numpy(2 * g.random(B)).float()
    d = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to(t).to(DEV)
    e = np.exp((l.double() - offset).numpy().astype(np.longdouble))
    for side in (-1, 1):
        nxt = mx.mxs_verify_tree(l.to(DEV), torch.zeros(B, dtype=torch.int64, device=DEV), d(np.arange(B + 1), torch.int32),
                                 d(border(e, 1, side), torch.float64), max_n=1)[2]
        assert bool((nxt == (0 if side < 0 else 1)).all()), (side, int((nxt != (0 if side < 0 else 1)).sum()))


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("scale,offset", [(1.0, 900.0), (1.0, -30000.0), (1e-6, 1e-4), (1e25, 1e26), (1e-40, 0.0)])
def test_logits_and_temperatures_of_any_size(mx, scale, offset, draft):
    """Temperatures at which logits are some 1e3 to 1e12 of them away from 0, next to each other or far apart."""
    for V in (300, 6000):
        temps = [scale * t for t in (1.0, 0.3, 1e-2, 1e-4, 1e-7, 3e-9, 1e-9, 1e-12)]
        c = Case([5] * 8, V, F32, draft, 5, "tree", temps, sharp=2.0)
        l = (c.t_logits.double() * scale + offset).float()
        c.t_logits.copy_(l)
        c.check(c.run(mx))


def test_tokens_and_parents_that_do_not_belong(mx):
    for draft in (True, False):
        c = Case([10] * 8, 300, F32, draft, 12, "tree", None, sharp=1.0)
        c.tokens[3::7] = -1
        c.tokens[4::7] = 300
        c.tokens[5::11] = 2 ** 40
        c.parents[6::9] = 9
        c.parents[7::9] = -4
        c.parents[8::13] = 2 ** 31 - 1
        for b in range(8):                                        # a parent that is not before its child is none
            for i in range(1, 10):
                if not 0 <= c.parents[10 * b + i] < i:
                    c.parents[10 * b + i] = -1
        kept = c.parents.copy()
        want = c.run(mx)
        c.check(want)
        c.parents = np.where(kept < 0, 50, kept).astype(np.int32)
        for x, y in zip(c.run(mx), want):
            assert torch.equal(x, y)


def test_identical_draft_is_always_accepted(mx):
    """A draft of the target's own probabilities: rejection has no room but rounding's."""
    c = Case([5] * 40, 4096, F32, True, 4, "chain", None, alike=0.0)
    path, count, nxt = c.run(mx)
    c.check((path, count, nxt))
    assert count.tolist() == [5] * 40


def test_siblings_that_use_the_draft_up(mx):
    """All tokens of a draft's support rejected: nothing is left of it, later children change nothing."""
    V = 64
    c = Case([6], V, F32, True, 2, "tree")
    c.parents[:] = [-1, 0, 0, 0, 0, 0]
    q = np.zeros((6, V), np.float32)
    q[:, [3, 9]] = 0.5
    c.draft = q
    c.t_draft.copy_(torch.from_numpy(q))
    c.tokens[:] = [0, 3, 9, 3, 20, 9]
    c.t_logits[:, 3] = -20.0
    c.t_logits[:, 9] = -20.0
    c.u[:] = 0.999
    got = c.run(mx)
    c.check(got)
    assert got[1].tolist() == [1]


def test_trees_longer_than_the_bound(mx):
    for draft in (True, False):
        c = Case([30, 5, 17], 200, F32, draft, 6, "chain", None, alike=0.1)
        for c.max_n in (1, 6, 16, 30):
            c.check(c.run(mx))
    c = Case([1024, 700], 130, F32, False, 7, "tree", [0.0, 0.9])
    c.check(c.run(mx))
    with pytest.raises(mx.MxsError):
        c.run(mx, max_n=1025)


def test_batches_of_many_rows_without_a_bound(mx):
    """max_n left out: more than 1024 rows in all, and a tree of more than 1024 nodes, cut off there."""
    for ns in ([64] * 32, [3, 1100, 20]):
        c = Case(ns, 60, BF, False, 3)
        c.max_n = 1024
        c.check(c.run(mx, max_n=None))


def test_empty_batches(mx):
    c = Case([0, 0], 10, F32, True, 1)
    c.t_logits, c.t_draft = (torch.zeros(0, 10, device=DEV) for _ in range(2))
    path, count, nxt = c.run(mx)
    assert count.tolist() == [0, 0] and nxt.tolist() == [-1, -1] and path.numel() == 0
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    out = mx.mxs_verify_tree(torch.zeros(0, 10, device=DEV), none, torch.zeros(1, dtype=torch.int32, device=DEV),
                             none.double())
    assert [x.numel() for x in out] == [0, 0, 0]


def test_rows_past_32_bit_offsets(mx):
    """Logits of more than 2^32 bytes: the last sequences read theirs."""
    V, total = 131072, 17000
    ns = [total - 9, 5, 4]
    l = torch.zeros(total, V, dtype=BF, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    l[-9:] = (torch.randn(9, V, generator=g, device=DEV) * 3).to(BF)
    c = Case([5, 4], V, BF, False, 3, "chain", [0.8, 0.0])
    c.t_logits = l[-9:]
    want = c.run(mx)
    c.check(want)
    tokens, u = torch.zeros(total, dtype=torch.int64, device=DEV), torch.zeros(total, dtype=torch.float64, device=DEV)
    tokens[-9:], u[-9:] = torch.from_numpy(c.tokens).to(DEV), torch.from_numpy(c.u).to(DEV)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(ns)]), dtype=torch.int32, device=DEV)
    path, count, nxt = mx.mxs_verify_tree(l, tokens, cu, u, max_n=5,
                                          temperature=torch.tensor([0.0, 0.8, 0.0], device=DEV))
    assert torch.equal(path[-9:], want[0]) and torch.equal(count[1:], want[1]) and torch.equal(nxt[1:], want[2])


@pytest.mark.parametrize("draft", [True, False])
def test_replays_of_a_graph(mx, draft):
    cases = [Case([9, 4, 7], 3001, BF, draft, s, "tree", [0.9, 0.0, 0.7]) for s in range(5)]
    c = cases[0]
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)
    buf = dict(l=c.t_logits.clone(), q=c.t_draft.clone() if draft else None, t=d(c.tokens), p=d(c.parents), u=d(c.u))
    cu, temps = d(c.cu.astype(np.int32)), d(np.array(c.temps, np.float32))
    path, count, nxt = d(np.zeros(c.total, np.int32)), d(np.zeros(3, np.int32)), d(np.zeros(3, np.int64))
    ws = torch.empty(mx.mxs_verify_tree_workspace(3, c.total, c.max_n, c.V), dtype=torch.uint8, device=DEV)

    def call():
        mx.mxs_verify_tree(buf["l"], buf["t"], cu, buf["u"], parents=buf["p"], draft=buf["q"], temperature=temps,
                           max_n=c.max_n, path=path, count=count, next_token=nxt, ws=ws)
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for x in cases + cases[:2]:
        buf["l"].copy_(x.t_logits)
        if draft:
            buf["q"].copy_(x.t_draft)
        for k, v in (("t", x.tokens), ("p", x.parents), ("u", x.u)):
            buf[k].copy_(d(v))
        for y in (path, count, nxt):
            y.fill_(55)
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        x.check((path, count, nxt))


def test_on_a_stream_of_the_callers(mx):
    s = torch.cuda.Stream()
    c = Case([9, 4, 7], 3001, BF, True, 2, "tree", [0.9, 0.0, 0.7])
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        got = c.run(mx)
    s.synchronize()
    c.check(got)


@pytest.mark.parametrize("kids", [2, 63, 64, 200])
def test_the_same_token_proposed_again(mx, kids):
    """Without a draft's distribution: a child whose token an elder sibling had is rejected, wherever it stands among
    them, and takes nothing out of the row again."""
    V, B = 400, 40
    c = Case([kids + 1] * B, V, F32, False, kids, "tree", sharp=1.0)
    g = np.random.default_rng(kids)
    c.parents = np.tile(np.array([-1] + [0] * kids, np.int32), B)
    c.tokens = g.integers(0, max(2, kids // 2), c.total).astype(np.int64)
    for u in (None, 1 - 2.0 ** -53):
        c.u = g.random(c.total) if u is None else np.where(np.arange(c.total) % (kids + 1), u, g.random(c.total))
        c.check(c.run(mx))
