"""Pages of the 4-bit cache on the GPU: tokens copied, sequences forked, room
reserved, accepted tokens moved together, pages given back. Everything is
whole numbers and moved bytes, so every comparison is exact. The model beside
it does one thing after the other in plain Python."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
PLANES = ("kc", "ks", "vc", "vs")


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import bit_gemm_hdiag_amd as mx
    return mx


def dev(x, t=torch.int32):
    return torch.tensor(x, dtype=t, device=DEV)


class Pool:
    """A pool with a page table, and its model on the host."""

    def __init__(self, mx, pages, page, H, D, rows, width, seed):
        self.mx, self.page, self.rng = mx, page, np.random.default_rng(seed)
        g = torch.Generator(device=DEV).manual_seed(seed)
        self.cache = mx.kv4_cache_alloc(pages, page, H, D)
        for k in PLANES:
            t = getattr(self.cache, k)
            t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
        self.refs, self.table = torch.zeros(pages, dtype=torch.int32), torch.full((rows, width), -1, dtype=torch.int32)
        self.lens = torch.zeros(rows, dtype=torch.int32)
        self.h = {k: getattr(self.cache, k).flatten(0, 1).cpu().numpy() for k in PLANES}
        self.m_refs, self.m_table, self.m_lens = (x.numpy().copy() for x in (self.refs, self.table, self.lens))
        self.refs, self.table, self.lens = (x.to(DEV) for x in (self.refs, self.table, self.lens))

    def same(self):
        assert np.array_equal(self.refs.cpu().numpy(), self.m_refs)
        assert np.array_equal(self.table.cpu().numpy(), self.m_table)
        assert np.array_equal(self.lens.cpu().numpy(), self.m_lens)
        for k in PLANES:
            assert np.array_equal(getattr(self.cache, k).flatten(0, 1).cpu().numpy(), self.h[k]), k

    def fork(self, src, dst):
        self.mx.mxs_kv4_fork(self.cache, self.refs, self.table, self.lens, dev(src), dev(dst))
        B = len(self.m_table)
        for s, d in zip(src, dst):
            if 0 <= s < B and 0 <= d < B and s != d:
                for j in range(self.m_table.shape[1]):
                    p = self.m_table[s, j] if j * self.page < self.m_lens[s] else -1
                    self.m_table[d, j] = p if 0 <= p < len(self.m_refs) else -1
                    if self.m_table[d, j] >= 0:
                        self.m_refs[p] += 1
                self.m_lens[d] = self.m_lens[s]

    def reserve(self, ns, alias=True, extra=0):
        """Slots of the model; compares the call's."""
        B, width = self.m_table.shape
        cu = np.concatenate([[0], np.cumsum(ns)])
        want = np.full(cu[-1] + extra, -7)
        free = [p for p in range(len(self.m_refs)) if self.m_refs[p] == 0]
        was, taken, asked = self.m_refs.copy(), 0, 0
        grown = self.m_lens.copy()
        for b, n in enumerate(ns):
            L = int(self.m_lens[b])
            rows = slice(cu[b], cu[b + 1])
            if L < 0 or L + n > width * self.page:
                want[rows] = -1
                continue
            j0, j1 = (L // self.page, (L + n - 1) // self.page + 1) if n else (0, 0)
            held = lambda j: 0 <= self.m_table[b, j] < len(was)
            takes = [j for j in range(j0, j1) if not held(j) or was[self.m_table[b, j]] > 1]
            for j in range(j0, j1):
                if not held(j):
                    self.m_table[b, j] = -1
            asked += len(takes)
            if takes and asked > len(free):
                want[rows] = -1
                continue
            for j in takes:
                p, old = free[taken], self.m_table[b, j]
                taken += 1
                if old >= 0:
                    self.m_refs[old] -= 1
                    k = L - j * self.page
                    if k > 0:
                        for x in self.h.values():
                            x[p * self.page:p * self.page + k] = x[old * self.page:old * self.page + k]
                self.m_table[b, j] = p
                self.m_refs[p] = 1
            want[rows] = [self.m_table[b, t // self.page] * self.page + t % self.page for t in range(L, L + n)]
            grown[b] = L + n
        self.m_lens = grown
        slots = torch.full((len(want),), -7, dtype=torch.int64, device=DEV)
        out = self.lens if alias else torch.full_like(self.lens, -9)
        got, lens = self.mx.mxs_kv4_reserve(self.cache, self.refs, self.table, self.lens, dev(cu), slots=slots,
                                            lens_out=out)
        assert got is slots and lens is out
        self.lens = out
        assert np.array_equal(slots.cpu().numpy(), want)
        return want

    def write(self, slots):
        """Other bytes in the new slots, as an append leaves them."""
        s = dev([x for x in slots if x >= 0], torch.int64)
        for k in PLANES:
            t = getattr(self.cache, k).flatten(0, 1)
            new = torch.randint(0, 256, (len(s), *t.shape[1:]), device=DEV, dtype=torch.uint8)
            t[s] = new
            self.h[k][s.cpu().numpy()] = new.cpu().numpy()

    def compact(self, ns, paths, alias=True):
        cu = np.concatenate([[0], np.cumsum(ns)])
        path = np.full(cu[-1], -1)
        for b, p in enumerate(paths):
            path[cu[b]:cu[b] + len(p)] = p
        for b, n in enumerate(ns):
            if self.m_lens[b] < n:
                continue
            base = int(self.m_lens[b]) - n
            at = lambda t: self.m_table[b, t // self.page] * self.page + t % self.page
            for x in self.h.values():
                rows = [x[at(base + f)].copy() for f in paths[b]]
                for i, r in enumerate(rows):
                    x[at(base + i)] = r
            self.m_lens[b] = base + len(paths[b])
        out = self.lens if alias else torch.full_like(self.lens, -9)
        got = self.mx.mxs_kv4_compact(self.cache, self.table, self.lens, dev(cu), dev(path),
                                      dev([len(p) for p in paths]), lens_out=out)
        assert got is out
        self.lens = out

    def release(self, keep, alias=True):
        out = self.lens if alias else torch.full_like(self.lens, -9)
        self.mx.mxs_kv4_release(self.cache, self.refs, self.table, self.lens, dev(keep), lens_out=out)
        self.lens = out
        for b, k in enumerate(keep):
            if k < 0:
                continue
            for j in range(self.m_table.shape[1]):
                if j * self.page >= k:
                    p = self.m_table[b, j]
                    if 0 <= p < len(self.m_refs):
                        self.m_refs[p] -= 1
                    self.m_table[b, j] = -1
            self.m_lens[b] = min(self.m_lens[b], k)

    def paths(self, ns):
        return [[0] + sorted(self.rng.choice(np.arange(1, n), self.rng.integers(0, n), replace=False).tolist())
                if n else [] for n in ns]


SHAPES = [(40, 16, 2, 64, 5, 12), (300, 17, 3, 96, 9, 25), (70, 1, 1, 32, 3, 60), (12, 256, 8, 128, 4, 3),
          (5000, 16, 1, 32, 70, 66), (9000, 3, 5, 32, 20, 500)]


@pytest.mark.parametrize("pages,page,H,D,rows,width", SHAPES)
def test_steps_of_a_server(mx, pages, page, H, D, rows, width):
    """Prompts, forks, drafted steps, accepted paths and sequences that end, until the pool has run out."""
    p = Pool(mx, pages, page, H, D, rows, width, pages + page)
    room = pages * page // rows
    p.write(p.reserve([int(p.rng.integers(0, max(2, room // 2))) if b % 3 != 2 else 0 for b in range(rows)]))
    p.same()
    for step in range(8):
        empty = [b for b in range(rows) if p.m_lens[b] == 0 and (p.m_table[b] < 0).all()]
        full = [b for b in range(rows) if p.m_lens[b] > 0]
        if full and empty:
            k = int(p.rng.integers(1, len(empty) + 1))
            p.fork(p.rng.choice(full, k).tolist(), empty[:k])
        ns = [int(p.rng.integers(0, 2 + step * 4)) if p.m_lens[b] or b % 2 else 0 for b in range(rows)]
        before = p.m_lens.copy()
        slots = p.reserve(ns, alias=step % 2 == 0, extra=step % 3)
        p.write(slots)
        ns = [n if p.m_lens[b] == before[b] + n else 0 for b, n in enumerate(ns)]    # what has room
        p.compact(ns, p.paths(ns), alias=step % 2 == 1)
        keep = [int(p.m_lens[b]) if p.rng.random() < 0.3 else -1 for b in range(rows)]
        keep[int(p.rng.integers(rows))] = 0
        b = int(p.rng.integers(rows))
        keep[b] = int(p.m_lens[b]) // 2
        p.release(keep, alias=step % 2 == 0)
        p.same()
    p.release([0] * rows)
    p.same()
    assert not p.m_refs.any() and not p.m_lens.any()


def test_reserve_takes_the_lowest_free_pages_across_chunks(mx):
    """Free pages far apart, chunks without any, pages kept back by a negative count."""
    p = Pool(mx, 30000, 2, 1, 32, 3, 900, 5)
    m = np.ones(30000, dtype=np.int32)
    free = np.unique(p.rng.integers(0, 30000, 900))
    free = free[(free < 4096) | (free > 3 * 4096)]
    m[free] = 0
    m[free[::7]] = -1
    p.m_refs, p.refs = m, torch.from_numpy(m.copy()).to(DEV)
    slots = p.reserve([300, 1, 500])
    p.same()
    given = np.unique(slots // 2)
    assert len(given) == 401 and (p.m_refs[given] == 1).all() and not np.isin(free[::7], given).any()


def test_reserve_of_many_pages_at_once(mx):
    """More pages than a workgroup notes in LDS, for one sequence and for the next, over several chunks."""
    p = Pool(mx, 7000, 1, 1, 32, 4, 2500, 15)
    p.write(p.reserve([257, 0, 1500, 3]))
    p.release([100, -1, 700, 0])
    p.fork([2], [1])
    slots = p.reserve([2000, 256, 1300, 1])
    p.same()
    assert len(set(slots.tolist())) == len(slots) and (slots >= 0).all()


def test_pool_that_runs_out(mx):
    """The first sequence that does not fit and later ones that need pages get none; one with room is served."""
    p = Pool(mx, 10, 4, 2, 64, 5, 8, 6)
    p.write(p.reserve([5, 0, 0, 9, 0]))                          # 2 + 3 pages
    want = p.reserve([8, 13, 4, 3, 0])                           # 2 of 5, then 4 of 3, 1 (refused after it), none
    p.same()
    assert (want[:8] >= 0).all() and (want[8:25] == -1).all() and (want[25:] >= 0).all()
    assert p.m_lens.tolist() == [13, 0, 0, 12, 0]
    # a shared page cannot be copied without a free one: nothing changes
    p.release([-1, -1, 0, 10, -1])
    p.fork([3], [2])
    p.reserve([11, 0, 0, 0, 0])
    p.same()
    want = p.reserve([0, 0, 20, 20, 0])
    assert (want == -1).all() and (p.m_refs > 1).any()
    p.same()


def test_rows_too_short_and_broken_lengths(mx):
    p = Pool(mx, 20, 4, 1, 32, 4, 3, 7)
    p.write(p.reserve([12, 13, 0, 3]))
    p.m_lens[1] = -5
    p.lens[1] = -5
    want = p.reserve([1, 2, 0, 9])
    assert want.tolist()[:3] == [-1] * 3 and (want[3:] >= 0).all()
    p.same()


def test_all_holders_of_a_page_write(mx):
    """Three forks of one sequence take a copy each; the page they shared is free afterwards."""
    p = Pool(mx, 20, 8, 2, 64, 4, 4, 8)
    p.write(p.reserve([13, 0, 0, 0]))
    shared = int(p.m_table[0, 1])
    p.fork([0, 0, 0], [1, 2, 3])
    assert p.m_refs[shared] == 4
    slots = p.reserve([2, 2, 2, 2])
    p.same()
    assert p.m_refs[shared] == 0 and len(set(slots.tolist())) == 8
    p.reserve([0, 4, 0, 0])                                       # no longer shared: in place, and one page more
    p.same()


def test_truncated_into_a_shared_page(mx):
    """A length cut back into pages that are shared: they are replaced before they are written, whole ones without a copy."""
    p = Pool(mx, 30, 4, 1, 32, 2, 8, 9)
    p.write(p.reserve([16, 0]))
    p.fork([0], [1])
    for t in (p.m_lens, p.lens):
        t[1] = 6
    p.reserve([0, 9])
    p.same()


def test_fork_pairs_that_are_skipped(mx):
    p = Pool(mx, 10, 4, 1, 32, 3, 4, 10)
    p.write(p.reserve([7, 0, 0]))
    p.fork([0, -1, 0, 5, 0], [0, 1, 3, 1, -2])
    p.same()
    p.fork([], [])
    p.fork([1], [2])                                              # nothing to share
    p.same()


@pytest.mark.parametrize("H,D,page,T", [(1, 32, 16, 1), (8, 128, 64, 3000), (3, 96, 17, 777), (5, 64, 1, 60),
                                        (2, 256, 300, 4000), (128, 128, 16, 100)])
@pytest.mark.parametrize("same", [False, True])
def test_copy(mx, H, D, page, T, same):
    n = -(-2 * T // page) + 1
    a = Pool(mx, n, page, H, D, 1, 1, T)
    b = a if same else Pool(mx, n + 3, page, H, D, 1, 1, T + 1)
    order = a.rng.permutation(n * page)
    src, dst = order[:T].copy(), order[T:2 * T].copy()            # disjoint, so also right within one pool
    if not same:
        dst = b.rng.permutation((n + 3) * page)[:T]
        if T > 4:
            src[3] = src[0]                                       # a source may repeat
    skip = a.rng.random(T) < 0.1
    src2, dst2 = src.copy(), dst.copy()
    src2[skip] = np.where(a.rng.random(skip.sum()) < 0.5, -1, n * page)
    dst2[a.rng.random(T) < 0.1] = -3
    ok = (src2 >= 0) & (src2 < n * page) & (dst2 >= 0)
    mx.mxs_kv4_copy(b.cache, dev(dst2, torch.int64), a.cache, dev(src2, torch.int64))
    for k in PLANES:
        x = a.h[k].copy()
        b.h[k][dst2[ok]] = x[src2[ok]]
    b.same()
    if not same:
        a.same()


@pytest.mark.parametrize("H,D,page,T", [(8, 128, 64, 40000), (3, 96, 17, 130000), (64, 1024, 3, 600), (33, 1024, 5, 5),
                                        (64, 1024, 3, 7)])
def test_copy_of_many_words(mx, H, D, page, T):
    """Four words a thread, tokens of more words than a workgroup takes, with scale bytes by eight and one by one."""
    test_copy(mx, H, D, page, T, False)


def test_copy_of_nothing(mx):
    a = Pool(mx, 2, 4, 1, 32, 1, 1, 1)
    none = dev([], torch.int64)
    mx.mxs_kv4_copy(a.cache, none, a.cache, none)
    a.same()


def test_compact_ignores_what_a_path_should_not_hold(mx):
    """Entries outside the tree, counts past it, sequences shorter than their tree, tokens in no page: in bounds, and
    no other sequence is touched."""
    p = Pool(mx, 30, 4, 1, 32, 5, 5, 11)
    p.write(p.reserve([10, 6, 3, 8, 5]))
    before = {k: v.copy() for k, v in p.h.items()}
    p.table[3, 1] = -1
    cu, path = [0, 4, 8, 12, 18, 18], [0, 9, -5, 2 ** 31 - 1] + [0, 1, 2, 3] + [0, 1, 3, 3] + [0, 2, 3, 4, 5, 5]
    out = mx.mxs_kv4_compact(p.cache, p.table, p.lens, dev(cu), dev(path), dev([4, -3, 2, 99, 7]))
    assert out.tolist() == [10, 2, 3, 8, 5]
    rows = lambda b, n: [int(p.m_table[b, t // 4]) * 4 + t % 4 for t in range(n)]
    for k in PLANES:
        now = getattr(p.cache, k).flatten(0, 1).cpu().numpy()
        for b, n in ((0, 10), (1, 6), (2, 3), (4, 5)):
            assert np.array_equal(now[rows(b, n)], before[k][rows(b, n)]), (k, b)


def test_step_in_a_graph(mx):
    """Fork, reserve, compact and release captured once; every replay as the eager calls."""
    ns, rows = [9, 4, 0, 6, 5, 3], 6
    keep = [40, 21, 5, 0, 0, 0]

    def make():
        p = Pool(mx, 400, 8, 2, 64, rows, 12, 12)
        p.write(p.reserve([40, 21, 5, 0, 0, 0]))
        return p

    def step(p, cu, path, count, src, dst, kp, ws, slots, grown, kept):
        mx.mxs_kv4_fork(p.cache, p.refs, p.table, p.lens, src, dst)
        mx.mxs_kv4_reserve(p.cache, p.refs, p.table, p.lens, cu, slots=slots, lens_out=grown, ws=ws)
        mx.mxs_kv4_compact(p.cache, p.table, grown, cu, path, count, lens_out=kept)
        mx.mxs_kv4_release(p.cache, p.refs, p.table, kept, kp, lens_out=kept)

    cu = np.concatenate([[0], np.cumsum(ns)])

    def fresh(i):
        path, count = np.full(cu[-1], -1), []
        r = np.random.default_rng(i)
        for b, n in enumerate(ns):
            q = [0] + sorted(r.choice(np.arange(1, n), r.integers(0, n), replace=False).tolist()) if n else []
            path[cu[b]:cu[b] + len(q)] = q
            count.append(len(q))
        return path, count
    state = []
    for _ in range(2):
        p = make()
        path, count = fresh(0)
        state.append((p, (dev(cu), dev(path), dev(count), dev([0, 1, 0]), dev([3, 4, 5]), dev(keep),
                          torch.empty(mx.mxs_kv4_reserve_workspace(400, rows), dtype=torch.uint8, device=DEV),
                          torch.empty(int(cu[-1]), dtype=torch.int64, device=DEV), dev([0] * rows), dev([0] * rows))))
    (e, ea), (c, ca) = state
    for k in PLANES:
        getattr(c.cache, k).copy_(getattr(e.cache, k))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, *ca)
    for i in range(5):
        path, count = fresh(i)
        for a in (ea, ca):
            a[1].copy_(dev(path))
            a[2].copy_(dev(count))
        step(e, *ea)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((e.refs, e.table, e.lens, ea[7], ea[8], ea[9]), (c.refs, c.table, c.lens, ca[7], ca[8], ca[9])):
            assert torch.equal(x, y), i
        for k in PLANES:
            assert torch.equal(getattr(e.cache, k), getattr(c.cache, k)), (i, k)


def test_on_a_stream_of_the_callers(mx):
    p = Pool(mx, 300, 17, 3, 96, 9, 25, 13)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        p.write(p.reserve([60, 0, 30, 0, 17, 0, 0, 0, 0]))
        p.fork([0, 0, 2], [1, 3, 5])
        ns = [3, 4, 5, 6, 7, 1, 0, 0, 0]
        p.write(p.reserve(ns))
        p.compact(ns, p.paths(ns))
        p.release([-1, 0, 20, -1, -1, -1, 0, -1, -1])
    s.synchronize()
    p.same()


def test_refused_sequences_keep_their_entries(mx):
    """Entries that name no page (any negative number, any past the pool) take pages where there is room; the table of a
    refused sequence is left as it was, shared pages and such entries among it."""
    p = Pool(mx, 7, 4, 1, 32, 5, 8, 1)
    p.write(p.reserve([9, 3, 0, 4, 0]))                           # 3 + 1 + 1 of 7 pages
    p.fork([0], [4])
    big = 2 ** 31 - 1
    odd = {(0, 3): -7, (0, 4): 7, (0, 5): 1 << 30, (1, 1): -2 ** 31, (1, 2): -2 ** 31 + 5, (1, 3): big, (2, 0): -3,
           (2, 1): 99, (3, 1): -2, (3, 2): -9}
    for at, v in odd.items():
        p.table[at] = v
    before, refs = p.table.clone(), p.refs.clone()
    ns = [16, 3, 0, 6, 5]                                         # wants 2 + 2 (shared), 1, 0, 2, 2 (shared, another)
    slots, lens = mx.mxs_kv4_reserve(p.cache, p.refs, p.table, p.lens, dev(np.concatenate([[0], np.cumsum(ns)])), total=30)
    assert lens.tolist() == [9, 3, 0, 4, 9] and bool((slots == -1).all())
    assert torch.equal(p.table, before) and torch.equal(p.refs, refs)
    ns = [0, 2, 8, 0, 0]
    slots, lens = mx.mxs_kv4_reserve(p.cache, p.refs, p.table, p.lens, dev(np.concatenate([[0], np.cumsum(ns)])), total=10)
    assert lens.tolist() == [9, 5, 0, 4, 9]                       # one of the two free pages, then two of one
    assert slots[:2].tolist() == [int(p.table[1, 0]) * 4 + 3, int(p.table[1, 1]) * 4] and bool((slots[2:] == -1).all())
    assert int(p.table[1, 1]) == 5 and torch.equal(p.table[[0, 2, 3, 4]], before[[0, 2, 3, 4]])
    assert p.table[1, 2:].tolist() == before[1, 2:].tolist()
    mx.mxs_kv4_release(p.cache, p.refs, p.table, lens, dev([0, -1, -1, -1, 0]), lens_out=lens)
    slots, lens = mx.mxs_kv4_reserve(p.cache, p.refs, p.table, lens, dev([0, 0, 0, 8, 13, 13]), total=13)
    assert lens.tolist() == [0, 5, 8, 9, 0] and bool((slots >= 0).all()) and len(set(slots.tolist())) == 13
    assert bool((p.table[2, :2] >= 0).all()) and bool((p.table[2, :2] < 7).all()) and p.table[3, 2] in range(7)
    held = p.table[(p.table >= 0) & (p.table < 7)]
    assert torch.equal(torch.bincount(held, minlength=7).int(), p.refs)


@pytest.mark.parametrize("graph", [False, True])
def test_refused_sequences_keep_their_tokens(mx, graph):
    """A step whose cu is never looked at on the host, over a pool that runs out: sequences that were refused, forks of
    one another among them, keep table, length and tokens; the others are compacted; the step is repeated with room."""
    p = Pool(mx, 12, 4, 2, 64, 6, 10, 21)
    p.write(p.reserve([6, 14, 9, 0, 3, 0]))                       # 2 + 4 + 3 + 1 of 12 pages
    p.fork([1], [3])
    ns, paths = [2, 4, 4, 5, 1, 3], [[0, 1], [0, 2], [0, 2, 3], [0, 3, 4], [0], [0, 2]]
    cu = np.concatenate([[0], np.cumsum(ns)])
    path = np.full(cu[-1], -1)
    for b, x in enumerate(paths):
        path[cu[b]:cu[b] + len(x)] = x
    cu, path, count = dev(cu), dev(path), dev([len(x) for x in paths])
    total = int(path.numel())
    g = torch.Generator(device=DEV).manual_seed(2)
    k, v, q = (torch.randn((total, h, 64), generator=g, device=DEV) for h in (2, 2, 4))
    logits = torch.randn((total, 50), generator=g, device=DEV)
    tokens, u = torch.zeros(total, dtype=torch.int64, device=DEV), torch.rand(total, dtype=torch.float64, device=DEV)
    ws = torch.empty(mx.mxs_kv4_reserve_workspace(12, 6), dtype=torch.uint8, device=DEV)
    slots, grown = torch.empty(total, dtype=torch.int64, device=DEV), dev([0] * 6)

    def step():
        mx.mxs_kv4_reserve(p.cache, p.refs, p.table, p.lens, cu, slots=slots, lens_out=grown, ws=ws)
        mx.mxs_kv4_append(p.cache, k, v, slots)
        mx.mxs_kv4_compact_granted(p.cache, p.table, grown, cu, path, count, slots, lens_out=p.lens)
        mx.mxs_kv4_release(p.cache, p.refs, p.table, p.lens, p.lens, lens_out=p.lens)

    def tokens_of(b, n):
        row = p.table[b].tolist()
        at = [row[t // 4] * 4 + t % 4 for t in range(n)]
        return [getattr(p.cache, x).flatten(0, 1)[at].clone() for x in PLANES]

    def same(x, y):
        return all(torch.equal(a, b) for a, b in zip(x, y))
    lens = p.lens.tolist()
    before = [tokens_of(b, n) for b, n in enumerate(lens)]
    if graph:
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            step()
        once = captured.replay
    else:
        once = step
    # 0 has room; 1 and 3 share a page that each would copy: 1 takes the last two, 2, 3 and 5 are refused; 4 has room
    once()
    torch.cuda.synchronize()
    first = slots[cu[:-1].long()].tolist()
    assert [x < 0 for x in first] == [False, False, True, True, False, True]
    assert p.lens.tolist() == [8, 16, 9, 14, 4, 0]
    for b, n in enumerate(lens):
        assert same(tokens_of(b, n), before[b]), b
    for b in (0, 1):                                              # the accepted ones, in their new places
        a = torch.arange(len(paths[b]), device=DEV)
        new = mx.mxs_kv4_read(p.cache, torch.tensor([int(p.table[b, (lens[b] + i) // 4]) * 4 + (lens[b] + i) % 4
                                                     for i in a.tolist()], device=DEV), torch.float32)
        other = mx.kv4_cache_alloc(2, 4, 2, 64)
        rows = [int(cu[b]) + i for i in paths[b]]
        mx.mxs_kv4_append(other, k[rows].contiguous(), v[rows].contiguous(), a)
        want = mx.mxs_kv4_read(other, a, torch.float32)
        assert torch.equal(new[0], want[0]) and torch.equal(new[1], want[1])
    held = p.table[p.table >= 0]
    assert torch.equal(torch.bincount(held, minlength=12).int(), p.refs)
    # the calls that read change nothing for a refused sequence (the pool's bytes are any, NaN among them)
    now = [getattr(p.cache, x).clone() for x in PLANES] + [p.table.clone(), p.lens.clone()]
    out = mx.mxs_attend_kv4_tree(q, p.cache, p.table, grown, cu, 0.125, max_q=5)
    mx.mxs_verify_tree(logits, tokens, cu, u)
    assert out.shape == q.shape and same(now, [getattr(p.cache, x) for x in PLANES] + [p.table, p.lens])
    # room again: the first two end
    mx.mxs_kv4_release(p.cache, p.refs, p.table, p.lens, dev([0, 0, -1, -1, -1, -1]), lens_out=p.lens)
    cu[:3] = 0                                                    # nothing more of theirs
    p.lens[:2] = 0
    shared = tokens_of(2, 9), tokens_of(3, 14)
    path[:4] = torch.tensor([0, 2, 3, -1], device=DEV)
    path[4:9] = torch.tensor([0, 3, 4, -1, -1], device=DEV)
    path[9:13] = torch.tensor([0, 0, 2, -1], device=DEV)
    cu[2:] = torch.tensor([0, 4, 9, 10, 13], device=DEV)
    once()
    torch.cuda.synchronize()
    assert p.lens.tolist() == [0, 0, 12, 17, 5, 2]
    assert same(tokens_of(2, 9), shared[0]) and same(tokens_of(3, 14), shared[1])
    held = p.table[p.table >= 0]
    assert torch.equal(torch.bincount(held, minlength=12).int(), p.refs)
