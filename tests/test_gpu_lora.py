"""Adapters beside a shared projection on the GPU against 64-bit forms.

Inputs of small whole numbers have exact results (every partial sum is below
2^24), so those comparisons are for equality. Otherwise, with u = 2^-24 and one
rounding within 2 u for a sum of the matrix cores: V = A x is a K-term sum of
exact products, added up over waves and slices (less than 32 more),
2 (K + 32) u sum |a x|; B V a sum of 3 R exact products (V in three parts),
2 (3 R + 8) u sum |b V|; the scale's product and the addition to Y round once each.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import bit_gemm_hdiag_amd as mx
    return mx


class Case:
    def __init__(self, mx, M, K, N, R, n, dtype, seed, whole, ranks=True, used=None, runs=False, ldx=0, ldy=0, scale=True):
        self.mx, self.M, self.K, self.N = mx, M, K, N
        g = torch.Generator().manual_seed(seed)
        if whole:
            make = lambda *s, top: torch.randint(-top, top + 1, s, generator=g).float()
        else:
            make = lambda *s, top: torch.randn(s, generator=g) * top
        self.x0 = make(M, K, top=2 if whole else 1)
        self.A = make(n, R, K, top=2 if whole else 0.05).to(dtype).to(DEV)
        self.B = make(n, N, R, top=1 if whole else 0.3).to(dtype).to(DEV)
        xs = torch.zeros(M, K + ldx, dtype=dtype)
        xs[:, ldx // 2:ldx // 2 + K] = self.x0.to(dtype)
        self.X = xs.to(DEV)[:, ldx // 2:ldx // 2 + K]
        self.rank = torch.randint(0 if n > 2 else 1, R + 1, (n,), generator=g, dtype=torch.int32).to(DEV) if ranks else None
        if ranks:                                                # what lies behind a rank does not matter
            for a, r in enumerate(self.rank.tolist()):
                self.A[a, r:] = float("nan")
                self.B[a, :, r:] = float("nan")
        self.scale = (2.0 ** torch.randint(-2, 3, (n,), generator=g).float()).to(DEV) if scale else None
        used = n if used is None else used
        which = torch.randperm(n, generator=g)[:used]
        ids = which[torch.randint(0, used, (M,), generator=g)]
        if runs:
            ids = which[torch.arange(M) * used // M]
        ids = ids.to(torch.int32)
        if M > 4 and not runs:
            out = torch.rand(M, generator=g) < 0.15
            ids[out] = torch.randint(0, 3, (int(out.sum()),), generator=g, dtype=torch.int32) * -1000 - 1
            ids[M // 2] = n
        self.ids = ids.to(DEV)
        ys = torch.zeros(M, N + ldy, dtype=F32)
        ys[:, :N] = make(M, N, top=3)
        self.ys = ys.to(DEV)
        self.Y = self.ys[:, ldy // 2:ldy // 2 + N] if ldy else self.ys
        self.set = mx.LoraSet(self.A, self.B, self.scale, self.rank)

    def reference(self):
        """(Y float64, bound of the rounding)"""
        y = self.Y.double().cpu().numpy()
        tol = np.zeros_like(y)
        x = self.X.double().cpu().numpy()
        for a in range(self.set.A.shape[0]):
            rows = (self.ids == a).nonzero().flatten().cpu().numpy()
            R = self.A.shape[1] if self.rank is None else int(self.rank[a])
            if len(rows) == 0 or R == 0:
                continue
            s = 1.0 if self.scale is None else float(self.scale[a])
            A, B = self.A[a, :R].double().cpu().numpy(), self.B[a, :, :R].double().cpu().numpy()
            V = x[rows] @ A.T
            add = s * (V @ B.T)
            vtol = 2 * (self.K + 32) * U * (np.abs(x[rows]) @ np.abs(A).T)
            y[rows] += add
            tol[rows] = abs(s) * (vtol @ np.abs(B).T + 2 * (3 * R + 8) * U * (np.abs(V) @ np.abs(B).T)) \
                + U * (np.abs(add) + np.abs(y[rows]))
        return y, tol

    def run(self, **kw):
        return self.mx.mxs_lora_add(self.Y, self.X, self.ids, self.set, **kw)


SIZES = [(1, 32, 1, 1, 1), (1, 8192, 512, 16, 3), (2, 64, 3, 3, 2), (7, 96, 65, 8, 5), (16, 416, 64, 16, 4),
         (17, 1024, 63, 24, 1), (33, 160, 130, 27, 3), (63, 512, 200, 64, 40), (64, 2048, 1001, 128, 2),
         (65, 512, 256, 16, 7), (200, 96, 70, 100, 300), (300, 1056, 129, 33, 2), (1000, 256, 96, 40, 60),
         (2050, 640, 300, 16, 5), (130, 32, 17, 5, 8192), (64, 64, 30000, 64, 20), (50, 96, 9001, 100, 30),
         (700, 64, 17003, 24, 6), (300, 64, 30001, 8, 9), (33, 2080, 66, 48, 1)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K,N,R,n", SIZES)
def test_whole_numbers_are_exact(mx, M, K, N, R, n, dtype):
    for k, kw in enumerate((dict(), dict(ranks=False, scale=False), dict(ldx=6, ldy=10), dict(runs=True, used=max(1, n // 2)))):
        c = Case(mx, M, K, N, R, n, dtype, M * 7 + k, True, **kw)
        ref, _ = c.reference()
        around = c.ys.clone()
        got = c.run()
        assert got is c.Y
        assert np.array_equal(got.double().cpu().numpy(), ref), kw
        if kw.get("ldy"):
            assert torch.equal(c.ys[:, :5], around[:, :5]) and torch.equal(c.ys[:, 5 + N:], around[:, 5 + N:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,K,N,R,n", SIZES)
def test_against_64_bits(mx, M, K, N, R, n, dtype):
    c = Case(mx, M, K, N, R, n, dtype, M * 5 + K, False)
    ref, tol = c.reference()
    assert (np.abs(c.run().double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M", [40, 400])
def test_rows_do_not_see_each_other(mx, M, dtype):
    """NaN and infinities in some rows of X stay in those rows; a row's result does not depend on what the others hold
    or on which adapters they take."""
    K, N, R, n = 512, 130, 24, 6
    c = Case(mx, M, K, N, R, n, dtype, 1, False, ranks=False)
    d = Case(mx, M, K, N, R, n, dtype, 1, False, ranks=False)
    bad = torch.arange(0, M, 5, device=DEV)
    d.X[bad[0::2]] = float("nan")
    d.X[bad[1::2], 3] = float("inf")
    d.ids[bad] = (d.ids[bad] + 1) % n
    c.run()
    d.run()
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[bad] = False
    assert torch.equal(c.Y[keep], d.Y[keep]) and torch.isfinite(c.Y).all()
    on = (d.ids[bad[0::2]] >= 0) & (d.ids[bad[0::2]] < n)
    assert torch.isnan(d.Y[bad[0::2]][on]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinite_products(mx, dtype):
    """A V of infinity times B: infinity of the right sign, NaN where B is 0, as the formula has it."""
    c = Case(mx, 3, 64, 20, 1, 1, dtype, 2, True, ranks=False, scale=False)
    c.A.fill_(1.0)
    c.X.zero_()
    c.X[:, 5] = torch.tensor([float("inf"), -float("inf"), 1.0], device=DEV).to(dtype)
    c.B[0, :, 0] = torch.tensor([1.0, -2.0, 0.0, 0.5] * 5, device=DEV).to(dtype)
    c.ids.zero_()
    c.Y.zero_()
    c.run()
    inf, nan = float("inf"), float("nan")
    want = torch.tensor([[inf, -inf, nan, inf] * 5, [-inf, inf, nan, -inf] * 5, [1.0, -2.0, 0.0, 0.5] * 5], device=DEV)
    assert torch.equal(torch.nan_to_num(c.Y, nan=7.0), torch.nan_to_num(want, nan=7.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,N,R,n", [(3, 20, 1, 1), (5, 70, 3, 2), (40, 64, 24, 3), (90, 200, 40, 2), (70, 15000, 8, 9),
                                     (33, 300, 100, 1), (70, 15000, 40, 9), (70, 15000, 128, 9), (200, 15001, 12, 9)])
def test_infinite_adapters(mx, M, N, R, n, dtype):
    """Infinities in B: of V's sign where V is not 0, whatever bits V has, NaN where it is; other elements as ever."""
    c = Case(mx, M, 64, N, R, n, dtype, M + R, True, ranks=False, scale=False)
    at = torch.rand(c.B.shape, generator=torch.Generator().manual_seed(R))
    c.B[(at < 0.15 / R).to(DEV)] = float("inf")
    c.B[(at > 1 - 0.15 / R).to(DEV)] = -float("inf")
    if M > 4:
        c.X[3, 5], c.X[4, 6] = float("inf"), -float("inf")
    want, x = c.Y.double().cpu().numpy(), c.X.double().cpu().numpy()
    A, B = c.A.double().cpu().numpy(), c.B.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        for t, a in enumerate(c.ids.tolist()):
            if 0 <= a < n:
                want[t] += (B[a] * (A[a] * x[t]).sum(1)).sum(1)
    assert np.isinf(want).any() and np.isfinite(want).any()
    assert np.array_equal(c.run().double().cpu().numpy(), want, equal_nan=True)


def test_values_of_v_near_the_largest(mx):
    """V up to the largest fp32 numbers: no part of it overflows."""
    c = Case(mx, 4, 32, 8, 2, 1, BF, 2, True, ranks=False, scale=False)
    c.A.zero_()
    c.A[0, 0, 0] = 1.0
    big = torch.tensor([3.38e38, -3.38e38, 1.0, 2.0 ** -120], device=DEV).to(BF)
    c.X.zero_()
    c.X[:, 0] = big
    c.B.zero_()
    c.B[0, :, 0] = 1.0
    c.ids.zero_()
    c.Y.zero_()
    c.run()
    assert torch.equal(c.Y, big.float()[:, None].expand(4, 8))


def test_every_bit_of_v_near_the_largest(mx):
    """V of more bits than bf16 has, above the largest bf16 number: a first part that is rounded would be infinite."""
    c = Case(mx, 4, 32, 8, 2, 1, BF, 2, True, ranks=False, scale=False)
    top = torch.tensor([0x7F7F], dtype=torch.int16).view(BF).item()
    x = torch.tensor([[top, 0.75 * 2.0 ** 120], [-top, -0.75 * 2.0 ** 120], [1.0, 2.0 ** -20], [-3.0, 2.0 ** -16]])
    want = x.double().sum(1).float()
    assert torch.equal(want.double(), x.double().sum(1)) and torch.isfinite(want).all()
    assert torch.isinf(want[:2].to(BF)).all()
    c.A.zero_()
    c.A[0, 0, :2] = 1.0
    c.X.zero_()
    c.X[:, :2] = x.to(BF).to(DEV)
    assert torch.equal(c.X[:, :2].float().cpu(), x)
    c.B.zero_()
    c.B[0, :, 0] = 1.0
    c.ids.zero_()
    c.Y.zero_()
    assert torch.equal(c.run().cpu(), want[:, None].expand(4, 8))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_small_values_of_v(mx, dtype):
    """bf16: bits of V below 2^-133, the smallest number of a part, are cut; above them it is whole, X, A and B below
    2^-126 among them. fp32: whole down to 2^-149."""
    c = Case(mx, 8, 32, 4, 2, 1, dtype, 2, True, ranks=False, scale=False)
    for t in (c.A, c.X, c.B, c.Y, c.ids):
        t.zero_()
    c.A[0, 0, :3] = torch.tensor([2.0 ** -60, 1.0, 2.0 ** 60], device=DEV).to(dtype)
    c.X[0, 0], c.X[1, 0], c.X[2, 0], c.X[3, 1] = 2.0 ** -66, 1.5 * 2.0 ** -60, 2.0 ** -73, 2.0 ** -130
    c.X[4, 2] = 2.0 ** -130
    c.X[5, 0], c.X[5, 1] = 2.0 ** -50, 2.0 ** -133
    c.X[6, 0], c.X[6, 1] = 2.0 ** -74, 2.0 ** -133                # V = 1.5 * 2^-133
    c.X[7, 0] = -2.0 ** -85
    c.B[0, 0, 0], c.B[0, 1, 0], c.B[0, 2, 0] = 2.0 ** 100, 1.0, -2.0 ** 90
    v = (c.A[0, 0].double() * c.X.double()).sum(1).cpu()
    got, want = c.run().double().cpu(), v[:, None] * c.B[0, :, 0].double().cpu()
    cut = 2.0 ** -133 if dtype is BF else 0.0
    assert torch.equal(got[:6, [0, 2]], want[:6, [0, 2]])
    assert bool(((got - want).abs() <= cut * c.B[0, :, 0].double().abs().cpu()).all())


@pytest.mark.parametrize("M", [50, 900])
def test_the_same_call_twice_gives_the_same_bits(mx, M):
    c = Case(mx, M, 2048, 300, 40, 9, BF, 3, False)
    y0 = c.Y.clone()
    first = c.run().clone()
    for fill in (0, 255):
        ws = torch.full((mx.mxs_lora_add_workspace(M, c.set),), fill, dtype=torch.uint8, device=DEV)
        c.Y.copy_(y0)
        assert torch.equal(c.run(ws=ws), first)


@pytest.mark.parametrize("K,N,R,n,most", [(8192, 256, 64, 48, 910), (8192, 256, 16, 16, 8128), (2048, 300, 40, 9, 400)])
def test_one_workspace_for_all_batches(mx, K, N, R, n, most):
    """A workspace of the size asked for the largest batch, with other bytes behind it, which stay."""
    need = mx.mxs_lora_add_workspace(most, Case(mx, 1, K, N, R, n, BF, 1, True).set)
    ws = torch.full((need + 4096,), 170, dtype=torch.uint8, device=DEV)
    for M in (most, most - 1, most // 2 + 1, 65, 64, 63, 1):
        c = Case(mx, M, K, N, R, n, BF, M, True)
        ref, _ = c.reference()
        assert np.array_equal(c.run(ws=ws[:need]).double().cpu().numpy(), ref), M
        assert bool((ws[need:] == 170).all()), M


def test_nothing_to_add(mx):
    for M in (8, 200):
        c = Case(mx, M, 64, 40, 8, 4, BF, 4, True, ranks=False)
        before = c.Y.clone()
        c.ids.fill_(-1)
        assert torch.equal(c.run(), before)
        c.ids.fill_(2)
        s = mx.LoraSet(c.A, c.B, None, torch.zeros(4, dtype=torch.int32, device=DEV))
        assert torch.equal(mx.mxs_lora_add(c.Y, c.X, c.ids, s), before)
    none = mx.LoraSet(c.A[:0].contiguous(), c.B[:0].contiguous())
    assert torch.equal(mx.mxs_lora_add(c.Y, c.X, c.ids, none), before)
    assert mx.mxs_lora_add(c.Y[:0], c.X[:0], c.ids[:0], c.set).numel() == 0


def test_many_rows_past_32_bit_offsets(mx):
    """X and Y of more than 2^31 elements: the last rows read and add theirs."""
    M, K, N = 140000, 16384, 16384
    g = torch.Generator(device=DEV).manual_seed(1)
    X, Y = torch.zeros(M, K, dtype=BF, device=DEV), torch.zeros(M, N, dtype=F32, device=DEV)
    A = torch.randint(-2, 3, (3, 4, K), generator=g, device=DEV).to(BF)
    B = torch.randint(-1, 2, (3, N, 4), generator=g, device=DEV).to(BF)
    X[-70:] = torch.randint(-2, 3, (70, K), generator=g, device=DEV).to(BF)
    ids = torch.full((M,), -1, dtype=torch.int32, device=DEV)
    ids[-70:] = torch.arange(70, device=DEV, dtype=torch.int32) % 3
    mx.mxs_lora_add(Y, X, ids, mx.LoraSet(A, B))
    x = X[-70:].float()
    for a in range(3):
        assert torch.equal(Y[-70:][a::3], (x[a::3] @ A[a].float().t()) @ B[a].float().t())
    assert not Y[:-70].any()


@pytest.mark.parametrize("M", [24, 500])
def test_replays_of_a_graph(mx, M):
    c = Case(mx, M, 512, 192, 16, 8, BF, 5, True)
    ws = torch.empty(mx.mxs_lora_add_workspace(M, c.set), dtype=torch.uint8, device=DEV)
    c.run(ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(ws=ws)
    for seed in range(5):
        d = Case(mx, M, 512, 192, 16, 8, BF, 50 + seed, True)
        for k in ("A", "B", "X", "ids", "Y", "scale", "rank"):
            getattr(c, k).copy_(getattr(d, k))
        ref, _ = c.reference()
        ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(c.Y.double().cpu().numpy(), ref), seed
        d.run()
        assert torch.equal(c.Y, d.Y)


def test_beside_the_mixed_product(mx):
    """Adapters added to mxs_mixed_gemm's output: the quantised product plus the adapters' own, on a stream of the caller's."""
    from bit_gemm_hdiag_amd import synth
    M, N, K = 40, 96, 256
    X = synth.activations(M, K, 1, synth.outlier_gains(K, 2, 2, 10), dtype=BF, device=DEV)
    W = synth.weights(N, K, 3, dtype=BF, device=DEV)
    perm = torch.randperm(K, generator=torch.Generator().manual_seed(4)).to(torch.int32).to(DEV)
    Wq = mx.mxs_quantize(W, perm, 1, 1, 6)
    c = Case(mx, M, K, N, 12, 3, BF, 6, False)
    c.X = X
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        c.Y = mx.mxs_mixed_gemm_fused(X, perm, Wq)
        base = c.Y.clone()
        c.run()
    s.synchronize()
    got, c.Y = c.Y, base
    ref, tol = c.reference()
    assert (np.abs(got.double().cpu().numpy() - ref) <= tol).all() and not torch.equal(got, base)
