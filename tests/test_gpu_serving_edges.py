"""The serving calls at the ends of what a cache can hold."""
import numpy as np
import pytest
import torch

from test_gpu_serving import BF, DEV, F32, Batch, n64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import bit_gemm_hdiag_amd as mx
    return mx


# ----------------------------------------------- blocks marked 0xFF that hold codes
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [40, 9000])                        # one and four words a thread
def test_read_of_marked_blocks_is_nan_whatever_their_codes(mx, dtype, T):
    H, D = 8, 128
    c = mx.kv4_cache_alloc(-(-T // 16), 16, H, D)
    g = torch.Generator(device=DEV).manual_seed(T)
    for t in (c.kc, c.vc):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    marked = []
    for t in (c.ks, c.vs):
        m = torch.rand(t.shape, generator=g, device=DEV) < 0.25
        t.copy_(torch.where(m, 255, 120))
        marked.append(m.view(-1, H, D // 32)[:T].repeat_interleave(32, -1))
    for got, m in zip(mx.mxs_kv4_read(c, torch.arange(T, device=DEV), dtype), marked):
        assert int((torch.isnan(got) != m).sum()) == 0
        assert int((~torch.isfinite(got[~m])).sum()) == 0


@pytest.mark.parametrize("D", [64, 96, 128, 256])
@pytest.mark.parametrize("n,G", [(1, 1), (1, 8), (3, 8), (12, 8), (40, 8)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_of_marked_blocks_is_nan_whatever_their_codes(mx, dtype, n, G, D):
    """Blocks with byte 0xFF and codes of either sign, in the context and among the drafted tokens."""
    b = Batch(mx, [700, 90, 60], [n, min(n, 5), min(n, 5)], 2 * G, 2, D, 16, dtype, "causal", 50 + D)
    c = b.cache
    last = lambda plane, s, t: plane[int(b.table[s, t // 16]), t % 16]
    for s, t, head, planes in ((0, 333, 0, ("vs", "vc")), (0, 700 - 1, 1, ("vs", "vc")), (1, 17, 0, ("ks", "kc")),
                               (1, 89, 1, ("ks", "kc"))):
        last(getattr(c, planes[0]), s, t)[head, 1] = 255
        codes = last(getattr(c, planes[1]), s, t)[head, 16:32]
        codes.copy_(torch.tensor([0x11, 0x77, 0x99, 0xF8] * 4, dtype=torch.uint8, device=DEV))
    got = b.run(mx)
    ref, _ = b.reference()
    assert np.isnan(ref).any() and not np.isnan(ref).all()
    assert np.array_equal(np.isnan(n64(got)), np.isnan(ref))
    b.check(got)


# ------------------------------------------------------------------ one of the two read
@pytest.mark.parametrize("T", [9, 9000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_read_of_keys_or_of_values_alone(mx, T, dtype):
    H, D = 3, 96
    c = mx.kv4_cache_alloc(-(-T // 17), 17, H, D)
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(T, generator=g).to(DEV)
    k, v = (torch.randn(T, H, D, generator=g).to(DEV) for _ in range(2))
    mx.mxs_kv4_append(c, k, v, slots)
    both = mx.mxs_kv4_read(c, slots, dtype)
    ko, none = mx.mxs_kv4_read(c, slots, dtype, values=False)
    assert none is None and torch.equal(ko, both[0])
    none, vo = mx.mxs_kv4_read(c, slots, dtype, keys=False)
    assert none is None and torch.equal(vo, both[1])
    rows = torch.full((T, 2 * H, D), 7.0, dtype=dtype, device=DEV)        # the other half is left as it was
    mx.mxs_kv4_read(c, slots, v_out=rows[:, H:], keys=False)
    assert torch.equal(rows[:, H:], both[1]) and bool((rows[:, :H] == 7.0).all())
    for bad in (dict(keys=False, values=False), dict(keys=False, k_out=rows[:, :H]),
                dict(values=False, v_out=rows[:, H:])):
        with pytest.raises(ValueError):
            mx.mxs_kv4_read(c, slots, **bad)


# --------------------------------------------------------------- values near the largest
@pytest.mark.parametrize("rows", [1, 8, 24, 40, 300])
@pytest.mark.parametrize("byte", [240, 250, 252, 254])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_of_large_values_is_finite(mx, dtype, D, byte, rows):
    """Codes of 1 and 0 at scales up to 2^127: over equal scores the output is the value itself, while
    sums of p 2^s are up to 60 times 2^127 (and of p 2^(s - 9), which the kernels keep, below 2^127)."""
    L = 60
    n = min(rows, L)
    G = rows // n
    B = 260 if rows == 24 else 3                                 # 24 rows: a kernel for few sequences, one for many
    b = Batch(mx, [L] * B, [n] * B, G, 1, D, 16, dtype, "causal", 4)
    b.q.zero_()
    c = b.cache
    c.vs.fill_(byte)
    c.vc.fill_(0x01)                                             # even dims 1, odd dims 0
    out = b.run(mx).double()
    assert int((~torch.isfinite(out)).sum()) == 0
    # sums of up to 60 weights of 1, exact; division and product round twice, then the output
    want = 2.0 ** (byte - 127)
    assert ((out[..., 0::2] - want).abs() <= (2 * 2.0 ** -24 + 2.0 ** -8 * (dtype == BF)) * want).all()
    assert not out[..., 1::2].any()


@pytest.mark.parametrize("rows", [1, 8, 24, 40, 300])
@pytest.mark.parametrize("byte", [0, 1, 2, 3, 4, 6, 9, 20])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_of_tiny_values(mx, dtype, byte, rows):
    """Codes 0 to 7 at the smallest scales, the same in every token, over equal scores."""
    L, D = 40, 64
    n = min(rows, L)
    B = 260 if rows == 24 else 3
    b = Batch(mx, [L] * B, [n] * B, rows // n, 1, D, 16, dtype, "causal", 4)
    b.q.zero_()
    c = b.cache
    c.vs.fill_(byte)
    codes = torch.arange(D, device=DEV) % 8
    c.vc.copy_((codes[0::2] | codes[1::2] << 4).to(torch.uint8))
    out = b.run(mx).double()
    want = codes.double() * 2.0 ** (byte - 127)
    # bytes 0 to 2 are read to multiples of 2^-124; a type's subnormals have one step
    low = 2.0 ** -125 if byte < 3 else 0.0
    step = {BF: 2.0 ** -134, F32: 2.0 ** -150}[dtype]
    assert ((out - want).abs() <= low + step + (2 * 2.0 ** -24 + 2.0 ** -8 * (dtype == BF)) * (want + low)).all()


# ------------------------------------------------------------ caches that others wrote
@pytest.mark.parametrize("Hq,Hkv,D,n", [(1, 1, 32, 1), (8, 2, 64, 1), (16, 2, 128, 1), (6, 2, 96, 9), (16, 1, 128, 12),
                                        (8, 2, 160, 7), (4, 1, 256, 3), (16, 2, 128, 40)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attention_over_any_codes(mx, dtype, Hq, Hkv, D, n):
    """Every code, -8 among them, which no quantised block holds, and blocks of differing scales."""
    b = Batch(mx, [300, 70], [n, n], Hq, Hkv, D, 16, dtype, "tree", 60 + D)
    g = torch.Generator(device=DEV).manual_seed(D)
    for t in (b.cache.kc, b.cache.vc):
        t.copy_(torch.randint(0, 256, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    for t in (b.cache.ks, b.cache.vs):
        t.copy_(torch.randint(118, 127, t.shape, generator=g, device=DEV, dtype=torch.uint8))
    b.check(b.run(mx))


def test_attention_over_no_pages(mx):
    """A table without columns: nothing is cached, every row is 0."""
    b = Batch(mx, [40, 3], [2, 1], 4, 2, 64, 16, BF, "causal", 3)
    out = torch.full_like(b.q, 5.0)
    none = torch.empty(2, 0, dtype=torch.int32, device=DEV)
    got = mx.mxs_attend_kv4_tree(b.q, b.cache, none, b.dev([0, 0]), b.dev([0, 2, 3]), 0.125, out=out)
    assert got is out and not out.any()
