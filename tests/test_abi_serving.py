"""Contract checks of the serving calls that need no GPU: rotary frequencies
(host code) against the formulas, and bad arguments refused before any device
work (every call below fails validation, so nothing is enqueued)."""
import ctypes
import math

import pytest

from ctypes import c_double, c_float, c_int32, c_int64, c_size_t, c_void_p

P = c_void_p
A = P(0x10000)            # never dereferenced: every call below fails validation
OK, ARG, SHAPE, WORKSPACE, UNSUPPORTED = 0, -1, -2, -4, -6


class Cache(ctypes.Structure):
    _fields_ = [("pages", c_int64), ("page_size", c_int32), ("H", c_int32), ("D", c_int32), ("reserved", c_int32),
                ("kc", P), ("ks", P), ("vc", P), ("vs", P)]


def cache(**kw):
    d = dict(pages=10, page_size=16, H=2, D=64, reserved=0, kc=A, ks=A, vc=A, vs=A)
    d.update(kw)
    return ctypes.byref(Cache(*d.values()))


BAD_CACHES = [(dict(pages=0), SHAPE), (dict(page_size=0), SHAPE), (dict(H=0), SHAPE), (dict(D=48), SHAPE),
              (dict(D=0), SHAPE), (dict(reserved=1), ARG), (dict(kc=None), ARG), (dict(vs=None), ARG),
              (dict(kc=P(0x10008)), UNSUPPORTED), (dict(ks=P(0x10004)), UNSUPPORTED), (dict(vc=P(0x10004)), UNSUPPORTED),
              (dict(pages=1 << 28), UNSUPPORTED), (dict(H=20000), UNSUPPORTED)]


@pytest.fixture(scope="module")
def lib():
    import os
    from bit_gemm_hdiag_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    lib = ctypes.CDLL(build.LIB)
    i64, i32 = c_int64, c_int32
    sig = {"mxs_rope_frequencies": [i32, c_double, i32, c_double, c_double, c_double, c_double, P],
           "mxs_rope": [P, i32, i64, i64, i64, i64, i64, P, P, i32, i32, c_float, P, i64, i64, P],
           "mxs_kv4_append": [P, P, P, i32, i64, i64, i64, i64, i64, P, P, P, i32, i32, c_float, P],
           "mxs_kv4_read": [P, P, i64, i32, P, i64, i64, P, i64, i64, P],
           "mxs_attend_kv4_tree": [P, i32, i64, P, P, i64, P, P, P, i64, i64, i64, i64, i64, i64, c_float, P, i64, P,
                                   c_size_t, P]}
    for n, a in sig.items():
        getattr(lib, n).argtypes = a
        getattr(lib, n).restype = c_int32
    w = lib.mxs_attend_kv4_tree_workspace
    w.argtypes, w.restype = [i32] + [i64] * 7, c_size_t
    lib.mxs_last_error.restype = ctypes.c_char_p
    return lib


def freqs(lib, rot, base=10000.0, scaling=0, factor=1.0, low=1.0, high=4.0, length=8192.0):
    out = (c_double * max(1, rot // 2))()
    s = lib.mxs_rope_frequencies(rot, base, scaling, factor, low, high, length, ctypes.cast(out, P))
    return s, list(out)


@pytest.mark.parametrize("rot,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (6, 7.5)])
def test_frequencies_follow_the_formulas(lib, rot, base):
    plain = [base ** (-2.0 * i / rot) for i in range(rot // 2)]

    def close(a, b):
        return all(math.isclose(x, y, rel_tol=1e-14) for x, y in zip(a, b)) and len(a) == len(b)
    assert close(freqs(lib, rot, base)[1], plain)
    assert close(freqs(lib, rot, base, 1, 8.0)[1], [f / 8.0 for f in plain])
    if rot > 2:
        b = base * 4.0 ** (rot / (rot - 2.0))
        got = freqs(lib, rot, base, 2, 4.0)[1]
        assert close(got, [b ** (-2.0 * i / rot) for i in range(rot // 2)])
        # the slowest pair turns exactly factor times slower, the fastest as before
        assert math.isclose(got[-1], plain[-1] / 4.0, rel_tol=1e-12) and got[0] == 1.0
    got = freqs(lib, rot, base, 3, 8.0, 1.0, 4.0, 8192.0)[1]
    for f, g in zip(plain, got):
        turns = 8192.0 * f / (2 * math.pi)
        if turns >= 4.0:
            assert g == f
        elif turns <= 1.0:
            assert math.isclose(g, f / 8.0, rel_tol=1e-14)
        else:
            k = (turns - 1.0) / 3.0
            assert math.isclose(g, k * f + (1 - k) * f / 8.0, rel_tol=1e-13)


def test_frequency_errors(lib):
    assert lib.mxs_rope_frequencies(64, 1e4, 0, 1.0, 1.0, 4.0, 8192.0, None) == ARG
    assert freqs(lib, 0)[0] == SHAPE and freqs(lib, 7)[0] == SHAPE
    assert freqs(lib, 2, scaling=2)[0] == SHAPE
    assert freqs(lib, 64, scaling=4)[0] == ARG and freqs(lib, 64, scaling=-1)[0] == ARG
    for bad in (0.0, -1.0, float("nan"), float("inf")):
        assert freqs(lib, 64, base=bad)[0] == ARG
        assert freqs(lib, 64, scaling=1, factor=bad)[0] == ARG
        assert freqs(lib, 64, scaling=3, length=bad)[0] == ARG
    assert freqs(lib, 64, scaling=3, low=4.0, high=4.0)[0] == ARG
    assert freqs(lib, 64, low=4.0, high=1.0, length=-1.0)[0] == OK          # read for the parts scaling only


def test_rope_errors(lib):
    def call(x=A, dt=1, T=4, H=2, D=64, ldt=128, ldh=64, pos=A, freq=A, rot=64, lay=0, y=P(0x90000), yt=128, yh=64):
        return lib.mxs_rope(x, dt, T, H, D, ldt, ldh, pos, freq, rot, lay, 1.0, y, yt, yh, None)
    assert call(T=0) == OK and call(H=0) == OK and call(T=0, x=None, y=None, pos=None) == OK
    assert call(dt=5) == ARG and call(lay=2) == ARG
    for k in ("x", "y", "pos", "freq"):
        assert call(**{k: None}) == ARG
    assert call(T=-1) == SHAPE and call(H=-1) == SHAPE and call(D=0) == SHAPE
    assert call(rot=0) == SHAPE and call(rot=63) == SHAPE and call(rot=66) == SHAPE
    assert call(ldt=32) == SHAPE and call(ldh=63) == SHAPE and call(ldt=-128) == SHAPE
    assert call(ldt=1 << 41) == SHAPE
    assert call(yt=96) == SHAPE                                  # rows of y overlap
    assert call(y=A, yt=256) == SHAPE                            # in place with other strides
    assert call(D=4098, ldt=1 << 14, ldh=4098, yt=1 << 14, yh=4098) == UNSUPPORTED
    assert call(H=65536) == UNSUPPORTED and call(T=1 << 31) == UNSUPPORTED
    assert call(x=P(0x10001)) == UNSUPPORTED and call(dt=0, y=P(0x90002)) == UNSUPPORTED
    assert call(pos=P(0x10004)) == UNSUPPORTED and call(freq=P(0x10004)) == UNSUPPORTED
    call(dt=5)
    assert b"dtype" in lib.mxs_last_error()


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches_are_refused_everywhere(lib, bad, status):
    c = cache(**bad)
    assert lib.mxs_kv4_append(c, A, A, 1, 4, 1 << 20, 64, 1 << 20, 64, A, None, None, 0, 0, 1.0, None) == status
    assert lib.mxs_kv4_read(c, A, 4, 1, A, 1 << 20, 64, A, 1 << 20, 64, None) == status
    assert lib.mxs_attend_kv4_tree(A, 1, 1 << 22, c, A, 10, A, A, None, 0, 1, 4, 4, 100, 20000, 1.0, A, 1 << 22, A,
                                   1 << 30, None) == status


def test_append_errors(lib):
    def call(c=cache(), k=A, v=A, dt=1, T=4, kt=128, kh=64, vt=128, vh=64, slots=A, pos=None, freq=None, rot=0, lay=0):
        return lib.mxs_kv4_append(c, k, v, dt, T, kt, kh, vt, vh, slots, pos, freq, rot, lay, 1.0, None)
    assert call(T=0) == OK and call(T=0, k=None, v=None, slots=None) == OK
    assert call(c=None) == ARG and call(dt=2) == ARG
    for k in ("k", "v", "slots"):
        assert call(**{k: None}) == ARG
    assert call(T=-1) == SHAPE and call(kt=63) == SHAPE and call(vh=32) == SHAPE and call(kh=-64) == SHAPE
    assert call(pos=A, freq=None, rot=64) == ARG and call(pos=A, freq=A, rot=64, lay=3) == ARG
    assert call(pos=A, freq=A, rot=0) == SHAPE and call(pos=A, freq=A, rot=66) == SHAPE
    assert call(pos=A, freq=A, rot=33) == SHAPE
    assert call(T=1 << 31) == UNSUPPORTED
    assert call(k=P(0x10001)) == UNSUPPORTED and call(dt=0, v=P(0x10002)) == UNSUPPORTED
    assert call(slots=P(0x10004)) == UNSUPPORTED and call(pos=P(0x10004), freq=A, rot=64) == UNSUPPORTED


def test_read_errors(lib):
    def call(c=cache(), slots=A, T=4, dt=1, k=A, kt=128, kh=64, v=A, vt=128, vh=64):
        return lib.mxs_kv4_read(c, slots, T, dt, k, kt, kh, v, vt, vh, None)
    assert call(T=0) == OK and call(T=0, k=None, v=None) == OK
    assert call(c=None) == ARG and call(dt=-1) == ARG and call(slots=None) == ARG and call(k=None, v=None) == ARG
    assert call(T=-1) == SHAPE and call(kt=32) == SHAPE and call(vh=60) == SHAPE
    assert call(kt=96) == SHAPE                                   # rows overlap
    assert call(k=None, kt=0, kh=0, vt=96) == SHAPE               # strides of the output that is there
    assert call(T=1 << 31) == UNSUPPORTED and call(k=P(0x10001)) == UNSUPPORTED
    assert call(slots=P(0x10004)) == UNSUPPORTED


def test_more_tokens_than_a_grid_holds_are_refused(lib):
    big = 1 << 24                # one token a workgroup of 256 threads would pass 2^32 threads
    assert lib.mxs_rope(A, 1, big, 2, 64, 128, 64, A, A, 64, 0, 1.0, P(0x90000), 128, 64, None) == UNSUPPORTED
    assert lib.mxs_kv4_append(cache(), A, A, 1, big, 128, 64, 128, 64, A, None, None, 0, 0, 1.0, None) == UNSUPPORTED
    assert lib.mxs_kv4_read(cache(), A, big, 1, A, 128, 64, A, 128, 64, None) == UNSUPPORTED


def test_tree_attention_errors(lib):
    def call(q=A, dt=1, ldq=256, c=cache(), table=A, ldt=10, lens=A, cu=A, mask=None, words=0, B=2, tq=4, mq=4, ml=160,
             Hq=4, s=0.125, out=A, ldo=256, ws=A, n=1 << 30):
        return lib.mxs_attend_kv4_tree(q, dt, ldq, c, table, ldt, lens, cu, mask, words, B, tq, mq, ml, Hq, s, out, ldo,
                                       ws, n, None)
    assert call(B=0) == OK and call(tq=0) == OK and call(mq=0) == OK
    assert call(B=0, q=None, out=None, table=None, lens=None, cu=None, ws=None, n=0) == OK
    assert call(c=None) == ARG and call(dt=9) == ARG
    assert call(s=float("nan")) == ARG and call(s=float("inf")) == ARG
    for k in ("q", "out", "table", "lens", "cu"):
        assert call(**{k: None}) == ARG
    for k in ("B", "tq", "mq", "ml", "ldt"):
        assert call(**{k: -1}) == SHAPE
    assert call(Hq=3) == SHAPE and call(Hq=1) == SHAPE and call(mask=A, words=0) == SHAPE
    assert call(mask=A, words=-1) == SHAPE
    assert call(ml=161) == SHAPE                                  # table too narrow
    assert call(ldq=255) == SHAPE and call(ldo=128) == SHAPE
    assert call(c=cache(D=288)) == UNSUPPORTED
    assert call(B=65536) == UNSUPPORTED and call(tq=(1 << 24) + 1) == UNSUPPORTED
    assert call(mq=(1 << 20) + 1) == UNSUPPORTED and call(ldt=1 << 27, ml=(1 << 30) + 1) == UNSUPPORTED
    assert call(q=P(0x10001)) == UNSUPPORTED and call(lens=P(0x10002)) == UNSUPPORTED
    assert call(cu=P(0x10002)) == UNSUPPORTED and call(table=P(0x10001)) == UNSUPPORTED
    assert call(mask=P(0x10004), words=1) == UNSUPPORTED
    assert call(B=65535, mq=1 << 20, tq=1 << 24, Hq=64, ldq=64 * 64, ldo=64 * 64) == UNSUPPORTED      # grid
    big = cache(pages=10000)
    need = lib.mxs_attend_kv4_tree_workspace(1, 2, 4, 4, 160000, 4, 2, 64)
    assert need > 0
    assert call(c=big, ldt=10000, ml=160000, n=need - 1) == WORKSPACE
    assert call(c=big, ldt=10000, ml=160000, ws=None) == WORKSPACE
    assert call(c=big, ldt=10000, ml=160000, ws=P(0x10008), n=need) == WORKSPACE


def test_tree_workspace(lib):
    w = lib.mxs_attend_kv4_tree_workspace
    assert w(1, 64, 64, 1, 160, 4, 2, 64) == 0                    # short contexts: nothing to join
    for bad in ((7, 1, 1, 1, 1 << 20, 4, 2, 64), (1, 0, 1, 1, 1 << 20, 4, 2, 64), (1, 1, 0, 1, 1 << 20, 4, 2, 64),
                (1, 1, 1, 0, 1 << 20, 4, 2, 64), (1, 1, 1, 1, -1, 4, 2, 64), (1, 1, 1, 1, 1 << 20, 3, 2, 64),
                (1, 1, 1, 1, 1 << 20, 4, 2, 48), (1, 1, 1, 1, 1 << 20, 4, 2, 288), (1, 1, 1, 1, 1 << 20, 4, 0, 64)):
        assert w(*bad) == 0
    # pieces are kept per workgroup, not per row and range: bounded for any batch
    for args in ((1, 1, 3, 3, 100000, 8, 2, 128), (1, 256, 1 << 16, 256, 1 << 17, 64, 8, 128),
                 (0, 64, 1 << 14, 256, 1 << 20, 128, 8, 256)):
        assert 0 < w(*args) < 1 << 28


def test_binding_refuses_host_tensors():
    import torch
    import bit_gemm_hdiag_amd as mx
    x = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError):
        mx.mxs_rope(x, torch.zeros(2, dtype=torch.int64), torch.zeros(32, dtype=torch.float64))
    with pytest.raises(ValueError):
        mx.mxs_rope_frequencies(64, scaling="other", device="cpu")
    with pytest.raises(mx.MxsError):
        mx.mxs_rope_frequencies(63, device="cpu")
    assert mx.mxs_rope_frequencies(64, device="cpu").shape == (32,)
    with pytest.raises(ValueError):
        mx.kv4_cache_alloc(2, 16, 2, 48, device="cpu")
    with pytest.raises(ValueError):
        mx.kv4_cache_alloc(2, 16, 2, 64, device="cpu")
    with pytest.raises(ValueError):
        mx.mxs_attend_kv4_tree(x, None, None, None, None, 1.0)


def test_work_that_wraps_64_bits_is_refused(lib):
    """Every size is allowed by itself; the count of work units is past 2^64, and
    wraps to a negative number, to zero or to a few units."""
    def call(B, Hq, H, max_q, max_len, dt=1):
        c = cache(pages=1 << 20, H=H, D=32)
        return lib.mxs_attend_kv4_tree(A, dt, Hq * 32, c, A, 1 << 26, A, A, None, 0, B, 1 << 24, max_q, max_len, Hq, 1.0, A,
                                       Hq * 32, A, 1 << 40, None)
    assert call(65535, 16383, 16383, 1 << 20, 1 << 30) == UNSUPPORTED
    assert call(1 << 15, 1 << 13, 1 << 13, 1 << 20, 1 << 30) == UNSUPPORTED       # 2^64 units
    assert call(1 << 15, 1 << 13, 1 << 13, 1 << 20, (1 << 30) - 64) == UNSUPPORTED
    for dt in (0, 1):
        for B in (1 << 12, 1 << 14, 65535):
            for heads in (1 << 12, 12345, 16383):
                for max_q in (1, 300, 1 << 20):
                    assert call(B, heads, heads, max_q, 1 << 30, dt) == UNSUPPORTED, (dt, B, heads, max_q)
    w = lib.mxs_attend_kv4_tree_workspace
    big = (1 << 63) - 1
    assert w(1, 1, 1, 1 << 14, 1 << 30, 65535, 1, 32) == 0 and w(1, 1, 1, 1 << 10, 1 << 16, 65535, 1, 32) > 0
    for bad in ((1, big, 1, 1, 1 << 30, 4, 2, 64), (1, 1, big, 1, 1 << 30, 4, 2, 64), (1, 1, 1, big, 1 << 30, 4, 2, 64),
                (1, 1, 1, 1, big, 4, 2, 64), (1, 1, 1, 1, 1 << 30, big - 1, 2, 64), (1, 1, 1, 1, 1 << 30, big, big, 64)):
        assert w(*bad) == 0                                       # sizes that the call refuses
