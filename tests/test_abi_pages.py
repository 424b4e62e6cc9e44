"""Contract checks of the calls on pages of the cache that need no GPU: bad
arguments are refused before any device work (every call below fails
validation or has nothing to do, so nothing is enqueued)."""
import ctypes
from ctypes import c_int32, c_int64, c_size_t

import pytest

from test_abi_serving import A, ARG, BAD_CACHES, OK, SHAPE, UNSUPPORTED, WORKSPACE, P, cache


@pytest.fixture(scope="module")
def lib():
    import os
    from bit_gemm_hdiag_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    lib = ctypes.CDLL(build.LIB)
    i64 = c_int64
    sig = {"mxs_kv4_copy": [P, P, P, P, i64, P],
           "mxs_kv4_fork": [P, P, P, i64, i64, P, P, P, i64, P],
           "mxs_kv4_reserve": [P, P, P, i64, i64, P, P, i64, P, P, P, c_size_t, P],
           "mxs_kv4_compact": [P, P, i64, i64, P, P, P, P, i64, P, P],
           "mxs_kv4_release": [P, P, P, i64, i64, P, P, P, P]}
    for n, a in sig.items():
        getattr(lib, n).argtypes = a
        getattr(lib, n).restype = c_int32
    lib.mxs_kv4_reserve_workspace.argtypes, lib.mxs_kv4_reserve_workspace.restype = [i64, i64], c_size_t
    return lib


MIS4, MIS8 = P(0x10002), P(0x10004)


def copy(lib, dst=None, ds=A, src=None, ss=A, T=4):
    return lib.mxs_kv4_copy(dst or cache(), ds, src or cache(), ss, T, None)


def fork(lib, c=None, refs=A, table=A, ldt=10, B=4, lens=A, src=A, dst=A, n=2):
    return lib.mxs_kv4_fork(c or cache(), refs, table, ldt, B, lens, src, dst, n, None)


def reserve(lib, c=None, refs=A, table=A, ldt=10, B=4, lens=A, cu=A, total=8, slots=A, out=A, ws=A, n=1 << 20):
    return lib.mxs_kv4_reserve(c or cache(), refs, table, ldt, B, lens, cu, total, slots, out, ws, n, None)


def compact(lib, c=None, table=A, ldt=10, B=4, lens=A, cu=A, path=A, count=A, total=8, out=A):
    return lib.mxs_kv4_compact(c or cache(), table, ldt, B, lens, cu, path, count, total, out, None)


def release(lib, c=None, refs=A, table=A, ldt=10, B=4, lens=A, keep=A, out=A):
    return lib.mxs_kv4_release(c or cache(), refs, table, ldt, B, lens, keep, out, None)


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_bad_caches_are_refused(lib, bad, status):
    c = cache(**bad)
    for call in (fork, reserve, compact, release):
        assert call(lib, c=c) == status
    assert copy(lib, dst=c) == status and copy(lib, src=c) == status


def test_copy_errors(lib):
    assert copy(lib, T=0) == OK and copy(lib, T=0, ds=None, ss=None) == OK
    assert lib.mxs_kv4_copy(None, A, cache(), A, 4, None) == ARG
    assert lib.mxs_kv4_copy(cache(), A, None, A, 4, None) == ARG
    assert copy(lib, ds=None) == ARG and copy(lib, ss=None) == ARG
    assert copy(lib, T=-1) == SHAPE and copy(lib, dst=cache(H=3)) == SHAPE and copy(lib, src=cache(D=96)) == SHAPE
    assert copy(lib, T=1 << 24) == UNSUPPORTED
    assert copy(lib, ds=MIS8) == UNSUPPORTED and copy(lib, ss=MIS8) == UNSUPPORTED


@pytest.mark.parametrize("call,needs", [(fork, ("refs", "table", "lens", "src", "dst")),
                                        (reserve, ("refs", "table", "lens", "cu", "slots", "out")),
                                        (compact, ("table", "lens", "cu", "path", "count", "out")),
                                        (release, ("refs", "table", "lens", "keep", "out"))])
def test_table_errors(lib, call, needs):
    assert call(lib, B=0) == OK and call(lib, B=0, **{k: None for k in needs}) == OK
    for k in needs:
        assert call(lib, **{k: None}) == ARG, k
        assert call(lib, **{k: MIS4}) == UNSUPPORTED, k
    assert call(lib, B=-1) == SHAPE and call(lib, ldt=-1) == SHAPE
    assert call(lib, B=65536) == UNSUPPORTED and call(lib, ldt=(1 << 30) + 1) == UNSUPPORTED


def test_sizes(lib):
    assert fork(lib, n=0) == OK and fork(lib, n=0, src=None, dst=None) == OK
    assert fork(lib, n=-1) == SHAPE and fork(lib, n=65536) == UNSUPPORTED
    for call in (reserve, compact):
        assert call(lib, total=-1) == SHAPE and call(lib, total=1 << 24) == UNSUPPORTED
    assert reserve(lib, slots=MIS8) == UNSUPPORTED
    assert reserve(lib, c=cache(pages=(1 << 24) + 1)) == UNSUPPORTED


def test_reserve_workspace(lib):
    w = lib.mxs_kv4_reserve_workspace
    for bad in ((0, 4), (-1, 4), ((1 << 24) + 1, 4), (10, 0), (10, -1), (10, 65536)):
        assert w(*bad) == 0
    need = w(10, 4)
    assert 0 < need < w(5000, 4) < w(1 << 24, 65535) < 1 << 28
    assert reserve(lib, n=need - 1) == WORKSPACE and reserve(lib, ws=None) == WORKSPACE
    assert reserve(lib, ws=P(0x10008), n=need) == WORKSPACE


def test_binding_refuses_wrong_tensors(monkeypatch):
    import torch
    import bit_gemm_hdiag_amd as mx
    from bit_gemm_hdiag_amd import binding
    from test_binding_workspace import Device

    def reached(*args):
        raise AssertionError("reached the library")
    monkeypatch.setattr(binding, "_call", reached)
    I32, I64 = torch.int32, torch.int64
    c = mx.KV4Cache(*(Device((6, 16, 2, w), torch.uint8) for w in (32, 2, 32, 2)))
    d = lambda n, t=I32: Device((n,), t)
    table, refs, lens, cu = Device((3, 5), I32), d(6), d(3), d(4)
    ws = Device((1 << 16,), torch.uint8)
    bad = [lambda: mx.mxs_kv4_copy(c, d(4), c, d(4, I64)), lambda: mx.mxs_kv4_copy(c, d(4, I64), c, d(5, I64)),
           lambda: mx.mxs_kv4_fork(c, d(5), table, lens, d(1), d(1)),
           lambda: mx.mxs_kv4_fork(c, refs, table, lens, d(1), d(2)),
           lambda: mx.mxs_kv4_fork(c, refs, Device((3, 5), I64), lens, d(1), d(1)),
           lambda: mx.mxs_kv4_reserve(c, refs, table, lens, cu, ws=ws),
           lambda: mx.mxs_kv4_reserve(c, refs, table, lens, cu, total=3, slots=d(4, I64), lens_out=lens, ws=ws),
           lambda: mx.mxs_kv4_reserve(c, refs, table, lens, d(3), slots=d(4, I64), lens_out=lens, ws=ws),
           lambda: mx.mxs_kv4_reserve(c, refs, table, lens, cu, slots=d(4), lens_out=lens, ws=ws),
           lambda: mx.mxs_kv4_compact(c, table, lens, cu, d(8, I64), d(3), lens_out=lens),
           lambda: mx.mxs_kv4_compact(c, table, lens, cu, d(8), d(4), lens_out=lens),
           lambda: mx.mxs_kv4_compact(c, Device((4, 5), I32), lens, cu, d(8), d(3), lens_out=lens),
           lambda: mx.mxs_kv4_release(c, refs, table, lens, d(3, I64), lens_out=lens),
           lambda: mx.mxs_kv4_release(c, refs, table, lens, d(3), lens_out=d(2))]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def test_compaction_with_the_slots_of_a_reservation(lib):
    f = lib.mxs_kv4_compact_granted
    f.argtypes, f.restype = [P, P, c_int64, c_int64, P, P, P, P, P, c_int64, P, P], c_int32

    def call(c=None, table=A, ldt=10, B=4, lens=A, cu=A, path=A, count=A, slots=A, total=8, out=A):
        return f(c or cache(), table, ldt, B, lens, cu, path, count, slots, total, out, None)
    for bad, status in BAD_CACHES:
        assert call(c=cache(**bad)) == status
    assert call(B=0) == OK and call(B=0, slots=None, path=None) == OK
    for k in ("table", "lens", "cu", "path", "count", "slots", "out"):
        assert call(**{k: None}) == ARG, k
        assert call(**{k: MIS4}) == UNSUPPORTED, k
    assert call(slots=MIS8) == UNSUPPORTED
    assert call(B=-1) == SHAPE and call(ldt=-1) == SHAPE and call(total=-1) == SHAPE
    assert call(B=65536) == UNSUPPORTED and call(total=1 << 24) == UNSUPPORTED


def test_binding_passes_the_slots_of_a_reservation(monkeypatch):
    import torch
    import bit_gemm_hdiag_amd as mx
    from bit_gemm_hdiag_amd import binding
    from test_binding_workspace import Device
    calls = []
    monkeypatch.setattr(binding, "_call", lambda gpu, fn, name, *args: calls.append((name, args)))
    I32, I64 = torch.int32, torch.int64
    c = mx.KV4Cache(*(Device((6, 16, 2, w), torch.uint8) for w in (32, 2, 32, 2)))
    d = lambda n, t=I32: Device((n,), t)
    args = c, Device((3, 5), I32), d(3), d(4), d(8), d(3)
    mx.mxs_kv4_compact(*args, lens_out=d(3))
    mx.mxs_kv4_compact_granted(*args, d(8, I64), lens_out=d(3))
    assert [n for n, _ in calls] == ["mxs_kv4_compact", "mxs_kv4_compact_granted"]
    assert [len(a) for _, a in calls] == [10, 11]
    for slots in (d(7, I64), d(8)):
        with pytest.raises(ValueError):
            mx.mxs_kv4_compact_granted(*args, slots, lens_out=d(3))
    assert len(calls) == 2
