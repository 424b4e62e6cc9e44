"""Contract checks of the verification of drafted tokens that need no GPU: bad
arguments are refused before any device work."""
import ctypes
from ctypes import c_int32, c_int64, c_size_t

import pytest

from test_abi_serving import A, ARG, OK, SHAPE, UNSUPPORTED, WORKSPACE, P


@pytest.fixture(scope="module")
def lib():
    import os
    from bit_gemm_hdiag_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    lib = ctypes.CDLL(build.LIB)
    i64, i32 = c_int64, c_int32
    lib.mxs_verify_tree.argtypes = [P, i32, i64, i64, P, P, P, i64, i64, i64, P, i64, i32, P, P, P, P, P, P, c_size_t, P]
    lib.mxs_verify_tree.restype = i32
    lib.mxs_verify_tree_workspace.argtypes, lib.mxs_verify_tree_workspace.restype = [i64] * 4, c_size_t
    return lib


def call(lib, logits=A, dt=1, ldl=1000, V=1000, tokens=A, parents=A, cu=A, B=2, total=10, max_n=8, draft=A, ldd=1000,
         rep=0, temp=A, u=A, path=A, count=A, nxt=A, ws=A, n=1 << 24):
    return lib.mxs_verify_tree(logits, dt, ldl, V, tokens, parents, cu, B, total, max_n, draft, ldd, rep, temp, u, path,
                               count, nxt, ws, n, None)


def test_errors(lib):
    assert call(lib, B=0) == OK and call(lib, B=0, logits=None, cu=None, count=None, nxt=None, ws=None, n=0) == OK
    assert call(lib, dt=2) == ARG and call(lib, rep=2) == ARG and call(lib, rep=-1) == ARG
    for k in ("logits", "tokens", "cu", "u", "path", "count", "nxt"):
        assert call(lib, **{k: None}) == ARG, k
    for k in ("B", "total", "max_n"):
        assert call(lib, **{k: -1}) == SHAPE, k
    assert call(lib, V=0) == SHAPE and call(lib, ldl=999) == SHAPE and call(lib, ldd=999) == SHAPE
    assert call(lib, ldl=(1 << 40) + 1) == SHAPE
    assert call(lib, B=65536) == UNSUPPORTED and call(lib, total=(1 << 22) + 1) == UNSUPPORTED
    assert call(lib, max_n=1025) == UNSUPPORTED
    assert call(lib, V=(1 << 20) + 1, ldl=1 << 21, ldd=1 << 21) == UNSUPPORTED
    for k, p in (("logits", 0x10001), ("tokens", 0x10004), ("parents", 0x10002), ("cu", 0x10002), ("draft", 0x10002),
                 ("temp", 0x10002), ("u", 0x10004), ("path", 0x10002), ("count", 0x10002), ("nxt", 0x10004)):
        assert call(lib, **{k: P(p)}) == UNSUPPORTED, k
    assert call(lib, dt=0, logits=P(0x10002)) == UNSUPPORTED
    need = lib.mxs_verify_tree_workspace(2, 10, 8, 1000)
    assert need > 0
    assert call(lib, n=need - 1) == WORKSPACE and call(lib, ws=None) == WORKSPACE
    assert call(lib, ws=P(0x10008), n=need) == WORKSPACE


def test_workspace(lib):
    w = lib.mxs_verify_tree_workspace
    for bad in ((0, 10, 8, 1000), (65536, 10, 8, 1000), (2, -1, 8, 1000), (2, (1 << 22) + 1, 8, 1000), (2, 10, -1, 1000),
                (2, 10, 1025, 1000), (2, 10, 8, 0), (2, 10, 8, (1 << 20) + 1)):
        assert w(*bad) == 0
    assert 0 < w(2, 10, 8, 1000) < w(2, 10, 8, 100000) < w(2, 1000, 8, 100000)
    assert w(65535, 1 << 22, 1024, 1 << 20) < 1 << 37


def test_binding_refuses_wrong_tensors(monkeypatch):
    import torch
    import bit_gemm_hdiag_amd as mx
    from bit_gemm_hdiag_amd import binding
    from test_binding_workspace import Device

    def reached(*args):
        raise AssertionError("reached the library")
    monkeypatch.setattr(binding, "_call", reached)
    F32, F64, I32, I64, BF = torch.float32, torch.float64, torch.int32, torch.int64, torch.bfloat16
    d = lambda n, t: Device((n,), t)
    ok = dict(logits=Device((6, 100), BF), tokens=d(6, I64), cu=d(3, I32), uniform=d(6, F64), parents=d(6, I32),
              draft=Device((6, 100), F32), temperature=d(2, F32), path=d(6, I32), count=d(2, I32), next_token=d(2, I64),
              ws=d(1 << 16, torch.uint8))
    with pytest.raises(AssertionError):
        mx.mxs_verify_tree(**ok)
    for bad in (dict(logits=Device((6, 100), F64)), dict(logits=Device((600,), BF)), dict(tokens=d(6, I32)),
                dict(tokens=d(5, I64)), dict(cu=d(3, I64)), dict(uniform=d(6, F32)), dict(uniform=d(7, F64)),
                dict(parents=d(5, I32)), dict(draft=Device((6, 100), BF)), dict(draft=Device((6, 99), F32)),
                dict(temperature=d(3, F32)), dict(temperature=d(2, F64)), dict(path=d(5, I32)), dict(count=d(3, I32)),
                dict(next_token=d(2, I32))):
        with pytest.raises((ValueError, TypeError)):
            mx.mxs_verify_tree(**{**ok, **bad})


@pytest.mark.parametrize("total", [6, 1024, 1025, 9000])
def test_default_bound_of_a_tree(monkeypatch, total):
    """Without max_n a batch of any number of rows is taken; its trees hold at most 1024 nodes."""
    import torch
    import bit_gemm_hdiag_amd as mx
    from bit_gemm_hdiag_amd import binding
    from test_binding_workspace import Device
    seen = []
    monkeypatch.setattr(binding, "_call", lambda gpu, fn, name, *args: seen.append(args))
    F64, I32, I64 = torch.float64, torch.int32, torch.int64
    d = lambda n, t: Device((n,), t)
    args = Device((total, 100), torch.bfloat16), d(total, I64), d(3, I32), d(total, F64)
    outs = dict(path=d(total, I32), count=d(2, I32), next_token=d(2, I64), ws=d(1 << 16, torch.uint8))
    mx.mxs_verify_tree(*args, **outs)
    mx.mxs_verify_tree(*args, **outs, max_n=4)
    assert [x[9] for x in seen] == [min(total, 1024), 4]
    assert mx.mxs_verify_tree_workspace(2, total, seen[0][9], 100) > 0
