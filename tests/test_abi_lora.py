"""Contract checks of the adapters beside a projection that need no GPU: bad
arguments are refused before any device work."""
import ctypes
from ctypes import c_int32, c_int64, c_size_t

import pytest

from test_abi_serving import A, ARG, OK, SHAPE, UNSUPPORTED, WORKSPACE, P


class Set(ctypes.Structure):
    _fields_ = [("K", c_int64), ("N", c_int64), ("n", c_int32), ("R", c_int32), ("dtype", c_int32),
                ("reserved", c_int32), ("A", P), ("B", P), ("scale", P), ("rank", P)]


def adapters(**kw):
    d = dict(K=256, N=100, n=4, R=16, dtype=1, reserved=0, A=A, B=A, scale=A, rank=A)
    d.update(kw)
    return ctypes.byref(Set(*d.values()))


@pytest.fixture(scope="module")
def lib():
    import os
    from bit_gemm_hdiag_amd import build
    if not os.path.exists(build.LIB):
        build.build()
    lib = ctypes.CDLL(build.LIB)
    i64 = c_int64
    lib.mxs_lora_add.argtypes, lib.mxs_lora_add.restype = [P, i64, i64, P, P, P, i64, P, c_size_t, P], c_int32
    lib.mxs_lora_add_workspace.argtypes, lib.mxs_lora_add_workspace.restype = [i64, P], c_size_t
    return lib


def call(lib, X=A, M=8, ldx=256, ids=A, s=None, Y=A, ldy=100, ws=A, n=1 << 30):
    return lib.mxs_lora_add(X, M, ldx, ids, s or adapters(), Y, ldy, ws, n, None)


def test_errors(lib):
    for empty in (dict(M=0), dict(s=adapters(N=0)), dict(s=adapters(n=0))):
        assert call(lib, **empty) == OK and call(lib, **empty, X=None, ids=None, Y=None, ws=None, n=0) == OK
    assert lib.mxs_lora_add(A, 8, 256, A, None, A, 100, A, 1 << 30, None) == ARG
    for k in ("X", "ids", "Y"):
        assert call(lib, **{k: None}) == ARG
    for bad in (dict(reserved=1), dict(dtype=2), dict(A=None), dict(B=None)):
        assert call(lib, s=adapters(**bad)) == ARG, bad
    for bad in (dict(K=0), dict(K=40), dict(K=-32), dict(N=-1), dict(n=-1), dict(R=0), dict(R=-4)):
        assert call(lib, s=adapters(**bad)) == SHAPE, bad
    assert call(lib, M=-1) == SHAPE and call(lib, ldx=255) == SHAPE and call(lib, ldy=99) == SHAPE
    assert call(lib, ldx=(1 << 40) + 1) == SHAPE
    for bad in (dict(R=129), dict(n=8193), dict(K=1 << 25), dict(N=(1 << 24) + 1)):
        assert call(lib, ldx=1 << 30, ldy=1 << 30, s=adapters(**bad)) == UNSUPPORTED, bad
    assert call(lib, M=(1 << 22) + 1) == UNSUPPORTED
    assert call(lib, X=P(0x10001)) == UNSUPPORTED and call(lib, Y=P(0x10002)) == UNSUPPORTED
    assert call(lib, ids=P(0x10002)) == UNSUPPORTED and call(lib, X=P(0x10002), s=adapters(dtype=0)) == UNSUPPORTED
    for k, p in (("A", 0x10008), ("B", 0x10008), ("scale", 0x10002), ("rank", 0x10002)):
        assert call(lib, s=adapters(**{k: P(p)})) == UNSUPPORTED, k
    for M in (8, 800):
        need = lib.mxs_lora_add_workspace(M, adapters())
        assert need > 0
        assert call(lib, M=M, n=need - 1) == WORKSPACE and call(lib, M=M, ws=None) == WORKSPACE
        assert call(lib, M=M, ws=P(0x10010), n=need) == WORKSPACE


def test_workspace(lib):
    w = lib.mxs_lora_add_workspace
    assert w(8, None) == 0
    for bad in (dict(dtype=5), dict(K=40), dict(R=0), dict(R=129), dict(n=8193), dict(N=0), dict(n=0), dict(n=-1)):
        assert w(8, adapters(**bad)) == 0, bad
    assert w(0, adapters()) == 0 and w(-1, adapters()) == 0 and w((1 << 22) + 1, adapters()) == 0
    assert 0 < w(8, adapters()) < w(8, adapters(R=128)) < w(5000, adapters(R=128))
    assert w(1 << 22, adapters(K=1 << 24, N=1 << 24, R=128, n=8192)) < 1 << 34


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("K,N,R,n", [(8192, 28672, 64, 48), (8192, 8192, 16, 16), (4096, 1001, 27, 9), (32, 100, 1, 1),
                                     (14336, 4096, 128, 300), (1 << 20, 64, 8, 8192), (416, 64, 33, 2)])
def test_workspace_for_the_largest_batch_serves_smaller_ones(lib, K, N, R, n, dtype):
    s = adapters(K=K, N=N, R=R, n=n, dtype=dtype)
    sizes = list(range(1, 9000)) + [x + d for k in range(14, 23) for x in (1 << k, 3 << k - 2) for d in (-1, 0, 1)]
    last = 0
    for M in sorted(x for x in sizes if x <= 1 << 22):
        need = lib.mxs_lora_add_workspace(M, s)
        assert need >= last, M
        last = need


def test_binding_refuses_wrong_tensors(monkeypatch):
    import torch
    import bit_gemm_hdiag_amd as mx
    from bit_gemm_hdiag_amd import binding
    from test_binding_workspace import Device

    def reached(*args):
        raise AssertionError("reached the library")
    monkeypatch.setattr(binding, "_call", reached)
    F32, I32, BF = torch.float32, torch.int32, torch.bfloat16
    t = lambda *shape, dt=BF: Device(shape, dt)
    for bad in ((t(4, 8, 64), t(4, 100, 9)), (t(4, 8, 64), t(3, 100, 8)), (t(4, 8, 64), t(4, 100, 8, dt=F32)),
                (t(8, 64), t(100, 8)), (t(4, 8, 64), t(4, 100, 8), t(3, dt=F32)),
                (t(4, 8, 64), t(4, 100, 8), t(4)), (t(4, 8, 64), t(4, 100, 8), None, t(4, dt=F32))):
        with pytest.raises(ValueError):
            mx.LoraSet(*bad)
    with pytest.raises(ValueError):
        mx.LoraSet(torch.zeros(1, 8, 64), torch.zeros(1, 5, 8))
    s = mx.LoraSet(t(4, 8, 64), t(4, 100, 8), t(4, dt=F32), t(4, dt=I32))
    ok = dict(Y=t(6, 100, dt=F32), X=t(6, 64), ids=t(6, dt=I32), adapters=s, ws=t(1 << 16, dt=torch.uint8))
    with pytest.raises(AssertionError):
        mx.mxs_lora_add(**ok)
    for bad in (dict(Y=t(6, 100)), dict(Y=t(6, 99, dt=F32)), dict(X=t(6, 64, dt=F32)), dict(X=t(6, 65)),
                dict(X=t(5, 64)), dict(ids=t(6, dt=torch.int64)), dict(ids=t(7, dt=I32))):
        with pytest.raises((ValueError, TypeError)):
            mx.mxs_lora_add(**{**ok, **bad})
