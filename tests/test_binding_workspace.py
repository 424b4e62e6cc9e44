"""A workspace that the binding allocates for a call lives until the library
function has returned: a call of two launches leaves its pieces there between
them, and a block given back earlier could go to a call of another thread on
the same stream. Checked without a GPU, with stubs in place of the library and
of device tensors."""
import gc
import weakref

import pytest
import torch

BYTES = 4096


class Device:
    """A contiguous device tensor as the binding sees one."""

    def __init__(self, shape, dtype):
        self.shape, self.dtype, self.device, self.is_cuda = torch.Size(shape), dtype, "cuda:0", True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return torch.empty(0, dtype=self.dtype).element_size()

    def stride(self, i=None):
        s = [1]
        for n in reversed(self.shape[1:]):
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def is_contiguous(self):
        return True

    def get_device(self):
        return 0

    def data_ptr(self):
        return id(self)


class Library:
    """Workspace queries answer BYTES; any other function notes whether the
    workspaces allocated so far are still there and were passed."""

    def __init__(self, made):
        self.made, self.calls = made, 0

    def __getattr__(self, name):
        if name.endswith("_workspace"):
            return lambda *a: BYTES

        def function(*args):
            gc.collect()
            assert self.made, name
            for tensor in self.made:
                assert tensor() is not None, name + ": workspace given back before the call"
                assert id(tensor()) in args and BYTES in args, name
            self.calls += 1
            return 0
        return function


@pytest.fixture
def stubbed(monkeypatch):
    from bit_gemm_hdiag_amd import binding
    made = []                                     # workspaces, by weak reference
    real = torch.empty

    def empty(*shape, dtype=None, device=None):
        if str(device) == "cpu" or device is None:
            return real(*shape, dtype=dtype)
        t = Device(shape[0] if isinstance(shape[0], (tuple, list)) else shape, dtype)
        if dtype is torch.uint8 and t.shape == (BYTES,):
            made.append(weakref.ref(t))
        return t

    lib = Library(made)
    monkeypatch.setattr(binding, "_lib", lib)
    monkeypatch.setattr(binding, "_stream", lambda dev: 0)
    monkeypatch.setattr(binding, "_call", lambda gpu, fn, name, *args: fn(*args, 0))
    monkeypatch.setattr(binding.torch, "empty", empty)
    monkeypatch.setattr(binding.torch, "zeros", empty)
    yield binding, lib
    assert lib.calls == 1


def qmat(binding, rows, K=64):
    d = lambda w, t=torch.uint8: Device((rows, w), t)
    return binding.QMat(rows, K, 1, 0, 1, d(32, torch.int8), d(0), d(16), d(K // 32))


F32, F64, I32 = torch.float32, torch.float64, torch.int32


def cache(binding):
    c = [Device((2, 16, 2, w), torch.uint8) for w in (32, 2, 32, 2)]
    return binding.KV4Cache(*c)


CALLS = {
    "calibrate": lambda b: b.mxs_calibrate(Device((8, 64), F32)),
    "score": lambda b: b.mxs_score(Device((8, 64), F32), Device((64,), F64)),
    "mixed_gemm": lambda b: b.mxs_mixed_gemm(qmat(b, 4), qmat(b, 8)),
    "mixed_gemm_mx": lambda b: b.mxs_mixed_gemm_mx(qmat(b, 4), qmat(b, 8)),
    "mixed_gemm_prepared": lambda b: b.mxs_mixed_gemm_prepared(qmat(b, 4), qmat(b, 8), Device((9,), torch.uint8)),
    "mixed_gemm_fused": lambda b: b.mxs_mixed_gemm_fused(Device((4, 64), F32), None, qmat(b, 8)),
    "mixed_gemm_fused_prepared": lambda b: b.mxs_mixed_gemm_fused_prepared(Device((4, 64), F32), None, qmat(b, 8),
                                                                           Device((9,), torch.uint8)),
    "output_error": lambda b: b.mxs_output_error(Device((4, 64), F32), Device((8, 64), F32), Device((4, 8), F32)),
    "attend_kv4": lambda b: b.mxs_attend_kv4(Device((4, 64), F32), [Device((9, 2, w), torch.uint8) for w in (32, 2)],
                                             [Device((9, 2, w), torch.uint8) for w in (32, 2)], 0.125),
    "attend_kv4_tree": lambda b: b.mxs_attend_kv4_tree(Device((3, 4, 64), F32), cache(b), Device((1, 2), I32),
                                                       Device((1,), I32), Device((2,), I32), 0.125),
}


@pytest.mark.parametrize("name", CALLS)
def test_workspace_of_the_binding_outlives_the_call(stubbed, name):
    binding, _ = stubbed
    CALLS[name](binding)
