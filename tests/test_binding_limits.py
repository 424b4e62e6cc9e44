"""Sizes that the C interface takes as 32-bit numbers: the binding refuses
larger ones, which would arrive without their upper half (2^32 + 16 as 16).
No GPU: device tensors are stubs, and no library function is reached."""
import pytest
import torch

from test_binding_workspace import Device

BIG = 2 ** 32


def planes(pages, page, H, D):
    return [Device((pages, page, H, D // w), torch.uint8) for w in (2, 32, 2, 32)]


@pytest.mark.parametrize("shape", [(1, BIG + 16, 1, 32), (0, BIG + 16, 1, 32), (1, 2 ** 31, 1, 32), (1, 16, BIG + 2, 32),
                                   (1, 16, 2, BIG + 64)])
def test_cache_sizes_past_32_bits_are_refused(shape):
    import bit_gemm_hdiag_amd as mx
    with pytest.raises(ValueError):
        mx.KV4Cache(*planes(*shape))
    c = mx.KV4Cache(*planes(3, 16, 2, 64))
    assert (c._c.pages, c._c.page_size, c._c.H, c._c.D) == (3, 16, 2, 64)


def test_rotated_dims_past_32_bits_are_refused(monkeypatch):
    import bit_gemm_hdiag_amd as mx
    from bit_gemm_hdiag_amd import binding

    def reached(*args):
        raise AssertionError("reached the library")
    monkeypatch.setattr(binding, "_call", reached)
    x, pos = Device((1, 2, 128), torch.float32), Device((1,), torch.int64)
    freq = Device((BIG // 2 + 32,), torch.float64)                # 2^32 + 64 dims
    with pytest.raises(ValueError):
        mx.mxs_rope(x, pos, freq, out=x)
    c = mx.KV4Cache(*planes(3, 16, 2, 128))
    with pytest.raises(ValueError):
        mx.mxs_kv4_append(c, x, x, pos, pos, freq)
    with pytest.raises(ValueError):
        mx.mxs_rope_frequencies(BIG + 64, device="meta")
