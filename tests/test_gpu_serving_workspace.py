"""A workspace is scratch: what it holds before a call does not reach the
result, whatever bytes they are, where a call has a list entry for every tile
and where it has one for every workgroup (more tiles than workgroups)."""
import numpy as np
import pytest
import torch

from test_gpu_serving import BF, DEV, F32, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import bit_gemm_hdiag_amd as mx
    return mx


# (sequences, cached tokens at most, query tokens at most, heads, KV heads, head dimension, bounds)
SHAPES = {
    "whole tiles, bounds of several": (67, 3, 1, 4, 2, 64, dict(max_q=70, max_len=70)),
    "whole tiles, decode": (300, 500, 1, 8, 8, 128, dict(max_q=1, max_len=4000)),
    "pieces, more tiles than workgroups": (70, 900, 9, 16, 4, 64, {}),
    "pieces, decode, few lines": (150, 2000, 1, 4, 4, 128, {}),
    "pieces, an entry a tile": (3, 3000, 4, 8, 2, 128, {}),
    "wide rows": (90, 300, 70, 4, 2, 64, {}),
    "empty sequences": (280, 40, 2, 2, 2, 32, dict(max_len=700)),
}


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_workspace_may_hold_anything(mx, dtype, shape):
    B, L, n, Hq, Hkv, D, bounds = SHAPES[shape]
    rng = np.random.default_rng(B)
    lens = rng.integers(0 if shape == "empty sequences" else 1, L + 1, B)
    lens[0] = L
    ns = np.minimum(rng.integers(0 if n > 1 else 1, n + 1, B), lens)
    ns[0] = n
    b = Batch(mx, lens.tolist(), ns.tolist(), Hq, Hkv, D, 16, dtype, "causal", B)
    args = b.args()
    args.update(bounds)
    wide = -(-args["max_len"] // 16) - b.table.shape[1]
    if wide > 0:
        args["table"] = b.dev(np.pad(b.table, ((0, 0), (0, wide)), constant_values=-1))
    need = mx.mxs_attend_kv4_tree_workspace(dtype, B, b.q.shape[0], args["max_q"], args["max_len"], Hq, Hkv, D)
    assert need > 0
    ws = torch.zeros(need + 64, dtype=torch.uint8, device=DEV)
    run = lambda: mx.mxs_attend_kv4_tree(b.q, b.cache, ws=ws[:need], **args)
    ref = run()
    b.check(ref)
    words = ws[:need // 4 * 4].view(torch.int32)
    g = torch.Generator(device=DEV).manual_seed(1)
    for fill in (0, -1, -2, -2 ** 31, 2 ** 31 - 1, 5, -1082130432, None):
        if fill is None:
            words.copy_(torch.randint(-2 ** 31, 2 ** 31, words.shape, generator=g, device=DEV, dtype=torch.int64))
        else:
            words.fill_(fill)
        ws[need:].fill_(0xA5)
        assert torch.equal(run(), ref), fill
        assert bool((ws[need:] == 0xA5).all())                   # nothing written past it
