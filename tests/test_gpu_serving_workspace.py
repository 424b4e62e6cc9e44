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


def test_two_threads_on_one_stream(mx):
    """Calls without a workspace of their own, whose two launches interleave with the other thread's."""
    import threading
    bs = [Batch(mx, [3000], [4], 8, 2, 128, 64, BF, "tree", 80 + i) for i in range(2)]
    args = [b.args() for b in bs]
    refs = [mx.mxs_attend_kv4_tree(b.q, b.cache, **a) for b, a in zip(bs, args)]
    outs = [[torch.empty_like(b.q) for _ in range(50)] for b in bs]
    torch.cuda.synchronize()
    failed = []

    def work(i):
        try:
            for o in outs[i]:
                mx.mxs_attend_kv4_tree(bs[i].q, bs[i].cache, out=o, **args[i])
        except Exception as e:                                   # shown by the main thread
            failed.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    for got, ref in zip(outs, refs):
        assert all(torch.equal(o, ref) for o in got)


@pytest.mark.parametrize("B,n,Hq,Hkv,D", [(70, 9, 16, 4, 64), (150, 1, 4, 4, 128), (5, 40, 8, 2, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_graph_replays_of_ragged_batches(mx, dtype, B, n, Hq, Hkv, D):
    """Captured once; lengths, query counts and the workspace's bytes change between replays."""
    L = 900
    b = Batch(mx, [L] * B, [n] * B, Hq, Hkv, D, 16, dtype, "causal", B + D)
    args = b.args()
    need = mx.mxs_attend_kv4_tree_workspace(dtype, B, B * n, n, L, Hq, Hkv, D)
    ws, ews = (torch.zeros(need, dtype=torch.uint8, device=DEV) for _ in range(2))
    out, eager = torch.empty_like(b.q), torch.empty_like(b.q)
    run = lambda o, w: mx.mxs_attend_kv4_tree(b.q, b.cache, out=o, ws=w, **args)
    run(out, ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(out, ws)
    rng = np.random.default_rng(B)
    for rep, (lo, hi) in enumerate(((L, L), (0, 0), (0, L), (0, 70), (L - 3, L), (1, 2))):
        lens = rng.integers(lo, hi + 1, B)
        ns = np.minimum(rng.integers(0, n + 1, B), lens)
        args["lens"].copy_(b.dev(lens))
        args["cu"].copy_(b.dev(np.concatenate([[0], np.cumsum(ns)])))
        for w, byte in ((ws, 0x80 + rep), (ews, 0)):
            w.fill_(byte)
        for o in (out, eager):
            o.fill_(7.0)
        graph.replay()
        run(eager, ews)
        torch.cuda.synchronize()
        assert torch.equal(out, eager), rep
        assert bool((out[int(ns.sum()):] == 7.0).all())          # rows of no sequence
