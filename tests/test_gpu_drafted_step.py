"""The serving calls together, as a server uses them: quantised projections with
adapters beside them, rotary positions, pages reserved, keys and values appended,
attention of drafted trees, verification against the logits, the accepted tokens
moved together, unused pages given back, a sequence forked.

Greedy decoding gives the same tokens with drafts, right or wrong ones, as
without. The two runs differ by the rounding of fp32 sums alone (another kernel
for other row counts), so the test asks first that every choice of the run
without drafts is clear of the second best by far more than that."""
import numpy as np
import pytest
import torch

from bit_gemm_hdiag_amd import synth
from test_gpu_serving import pack_bits

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
E, HQ, H, D, V, PAGE = 256, 8, 2, 64, 1000, 16


@pytest.fixture(scope="module")
def mx():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import bit_gemm_hdiag_amd as mx
    return mx


def dev(x, t=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=t, device=DEV)


class Server:
    """One layer: logits = head (embedding + attention), all sequences in one batch."""

    def __init__(self, mx, prompts, adapters, forks, pages=60):
        g = torch.Generator(device=DEV).manual_seed(3)
        rnd = lambda *s: torch.randn(s, generator=g, device=DEV)
        self.mx, self.forks = mx, forks
        self.emb = rnd(V, E).to(torch.bfloat16)
        N = (HQ + 2 * H) * D
        self.W = mx.mxs_quantize(synth.weights(N, E, 5, dtype=torch.bfloat16, device=DEV),
                                 torch.arange(E, dtype=torch.int32, device=DEV), 1, 1, 6)
        self.lora = mx.LoraSet((rnd(3, 8, E) * 0.06).to(torch.bfloat16), (rnd(3, N, 8) * 0.3).to(torch.bfloat16),
                               dev([0.5, 1.0, 2.0], torch.float32), dev([8, 3, 5]))
        self.head, self.mix = rnd(E, V), rnd(HQ * D, E)
        self.freq = mx.mxs_rope_frequencies(D, 10000.0)
        B = len(prompts) + len(forks)
        self.cache = mx.kv4_cache_alloc(pages, PAGE, H, D)
        self.refs, self.table = dev([0] * pages), torch.full((B, 12), -1, dtype=torch.int32, device=DEV)
        self.lens = dev([0] * B)
        self.adapters = adapters
        self.tokens = [list(p) for p in prompts] + [[] for _ in forks]
        self.margin = np.inf
        # the prompts but for their last token, which roots the first tree
        self.forward([p[:-1] for p in prompts] + [[] for _ in forks], None)
        mx.mxs_kv4_fork(self.cache, self.refs, self.table, self.lens, dev(forks), dev(range(len(prompts), B)))
        for i, f in enumerate(forks):
            self.tokens[len(prompts) + i] = list(prompts[f])

    def forward(self, rows, parents):
        """Logits of the rows of every sequence, which are the last of its cached tokens afterwards."""
        mx = self.mx
        ns = [len(r) for r in rows]
        cu = dev(np.concatenate([[0], np.cumsum(ns)]))
        flat = [t for r in rows for t in r]
        x = self.emb[dev(flat, torch.int64)]
        y = mx.mxs_mixed_gemm_fused(x, None, self.W)
        ids = dev([a for a, n in zip(self.adapters, ns) for _ in range(n)])
        mx.mxs_lora_add(y, x, ids, self.lora)
        q, k, v = (t.view(len(flat), -1, D) for t in y.split([HQ * D, H * D, H * D], dim=1))
        before = self.lens.cpu().numpy()
        depth, total, n_max = [], len(flat), max(max(ns), 1)
        seen = np.zeros((total, n_max), dtype=bool)
        at = 0
        for b, n in enumerate(ns):
            for i in range(n):
                p = i - 1 if parents is None else parents[b][i]
                if i:
                    seen[at + i] = seen[at + p]
                seen[at + i, i] = True
                depth.append(int(seen[at + i].sum()) - 1 + int(before[b]))
            at += n
        pos = dev(depth, torch.int64)
        slots, self.lens = mx.mxs_kv4_reserve(self.cache, self.refs, self.table, self.lens, cu, total=total,
                                              lens_out=self.lens)
        assert int(slots.min()) >= 0
        mx.mxs_kv4_append(self.cache, k, v, slots, positions=pos, freq=self.freq)
        q = mx.mxs_rope(q, pos, self.freq)
        o = mx.mxs_attend_kv4_tree(q, self.cache, self.table, self.lens, cu, 0.125,
                                   mask=None if parents is None else pack_bits(seen), max_q=n_max)
        return (0.1 * x.float() + o.view(total, -1) @ self.mix) @ self.head, cu

    def step(self, drafts):
        """drafts: (tokens, parents) of every sequence, below its last token."""
        mx = self.mx
        rows = [[t[-1]] + d[0] for t, d in zip(self.tokens, drafts)]
        parents = [[-1] + d[1] for d in drafts]
        logits, cu = self.forward(rows, parents)
        total = logits.shape[0]
        top = logits.topk(2, dim=-1).values
        self.margin = min(self.margin, float((top[:, 0] - top[:, 1]).min()))
        path, count, nxt = mx.mxs_verify_tree(
            logits, dev([t for r in rows for t in r], torch.int64), cu, torch.zeros(total, dtype=torch.float64, device=DEV),
            parents=dev([p for r in parents for p in r]), temperature=torch.zeros(len(rows), device=DEV))
        mx.mxs_kv4_compact(self.cache, self.table, self.lens, cu, path, count, lens_out=self.lens)
        mx.mxs_kv4_release(self.cache, self.refs, self.table, self.lens, self.lens.clone(), lens_out=self.lens)
        path, count, nxt, at = path.tolist(), count.tolist(), nxt.tolist(), 0
        for b, r in enumerate(rows):
            self.tokens[b] += [r[i] for i in path[at + 1:at + count[b]]] + [nxt[b]]
            at += len(r)
        held = self.table[self.table >= 0]
        assert int(self.refs.sum()) == held.numel() and bool((self.refs >= 0).all())
        assert self.lens.tolist() == [len(t) - 1 for t in self.tokens]
        return count


def test_drafts_do_not_change_greedy_decoding(mx):
    g = np.random.default_rng(7)
    prompts = [g.integers(0, V, n).tolist() for n in (21, 5, 32, 1)]
    adapters, forks, new = [0, -1, 2, 1, 1, 0], [0, 2], 40
    plain = Server(mx, prompts, adapters, forks)
    none = [([], [])] * 6
    start = [len(t) for t in plain.tokens]
    for _ in range(new):
        assert plain.step(none) == [1] * 6
    assert plain.margin > 1e-2
    for a, b in ((0, 4), (2, 5)):                                # another adapter: another continuation
        assert plain.tokens[a] != plain.tokens[b]

    drafted = Server(mx, prompts, adapters, forks)
    steps, kept = 0, 0
    while min(len(t) - s for t, s in zip(drafted.tokens, start)) < new - 8:
        drafts = []
        for b, t in enumerate(drafted.tokens):
            truth = plain.tokens[b][len(t):]
            toks, pars, node = [], [], 0
            for x in truth[:int(g.integers(0, 5))]:              # right tokens, behind and before wrong siblings
                wrong = int(g.integers(V))
                for y in ([wrong, x] if g.random() < 0.5 else [x]) if g.random() < 0.9 else [wrong]:
                    toks.append(y)
                    pars.append(node)
                node = len(toks)
            drafts.append((toks, pars))
        count = drafted.step(drafts)
        steps, kept = steps + 1, kept + sum(c - 1 for c in count)
    assert kept > steps                                          # drafts were accepted
    for a, b in zip(plain.tokens, drafted.tokens):
        n = min(len(a), len(b))
        assert a[:n] == b[:n]
    # what both keep of a sequence is the same but for codes on a rounding border
    for b in range(6):
        n = min(len(plain.tokens[b]), len(drafted.tokens[b])) - 1
        kv = []
        for s in (plain, drafted):
            t = torch.arange(n, device=DEV)
            slots = s.table[b, t // PAGE].long() * PAGE + t % PAGE
            kv.append(torch.cat(mx.mxs_kv4_read(s.cache, slots, torch.float32)))
        assert float((kv[0] != kv[1]).float().mean()) < 1e-3
    drafted.mx.mxs_kv4_release(drafted.cache, drafted.refs, drafted.table, drafted.lens, dev([0] * 6))
    assert not drafted.refs.any() and bool((drafted.table == -1).all())
