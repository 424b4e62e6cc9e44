"""Measured cases of the serving calls around the attention of drafted tokens.

Three operators of a decode step of many requests:

* ``lora``    low-rank adapters of the requests beside a shared projection:
              Y[t] += scale[a] B[a] (A[a] X[t]), a = ids[t] (``mxs_lora_add``);
* ``verify``  drafted tokens, a chain or a tree a sequence, against the
              target's logits from given random numbers
              (``mxs_verify_tree``);
* ``pages``   pages of the 4-bit K/V cache: sequences forked, room made for
              drafted tokens (shared pages copied first), the accepted ones
              moved together, pages freed (``mxs_kv4_fork``,
              ``mxs_kv4_reserve``, ``mxs_kv4_compact``, ``mxs_kv4_release``),
              and ``copy``, tokens moved to another pool (``mxs_kv4_copy``).

``own`` selects the library's kernels; otherwise the operators run in their
plain form. ``exact`` evaluates the definition in 64 bits; of the three, only
the adapters give computed numbers (tokens, indexes and moved bytes are whole).
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ----------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step of eight requests on four adapters, 70B q_proj: latency
        dict(name="lora_decode8", op="lora", M=8, K=8192, N=8192, R=16, n=16, used=4, dtype="bf16", order="mixed"),
        # 64 decode tokens, 32 adapters of rank 64 on the 70B up projection: adapter bytes are what counts
        dict(name="lora_decode64", op="lora", M=64, K=8192, N=28672, R=64, n=48, used=32, dtype="bf16", order="mixed"),
        # fp32, odd rows and ranks below an odd stored rank, some tokens without an adapter
        dict(name="lora_odd_f32", op="lora", M=301, K=4096, N=1001, R=27, n=9, used=7, dtype="f32", order="mixed"),
        # prompts of eight requests, each a run of rows, 70B q_proj: X and Y are what counts
        dict(name="lora_prompt4096", op="lora", M=4096, K=8192, N=8192, R=16, n=16, used=8, dtype="bf16",
             order="runs"),
        # one user, four drafted tokens in a chain, a small vocabulary: latency
        dict(name="verify_chain5", op="verify", B=1, n=5, V=32000, dtype="f32", tree="chain", draft=True,
             greedy=False, masked=False),
        # 32 users, chains of seven drafted tokens with their distributions, a large vocabulary
        dict(name="verify_chain32", op="verify", B=32, n=8, V=128000, dtype="bf16", tree="chain", draft=True,
             greedy=False, masked=False),
        # odd vocabulary with masked tokens, trees whose siblings are drawn without replacement, greedy users among them
        dict(name="verify_tree_odd", op="verify", B=5, n=13, V=50021, dtype="f32", tree="tree", draft=True,
             greedy=True, masked=True),
        # sixteen users with trees of 64 tokens proposed without a distribution: logit bytes are what counts
        dict(name="verify_tree64", op="verify", B=16, n=64, V=128000, dtype="bf16", tree="tree", draft=False,
             greedy=True, masked=False),
        # one user forks once and both draft eight tokens: latency of the four calls
        dict(name="pages_fork1", op="pages", B=1, forks=1, n=8, L=500, H=8, D=128, page=64, pages=64),
        # 64 users, 32 of them forked, trees of 26 tokens over long contexts, a large pool
        dict(name="pages_step96", op="pages", B=64, forks=32, n=26, L=8192, H=8, D=128, page=64, pages=16384),
        # odd heads and dimension, pages of 17 tokens, moved to another pool
        dict(name="copy_odd", op="copy", T=1901, H=3, D=96, page=17),
        # the cache of a long prompt moved to another pool
        dict(name="copy_long131072", op="copy", T=131072, H=8, D=128, page=64),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["lora", "lora", "verify", "verify", "pages", "copy"])
    if op == "lora":
        order = rng.choice(["mixed", "mixed", "runs"])
        n = _log_int(rng, 1, 64)
        R = rng.choice([4, 8, 16, 16, 27, 32, 64, 128])
        M = _log_int(rng, 1, 256) if order == "mixed" else _log_int(rng, 64, 3000)
        return dict(op=op, M=M, K=32 * _log_int(rng, 16, 256), N=_log_int(rng, 500, 8192), R=R, n=n,
                    used=rng.randint(1, n), dtype=rng.choice(["bf16", "bf16", "f32"]), order=order)
    if op == "verify":
        tree = rng.choice(["chain", "tree"])
        B, n = _log_int(rng, 1, 24), _log_int(rng, 1, 32 if tree == "tree" else 9)
        return dict(op=op, B=B, n=n, V=_log_int(rng, 1000, 128000), dtype=rng.choice(["bf16", "f32"]), tree=tree,
                    draft=rng.random() < 0.5, greedy=rng.random() < 0.5, masked=rng.random() < 0.3)
    H, D, page = rng.choice([1, 3, 8, 8]), rng.choice([32, 64, 96, 128, 128, 256]), rng.choice([16, 17, 64, 256])
    if op == "copy":
        return dict(op=op, T=_log_int(rng, 1, 60000), H=H, D=D, page=page)
    B, L, n = _log_int(rng, 1, 48), _log_int(rng, 20, 4000), _log_int(rng, 1, 64)
    forks = rng.randint(0, B)
    return dict(op=op, B=B, forks=forks, n=n, L=L, H=H, D=D, page=page,
                pages=(B + forks + 1) * (-(-(L + n) // page) + 2) + rng.randint(0, 2000))


def _ragged(count, most, least=1):
    """`count` sizes between half of most and most, fixed by the case."""
    return [max(least, int(round(most * (1.0 - 0.5 * ((b * 0.6180339887498949) % 1.0))))) for b in range(count)]


# ---------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(shape, g):
    return torch.randn(shape, generator=g, device="cuda")


def _prepare_lora(case, g, cpu):
    M, K, N, R, n, used = (case[k] for k in ("M", "K", "N", "R", "n", "used"))
    dt = DTYPES[case["dtype"]]
    which = torch.randperm(n, generator=cpu)[:used]
    if case["order"] == "runs":                       # prompts: every request a run of rows
        pick = torch.arange(M) * used // M
    else:                                             # decode tokens in any order, popular adapters first
        pick = (torch.rand(M, generator=cpu).square() * used).long()
        pick[torch.randperm(M, generator=cpu)[:min(M, used)]] = torch.arange(min(M, used))
    ids = which[pick].to(torch.int32)
    if case["order"] == "mixed" and M > 100:
        ids[torch.rand(M, generator=cpu) < 0.05] = -1
    rank = torch.full((n,), R, dtype=torch.int32)
    if R % 8:
        rank = torch.randint(1, R + 1, (n,), generator=cpu, dtype=torch.int32)
    st = dict(ids=ids.cuda(), rank=rank.cuda(), x=_randn((M, K), g).to(dt), y=_randn((M, N), g),
              A=(_randn((n, R, K), g) / math.sqrt(K)).to(dt), B=(_randn((n, N, R), g) / math.sqrt(R)).to(dt),
              scale=torch.rand(n, generator=cpu).cuda() + 0.5)
    # the requests of each adapter, as the scheduler knows them
    st["host"] = [(int(a), int(rank[a]), (ids == a).nonzero().flatten().cuda()) for a in which.tolist()
                  if bool((ids == a).any())]
    if own:
        import bit_gemm_hdiag_amd as mx
        st["set"] = mx.LoraSet(st["A"], st["B"], st["scale"], st["rank"])
    return st


def _prepare_verify(case, g, cpu):
    B, n, V = case["B"], case["n"], case["V"]
    ns = _ragged(B, n)
    total, cu = sum(ns), torch.tensor([0] + ns).cumsum(0)
    # a peaked distribution over a long tail; the draft's is the target's with errors
    tail = _randn((total, V), g) * 2.0
    top = torch.randint(0, V, (total, 12), generator=g, device="cuda")
    logits = tail.scatter(1, top, 9.0 + 4.0 * torch.rand((total, 12), generator=g, device="cuda"))
    q = torch.softmax(logits + 0.7 * _randn((total, V), g), -1)
    if case["masked"]:                                # masked tokens: the lowest value and minus infinity
        hide = torch.rand((total, V), generator=g, device="cuda")
        logits = torch.where(hide < 0.3, torch.full_like(logits, torch.finfo(DTYPES[case["dtype"]]).min), logits)
        logits = torch.where(hide > 0.8, torch.full_like(logits, -math.inf), logits)
    parents, tokens = torch.full((total,), -1, dtype=torch.int32), torch.zeros(total, dtype=torch.int64)
    # up to 64 draws of every row, no token twice: the largest of q / Exp(1)
    w = q / torch.empty_like(q).exponential_(generator=g)
    drawn = w.topk(min(64, V), dim=-1).indices.cpu()
    for b in range(B):
        children = [0] * ns[b]
        for i in range(1, ns[b]):
            p = i - 1 if case["tree"] == "chain" else int(torch.randint(max(0, (i - 1) // 3), i, (1,), generator=cpu))
            r = int(cu[b]) + i
            parents[r] = p
            tokens[r] = drawn[int(cu[b]) + p, children[p] % drawn.shape[1]]
            children[p] += 1
    temperature = 0.6 + 0.6 * torch.rand(B, generator=cpu)
    if case["greedy"]:
        temperature[::2] = 0.0
    st = dict(logits=logits.to(DTYPES[case["dtype"]]), draft=q.contiguous() if case["draft"] else None,
              tokens=tokens.cuda(), parents=parents.cuda(), cu=cu.to(torch.int32).cuda(),
              temperature=temperature.cuda(),
              uniform=torch.rand(total, generator=cpu, dtype=torch.float64).cuda(), max_n=max(ns))
    if own:
        import bit_gemm_hdiag_amd as mx
        st["ws"] = torch.empty(max(1, mx.mxs_verify_tree_workspace(B, total, max(ns), V)), dtype=torch.uint8,
                               device="cuda")
        st["path"] = torch.empty(total, dtype=torch.int32, device="cuda")
        st["count"] = torch.empty(B, dtype=torch.int32, device="cuda")
        st["next"] = torch.empty(B, dtype=torch.int64, device="cuda")
    return st


def _planes(pages, page, H, D, g):
    """Any codes, and the scale bytes of ordinary keys and values."""
    kw = dict(generator=g, device="cuda", dtype=torch.uint8)
    return [torch.randint(lo, hi, (pages, page, H, D // w), **kw)
            for lo, hi, w in ((0, 256, 2), (115, 130, 32), (0, 256, 2), (115, 130, 32))]


def _prepare_pages(case, g, cpu):
    B, F, page, pages = case["B"], case["forks"], case["page"], case["pages"]
    rows = B + F
    lens = torch.tensor(_ragged(B, case["L"]) + [0] * F, dtype=torch.int32)
    ns = _ragged(rows, case["n"])
    width = -(-(case["L"] + case["n"]) // page)
    order, at = torch.randperm(pages, generator=cpu).to(torch.int32), 0
    table = torch.full((rows, width), -1, dtype=torch.int32)
    for b in range(B):
        k = -(-int(lens[b]) // page)
        table[b, :k] = order[at:at + k]
        at += k
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[order[:at].long()] = 1
    cu = torch.tensor([0] + ns).cumsum(0).to(torch.int32)
    path, count = torch.zeros(sum(ns), dtype=torch.int32), torch.zeros(rows, dtype=torch.int32)
    for b, n in enumerate(ns):                        # the root and a path below it
        kept = [0] + [i for i in range(1, n) if float(torch.rand(1, generator=cpu)) < 0.4]
        path[int(cu[b]):int(cu[b]) + len(kept)] = torch.tensor(kept, dtype=torch.int32)
        count[b] = len(kept)
    st = dict(planes=_planes(pages, page, case["H"], case["D"], g), table=table.cuda(), lens=lens.cuda(),
              refs=refs.cuda(), cu=cu.cuda(), path=path.cuda(), count=count.cuda(),
              src=torch.arange(F, dtype=torch.int32).cuda(), dst=torch.arange(B, rows, dtype=torch.int32).cuda(),
              keep=lens.cuda(), grown=torch.empty(rows, dtype=torch.int32, device="cuda"),
              kept=torch.empty(rows, dtype=torch.int32, device="cuda"),
              left=torch.empty(rows, dtype=torch.int32, device="cuda"),
              slots=torch.empty(sum(ns), dtype=torch.int64, device="cuda"))
    if own:
        import bit_gemm_hdiag_amd as mx
        st["cache"] = mx.KV4Cache(*st["planes"])
        st["ws"] = torch.empty(max(1, mx.mxs_kv4_reserve_workspace(pages, rows)), dtype=torch.uint8, device="cuda")
    return st


def _prepare_copy(case, g, cpu):
    T, page = case["T"], case["page"]
    need = -(-T // page)
    st = dict(planes=_planes(need + 2, page, case["H"], case["D"], g),
              other=_planes(need + 3, page, case["H"], case["D"], g))
    for name, pages in (("src", need + 2), ("dst", need + 3)):
        order, t = torch.randperm(pages, generator=cpu)[:need], torch.arange(T)
        st[name] = (order[t // page] * page + t % page).cuda()
    if own:
        import bit_gemm_hdiag_amd as mx
        st["from"], st["to"] = mx.KV4Cache(*st["planes"]), mx.KV4Cache(*st["other"])
    return st


def prepare(case, seed):
    g, cpu = _gen(seed), torch.Generator().manual_seed(int(seed) + 1)
    make = {"lora": _prepare_lora, "verify": _prepare_verify, "pages": _prepare_pages, "copy": _prepare_copy}
    return dict(make[case["op"]](case, g, cpu), case=case)


# ------------------------------------------------------------------ plain forms
def _plain_lora(st):
    y = st["y"]
    for a, r, rows in st["host"]:
        v = st["x"][rows].float() @ st["A"][a, :r].float().t()
        y[rows] += st["scale"][a] * (v @ st["B"][a, :, :r].float().t())
    return y


def _plain_verify(st):
    """All sequences at once, node by node; 64 bits, because a token is chosen by where sums cross a number."""
    cu = st["cu"].long()
    first, n = cu[:-1], cu[1:] - cu[:-1]
    B, V = n.numel(), st["logits"].shape[1]
    seq = torch.repeat_interleave(torch.arange(B, device=n.device), n)
    l = st["logits"].double()
    best = l.argmax(-1)
    m = l.gather(1, best[:, None])
    temp = st["temperature"].double()
    greedy = temp <= 0
    e = torch.exp((l - m) / torch.where(greedy, 1.0, temp)[seq][:, None])
    hot = torch.zeros_like(e).scatter_(1, best[:, None], 1.0)
    e = torch.where(greedy[seq][:, None], hot, e)
    draft, tokens, uniform = st["draft"], st["tokens"], st["uniform"]
    up = first[seq] + st["parents"].long()             # row of the parent
    cur, S, left = first.clone(), torch.zeros(B, 1, dtype=torch.float64, device=n.device), torch.ones_like(temp)
    R = e[cur].sum(-1)
    path, count = torch.full_like(st["parents"], -1), torch.ones_like(n)
    path[first] = 0
    for i in range(1, st["max_n"]):
        row = (first + i).clamp(max=tokens.numel() - 1)
        live = (i < n) & (up[row] == cur)
        x = tokens[row]
        q = draft[cur, x].double() if draft is not None else torch.ones_like(temp)
        w = (e[cur, x] - S[:, 0] * q).clamp(min=0) if draft is not None else e[cur, x]
        ok = live & torch.where(greedy, w > 0, uniform[row] * q * R < w * left)
        lost = live & ~ok & ~greedy
        path[(first + count).clamp(max=tokens.numel() - 1)[ok]] = i
        count += ok
        if draft is not None:
            S = torch.where(lost[:, None], S + (R / left)[:, None], S)
            left = torch.where(lost, left - q, left)
        else:
            e[cur, x] = torch.where(lost, 0.0, e[cur, x])
        cur = torch.where(ok, row, cur)
        S, left = torch.where(ok[:, None], 0.0, S), torch.where(ok, 1.0, left)
        rest = e[cur] if draft is None else (e[cur] - S * draft[cur].double()).clamp(min=0)
        R = torch.where(ok | lost, rest.sum(-1), R)
    rest = e[cur] if draft is None else torch.where(greedy[:, None], e[cur],
                                                    (e[cur] - S * draft[cur].double()).clamp(min=0))
    cum = rest.cumsum(-1)
    over = (cum > (uniform[first] * cum[:, -1])[:, None]) & (rest > 0)
    nxt = torch.where(over.any(-1), over.to(torch.uint8).argmax(-1), V - 1 - (rest > 0).flip(-1).to(torch.uint8).argmax(-1))
    return path, count.to(torch.int32), nxt


def _plain_pages(st):
    page, pages = st["case"]["page"], st["case"]["pages"]
    table, refs, lens, cu = st["table"], st["refs"], st["lens"], st["cu"].long()
    rows, width = table.shape
    j = torch.arange(width, device=table.device)
    # fork: the children hold the pages of their parents' tokens
    src, dst = st["src"].long(), st["dst"].long()
    shared = j[None] * page < lens[src][:, None]
    table[dst] = torch.where(shared, table[src], -1)
    refs.index_add_(0, table[src].clamp(min=0).flatten().long(), shared.flatten().to(torch.int32))
    lens[dst] = lens[src]
    # reserve: pages for the tokens behind lens, the lowest free ones, in order; shared pages are replaced
    n = cu[1:] - cu[:-1]
    old = table.clone()
    wanted = ((j[None] + 1) * page > lens[:, None]) & (j[None] * page < (lens + n)[:, None])
    held = old >= 0
    replaced = wanted & held & (refs[old.clamp(min=0).long()] > 1)
    takes = wanted & (~held | replaced)
    free = torch.argsort((refs != 0).to(torch.uint8), stable=True)
    rank = (takes.flatten().long().cumsum(0) - 1).view(rows, width)
    table.copy_(torch.where(takes, free[rank.clamp(min=0)].to(torch.int32), old))
    refs.index_add_(0, old.clamp(min=0).flatten().long(), -replaced.flatten().to(torch.int32))
    refs.index_add_(0, table.clamp(min=0).flatten().long(), takes.flatten().to(torch.int32))
    seq = torch.repeat_interleave(torch.arange(rows, device=n.device), n)
    t = lens[seq] + torch.arange(seq.numel(), device=n.device) - cu[seq]
    st["slots"].copy_(table[seq, t // page].long() * page + t % page)
    torch.add(lens, n.to(torch.int32), out=st["grown"])
    b = torch.arange(rows, device=n.device)
    k = torch.arange(page, device=n.device)
    last = (lens // page).clamp(max=width - 1).long()
    copied = (replaced[b, last] & (lens % page > 0))[:, None] & (k[None] < (lens % page)[:, None])
    where = copied.nonzero()
    a, z = (x[where[:, 0], last[where[:, 0]]].long() * page + where[:, 1] for x in (old, table))
    # compact: token path[i] of the last n becomes number i of them
    keep = torch.arange(seq.numel(), device=n.device) - cu[seq] < st["count"][seq]
    base, i = lens[seq][keep], (torch.arange(seq.numel(), device=n.device) - cu[seq])[keep]
    s, d = base + st["path"][keep], base + i
    s, d = (table[seq[keep], v // page].long() * page + v % page for v in (s, d))
    for x in st["planes"]:
        flat = x.flatten(0, 1)
        flat[z] = flat[a]
        flat[d] = flat[s]
    torch.add(lens, st["count"], out=st["kept"])
    # release: every page behind keep tokens
    drop = (j[None] * page >= st["keep"][:, None]) & (table >= 0)
    refs.index_add_(0, table.clamp(min=0).flatten().long(), -drop.flatten().to(torch.int32))
    table.masked_fill_(drop, -1)
    torch.minimum(st["kept"], st["keep"], out=st["left"])
    return [st["slots"], st["grown"], st["kept"], st["left"], refs, table, *st["planes"]]


def _plain_copy(st):
    for a, b in zip(st["planes"], st["other"]):
        b.flatten(0, 1)[st["dst"]] = a.flatten(0, 1)[st["src"]]
    return st["other"]


# ----------------------------------------------------------------------- one pass
def run(st):
    """Caches come back as the bytes that were moved: no call here reads them as numbers."""
    op = st["case"]["op"]
    if not own:
        return {"lora": _plain_lora, "verify": _plain_verify, "pages": _plain_pages, "copy": _plain_copy}[op](st)
    import bit_gemm_hdiag_amd as mx
    if op == "lora":
        return mx.mxs_lora_add(st["y"], st["x"], st["ids"], st["set"])
    if op == "verify":
        return mx.mxs_verify_tree(st["logits"], st["tokens"], st["cu"], st["uniform"], parents=st["parents"],
                                  draft=st["draft"], temperature=st["temperature"], max_n=st["max_n"],
                                  path=st["path"], count=st["count"], next_token=st["next"], ws=st["ws"])
    if op == "copy":
        mx.mxs_kv4_copy(st["to"], st["dst"], st["from"], st["src"])
        return st["other"]
    cache, refs, table = st["cache"], st["refs"], st["table"]
    if st["src"].numel():
        mx.mxs_kv4_fork(cache, refs, table, st["lens"], st["src"], st["dst"])
    mx.mxs_kv4_reserve(cache, refs, table, st["lens"], st["cu"], slots=st["slots"], lens_out=st["grown"], ws=st["ws"])
    mx.mxs_kv4_compact(cache, table, st["grown"], st["cu"], st["path"], st["count"], lens_out=st["kept"])
    mx.mxs_kv4_release(cache, refs, table, st["kept"], st["keep"], lens_out=st["left"])
    return [st["slots"], st["grown"], st["kept"], st["left"], refs, table, *st["planes"]]


def work(case):
    if case["op"] == "lora":
        es = 2 if case["dtype"] == "bf16" else 4
        M, K, N, R = case["M"], case["K"], case["N"], case["R"]
        active = min(M, case["used"])
        return {"bytes": M * K * es + 8 * M * N + active * R * (K + N) * es + 4 * M, "flops": 2 * M * R * (K + N)}
    if case["op"] == "verify":
        es = 2 if case["dtype"] == "bf16" else 4
        total, V = sum(_ragged(case["B"], case["n"])), case["V"]
        # the logits of every node; a draft's distribution for one node a sequence
        return {"bytes": total * (V * es + 28) + (4 * case["B"] * V if case["draft"] else 0), "flops": 4 * total * V}
    row = 2 * case["H"] * (case["D"] // 2 + case["D"] // 32)
    if case["op"] == "copy":
        return {"bytes": case["T"] * (2 * row + 16), "flops": 0}
    ns, lens = _ragged(case["B"] + case["forks"], case["n"]), _ragged(case["B"], case["L"])
    # two fifths of the drafted tokens move; the last page of a forked sequence is copied for both
    moved = 0.4 * sum(ns) + 2 * sum(L % case["page"] for L in lens[:case["forks"]])
    return {"bytes": 2 * row * moved + 4 * case["pages"] + 24 * sum(ns), "flops": 0}


# ------------------------------------------------------------- definitions, 64 bits
def exact(case, seed):
    if case["op"] != "lora":
        return None
    st = prepare(case, seed)
    y = st["y"].double()
    ids, rank = st["ids"].tolist(), st["rank"].tolist()
    for a in sorted(set(ids) - {-1}):
        rows = torch.tensor([t for t, i in enumerate(ids) if i == a], device="cuda")
        A, B = st["A"][a].double(), st["B"][a].double()
        A[rank[a]:], B[:, rank[a]:] = 0, 0
        both = st["scale"][a].double() * torch.linalg.multi_dot([st["x"][rows].double(), A.t(), B.t()])
        y.index_add_(0, rows, both)
    return y
