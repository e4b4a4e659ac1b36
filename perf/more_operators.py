"""Drafted tokens over the paged cache, and the norms in front of attention,
as they are measured.

A model served with drafted tokens checks several of them in one step.  The
drafts of a row form a tree: its first token is the newest one that stands
already, every other token continues an earlier one (its parent).  Token j of
a row's tree lies in the cache behind the row's n cached tokens, at slot n + j,
though its position in the text is n + its depth.  Four operators:

  norm     scales every head of queries and keys to unit mean square, times a
           learned weight, and rotates it by the token's position; in training
           with its gradient
  tree     attention of the drafted tokens over the cached ones and those
           drafted tokens that lie on their own path; over all cached keys or
           over 16 blocks of 128 that each token chose
  verify   walks down the tree: keeps drafted tokens by given random numbers so
           that what is kept is distributed as the target's probabilities say,
           and draws the token behind them
  compact  moves the kept tokens' keys and values together, behind the prefix
"""
import math

import torch

own = False

BLOCK = 128
SLOTS = 16
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # Queries and keys of one row's nine drafted tokens, of a small model: latency.
        dict(name="norm_one", op="norm", train=0, tokens=9, docs=1, start_hi=5000, heads=24, kv=8,
             dim=64, rot=64, inter=1, dtype="fp16"),
        # A training step's packed row of documents: forward and gradient, queries and keys cut
        # from one projection.
        dict(name="norm_train", op="norm", train=1, tokens=16384, docs=9, start_hi=0, heads=64, kv=4,
             dim=128, rot=64, inter=0, dtype="bf16"),
        # One conversation with a chain of seven drafts: latency.
        dict(name="tree_one", op="tree", rows=1, tree_lo=8, tree_hi=8, len_lo=2900, len_hi=2900,
             pad=0, page=64, heads=64, kv=4, dim=128, sparse=0, chain=1, dtype="bf16"),
        # A batch's step with trees of 10 to 32 tokens, every key.
        dict(name="tree_step", op="tree", rows=32, tree_lo=10, tree_hi=32, len_lo=500, len_hi=12000,
             pad=5, page=64, heads=64, kv=4, dim=128, sparse=0, chain=0, dtype="bf16"),
        # Trees of 16 behind longer contexts, each token over the blocks that it chose.
        dict(name="tree_blocks", op="tree", rows=16, tree_lo=16, tree_hi=16, len_lo=2000,
             len_hi=50000, pad=0, page=128, heads=64, kv=4, dim=128, sparse=1, chain=0,
             dtype="bf16"),
        # Short drafts of a small model in small pages, some rows with the standing token alone.
        dict(name="tree_ragged", op="tree", rows=43, tree_lo=1, tree_hi=7, len_lo=1, len_hi=9000,
             pad=0, page=16, heads=24, kv=8, dim=64, sparse=0, chain=0, dtype="fp16"),
        # The largest trees, or 64 tokens behind a cached prefix at once: the most arithmetic.
        dict(name="tree_large", op="tree", rows=8, tree_lo=64, tree_hi=64, len_lo=12000,
             len_hi=16384, pad=0, page=32, heads=64, kv=4, dim=128, sparse=0, chain=0,
             dtype="bf16"),
        # One row's chain of five drafts, with the probabilities that they were drawn by.
        dict(name="verify_one", op="verify", rows=1, tree_lo=6, tree_hi=6, vocab=32000, chain=1,
             draft=1),
        # Trees of a batch whose drafts are a model's best guesses: no probabilities of theirs.
        dict(name="verify_trees", op="verify", rows=40, tree_lo=9, tree_hi=25, vocab=100003, chain=0,
             draft=0),
        # The widest batch: drawn drafts, a large vocabulary.
        dict(name="verify_many", op="verify", rows=128, tree_lo=4, tree_hi=8, vocab=151000, chain=0,
             draft=1),
        # One row keeps a few of its drafts.
        dict(name="compact_one", op="compact", rows=1, tree_lo=8, tree_hi=8, len_lo=2900, len_hi=2900,
             page=64, kv=4, dim=128, dtype="bf16"),
        # A batch's trees, kept to every degree.
        dict(name="compact_step", op="compact", rows=128, tree_lo=16, tree_hi=64, len_lo=100,
             len_hi=4000, page=16, kv=8, dim=128, dtype="fp16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["norm", "tree", "tree", "verify", "compact"])
    kv = rng.choice([1, 2, 4, 8])
    dim = rng.choice([64, 128])
    dtype = rng.choice(["bf16", "fp16"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op == "norm":
        train = rng.randint(0, 1)
        return dict(op=op, train=train, tokens=_spread(rng, 1, 16384), docs=rng.randint(1, 12),
                    start_hi=0 if train else rng.choice([0, 100000]), heads=kv * rng.choice([1, 3, 7, 8]),
                    kv=kv, dim=dim, rot=rng.choice([dim, dim // 2, 32]), inter=rng.randint(0, 1),
                    dtype=dtype)
    tree_hi = _spread(rng, 1, 64)
    tree_lo = rng.randint(1, tree_hi)
    if op == "verify":
        rows = _spread(rng, 1, 128)
        vocab = _spread(rng, 1000, min(151000, 110000000 // (rows * tree_hi)))
        return dict(op=op, rows=rows, tree_lo=tree_lo, tree_hi=tree_hi, vocab=vocab,
                    chain=rng.randint(0, 1), draft=rng.randint(0, 1))
    rows = _spread(rng, 1, 128)
    if op == "compact":
        len_hi = _spread(rng, 1, 4000)
        return dict(op=op, rows=rows, tree_lo=tree_lo, tree_hi=tree_hi, len_lo=rng.randint(1, len_hi),
                    len_hi=len_hi, page=page, kv=kv, dim=dim, dtype=dtype)
    sparse = rng.randint(0, 1)
    kv = rng.choice([1, 2, 4])
    # rows x tree x length no more than the largest listed case's
    longest = min(131072, 8 * 64 * 16384 // (rows * tree_hi), 400000 // rows)
    len_hi = _spread(rng, min(longest, 20 * BLOCK if sparse else 1), longest)
    return dict(op=op, rows=rows, tree_lo=tree_lo, tree_hi=tree_hi, len_lo=rng.randint(1, len_hi),
                len_hi=len_hi, pad=rng.choice([0, 0, 3]), page=page, heads=kv * rng.choice([1, 3, 7, 8, 16]),
                kv=kv, dim=dim, sparse=sparse, chain=rng.randint(0, 1), dtype=dtype)


# ------------------------------------------------------------------ a case's sizes
def _ladder(n, lo, hi):
    """n whole numbers of [lo, hi], hi first, spread evenly in no order."""
    return [hi - int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _trees(case):
    return _ladder(case["rows"], case["tree_lo"], case["tree_hi"])


def _lens(case):
    # another order than that of the trees
    return _ladder(case["rows"], case["len_lo"], case["len_hi"])[::-1]


def _kept(case):
    """Tokens that each row of a compact case keeps: some, all or one."""
    return [1 + (i * 5 + 3) % ((n + 1) // 2) if n > 1 else 1 for i, n in enumerate(_trees(case))]


def work(case):
    op = case["op"]
    if op == "norm":
        values = case["tokens"] * (case["heads"] + case["kv"]) * case["dim"]
        passes = 5 if case["train"] else 2      # forward 1 in, 1 out; gradient 2 in, 1 out
        return dict(bytes=values * 2 * passes + case["tokens"] * 4,
                    flops=values * (20 if case["train"] else 7))
    trees, rows = _trees(case), case["rows"]
    if op == "verify":
        # the last kept token's distribution of every row is read whole
        return dict(bytes=rows * case["vocab"] * 4 + sum(trees) * 16, flops=rows * case["vocab"])
    if op == "compact":
        moved = sum(k - 1 for k in _kept(case))
        return dict(bytes=moved * 2 * 2 * case["kv"] * case["dim"] * 2 + sum(_kept(case)) * 4 + rows * 12,
                    flops=0)
    keys = pairs = 0
    for n, m in zip(_lens(case), trees):
        seen = n
        if case["sparse"]:
            blocks = -(-n // BLOCK)
            seen = min(blocks, SLOTS) * BLOCK - (blocks * BLOCK - n)
        keys += seen + m            # read at least once
        pairs += m * seen + m       # a token sees itself at least
    q = sum(trees) * case["heads"] * case["dim"]
    return dict(bytes=keys * case["kv"] * case["dim"] * 4 + q * 4 + sum(trees) * case["heads"] * 4,
                flops=4 * pairs * case["heads"] * case["dim"])


# ------------------------------------------------------------------ inputs
def _pages(gen, lens, page):
    """A shuffled pool that holds every row's tokens, and the page table:
    unused entries are -1, and it is wider than any row needs."""
    need = [-(-n // page) for n in lens]
    pool = sum(need) + 5
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    col = torch.arange(max(need) + 2, device="cuda")
    first = torch.cumsum(n, 0) - n
    at = (first[:, None] + col[None, :]).clamp(max=pool - 1)
    table = torch.where(col[None, :] < n[:, None], order[at], order.new_full((), -1))
    return pool, table.contiguous()


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _offsets(trees):
    offs = [0]
    for n in trees:
        offs.append(offs[-1] + n)
    return offs


def _parents(seed, trees, chain):
    """Parents of all rows' tokens, numbered within the row, the first token's
    -1; trees lie level by level."""
    state = seed * 2654435761 % (1 << 32) + 1
    out = []
    for n in trees:
        at = [-1]
        for j in range(1, n):
            state = state * 1664525 + 1013904223 & 0xffffffff
            at.append(j - 1 if chain else max(at[-1], 0, (j - 1) // 3) + (state >> 16) % 3)
            at[-1] = min(at[-1], j - 1)
        out += at
    return out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"norm": _prepare_norm, "tree": _prepare_tree, "verify": _prepare_verify,
            "compact": _prepare_compact}[case["op"]](case, seed, gen)


def _prepare_norm(case, seed, gen):
    T, heads, kv, dim, rot = (case[x] for x in ("tokens", "heads", "kv", "dim", "rot"))
    dt = DTYPES[case["dtype"]]
    st = dict(case=case)
    # a projection's output: queries, keys and values of a token side by side
    x = _normal(gen, (T, heads + 2 * kv, dim), dt)
    st["q"], st["k"] = x[:, :heads], x[:, heads:heads + kv]
    st["wq"] = 1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")
    st["wk"] = 1 + 0.2 * torch.randn(dim, generator=gen, device="cuda")
    # documents one after the other, positions from a start of their own
    docs = min(case["docs"], T)
    each = -(-T // docs)
    t = torch.arange(T, device="cuda")
    start = torch.randint(0, case["start_hi"] + 1, (docs,), generator=gen, device="cuda")
    st["pos"] = (start[t // each] + t % each).to(torch.int32)
    st["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / rot)
                      ).float()
    if case["train"]:
        st["gq"] = _normal(gen, (T, heads, dim), dt)
        st["gk"] = _normal(gen, (T, kv, dim), dt)
        for name in ("q", "k", "wq", "wk"):
            st[name] = st[name].detach().requires_grad_()
    return st


def _prepare_tree(case, seed, gen):
    trees, lens = _trees(case), _lens(case)
    dt = DTYPES[case["dtype"]]
    kv, dim, page = case["kv"], case["dim"], case["page"]
    offs = _offsets(trees)
    st = dict(case=case, offs=_int32(offs), lens=_int32(lens), scale=1.0 / math.sqrt(dim))
    st["parents"] = _int32(_parents(seed, trees, case["chain"]) + [-1] * case["pad"])
    pool, st["table"] = _pages(gen, [n + m for n, m in zip(lens, trees)], page)
    st["q"] = _normal(gen, (offs[-1] + case["pad"], case["heads"], dim), dt)
    st["k_cache"] = _normal(gen, (pool, page, kv, dim), dt)
    st["v_cache"] = _normal(gen, (pool, page, kv, dim), dt)
    st["q2k"] = _choose(gen, st, kv) if case["sparse"] else None
    if own:
        from block_sparse_gqa_msa_gb300 import api
        st["cache"] = api.PagedCache(st["k_cache"], st["v_cache"])
        st["workspace"] = torch.empty(
            api.paged_tree_workspace_bytes(st["cache"], case["rows"], st["q"].shape[0], case["heads"]),
            dtype=torch.uint8, device="cuda")
    return st


def _choose(gen, st, kv):
    """q2k [kv, tokens, 16]: the newest cached block, block 0 and 14 others,
    ascending; a row's tokens agree on most of them."""
    T = st["q"].shape[0]
    row = torch.searchsorted(st["offs"].long()[1:], torch.arange(T, device="cuda"), right=True)
    row = row.clamp(max=st["lens"].numel() - 1)
    n = (st["lens"].long() + BLOCK - 1) // BLOCK
    most = max(int(n.max()), SLOTS)
    v = torch.arange(most, device="cuda")
    key = torch.rand(kv, st["lens"].numel(), most, generator=gen, device="cuda")[:, row]
    few = torch.rand(kv, T, most, generator=gen, device="cuda")
    # a token's own view of the scores: most of the row's best stay among the best
    key = key + 0.3 * few * (SLOTS / n[row].clamp(min=SLOTS))[None, :, None]
    key = torch.where(v == n[row][:, None] - 1, key.new_full((), 3.0), key)
    key[:, :, 0] = 2.5
    key = torch.where(v < n[row][:, None], key, key.new_full((), -1.0))
    top, at = key.topk(SLOTS, dim=2)
    at = torch.where(top >= 0, at, at.new_full((), most)).sort(dim=2).values
    return torch.where(at < most, at, at.new_full((), -1)).to(torch.int32).contiguous()


def _prepare_verify(case, seed, gen):
    trees, V = _trees(case), case["vocab"]
    offs = _offsets(trees)
    T = offs[-1]
    parents = _parents(seed, trees, case["chain"])
    st = dict(case=case, offs=_int32(offs), parents=_int32(parents))
    # a model's logits: a few likely tokens, a long tail; the drafting model is near it
    logit = torch.randn(T, V, generator=gen, device="cuda") * 2.0
    logit.scatter_(1, torch.randint(0, V, (T, 4), generator=gen, device="cuda"),
                   math.log(V) + 2 + 2 * torch.rand(T, 4, generator=gen, device="cuda"))
    near = logit + 0.7 * torch.randn(T, V, generator=gen, device="cuda")
    st["target"] = torch.softmax(logit, dim=1)
    draft = torch.softmax(near, dim=1)
    del logit, near
    # every token behind a first one is drawn by the drafting model after its parent, or the
    # parent's best guesses in turn
    rank, seen = [], {}
    base = [b for b, n in zip(offs, trees) for _ in range(n)]
    for j, (p, b) in enumerate(zip(parents, base)):
        rank.append(seen.get((b, p), 0))
        seen[b, p] = rank[-1] + 1
    at = torch.tensor([b + max(p, 0) for p, b in zip(parents, base)], device="cuda")
    if case["draft"]:
        st["draft"] = draft
        u = torch.rand(T, 1, generator=gen, device="cuda", dtype=torch.float64)
        step = 64  # rows at a time: sums of the probabilities in 64 bits
        tok = [torch.searchsorted(torch.cumsum(draft[at[i:i + step]].double(), 1),
                                  u[i:i + step])[:, 0] for i in range(0, T, step)]
        tokens = torch.cat(tok).clamp(max=V - 1)
    else:
        st["draft"] = None
        best = draft.topk(max(rank) + 1, dim=1).indices
        tokens = best[at, torch.tensor(rank, device="cuda")]
    st["tokens"] = tokens.to(torch.int32)
    st["u"] = torch.rand(T, generator=gen, device="cuda")
    st["u_last"] = torch.rand(case["rows"], generator=gen, device="cuda")
    return st


def _prepare_compact(case, seed, gen):
    trees, lens, kept = _trees(case), _lens(case), _kept(case)
    dt = DTYPES[case["dtype"]]
    st = dict(case=case, lens=_int32(lens), count=_int32(kept))
    pool, st["table"] = _pages(gen, [n + m for n, m in zip(lens, trees)], case["page"])
    shape = (pool, case["page"], case["kv"], case["dim"])
    st["k_cache"], st["v_cache"] = _normal(gen, shape, dt), _normal(gen, shape, dt)
    # a path down the tree: tokens that stay where they are, then ones from further behind
    path, state = [], seed + 7
    for n, c in zip(trees, kept):
        state = state * 1664525 + 1013904223 & 0xffffffff
        stay = 1 + (state >> 16) % c
        room, need = n - c, c - stay
        skip = (state >> 20) % (room - need + 1) if need else 0
        at = list(range(stay)) + [c + skip + i for i in range(need)]
        path.append(at + [-1] * (case["tree_hi"] - c))
    st["path"] = _int32(path)
    if own:
        from block_sparse_gqa_msa_gb300 import api
        st["cache"] = api.PagedCache(st["k_cache"], st["v_cache"])
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return {"norm": _norm, "tree": _tree, "verify": _verify, "compact": _compact}[
        state["case"]["op"]](state)


def _norm(st):
    case = st["case"]
    inter = bool(case["inter"])
    if own:
        from block_sparse_gqa_msa_gb300 import api, autograd
        if not case["train"]:
            q, k = api.msa_norm_rope(st["q"], st["k"], st["wq"], st["wk"], st["pos"], st["inv_freq"],
                                     eps=EPS, interleaved=inter)
            return dict(q=q, k=k)
        leaves = (st["q"], st["k"], st["wq"], st["wk"])
        q, k = autograd.msa_norm_rope(*leaves, st["pos"], st["inv_freq"], eps=EPS, interleaved=inter)
        dq, dk, dwq, dwk = torch.autograd.grad((q, k), leaves, (st["gq"], st["gk"]))
        return dict(q=q.detach(), k=k.detach(), dq=dq, dk=dk, dwq=dwq, dwk=dwk)
    with torch.no_grad():
        return _norm_plain(st, inter)


def _norm_plain(st, inter):
    rot = st["case"]["rot"]
    angle = st["pos"].double()[:, None] * st["inv_freq"].double()[None, :]
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]

    def turn(x, s):
        out = x.clone()
        if inter:
            a, b = x[..., 0:rot:2], x[..., 1:rot:2]
            out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * s, b * cos + a * s
        else:
            a, b = x[..., :rot // 2], x[..., rot // 2:rot]
            out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * s, b * cos + a * s
        return out

    def forward(x, w):
        x = x.float()
        n = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        return turn(x * n * w, sin), x * n, n

    out = {}
    for name in ("q", "k"):
        x, w = st[name], st["w" + name]
        y, unit, n = forward(x, w)
        out[name] = y.to(x.dtype)
        if st["case"]["train"]:
            g = turn(st["g" + name].float(), -sin)
            gw = g * w
            dx = n * (gw - unit * (gw * unit).mean(-1, keepdim=True))
            out["d" + name] = dx.to(x.dtype)
            out["dw" + name] = (g * unit).sum((0, 1))
    return out


def _rows_of(offs, T):
    """Tokens that rows own, their rows and their numbers in the row."""
    offs = offs.long()
    t = torch.arange(T, device="cuda")
    t = t[t < offs[-1]]
    row = torch.searchsorted(offs[1:], t, right=True)
    return t, row, t - offs[row]


def _ancestors(parents, row, j, rows, most):
    """[rows, most, most]: whether token j of a row has token i on its path,
    itself included."""
    step = torch.zeros(rows, most, most, device="cuda")
    up = parents >= 0
    step[row[up], j[up], parents[up]] = 1
    reach = torch.eye(most, device="cuda").expand(rows, -1, -1) + step
    for _ in range(max(1, (most - 1).bit_length())):  # paths of twice the length
        reach = (torch.matmul(reach, reach) > 0).float()
    return reach > 0


def _tree(st):
    case, q = st["case"], st["q"]
    if own:
        from block_sparse_gqa_msa_gb300 import api
        o, lse = api.msa_paged_tree(st["cache"], q, st["table"], st["offs"], st["lens"], st["scale"],
                                    parents=None if case["chain"] else st["parents"], q2k=st["q2k"],
                                    workspace=st["workspace"])
        T = T_real(case)
        return dict(o=o[:T], lse=lse[:T])
    page, lens, rows = case["page"], st["lens"].long(), case["rows"]
    kv, dim, heads = case["kv"], case["dim"], case["heads"]
    t, row, j = _rows_of(st["offs"], q.shape[0])
    most = case["tree_hi"]
    there = _ancestors(st["parents"].long()[t], row, j, rows, most)
    qs = torch.zeros(rows, most, heads, dim, device="cuda")
    qs[row, j] = q[t].float()
    qs = qs.view(rows, most, kv, -1, dim).permute(0, 2, 1, 3, 4)            # [rows, kv, most, n, dim]
    pages = st["table"].long().clamp(min=0)
    k = st["k_cache"][pages].float().view(rows, -1, kv, dim).transpose(1, 2)  # [rows, kv, keys, dim]
    v = st["v_cache"][pages].float().view(rows, -1, kv, dim).transpose(1, 2)
    key = torch.arange(k.shape[2], device="cuda")
    node = key[None, :] - lens[:, None]                                      # [rows, keys]
    drafted = (node >= 0) & (node < most)
    seen = there.gather(2, node.clamp(0, most - 1)[:, None, :].expand(-1, most, -1))
    seen = torch.where(drafted[:, None, :], seen, (node < 0)[:, None, :])[:, None]  # [rows, 1, most, keys]
    if st["q2k"] is not None:
        chosen = torch.zeros(rows, kv, most, key.numel() // BLOCK + 2, dtype=torch.bool, device="cuda")
        blocks = st["q2k"].long()[:, t]                                      # [kv, tokens, 16]
        blocks = torch.where(blocks >= 0, blocks, chosen.shape[3] - 1)
        chosen[row[None, :, None], torch.arange(kv, device="cuda")[:, None, None],
               j[None, :, None], blocks] = True
        seen = seen & (chosen[..., key // BLOCK] | (node >= 0)[:, None, None, :])
    s = torch.matmul(qs.reshape(rows, kv, -1, dim), k.transpose(2, 3)) * st["scale"]
    s = s.view(rows, kv, most, heads // kv, -1)
    s = torch.where(seen[:, :, :, None, :], s, s.new_full((), -math.inf))
    top = s.amax(dim=4, keepdim=True).clamp(min=-1e30)
    p = torch.exp(s - top)
    total = p.sum(dim=4, keepdim=True)
    o = torch.matmul((p / total).view(rows, kv, -1, key.numel()), v).view(rows, kv, most, -1, dim)
    lse = (top + torch.log(total))[..., 0]
    o = o.permute(0, 2, 1, 3, 4).reshape(rows, most, heads, dim)[row, j].to(q.dtype)
    return dict(o=o, lse=lse.permute(0, 2, 1, 3).reshape(rows, most, heads)[row, j])


def T_real(case):
    """Tokens of a tree case that rows own."""
    return sum(_trees(case))


def _verify(st):
    case = st["case"]
    if own:
        from block_sparse_gqa_msa_gb300 import api
        path, count, last = api.msa_tree_verify(
            st["target"], st["tokens"], st["offs"], st["u"], st["u_last"], draft=st["draft"],
            parents=None if case["chain"] else st["parents"], max_path=case["tree_hi"])
        return dict(path=path, count=count, last=last)
    rows, most = case["rows"], case["tree_hi"]
    first, end = st["offs"].long()[:-1], st["offs"].long()[1:]
    every = torch.arange(rows, device="cuda")
    cur = torch.zeros(rows, dtype=torch.long, device="cuda")     # the last kept token
    count = torch.ones_like(cur)
    path = torch.full((rows, most + 1), -1, dtype=torch.long, device="cuda")
    path[:, 0] = 0
    rest = st["target"][first]                                   # what is left of its distribution
    whole = torch.ones(rows, dtype=torch.float64, device="cuda")  # the sum of that
    for j in range(1, most):
        at = torch.minimum(first + j, end - 1)
        tried = (first + j < end) & (st["parents"].long()[at] == cur)
        x, u = st["tokens"].long()[at], st["u"][at].double()
        mine = rest.gather(1, x[:, None])[:, 0].double()
        if st["draft"] is None:
            kept = tried & (mine > 0) & (u * whole < mine)
            lost = tried & ~kept
            whole = torch.where(lost, whole - mine, whole)
            gone = torch.where(lost, x, 0)
            rest[every, gone] = torch.where(lost, 0.0, rest[every, gone])
        else:
            q = st["draft"][first + cur]
            part = torch.where(whole > 0, 1 / whole, 0.0).float()
            kept = tried & (u * q.gather(1, x[:, None])[:, 0].double() < mine * part.double())
            lost = tried & ~kept
            left = (rest * part[:, None] - q).clamp(min=0)
            rest = torch.where(lost[:, None], left, rest)
            whole = torch.where(lost, rest.sum(1, dtype=torch.float64), whole)
        cur = torch.where(kept, j, cur)
        path[every, torch.where(kept, count, most)] = j
        count = count + kept
        rest = torch.where(kept[:, None], st["target"][first + cur], rest)
        whole = torch.where(kept, 1.0, whole)
    # nothing left: the distribution itself
    none = rest.amax(1, keepdim=True) <= 0
    rest = torch.where(none, st["target"][first + cur], rest)
    run_up = torch.cumsum(rest.double(), 1)
    goal = st["u_last"].double() * run_up[:, -1]
    last = torch.searchsorted(run_up, goal[:, None], right=True)[:, 0]
    path = path[:, :most]
    path = torch.where(torch.arange(most, device="cuda") < count[:, None], path, -1)
    return dict(path=path.to(torch.int32), count=count.to(torch.int32), last=last.to(torch.int32))


def _compact(st):
    case = st["case"]
    if own:
        from block_sparse_gqa_msa_gb300 import api
        length = api.msa_paged_compact(st["cache"], st["table"], st["lens"], st["path"], st["count"])
    else:
        i = torch.arange(st["path"].shape[1], device="cuda")
        row, i = torch.nonzero(i[None, :] < st["count"][:, None], as_tuple=True)
        lens, page = st["lens"].long(), case["page"]

        def place(pos):
            return st["table"].long()[row, pos // page], pos % page

        source = place(lens[row] + st["path"].long()[row, i])
        target = place(lens[row] + i)
        st["k_cache"][target] = st["k_cache"][source]
        st["v_cache"][target] = st["v_cache"][source]
        length = st["lens"] + st["count"]
    return dict(k_cache=st["k_cache"], v_cache=st["v_cache"], length=length)


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers alone
    st = prepare(case, seed)
    with torch.no_grad():
        return {"norm": _exact_norm, "tree": _exact_tree, "compact": _exact_compact}[case["op"]](st)


def _exact_norm(st):
    case = st["case"]
    rot = case["rot"]
    pair = torch.arange(rot // 2, device="cuda")
    lo, hi = (2 * pair, 2 * pair + 1) if case["inter"] else (pair, pair + rot // 2)
    turn = torch.polar(torch.ones(case["tokens"], rot // 2, dtype=torch.float64, device="cuda"),
                       st["pos"].double()[:, None] * st["inv_freq"].double())[:, None, :]

    def rotate(x, by):
        z = torch.complex(x[..., lo], x[..., hi]) * by
        x = x.clone()
        x[..., lo], x[..., hi] = z.real, z.imag
        return x

    outs = {}
    for name in ("q", "k"):
        w = st["w" + name].double()
        x = st[name].double()
        size = (x.pow(2).sum(-1, keepdim=True) / case["dim"] + EPS).sqrt()
        outs[name] = rotate(x / size * w, turn)
        if case["train"]:
            g = rotate(st["g" + name].double(), turn.conj())
            # of y = w x / size: dx = (w g) / size - x <w g, x> / (dim size^3)
            inner = (w * g * x).sum(-1, keepdim=True)
            outs["d" + name] = w * g / size - x * inner / (case["dim"] * size ** 3)
            outs["dw" + name] = torch.einsum("thd,thd->d", g, x / size)
    return outs


def _exact_tree(st):
    case = st["case"]
    page, kv, heads = case["page"], case["kv"], case["heads"]
    share = heads // kv
    offs, parents = st["offs"].tolist(), st["parents"].tolist()
    outs, logs = [], []
    for r, n in enumerate(st["lens"].tolist()):
        t0, m = offs[r], offs[r + 1] - offs[r]
        pages = st["table"][r, :-(-(n + m) // page)].long()
        k = st["k_cache"][pages].flatten(0, 1)[:n + m].double()
        v = st["v_cache"][pages].flatten(0, 1)[:n + m].double()
        line = [[False] * m for _ in range(m)]
        for j in range(m):
            up = parents[t0 + j]
            if up >= 0:
                line[j] = list(line[up])
            line[j][j] = True
        line = torch.tensor(line, device="cuda")
        o = torch.empty(m, heads, case["dim"], dtype=torch.float64, device="cuda")
        lse = torch.empty(m, heads, dtype=torch.float64, device="cuda")
        block = torch.arange(n, device="cuda") // BLOCK
        for g in range(kv):
            mine = slice(g * share, (g + 1) * share)
            s = torch.einsum("mhd,kd->mhk", st["q"][t0:t0 + m, mine].double(), k[:, g]) * st["scale"]
            hide = torch.zeros(m, n + m, dtype=torch.bool, device="cuda")
            hide[:, n:] = ~line
            if st["q2k"] is not None:
                chosen = st["q2k"][g, t0:t0 + m].long()
                hide[:, :n] = ~(block[None, :, None] == chosen[:, None, :]).any(2)
            s = s.masked_fill(hide[:, None, :], -math.inf)
            lse[:, mine] = torch.logsumexp(s, dim=2)
            o[:, mine] = torch.softmax(s, dim=2) @ v[:, g]
        outs.append(o)
        logs.append(lse)
    return dict(o=torch.cat(outs), lse=torch.cat(logs))


def _exact_compact(st):
    page = st["case"]["page"]
    before = dict(k_cache=st["k_cache"].clone(), v_cache=st["v_cache"].clone())
    after = {name: x.double() for name, x in before.items()}
    for r, (n, c) in enumerate(zip(st["lens"].tolist(), st["count"].tolist())):
        table = st["table"][r].tolist()
        for i, j in enumerate(st["path"][r, :c].tolist()):
            for name, x in after.items():
                x[table[(n + i) // page], (n + i) % page] = (
                    before[name][table[(n + j) // page], (n + j) % page].double())
    return dict(after, length=None)
