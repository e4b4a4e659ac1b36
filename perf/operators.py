"""The serving operators of the paged cache, as they are measured.

A model trained with block-sparse attention is served token by token from a
paged cache.  Four operators make one step of that:

  append   rotates the keys (and the queries) of new tokens by their positions
           and writes keys and values into the cache's pages
  index    writes the index keys of new tokens into their pages and renews
           the means of the 128-key blocks that they touch
  select   scores the cached blocks for one new token of each row and picks 16
  decode   attention of one new token of each row over the cache: over all of
           its keys, or over the selected blocks only

Rows are sequences.  Token j of row r lives in page page_table[r][j // S] at
slot j % S (S: the page size).
"""
import math

import torch

own = False

BLOCK = 128
SLOTS = 16
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # One sequence behind a long conversation gets its next token: latency.
        dict(name="append_one", op="append", rows=1, fresh_lo=1, fresh_hi=1, start_lo=90000,
             start_hi=90000, pad=0, page=64, heads=64, kv=4, dim=128, rot=64, inter=0, dtype="bf16",
             keep_k=0),
        # A decode step of a batch captured for 160 rows with 150 in use; every channel rotated
        # in neighbouring pairs.
        dict(name="append_step", op="append", rows=150, fresh_lo=1, fresh_hi=1, start_lo=100,
             start_hi=8192, pad=10, page=16, heads=64, kv=8, dim=128, rot=128, inter=1, dtype="fp16",
             keep_k=0),
        # Nine ragged prompts, about 17000 tokens together; the rotated keys are handed back for the
        # attention over the prompts themselves.
        dict(name="append_prompts", op="append", rows=9, fresh_lo=317, fresh_hi=3300, start_lo=0,
             start_hi=0, pad=0, page=128, heads=64, kv=4, dim=128, rot=64, inter=0, dtype="bf16",
             keep_k=1),
        # Index keys of one decode step of 96 rows, blocks filled to every degree.
        dict(name="index_step", op="index", rows=96, fresh_lo=1, fresh_hi=1, start_lo=1,
             start_hi=16383, pad=0, page=128, heads=4, dim=64),
        # Index keys of ragged prompts that continue cached prefixes.
        dict(name="index_prompts", op="index", rows=7, fresh_lo=129, fresh_hi=5000, start_lo=0,
             start_hi=1000, pad=0, page=32, heads=4, dim=128),
        # Selection for one long document's next token.
        dict(name="select_one", op="select", rows=1, len_lo=131072, len_hi=131072, page=128,
             heads=4, dim=64, force=1),
        # Selection for a batch from short to long contexts, no block kept by force.
        dict(name="select_step", op="select", rows=64, len_lo=900, len_hi=131072, page=64,
             heads=4, dim=128, force=0),
        # The smallest attention call: one row, a short context, every key.
        dict(name="decode_one_short", op="decode", rows=1, len_lo=1000, len_hi=1000, page=16,
             heads=64, kv=4, dim=128, sparse=0, dtype="bf16"),
        # The next token of one long document over its 16 selected blocks.
        dict(name="decode_one_blocks", op="decode", rows=1, len_lo=131001, len_hi=131001, page=128,
             heads=64, kv=4, dim=128, sparse=1, dtype="bf16"),
        # A decode step of 128 rows over their selected blocks.
        dict(name="decode_step_blocks", op="decode", rows=128, len_lo=500, len_hi=16384, page=64,
             heads=64, kv=4, dim=128, sparse=1, dtype="bf16"),
        # A dense layer's decode step: ragged contexts, a small head, odd sharing.
        dict(name="decode_step_ragged", op="decode", rows=77, len_lo=1, len_hi=12000, page=32,
             heads=24, kv=8, dim=64, sparse=0, dtype="fp16"),
        # Long contexts, every key: the largest read.
        dict(name="decode_long", op="decode", rows=9, len_lo=65536, len_hi=131072, page=128,
             heads=64, kv=4, dim=128, sparse=0, dtype="bf16"),
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "index", "select", "decode", "decode"])
    page = rng.choice([16, 32, 64, 128, 256])
    if op in ("append", "index"):
        if rng.random() < 0.5:  # a decode step
            rows, fresh_lo, fresh_hi = _spread(rng, 1, 512), 1, 1
        else:                   # prompts
            rows = _spread(rng, 1, 16)
            fresh_hi = _spread(rng, 2, 16384 // rows)
            fresh_lo = rng.randint(1, fresh_hi)
        start_hi = rng.choice([0, _spread(rng, 1, 30000 // rows + 100)])
        case = dict(op=op, rows=rows, fresh_lo=fresh_lo, fresh_hi=fresh_hi,
                    start_lo=rng.randint(0, start_hi), start_hi=start_hi,
                    pad=rng.choice([0, 0, 3]), page=page)
        if op == "index":
            return dict(case, heads=4, dim=rng.choice([8, 32, 64, 128]))
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 128])
        return dict(case, kv=kv, heads=kv * rng.choice([1, 3, 7, 8]), dim=dim,
                    rot=rng.choice([dim, dim // 2, 32]), inter=rng.randint(0, 1),
                    dtype=rng.choice(["bf16", "fp16"]), keep_k=rng.randint(0, 1))
    rows = _spread(rng, 1, 256)
    # at least one row of a selection has blocks to choose from (more than 16)
    shortest = 20 * BLOCK if op == "select" else 1
    len_hi = _spread(rng, shortest, min(131072, 1000000 // rows))
    case = dict(op=op, rows=rows, len_lo=rng.randint(1, len_hi), len_hi=len_hi, page=page)
    if op == "select":
        return dict(case, heads=4, dim=rng.choice([32, 64, 128]), force=rng.randint(0, 1))
    kv = rng.choice([1, 2, 4])
    return dict(case, kv=kv, heads=kv * rng.choice([1, 3, 7, 8, 16]), dim=rng.choice([64, 128]),
                sparse=rng.randint(0, 1), dtype=rng.choice(["bf16", "fp16"]))


# ------------------------------------------------------------------ a case's sizes
def _ladder(n, lo, hi):
    """n whole numbers of [lo, hi], hi first, spread evenly in no order."""
    return [hi - int((hi - lo) * ((i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _fresh(case):
    """New tokens and first position of each row."""
    return (_ladder(case["rows"], case["fresh_lo"], case["fresh_hi"]),
            _ladder(case["rows"], case["start_lo"], case["start_hi"]))


def _lens(case):
    return _ladder(case["rows"], case["len_lo"], case["len_hi"])


def _seen(case):
    """Keys that each row of a decode case attends, per key head."""
    if not case["sparse"]:
        return _lens(case)
    out = []
    for n in _lens(case):
        blocks = -(-n // BLOCK)
        out.append(min(blocks, SLOTS) * BLOCK - (blocks * BLOCK - n))  # the last block is one of them
    return out


def work(case):
    op, rows = case["op"], case["rows"]
    if op in ("append", "index"):
        fresh, start = _fresh(case)
        tokens = sum(fresh)
        if op == "append":
            per = case["dim"] * 2
            n = 2 * case["heads"] + 4 * case["kv"] + (case["kv"] if case["keep_k"] else 0)
            turned = case["heads"] + case["kv"]
            return dict(bytes=tokens * n * per + 12 * rows, flops=tokens * turned * case["rot"] * 3)
        width = case["heads"] * case["dim"]
        blocks = sum(-(-(s + f) // BLOCK) - s // BLOCK for f, s in zip(fresh, start))
        before = sum(s % BLOCK for s in start)
        return dict(bytes=tokens * width * 4 + before * width * 2 + blocks * width * 4 + 12 * rows,
                    flops=(tokens + before) * width)
    if op == "select":
        width = case["heads"] * case["dim"]
        scored = 0
        for n in _lens(case):
            blocks = -(-n // BLOCK)
            scored += 0 if blocks <= SLOTS else blocks - (2 if case["force"] else 0)
        return dict(bytes=scored * width * 4 + rows * (width * 2 + case["heads"] * SLOTS * 4 + 8),
                    flops=2 * scored * width)
    keys = sum(_seen(case))
    q = rows * case["heads"] * case["dim"]
    return dict(bytes=keys * case["kv"] * case["dim"] * 4 + q * 4 + rows * case["heads"] * 4 + 8 * rows
                + (rows * case["kv"] * SLOTS * 4 if case["sparse"] else 0),
                flops=4 * keys * case["heads"] * case["dim"])


# ------------------------------------------------------------------ inputs
def _pages(gen, lens, page):
    """A shuffled pool that holds every row's tokens, and the page table:
    unused entries are -1, and it is wider than any row needs."""
    need = [-(-n // page) for n in lens]
    pool = sum(need) + 5
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    width = max(need) + 2
    col = torch.arange(width, device="cuda")
    first = torch.cumsum(n, 0) - n
    at = (first[:, None] + col[None, :]).clamp(max=pool - 1)
    table = torch.where(col[None, :] < n[:, None], order[at], order.new_full((), -1))
    return pool, table.contiguous()


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _grid(gen, shape, unit):
    """Normal values on a grid of `unit`, four standard deviations at most:
    block means and scores on it are exact in 32 bits, so that which blocks
    are best does not depend on the order of a sum."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x.clamp(-4, 4) / unit).round() * unit


def _int32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, page = case["op"], case["page"]
    st = dict(case=case)
    if op in ("append", "index"):
        fresh, start = _fresh(case)
        pool, st["table"] = _pages(gen, [f + s for f, s in zip(fresh, start)], page)
        offs = [0]
        for f in fresh:
            offs.append(offs[-1] + f)
        T = offs[-1] + case["pad"]
        st["offs"], st["start"] = _int32(offs), _int32(start)
        if op == "append":
            dt = DTYPES[case["dtype"]]
            kv, dim, rot = case["kv"], case["dim"], case["rot"]
            st["q"] = _normal(gen, (T, case["heads"], dim), dt)
            st["k"] = _normal(gen, (T, kv, dim), dt)
            st["v"] = _normal(gen, (T, kv, dim), dt)
            st["k_cache"] = _normal(gen, (pool, page, kv, dim), dt)
            st["v_cache"] = _normal(gen, (pool, page, kv, dim), dt)
            st["q_out"] = torch.zeros_like(st["q"])
            st["k_out"] = torch.zeros_like(st["k"]) if case["keep_k"] else None
            st["inv_freq"] = (10000.0 ** (-torch.arange(0, rot, 2, device="cuda",
                                                        dtype=torch.float64) / rot)).float()
        else:
            heads, dim = case["heads"], case["dim"]
            st["ik"] = _grid(gen, (T, heads, dim), 0.25).bfloat16()
            st["keys"] = _grid(gen, (pool, page, heads, dim), 0.25).bfloat16()
            st["means"] = torch.zeros(pool * max(1, page // BLOCK), heads, dim, device="cuda")
    else:
        lens = _lens(case)
        pool, st["table"] = _pages(gen, lens, page)
        st["lens"] = _int32(lens)
        if op == "select":
            heads, dim = case["heads"], case["dim"]
            st["iq"] = _grid(gen, (case["rows"], heads, dim), 0.25).bfloat16()
            slots = pool * max(1, page // BLOCK)
            st["means"] = _grid(gen, (slots, heads, dim), 1.0 / 64) / 8  # of 128 keys: a grid of 1/512
            if own:  # the handle wants the keys' pages too; selection does not read them
                st["keys"] = torch.zeros(pool, page, heads, dim, dtype=torch.bfloat16, device="cuda")
        else:
            dt = DTYPES[case["dtype"]]
            kv, dim, rows = case["kv"], case["dim"], case["rows"]
            st["q"] = _normal(gen, (rows, case["heads"], dim), dt)
            st["k_cache"] = _normal(gen, (pool, page, kv, dim), dt)
            st["v_cache"] = _normal(gen, (pool, page, kv, dim), dt)
            st["scale"] = 1.0 / math.sqrt(dim)
            st["q2k"] = _choose(gen, lens, kv) if case["sparse"] else None
    if own:
        from block_sparse_gqa_msa_gb300 import api
        if op in ("append", "decode"):
            st["cache"] = api.PagedCache(st["k_cache"], st["v_cache"])
        else:
            st["index"] = api.PagedIndex(st["keys"], st["means"])
        if op == "decode":
            st["workspace"] = torch.empty(
                api.paged_decode_workspace_bytes(st["cache"], case["rows"], case["heads"]),
                dtype=torch.uint8, device="cuda")
    return st


def _choose(gen, lens, kv):
    """q2k [kv, rows, 16]: the newest block, block 0 and 14 others, ascending."""
    n = torch.tensor([-(-x // BLOCK) for x in lens], device="cuda")
    most = max(int(n.max()), SLOTS)
    v = torch.arange(most, device="cuda")
    key = torch.rand(kv, len(lens), most, generator=gen, device="cuda")
    key = torch.where(v[None, :] == n[:, None] - 1, key.new_full((), 3.0), key)
    key[:, :, 0] = 2.0
    key = torch.where(v[None, :] < n[:, None], key, key.new_full((), -1.0))
    top, at = key.topk(SLOTS, dim=2)
    at = torch.where(top >= 0, at, at.new_full((), most)).sort(dim=2).values
    return torch.where(at < most, at, at.new_full((), -1)).to(torch.int32).contiguous()


# ------------------------------------------------------------------ one pass
def run(state):
    return {"append": _append, "index": _index, "select": _select, "decode": _decode}[
        state["case"]["op"]](state)


def _places(st, T):
    """Real tokens of a call, their positions, pages and slots."""
    offs = st["offs"].long()
    t = torch.arange(T, device="cuda")
    t = t[t < offs[-1]]
    row = torch.searchsorted(offs[1:], t, right=True)
    pos = st["start"].long()[row] + t - offs[row]
    page = st["case"]["page"]
    return t, row, pos, st["table"].long()[row, pos // page], pos % page


def _append(st):
    if own:
        from block_sparse_gqa_msa_gb300 import api
        api.msa_paged_append(st["cache"], st["k"], st["v"], st["table"], st["offs"], st["start"],
                             inv_freq=st["inv_freq"], interleaved=bool(st["case"]["inter"]),
                             q=st["q"], q_out=st["q_out"], k_out=st["k_out"])
    else:
        t, _, pos, pg, slot = _places(st, st["k"].shape[0])
        angle = pos.double()[:, None] * st["inv_freq"].double()[None, :]
        cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
        rot, inter = st["case"]["rot"], st["case"]["inter"]

        def turn(x):
            x = x[t].float()
            out = x.clone()
            if inter:
                a, b = x[..., 0:rot:2], x[..., 1:rot:2]
                out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
            else:
                a, b = x[..., :rot // 2], x[..., rot // 2:rot]
                out[..., :rot // 2], out[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
            return out.to(st["k"].dtype)

        k = turn(st["k"])
        st["k_cache"][pg, slot] = k
        st["v_cache"][pg, slot] = st["v"][t]
        st["q_out"][t] = turn(st["q"])
        if st["k_out"] is not None:
            st["k_out"][t] = k
    out = dict(q=st["q_out"], k_cache=st["k_cache"], v_cache=st["v_cache"])
    if st["k_out"] is not None:
        out["k"] = st["k_out"]
    return out


def _index(st):
    if own:
        from block_sparse_gqa_msa_gb300 import api
        api.msa_paged_index(st["index"], st["ik"], st["table"], st["offs"], st["start"])
    else:
        t, row, pos, pg, slot = _places(st, st["ik"].shape[0])
        st["keys"][pg, slot] = st["ik"][t]
        # the last new token of each block that got one
        last = (pos % BLOCK == BLOCK - 1) | (t + 1 == st["offs"].long()[row + 1])
        row, pos, pg = row[last], pos[last], pg[last]
        page = st["case"]["page"]
        j = (pos // BLOCK * BLOCK)[:, None] + torch.arange(BLOCK, device="cuda")[None, :]
        there = j <= pos[:, None]
        j = torch.minimum(j, pos[:, None])
        x = st["keys"][st["table"].long()[row[:, None], j // page], j % page].float()
        total = torch.where(there[:, :, None, None], x, x.new_zeros(())).sum(1)
        mean = total / (pos % BLOCK + 1).float()[:, None, None]
        st["means"][_mean_slot(pg, pos, page)] = mean
    return dict(keys=st["keys"], means=st["means"])


def _mean_slot(pg, pos, page):
    """Where the mean of the block that holds pos (its last cached key) is kept."""
    return pg if page <= BLOCK else pg * (page // BLOCK) + pos % page // BLOCK


def _select(st):
    if own:
        from block_sparse_gqa_msa_gb300 import api
        return api.msa_paged_select(st["index"], st["iq"], st["table"], st["lens"],
                                    force_local=bool(st["case"]["force"]))
    page, table = st["case"]["page"], st["table"].long()
    lens = st["lens"].long()
    n = (lens + BLOCK - 1) // BLOCK
    v = torch.arange(max(SLOTS, table.shape[1] * page // BLOCK), device="cuda")
    last = torch.minimum(v[None, :] * BLOCK + BLOCK - 1, lens[:, None] - 1)
    slot = _mean_slot(table.gather(1, last // page), last, page)
    score = torch.einsum("rvhd,rhd->hrv", st["means"][slot], st["iq"].float())
    if st["case"]["force"]:
        score[:, :, 0] = math.inf
        score = torch.where(v[None, :] == n[:, None] - 1, score.new_full((), math.inf), score)
    there = v[None, :] < n[:, None]
    score = torch.where(there, score, score.new_full((), -math.inf))
    at = score.sort(dim=2, descending=True, stable=True).indices[:, :, :SLOTS]
    at = torch.where(at < n[None, :, None], at, at.new_full((), v.numel())).sort(dim=2).values
    return torch.where(at < v.numel(), at, at.new_full((), -1)).to(torch.int32)


def _decode(st):
    if own:
        from block_sparse_gqa_msa_gb300 import api
        o, lse = api.msa_paged_decode(st["cache"], st["q"], st["table"], st["lens"], st["scale"],
                                      q2k=st["q2k"], workspace=st["workspace"])
        return dict(o=o, lse=lse)
    case = st["case"]
    page, table, lens = case["page"], st["table"].long(), st["lens"].long()
    rows, kv, dim = case["rows"], case["kv"], case["dim"]
    q = st["q"].float().view(rows, kv, -1, dim)
    if st["q2k"] is None:
        j = torch.arange(table.shape[1] * page, device="cuda")
        seen = (j[None, :] < lens[:, None])[:, None, :]                          # [rows, 1, keys]
        pages = table.clamp(min=0)
        k = st["k_cache"][pages].float().view(rows, -1, kv, dim).transpose(1, 2)  # [rows, kv, keys, dim]
        v = st["v_cache"][pages].float().view(rows, -1, kv, dim).transpose(1, 2)
    else:
        block = st["q2k"].long().transpose(0, 1)                                  # [rows, kv, 16]
        j = (block[..., None] * BLOCK + torch.arange(BLOCK, device="cuda")).flatten(2)
        seen = (j >= 0) & (j < lens[:, None, None])
        j = torch.minimum(j.clamp(min=0), lens[:, None, None] - 1)
        pages = table.gather(1, (j // page).flatten(1)).view(j.shape)
        head = torch.arange(kv, device="cuda")[None, :, None]
        k = st["k_cache"][pages, j % page, head].float()
        v = st["v_cache"][pages, j % page, head].float()
    s = torch.matmul(q, k.transpose(2, 3)) * st["scale"]
    s = torch.where(seen[:, :, None, :], s, s.new_full((), -math.inf))
    top = s.amax(dim=3, keepdim=True)
    p = torch.exp(s - top)
    total = p.sum(dim=3, keepdim=True)
    o = torch.matmul(p / total, v).view(rows, -1, dim).to(st["q"].dtype)
    return dict(o=o, lse=(top + torch.log(total)).view(rows, -1))


# ------------------------------------------------------------------ in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "index": _exact_index, "select": lambda s: None,
            "decode": _exact_decode}[case["op"]](st)


def _exact_append(st):
    case = st["case"]
    page, rot = case["page"], case["rot"]
    freq = st["inv_freq"].double()
    outs = dict(q=st["q_out"].double(), k_cache=st["k_cache"].double(),
                v_cache=st["v_cache"].double())
    if case["keep_k"]:
        outs["k"] = st["k_out"].double()
    first = st["offs"].tolist()
    pair = torch.arange(rot // 2, device="cuda")
    lo, hi = (2 * pair, 2 * pair + 1) if case["inter"] else (pair, pair + rot // 2)
    for r, begin in enumerate(st["start"].tolist()):
        here = slice(first[r], first[r + 1])
        pos = begin + torch.arange(first[r + 1] - first[r], device="cuda")
        turn = torch.polar(torch.ones(len(pos), rot // 2, dtype=torch.float64, device="cuda"),
                           pos.double()[:, None] * freq)[:, None, :]
        done = {}
        for name in ("q", "k"):
            x = st[name][here].double()
            z = torch.complex(x[..., lo], x[..., hi]) * turn
            x[..., lo], x[..., hi] = z.real, z.imag
            done[name] = x
        where = st["table"][r].long()[pos // page], pos % page
        outs["q"][here] = done["q"]
        outs["k_cache"][where] = done["k"]
        outs["v_cache"][where] = st["v"][here].double()
        if case["keep_k"]:
            outs["k"][here] = done["k"]
    return outs


def _exact_index(st):
    case = st["case"]
    page = case["page"]
    keys, means = st["keys"].double(), st["means"].double()
    first = st["offs"].tolist()
    for r, begin in enumerate(st["start"].tolist()):
        end = begin + first[r + 1] - first[r]
        table = st["table"][r].long()
        pos = torch.arange(begin, end, device="cuda")
        keys[table[pos // page], pos % page] = st["ik"][first[r]:first[r + 1]].double()
        for lo in range(begin // BLOCK * BLOCK, end, BLOCK):
            hi = min(lo + BLOCK, end)
            pos = torch.arange(lo, hi, device="cuda")
            at = int(_mean_slot(table[(hi - 1) // page], hi - 1, page))
            means[at] = keys[table[pos // page], pos % page].mean(0)
    return dict(keys=keys, means=means)


def _exact_decode(st):
    case = st["case"]
    page, kv = case["page"], case["kv"]
    outs, logs = [], []
    for r, n in enumerate(st["lens"].tolist()):
        pages = st["table"][r, :-(-n // page)].long()
        k = st["k_cache"][pages].flatten(0, 1)[:n]
        v = st["v_cache"][pages].flatten(0, 1)[:n]
        o = torch.empty(case["heads"], case["dim"], dtype=torch.float64, device="cuda")
        lse = torch.empty(case["heads"], dtype=torch.float64, device="cuda")
        share = case["heads"] // kv
        for g in range(kv):
            mine = slice(g * share, (g + 1) * share)
            kg, vg = k[:, g], v[:, g]
            if st["q2k"] is not None:
                chosen = st["q2k"][g, r]
                pos = torch.arange(n, device="cuda") // BLOCK
                keep = torch.isin(pos, chosen[chosen >= 0].long())
                kg, vg = kg[keep], vg[keep]
            s = st["q"][r, mine].double() @ kg.double().T * st["scale"]
            lse[mine] = torch.logsumexp(s, dim=1)
            o[mine] = torch.softmax(s, dim=1) @ vg.double()
        outs.append(o)
        logs.append(lse)
    return dict(o=torch.stack(outs), lse=torch.stack(logs))
