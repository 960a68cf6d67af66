"""The paged-cache operators as they are measured: a decoding step over a cache of
keys and values in pages, from the block tables to the attention of drafted tokens
and the move of the accepted ones.

Four operators, one case kind each:

  plan    sparse_attn_cache_plan    block tables, slot map, positions and tree masks
                                    of a step, from the requests' lengths
  write   sparse_attn_cache_write   the new tokens' keys and values into their slots
  tree    sparse_attn_tree_fwd      attention of the new tokens (one token, a tree of
                                    drafted tokens, or a chunk of a prompt) over the
                                    cached tokens and one another
  accept  sparse_attn_cache_accept  the accepted drafts' rows moved to their final
                                    places, in every layer

Notation: request r has L_r tokens in the cache and T_r new ones; new token i of the
request takes the place L_r + i, page table[r, place // page] and slot
page_id * page + place % page. A new token sees all L_r cached tokens and the new
ones that its mask row names (its ancestors and itself; without a mask every new
token up to itself).

`own` is set from outside: False computes the operators in plain torch, True calls
the library.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a decoding step of a mid-size batch: one token for each request
        dict(name="plan_step_64", kind="plan", requests=64, ctx=8192, new=1, tree=False, page=64, ended=0),
        # drafted trees for a full batch, small pages, some requests ending
        dict(name="plan_tree_256x48", kind="plan", requests=256, ctx=16384, new=48, tree=True, page=16, ended=9),
        # prompts admitted in one go: long ragged counts
        dict(name="plan_prompts_9", kind="plan", requests=9, ctx=1, new=18800, tree=False, page=64, ended=2),
        # the rows of one decoding step, 8 key heads
        dict(name="write_step_64", kind="write", tokens=64, heads=8, d=128, page=64, dtype="bf16", headmajor=False),
        # a whole long prompt, given head by head as the block-sparse forward has it
        dict(name="write_prompt_29601", kind="write", tokens=29601, heads=24, d=128, page=64, dtype="bf16",
             headmajor=True),
        # plain decoding, one long-running request: the latency of a single call
        dict(name="tree_one_4096", kind="tree", requests=1, ctx=4096, ragged=False, new=1, mask=False, hq=24, hkv=24,
             d=128, page=64, dtype="bf16"),
        # plain decoding, a ragged batch with shared key heads
        dict(name="tree_step_64", kind="tree", requests=64, ctx=16384, ragged=True, new=1, mask=False, hq=32, hkv=8,
             d=128, page=64, dtype="fp16"),
        # small trees, odd sizes everywhere, heads of 64
        dict(name="tree_odd_7x13", kind="tree", requests=7, ctx=5003, ragged=True, new=13, mask=True, hq=12, hkv=4,
             d=64, page=32, dtype="bf16"),
        # drafted trees of 64 tokens for a batch, small pages
        dict(name="tree_16x64", kind="tree", requests=16, ctx=16384, ragged=True, new=64, mask=True, hq=32, hkv=8,
             d=128, page=16, dtype="bf16"),
        # a chunk of a prompt behind a long context: no mask, the tensor cores' case
        dict(name="tree_chunk_2x2048", kind="tree", requests=2, ctx=30000, ragged=True, new=2048, mask=False, hq=32,
             hkv=8, d=128, page=128, dtype="bf16"),
        # accepted drafts of a small batch in a shallow model
        dict(name="accept_16", kind="accept", requests=16, layers=4, heads=8, d=128, new=16, take=4, page=64,
             dtype="bf16"),
        # a full batch in a deep model
        dict(name="accept_96x32", kind="accept", requests=96, layers=32, heads=4, d=128, new=48, take=9, page=16,
             dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    kind = rng.choice(["plan", "write", "tree", "tree", "tree", "accept"])
    page = rng.choice([16, 32, 64, 128, 256])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "plan":
        requests = _log(rng, 1, 700)
        tree = rng.random() < 0.5
        return dict(kind=kind, requests=requests, ctx=_log(rng, 1, 20000),
                    new=_log(rng, 1, 64) if tree else _log(rng, 1, max(1, 110000 // requests)),
                    tree=tree, page=page, ended=rng.randrange(0, 1 + requests // 3))
    if kind == "write":
        return dict(kind=kind, tokens=_log(rng, 1, 29000), heads=rng.choice([1, 2, 3, 5, 8, 24]),
                    d=rng.choice([64, 128]), page=page, dtype=dtype, headmajor=rng.random() < 0.5)
    if kind == "accept":
        new = _log(rng, 1, 64)
        return dict(kind=kind, requests=_log(rng, 1, 90), layers=_log(rng, 1, 32), heads=rng.choice([1, 2, 3, 4]),
                    d=rng.choice([64, 128]), new=new, take=rng.randint(1, min(new, 12)), page=page, dtype=dtype)
    shape = rng.choice(["step", "tree", "chunk"])
    hkv = rng.choice([1, 2, 4, 8])
    hq = hkv * rng.choice([1, 2, 3, 4, 5, 8])
    if shape == "step":
        requests, new, ctx = _log(rng, 1, 96), 1, _log(rng, 1, 16384)
    elif shape == "tree":
        requests, new, ctx = _log(rng, 1, 24), _log(rng, 2, 100), _log(rng, 1, 16384)
    else:
        requests, new, ctx = rng.randint(1, 3), _log(rng, 100, 1500), _log(rng, 1, 16384)
    return dict(kind=kind, requests=requests, ctx=ctx, ragged=rng.random() < 0.7, new=new, mask=shape == "tree",
                hq=hq, hkv=hkv, d=rng.choice([64, 128]), page=page, dtype=dtype)


def _spread(n, top, ragged=True):
    """n lengths from 1 to top: all of them top, or spread evenly over the range in a fixed mixed order."""
    if not ragged:
        return [top] * n
    return [1 + int((top - 1) * (((i + 1) * 0.6180339887498949) % 1.0)) if i else top for i in range(n)]


def _counts(case):
    """(cached tokens, new tokens) of every request; a tree batch drafts the same number for each."""
    n = case["requests"]
    ctx = _spread(n, case["ctx"], case.get("ragged", True))
    new = _spread(n, case["new"]) if case["kind"] == "plan" and not case["tree"] else [case["new"]] * n
    return ctx, new


# ------------------------------------------------------------------ inputs

def _tree(n, gen):
    """Parents of a drafted tree of n tokens: a trunk of the most likely continuations first, then side
    branches that hang off any earlier token."""
    trunk = max(1, n // 4)
    pick = torch.rand(n, generator=gen)
    return [i - 1 if i < trunk else int(pick[i] * i) for i in range(n)]


def _mask_words(parents, words):
    """The visible new tokens of each new token of one request, 32 to a word, as signed words."""
    seen, rows = [], []
    for i, p in enumerate(parents):
        s = (1 << i) | (seen[p] if p >= 0 else 0)
        seen.append(s)
        row = [(s >> (32 * w)) & 0xffffffff for w in range(words)]
        rows.append([x - (1 << 32) if x >> 31 else x for x in row])
    return rows


def _ints(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


def _paged(case, ctx, new, gen, layers=None):
    """A cache that holds every request's tokens in pages of a pool in mixed order, and its block tables."""
    page = case["page"]
    need = [(c + t + page - 1) // page for c, t in zip(ctx, new)]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen).tolist()
    table = torch.zeros(len(ctx), max(need), dtype=torch.int32)
    for r, k in enumerate(need):
        table[r, :k] = torch.tensor([order.pop() for _ in range(k)], dtype=torch.int32)
    heads = case["hkv"] if case["kind"] == "tree" else case["heads"]
    shape = (pages, page, heads, case["d"])
    if layers is not None:
        shape = (layers,) + shape
    dev = torch.Generator(device="cuda")
    dev.manual_seed(int(torch.randint(1 << 30, (1,), generator=gen)))
    kv = [torch.empty(shape, dtype=_TYPES[case["dtype"]], device="cuda").normal_(generator=dev) for _ in range(2)]
    return kv[0], kv[1], table.cuda(), dev


def prepare(case, seed):
    gen = torch.Generator()
    gen.manual_seed(1009 * seed + 17)
    kind = case["kind"]
    state = dict(case=case)
    if kind == "plan":
        ctx, new = _counts(case)
        page, R = case["page"], case["requests"]
        ended = set(torch.randperm(R, generator=gen)[:case["ended"]].tolist())
        held = [(c + page - 1) // page + (1 if c % 3 == 0 else 0) for c in ctx]   # some hold a page of a past draft
        width = max((c + t + page - 1) // page + 1 for c, t in zip(ctx, new))
        pages = sum(held) + sum((t + page - 1) // page for t in new) + 1
        order = torch.randperm(pages, generator=gen).tolist()
        table = torch.zeros(R, width, dtype=torch.int32)
        for r in range(R):
            table[r, :held[r]] = torch.tensor([order.pop() for _ in range(held[r])], dtype=torch.int32)
        free = torch.zeros(pages, dtype=torch.int32)
        free[:len(order)] = torch.tensor(order, dtype=torch.int32)
        parents = [] if case["tree"] else None
        if case["tree"]:
            for r in range(R):
                if r not in ended:
                    parents += _tree(new[r], gen)
        n = sum(new) + 5                                            # the step's buffers hold every request, and more
        new = [-1 if r in ended else t for r, t in enumerate(new)]
        if parents is not None:
            parents = _ints(parents + [-1] * (n - len(parents)))
        state.update(lens=_ints(ctx), new=_ints(new), held=_ints(held), nfree=_ints([len(order)]), free=free.cuda(),
                     table=table.cuda(), parents=parents, n=n, page=page,
                     words=(case["new"] + 31) // 32 if case["tree"] else 0)
    elif kind == "write":
        n, H, d, page = case["tokens"], case["heads"], case["d"], case["page"]
        pages = (n + page - 1) // page + 2
        ids = torch.randperm(pages, generator=gen)
        place = torch.arange(n)
        slots = ids[place // page] * page + place % page
        slots[torch.rand(n, generator=gen) < 0.02] = -1             # rows of a padded batch
        dev = torch.Generator(device="cuda")
        dev.manual_seed(seed + 5)
        dt = _TYPES[case["dtype"]]
        shape = (H, n, d) if case["headmajor"] else (n, H, d)
        k, v = (torch.empty(shape, dtype=dt, device="cuda").normal_(generator=dev) for _ in range(2))
        if case["headmajor"]:
            k, v = k.transpose(0, 1), v.transpose(0, 1)
        kc, vc = (torch.zeros(pages, page, H, d, dtype=dt, device="cuda") for _ in range(2))
        state.update(k=k, v=v, slots=slots.to(torch.int32).cuda(), kc=kc, vc=vc)
    elif kind == "tree":
        ctx, new = _counts(case)
        kc, vc, table, dev = _paged(case, ctx, new, gen)
        n = sum(new)
        q = torch.empty(n, case["hq"], case["d"], dtype=_TYPES[case["dtype"]], device="cuda").normal_(generator=dev)
        q *= 1.5                                                     # scores of a trained model are not flat
        starts = [0]
        for t in new:
            starts.append(starts[-1] + t)
        mask = None
        if case["mask"]:
            words = (case["new"] + 31) // 32
            mask = _ints([row for t in new for row in _mask_words(_tree(t, gen), words)])
        state.update(q=q, kc=kc, vc=vc, table=table, lens=_ints(ctx), starts=_ints(starts), new=_ints(new), mask=mask,
                     ctx=ctx, count=new, scale=case["d"] ** -0.5)
    else:
        R, T = case["requests"], case["new"]
        ctx = _spread(R, 90)
        kc, vc, table, _ = _paged(case, ctx, [T] * R, gen, case["layers"])
        # every request accepts 1 to `take` tokens: along the trunk, then off it into a side branch
        taken, accepted = [], torch.full((R, case["take"]), -1, dtype=torch.int32)
        for r in range(R):
            m = 1 + int(torch.randint(case["take"], (1,), generator=gen))
            stay = int(torch.randint(m + 1, (1,), generator=gen)) if T > m else m
            stay = max(stay, m - (T - m))
            side = torch.randperm(T - m, generator=gen)[:m - stay].sort().values + m
            accepted[r, :m] = torch.cat([torch.arange(stay), side]).to(torch.int32)
            taken.append(m)
        state.update(kc=kc, vc=vc, table=table, lens=_ints(ctx), accepted=accepted.cuda(), taken=_ints(taken),
                     starts=_ints([T * r for r in range(R + 1)]), new=_ints([T] * R))
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    kind = state["case"]["kind"]
    if own:
        return _OWN[kind](state)
    return _PLAIN[kind](state)


def _own_plan(s):
    import free_block_sparse_mean_b200 as sa
    p = sa.sparse_attn_cache_plan(s["lens"], s["new"], s["table"], s["held"], s["free"], s["nfree"], s["n"],
                                  s["page"], parents=s["parents"], mask_words=s["words"])
    out = [p.table, p.free_pages, p.held, p.nfree, p.starts, p.granted, p.slots, p.positions]
    return out + ([p.mask] if s["parents"] is not None else [])


def _own_write(s):
    import free_block_sparse_mean_b200 as sa
    sa.sparse_attn_cache_write(s["k"], s["v"], s["slots"], s["kc"], s["vc"])
    return s["kc"], s["vc"]


def _cache_plan(s):
    import free_block_sparse_mean_b200 as sa
    return sa.CachePlan(table=s["table"], lens=s["lens"], starts=s["starts"], granted=s["new"], mask=s.get("mask"),
                        max_new=s["case"]["new"])


def _own_tree(s):
    import free_block_sparse_mean_b200 as sa
    return sa.sparse_attn_tree_fwd(s["q"], s["kc"], s["vc"], _cache_plan(s), scale=s["scale"])


def _own_accept(s):
    import free_block_sparse_mean_b200 as sa
    sa.sparse_attn_cache_accept(s["kc"], s["vc"], _cache_plan(s), s["accepted"], s["taken"])
    return s["kc"], s["vc"]


def _plain_plan(s):
    page, n = s["page"], s["n"]
    lens, new, held = s["lens"].long(), s["new"].long(), s["held"].long()
    table, free, nfree = s["table"], s["free"], s["nfree"].long()
    R, width = table.shape
    dev = table.device
    over = new < 0
    count = new.clamp(min=0)
    col = torch.arange(width, device=dev)
    # the pages of ended requests go back on the list, in request order
    back = torch.where(over, held, 0)
    at = nfree + (torch.cumsum(back, 0) - back)[:, None] + col
    put = over[:, None] & (col < held[:, None])
    free = torch.cat([free, free.new_zeros(1)])
    free.scatter_(0, torch.where(put, at, free.numel() - 1).reshape(-1), table.reshape(-1))
    top = nfree + back.sum()
    # pages are taken off the list's end, in request order, while they last
    need = torch.where(over, 0, ((lens + count + page - 1) // page - held).clamp(min=0))
    upto = torch.cumsum(need, 0)
    served = ~over & ((need == 0) | (upto <= top))
    need = torch.where(served, need, 0)
    taken = torch.where(served & (need > 0), upto, 0).max()
    grow = (col >= held[:, None]) & (col < (held + need)[:, None])
    src = top - 1 - ((upto - need)[:, None] + col - held[:, None])
    table = torch.where(grow, free[src.clamp(0, free.numel() - 1)], table)
    held_out = torch.where(over, 0, held + need)
    granted = torch.where(served, count, 0)
    starts = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)])
    # the new tokens
    i = torch.arange(n, device=dev)
    r = (torch.searchsorted(starts, i, right=True) - 1).clamp(max=R - 1)
    live = i < starts[-1]
    here = i - starts[r]
    place = lens[r] + here
    slot = table[r, (place // page).clamp(max=width - 1)].long() * page + place % page
    slots = torch.where(live & (granted[r] > 0), slot, -1)
    out = [table, free[:-1], held_out, top - taken, starts, granted, slots]
    if s["parents"] is None:
        return [x.to(torch.int32) for x in out + [torch.where(live, place, 0)]]
    words = s["words"]
    bit = torch.zeros(n, words, dtype=torch.int64, device=dev)
    node, depth = torch.where(live, here, -1), torch.full_like(here, -1)
    up = torch.cat([s["parents"].long(), s["parents"].new_full((1,), -1).long()])
    for _ in range(32 * words):
        on = node >= 0
        w = (node.clamp(min=0) // 32)[:, None] == torch.arange(words, device=dev)
        bit |= torch.where(on[:, None] & w, (1 << (node.clamp(min=0) % 32))[:, None], 0)
        depth += on
        node = torch.where(on, up[(starts[r] + node.clamp(min=0)).clamp(max=n)], -1)
    mask = torch.where(bit >= 1 << 31, bit - (1 << 32), bit)
    return [x.to(torch.int32) for x in out + [torch.where(live, lens[r] + depth, 0), mask]]


def _plain_write(s):
    kc, vc, slots = s["kc"], s["vc"], s["slots"].long()
    keep = torch.nonzero(slots >= 0)[:, 0]
    at = slots[keep]
    kc.view(-1, *kc.shape[2:])[at] = s["k"][keep]
    vc.view(-1, *vc.shape[2:])[at] = s["v"][keep]
    return kc, vc


def _plain_tree(s):
    q, kc, vc, table = s["q"], s["kc"], s["vc"], s["table"]
    page, hkv, d = kc.shape[1:]
    group = q.shape[1] // hkv
    out = torch.empty_like(q)
    first = 0
    for r, (ctx, t) in enumerate(zip(s["ctx"], s["count"])):
        total = ctx + t
        ids = table[r, :(total + page - 1) // page].long()
        rows = q[first:first + t].float().view(t, hkv, group, d).permute(1, 2, 0, 3)
        j = torch.arange(t, device=q.device)
        if s["mask"] is None:
            sees = j[None, :] <= j[:, None]
        else:
            words = s["mask"][first:first + t].long() & 0xffffffff
            sees = (words[:, j // 32] >> (j % 32)) & 1 == 1
        step = max(1, (1 << 30) // (group * t * total))              # heads at a time: 4 GB of scores
        for h in range(0, hkv, step):
            hs = slice(h, min(h + step, hkv))
            k = kc[ids, :, hs].reshape(-1, hs.stop - h, d)[:total].float().permute(1, 2, 0)
            v = vc[ids, :, hs].reshape(-1, hs.stop - h, d)[:total].float().permute(1, 0, 2)
            p = torch.matmul(rows[hs].reshape(hs.stop - h, group * t, d), k) * s["scale"]
            p = p.view(hs.stop - h, group, t, total)
            p[..., ctx:].masked_fill_(~sees, -math.inf)
            p = torch.exp(p - p.amax(-1, keepdim=True))
            o = torch.matmul(p.view(hs.stop - h, group * t, total), v) / p.sum(-1).view(hs.stop - h, group * t, 1)
            o = o.view(hs.stop - h, group, t, d).permute(2, 0, 1, 3)
            out[first:first + t].view(t, hkv, group, d)[:, hs] = o.to(q.dtype)
        first += t
    return out


def _plain_accept(s):
    kc, vc, table = s["kc"], s["vc"], s["table"].long()
    page = kc.shape[2]
    acc, lens = s["accepted"].long(), s["lens"].long()
    i = torch.arange(acc.shape[1], device=acc.device)
    r, c = torch.nonzero(i < s["taken"][:, None], as_tuple=True)
    src, dst = lens[r] + acc[r, c], lens[r] + c
    src = table[r, src // page] * page + src % page
    dst = table[r, dst // page] * page + dst % page
    for cache in (kc, vc):
        rows = cache.view(cache.shape[0], -1, *cache.shape[3:])
        rows[:, dst] = rows[:, src]
    return kc, vc


_PLAIN = dict(plan=_plain_plan, write=_plain_write, tree=_plain_tree, accept=_plain_accept)
_OWN = dict(plan=_own_plan, write=_own_write, tree=_own_tree, accept=_own_accept)


# ------------------------------------------------------------------ definition and work

def exact(case, seed):
    """The attention by its definition in 64 bits, one request and query head at a time; the other operators
    move and count whole values and have nothing to round."""
    if case["kind"] != "tree":
        return None
    s = prepare(case, seed)
    q, page = s["q"], case["page"]
    group = case["hq"] // case["hkv"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    starts = s["starts"].tolist()
    for r in range(case["requests"]):
        lo, hi, ctx = starts[r], starts[r + 1], s["ctx"][r]
        T = hi - lo
        place = torch.arange(ctx + T, device=q.device)
        where = s["table"][r].long()[place // page], place % page
        visible = torch.ones(T, ctx + T, dtype=torch.bool, device=q.device)
        if s["mask"] is None:
            visible[:, ctx:] = torch.ones(T, T, device=q.device).tril().bool()
        else:
            bits = [[(w >> b) & 1 for w in row for b in range(32)][:T] for row in s["mask"][lo:hi].tolist()]
            visible[:, ctx:] = torch.tensor(bits, device=q.device).bool()
        for h in range(case["hq"]):
            keys = s["kc"][where[0], where[1], h // group].double()
            values = s["vc"][where[0], where[1], h // group].double()
            for a in range(0, T, 1024):
                rows = slice(a, min(a + 1024, T))
                score = (q[lo:hi, h][rows].double() @ keys.T) / math.sqrt(case["d"])
                score = torch.where(visible[rows], score, -math.inf)
                out[lo:hi, h][rows] = torch.softmax(score, -1) @ values
    return out


def work(case):
    kind = case["kind"]
    if kind == "plan":
        ctx, new = _counts(case)
        page, R = case["page"], case["requests"]
        n = sum(new)
        grown = sum(max(0, (c + t + page - 1) // page - (c + page - 1) // page) for c, t in zip(ctx, new))
        words = (case["new"] + 31) // 32 if case["tree"] else 0
        # lengths, counts and held pages read; starts, grants and held pages written; each page's id read and
        # written; a slot and a position for each token, and for a tree its parent and its mask
        return {"bytes": 4 * (6 * R + 2 * grown + 2 * n + (1 + words) * n * case["tree"]), "flops": 0}
    size = 2
    if kind == "write":
        return {"bytes": 2 * 2 * size * case["tokens"] * case["heads"] * case["d"] + 4 * case["tokens"], "flops": 0}
    if kind == "accept":
        rows = case["requests"] * (1 + case["take"]) / 2 * case["layers"] * case["heads"]
        return {"bytes": int(2 * 2 * size * rows * case["d"] * 0.5), "flops": 0}    # about half of them move
    ctx, new = _counts(case)
    keys = sum(c + t for c, t in zip(ctx, new))
    pairs = sum(t * c + t * (t + 1) // 2 for c, t in zip(ctx, new))
    return {"bytes": size * case["d"] * (2 * keys * case["hkv"] + 2 * sum(new) * case["hq"]),
            "flops": 4 * pairs * case["hq"] * case["d"]}
