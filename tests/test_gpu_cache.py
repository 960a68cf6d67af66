"""Paged cache: step plan, write, attention of new tokens and accept against the plain
CPU implementation (oracle/paged_cache_oracle.py)."""
import math
import random

import pytest
import torch

from oracle import paged_cache_oracle as orc

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import free_block_sparse_mean_b200 as sa

BF, HF = torch.bfloat16, torch.float16


def dev_ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def no_device_error():
    torch.cuda.synchronize()
    assert sa.sparse_attn_device_error() == 0


# ------------------------------------------------------------------ step plan

def plan_case(rng, R, page, tree, ended, top_len=300, top_new=40, spare=0, words=None):
    lens = [rng.randint(0, top_len) for _ in range(R)]
    new = [rng.choice([0, 1, rng.randint(1, top_new)]) for _ in range(R)]
    held = [-(-c // page) + rng.choice([0, 0, 1, 3]) for c in lens]
    width = max(max(-(-(c + t) // page), h) for c, t, h in zip(lens, new, held)) + 1
    pages = sum(held) + sum(-(-t // page) for t in new) + 2 + spare
    ids = list(range(pages))
    rng.shuffle(ids)
    table = [[ids.pop() for _ in range(h)] + [-7] * (width - h) for h in held]
    free = list(ids) + [0] * (pages - len(ids))
    nfree = len(ids)
    for r in rng.sample(range(R), min(ended, R)):
        new[r] = -rng.randint(1, 3)
    parents = None
    if tree:
        parents = []
        for t in new:
            parents += [rng.randint(-1, i - 1) for i in range(max(t, 0))]
    n = max(1, sum(max(t, 0) for t in new) + rng.choice([0, 1, 9]))
    if tree:
        parents += [5] * (n - len(parents))
    return dict(lens=lens, new=new, held=held, nfree=nfree, free=free, table=table, parents=parents, page=page, n=n,
                words=words if words is not None else ((max(max(new), 1) + 31) // 32 if tree else 0))


def run_plan(c, out=None):
    free, table = dev_ints(c["free"]), dev_ints(c["table"])
    return sa.sparse_attn_cache_plan(dev_ints(c["lens"]), dev_ints(c["new"]), table, dev_ints(c["held"]), free,
                                     dev_ints([c["nfree"]]), c["n"], c["page"],
                                     parents=None if c["parents"] is None else dev_ints(c["parents"]),
                                     mask_words=c["words"], out=out)


def check_plan(p, c):
    ref = orc.plan(c["lens"], c["new"], c["held"], c["nfree"], c["free"], c["table"], c["parents"], c["page"], c["n"],
                   c["words"])
    for name, want in ref.items():
        if name == "mask" and not c["words"]:
            assert p.mask is None
            continue
        got = getattr(p, name).cpu().tolist()
        if name == "free_pages":          # behind the counts the list holds leftovers
            got, want = got[:ref["nfree"][0]], want[:ref["nfree"][0]]
        assert got == want, name
    return ref


@pytest.mark.parametrize("R,page,tree,ended", [
    (1, 16, False, 0), (1, 256, True, 0), (2, 64, True, 1), (7, 32, False, 3), (33, 16, True, 5), (64, 64, False, 0),
    (255, 128, True, 40), (256, 16, False, 256), (257, 16, True, 13), (700, 32, True, 200), (2100, 64, False, 7)])
def test_plan_matches_the_plain_one(R, page, tree, ended):
    rng = random.Random(R * 1000 + page)
    c = plan_case(rng, R, page, tree, ended)
    p = run_plan(c)
    no_device_error()
    check_plan(p, c)
    # a step's outputs feed the next: the unused pages of a table row come first
    c2 = dict(c, lens=[max(0, l + g // 2) if t >= 0 else 0 for l, g, t in zip(c["lens"], p.granted.tolist(), c["new"])],
              held=p.held.tolist(), nfree=int(p.nfree), free=p.free_pages.tolist(), table=p.table.tolist())
    check_plan(run_plan(c2), c2)
    no_device_error()


def test_plan_serves_in_order_while_pages_last():
    rng = random.Random(3)
    c = plan_case(rng, 40, 16, False, 4)
    # not enough pages for all: only part of the list is offered
    for nfree in (0, 1, c["nfree"] // 3, c["nfree"] - 1):
        d = dict(c, nfree=nfree)
        p = run_plan(d)
        check_plan(p, d)                 # the ended requests' pages may cover every need
    c = plan_case(rng, 40, 16, False, 0)
    refused = 0
    for nfree in (0, 1, 5, c["nfree"] // 3):
        d = dict(c, nfree=nfree)
        ref = check_plan(run_plan(d), d)
        refused += sum(g == 0 and t > 0 for g, t in zip(ref["granted"], c["new"]))
    assert refused > 0
    no_device_error()


def test_plan_chain_masks_and_long_trees():
    rng = random.Random(5)
    for tree in (False, True):
        c = plan_case(rng, 5, 32, tree, 1, top_new=1000, words=32)
        check_plan(run_plan(c), c)
    no_device_error()


def test_plan_repeats_with_the_same_inputs():
    rng = random.Random(8)
    c = plan_case(rng, 50, 16, True, 10)
    args = [dev_ints(c["lens"]), dev_ints(c["new"]), dev_ints(c["table"]), dev_ints(c["held"]), dev_ints(c["free"]),
            dev_ints([c["nfree"]]), c["n"], c["page"]]
    kw = dict(parents=dev_ints(c["parents"]), mask_words=c["words"])
    first = sa.sparse_attn_cache_plan(*args, **kw)
    keep = [getattr(first, k).clone() for k in ("table", "free_pages", "held", "nfree", "slots", "positions", "mask")]
    again = sa.sparse_attn_cache_plan(*args, **kw, out=first)
    assert again is first
    for k, x in zip(("table", "free_pages", "held", "nfree", "slots", "positions", "mask"), keep):
        assert torch.equal(getattr(first, k), x), k
    check_plan(first, c)
    no_device_error()


@pytest.mark.parametrize("fault", ["held", "short", "lens", "width", "words", "rows", "parent", "nfree"])
def test_plan_flags_what_is_out_of_range(fault):
    rng = random.Random(11)
    c = plan_case(rng, 12, 16, True, 0)
    c["new"] = [max(1, min(t, 9)) for t in c["new"]]
    c["n"] = sum(c["new"])
    c["parents"] = [max(-1, i - 1) for t in c["new"] for i in range(t)]
    c["words"] = 1
    r = 4
    if fault == "held":
        c["held"][r] = len(c["table"][0]) + 1
    elif fault == "short":
        c["held"][r] = 0
        c["lens"][r] = 100
    elif fault == "lens":
        c["lens"][r] = -1
    elif fault == "width":
        c["lens"][r] = c["held"][r] * 16
        c["new"][r] += 0
        c["held"][r] = len(c["table"][0])
        c["lens"][r] = c["held"][r] * 16
        c["table"][r] = list(range(len(c["table"][0])))
    elif fault == "words":
        c["n"] += 33 - c["new"][r]
        c["new"][r] = 33
        c["parents"] = [max(-1, i - 1) for t in c["new"] for i in range(t)]
    elif fault == "rows":
        c["n"] -= 1
        c["parents"] = c["parents"][:c["n"]]
    elif fault == "parent":
        c["parents"][sum(c["new"][:r])] = 0         # the root its own parent
    elif fault == "nfree":
        c["nfree"] = len(c["free"]) + 1
    p = run_plan(c)
    torch.cuda.synchronize()
    assert sa.sparse_attn_device_error() == 4
    if fault == "nfree":
        c["nfree"] = 0
    check_plan(p, c)


# ------------------------------------------------------------------ write

@pytest.mark.parametrize("n,H,d,page,dtype,layout", [
    (1, 1, 64, 16, BF, "rows"), (5, 3, 128, 32, HF, "rows"), (130, 8, 128, 64, BF, "heads"),
    (67, 5, 64, 256, HF, "fused"), (1000, 2, 128, 128, BF, "hnd")])
def test_write_puts_rows_into_their_slots(n, H, d, page, dtype, layout):
    g = torch.Generator().manual_seed(n)
    pages = -(-n // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:n]
    slots[torch.rand(n, generator=g) < 0.2] = -1
    if layout == "heads":
        k, v = (torch.randn(H, n, d, generator=g).to(dtype).cuda().transpose(0, 1) for _ in range(2))
    elif layout == "fused":
        kv = torch.randn(n, 4 * H, d, generator=g).to(dtype).cuda()
        k, v = kv[:, H:2 * H], kv[:, 3 * H:]
    else:
        k, v = (torch.randn(n, H, d, generator=g).to(dtype).cuda() for _ in range(2))
    shape = (pages, H, page, d) if layout == "hnd" else (pages, page, H, d)
    kc, vc = (torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2))
    if layout == "hnd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    want = []
    for rows, cache in ((k, kc), (v, vc)):
        w = cache.cpu().clone()
        for i, s in enumerate(slots.tolist()):
            if s >= 0:
                w[s // page, s % page] = rows[i].cpu()
        want.append(w)
    sa.sparse_attn_cache_write(k, v, slots.to(torch.int32).cuda(), kc, vc)
    no_device_error()
    assert torch.equal(kc.cpu(), want[0]) and torch.equal(vc.cpu(), want[1])


def test_write_leaves_out_slots_outside_the_pool():
    kc = torch.zeros(2, 16, 2, 64, dtype=BF, device="cuda")
    vc = kc.clone()
    k = torch.ones(4, 2, 64, dtype=BF, device="cuda")
    sa.sparse_attn_cache_write(k, k, dev_ints([32, 3, -2, -1]), kc, vc)
    torch.cuda.synchronize()
    assert sa.sparse_attn_device_error() == 2
    assert float(kc.float().sum()) == 128 and float(kc[0, 3].float().sum()) == 128 and torch.equal(kc, vc)


# ------------------------------------------------------------------ attention

def cache_of(ctx, new, page, Hkv, d, dtype, seed, layout="nhd", extra_pages=2, fill=None):
    """A pool holding every request's places in mixed pages; other places hold `fill`."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-(c + t) // page) for c, t in zip(ctx, new)]
    pages = sum(need) + extra_pages
    ids = torch.randperm(pages, generator=g).tolist()
    width = max(need) + 1
    table = [[ids.pop() for _ in range(k)] + [-1] * (width - k) for k in need]
    shape = (pages, Hkv, page, d) if layout == "hnd" else (pages, page, Hkv, d)
    kc, vc = (torch.randn(shape, generator=g).to(dtype) for _ in range(2))
    if layout == "hnd":
        kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    if fill is not None:
        used = torch.zeros(pages, page, dtype=torch.bool)
        for r, row in enumerate(table):
            for at in range(ctx[r] + new[r]):
                used[row[at // page], at % page] = True
        kc[~used] = fill
        vc[~used] = fill
    return kc, vc, table


def random_mask(new, words, seed, kind="tree"):
    rng = random.Random(seed)
    rows = []
    for T in new:
        seen = []
        for t in range(T):
            if kind == "tree":
                up = rng.randint(-1, t - 1)
                s = (1 << t) | (seen[up] if up >= 0 else 0)
            elif kind == "any":
                s = rng.getrandbits(T)
            else:
                s = 0
            seen.append(s)
            rows.append([((s >> (32 * w)) & 0xffffffff) for w in range(words)])
    return [[x - (1 << 32) if x >> 31 else x for x in row] for row in rows]


def tolerance(o, a, smax, d, keys, vmax, dtype):
    """Bound of the kernel's error. Half a step u = eps/2 of the type rounds each P (the sum
    l keeps them unrounded): u * sum p|v| / l = u * a. The result's rounding: u * |o|.
    A score's fp32 sum of d products and its scaling err by at most (d + 3) 2^-23 of
    sum |q||k| scale (a truncating adder loses up to a whole step), ex2.approx adds 2^-22; a relative
    error e of every p moves o by at most 2 e a. fp16 P below 2^-14 (of the row's maximum,
    where l >= 1) err by 2^-25 each. fp32 sums over the keys: keys 2^-23 of a."""
    u = torch.finfo(dtype).eps / 2
    e = (d + 3) * 2.0 ** -23 * smax[..., None] + 2.0 ** -22
    tol = u * a * (1 + u) + u * (o.abs() + u * a) + 2 * e * a + keys * 2.0 ** -23 * a + 1e-30
    if dtype == HF:
        tol = tol + keys * 2.0 ** -25 * vmax + 2.0 ** -25     # ... and o itself below 2^-14
    return tol


def check_attention(ctx, new, page, Hq, Hkv, d, dtype, *, mask=None, words=0, seed=0, layout="nhd", scale=None,
                    qscale=1.0, fill=math.nan, granted=None, pad=0, max_new=0, q=None, caches=None, want_errors=0,
                    qlayout="rows"):
    kc, vc, table = caches if caches is not None else cache_of(ctx, new, page, Hkv, d, dtype, seed, layout, fill=fill)
    starts = [0]
    for t in new:
        starts.append(starts[-1] + t)
    n = starts[-1] + pad
    g = torch.Generator().manual_seed(seed + 77)
    if q is None:
        q = (torch.randn(n, Hq, d, generator=g) * qscale).to(dtype)
    m = None
    if mask is not None:
        m = mask + [[-1] * words] * pad
    scale = d ** -0.5 if scale is None else scale
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints(ctx), starts=dev_ints(starts),
                        granted=None if granted is None else dev_ints(granted),
                        mask=None if m is None else dev_ints(m), max_new=max_new)
    out = torch.full((n, Hq, d), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((n, Hq), 7.0, device="cuda")
    def gpu(x):   # keep the layout
        return x.transpose(1, 2).contiguous().cuda().transpose(1, 2) if layout == "hnd" else x.cuda()
    qg = q.cuda()
    if qlayout == "heads":
        qg = q.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    elif qlayout == "fused":
        big = torch.randn(n, Hq + 2 * Hkv, d, dtype=dtype, device="cuda")
        big[:, :Hq] = qg
        qg = big[:, :Hq]
    got = sa.sparse_attn_tree_fwd(qg, gpu(kc), gpu(vc), plan, scale, out=out, lse=lse)
    assert got is out
    torch.cuda.synchronize()
    assert sa.sparse_attn_device_error() == want_errors
    counts = [min(t, x) for t, x in zip(new, granted)] if granted is not None else new
    o, ref_lse, a, smax = orc.tree_attention(q, kc, vc, table, ctx, starts, counts, m, scale)
    got, glse = out.cpu().double(), lse.cpu().double()
    real = ~torch.isnan(ref_lse)
    assert torch.all(got[~real] == 7.0) and torch.all(glse[~real] == 7.0), "rows that do not exist were written"
    finite = vc[torch.isfinite(vc)]
    vmax = float(finite.abs().max()) if finite.numel() else 0.0
    tol = tolerance(o, a, smax, d, max(c + t for c, t in zip(ctx, new)), vmax, dtype)
    err = (got - o).abs()[real]
    assert torch.all(err <= tol[real]), f"worst {float((err / tol[real]).max()):.3f} of the bound"
    none = torch.isinf(ref_lse) & real
    assert torch.all(got[none] == 0) and torch.all(glse[none] == -math.inf)
    some = real & ~none
    e = (d + 3) * 2.0 ** -23 * smax[some] + (max(ctx) + max(new) + 8) * 2.0 ** -23 + 2.0 ** -22 * ref_lse[some].abs()
    assert torch.all((glse - ref_lse)[some].abs() <= e)
    return got


ATTENTION = [
    # ctx, new, page, Hq, Hkv, d, dtype, mask kind
    ([0], [1], 16, 1, 1, 64, BF, None),
    ([1], [1], 64, 1, 1, 128, BF, None),
    ([63], [1], 64, 4, 2, 128, HF, None),
    ([64], [1], 32, 8, 1, 64, HF, None),
    ([129, 0, 500], [1, 1, 1], 128, 6, 2, 128, BF, None),
    ([4096], [1], 256, 24, 24, 128, BF, None),
    ([1000, 3, 77, 2049], [1, 1, 1, 1], 16, 32, 8, 128, HF, None),
    ([40, 0, 200], [5, 13, 1], 32, 12, 4, 64, BF, "tree"),
    ([333, 17], [64, 64], 16, 32, 8, 128, BF, "tree"),
    ([1, 700], [33, 100], 64, 7, 1, 128, HF, "tree"),
    ([0, 10], [9, 70], 16, 5, 5, 64, BF, "any"),
    ([0, 0, 5], [3, 64, 2], 32, 2, 1, 128, BF, "none"),
    ([100], [300], 128, 8, 2, 128, BF, None),
    ([0, 513], [129, 257], 16, 10, 2, 64, HF, None),
    ([31], [500], 64, 4, 4, 128, BF, "any"),
    ([65, 900], [40, 3], 256, 128, 1, 128, BF, None),
    ([2000, 5], [2, 9], 64, 33, 11, 64, HF, "tree"),
]


@pytest.mark.parametrize("ctx,new,page,Hq,Hkv,d,dtype,kind", ATTENTION)
def test_attention_matches_the_definition(ctx, new, page, Hq, Hkv, d, dtype, kind):
    words = (max(new) + 31) // 32 if kind else 0
    mask = random_mask(new, words, 5, kind) if kind else None
    check_attention(ctx, new, page, Hq, Hkv, d, dtype, mask=mask, words=words)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("T,G", [(1, 1), (1, 8), (3, 4), (9, 3), (32, 1), (33, 1), (5, 16), (64, 2), (129, 1)])
def test_attention_tile_shapes(T, G, d, dtype):
    """Row counts around the 32-row and 128-row limits, tiles sized for the step's tokens."""
    check_attention([130, 7], [T, max(1, T // 2)], 64, 2 * G, 2, d, dtype, max_new=T, seed=T)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("layout,qlayout", [("nhd", "heads"), ("hnd", "fused")])
def test_attention_layouts_and_pages(page, layout, qlayout):
    """Pages that end inside a 64-key block, both cache layouts, strided queries."""
    check_attention([page - 1, 3 * page + 5, 0], [2, 4, 7], page, 6, 3, 128, BF, layout=layout, qlayout=qlayout,
                    mask=random_mask([2, 4, 7], 1, 3), words=1, seed=page)


@pytest.mark.parametrize("ctx,new,Hq,Hkv,kind", [
    ([20000], [1], 4, 2, None), ([9000, 3, 400], [4, 1, 2], 4, 4, "tree"), ([6000], [200], 2, 1, None),
    ([7001, 7002], [40, 40], 2, 2, "any")])
def test_attention_split_over_the_keys(ctx, new, Hq, Hkv, kind):
    """Long caches and few rows: many pieces to a row, joined by the second kernel."""
    words = (max(new) + 31) // 32 if kind else 0
    check_attention(ctx, new, 64, Hq, Hkv, 64, BF, mask=random_mask(new, words, 9, kind) if kind else None,
                    words=words, max_new=max(new), seed=1)


def test_attention_with_growing_and_peaked_scores():
    """Maxima that rise from block to block (the running maximum is corrected), and rows
    where one key holds everything."""
    for seed, ramp in ((1, True), (2, False)):
        ctx, new, page, H, d = [700], [40], 64, 2, 128
        kc, vc, table = cache_of(ctx, new, page, H, d, BF, seed)
        q = torch.randn(40, H, d, generator=torch.Generator().manual_seed(seed)).abs().to(BF)
        for at in range(740):
            scale = at / 200 if ramp else (40.0 if at == 333 else 0.1)
            kc[table[0][at // page], at % page] = (torch.ones(H, d) * scale * (1 if ramp else d ** -0.5)).to(BF)
        check_attention(ctx, new, page, H, H, d, BF, q=q, caches=(kc, vc, table), seed=seed)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("new,kind", [([64], "tree"), ([9, 30], "any"), ([150], None)])
def test_attention_keeps_unseen_values_out(bad, new, kind):
    """Keys and values that are not finite in new tokens that a row does not see: the row
    is as if they were not there; a row that sees such a value gets it."""
    ctx = [100] * len(new)
    words = (max(new) + 31) // 32 if kind else 0
    mask = random_mask(new, words, 4, kind) if kind else None
    page, Hkv, d = 32, 2, 128
    kc, vc, table = cache_of(ctx, new, page, Hkv, d, BF, 6, fill=bad)
    hurt = {}
    for r, T in enumerate(new):
        j = T - 1 if kind is None else T // 2
        at = ctx[r] + j
        vc[table[r][at // page], at % page, 1, 5] = bad
        vc[table[r][at // page], at % page, 0, 127] = bad
        hurt[r] = j
    starts = [0]
    for t in new:
        starts.append(starts[-1] + t)
    n, Hq = starts[-1], 4
    q = torch.randn(n, Hq, d, generator=torch.Generator().manual_seed(3)).to(BF)
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints(ctx), starts=dev_ints(starts),
                        mask=None if mask is None else dev_ints(mask))
    o = sa.sparse_attn_tree_fwd(q.cuda(), kc.cuda(), vc.cuda(), plan).cpu()
    no_device_error()
    clean = vc.clone()
    clean[~torch.isfinite(clean)] = 0
    ref, _, _, _ = orc.tree_attention(q, kc, clean, table, ctx, starts, new, mask, d ** -0.5)
    for r, T in enumerate(new):
        for t in range(T):
            row = o[starts[r] + t].clone()
            if orc.visible(None if mask is None else mask[starts[r] + t], t, T)[hurt[r]]:
                for h, x in ((0, 127), (1, 127), (2, 5), (3, 5)):
                    got = row[h, x]
                    assert torch.isnan(got) if math.isnan(bad) else got == bad
                    row[h, x] = ref[starts[r] + t, h, x].to(BF)
            assert torch.isfinite(row).all()
            assert (row.double() - ref[starts[r] + t]).abs().max() < 0.05


def test_attention_unseen_keys_that_are_not_finite():
    kc, vc, table = cache_of([70], [20], 16, 2, 64, HF, 8, fill=math.inf)
    mask = random_mask([20], 1, 2)
    for bad_at in (11, 19):
        rows = [i for i in range(20) if not (mask[i][0] >> bad_at) & 1]
        k2 = kc.clone()
        at = 70 + bad_at
        k2[table[0][at // 16], at % 16] = math.nan
        q = torch.randn(20, 2, 64).to(HF).cuda()
        plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([70]), starts=dev_ints([0, 20]), mask=dev_ints(mask))
        a = sa.sparse_attn_tree_fwd(q, kc.cuda(), vc.cuda(), plan)
        b = sa.sparse_attn_tree_fwd(q, k2.cuda(), vc.cuda(), plan)
        assert torch.equal(a[rows], b[rows]) and bool(torch.isnan(b).any())
    no_device_error()


def test_attention_leaves_other_rows_alone():
    """Requests that were granted fewer tokens or none, and rows behind the last request."""
    check_attention([50, 60, 0, 9], [4, 3, 5, 2], 32, 4, 2, 128, BF, granted=[4, 0, 2, 2], pad=7)
    check_attention([50, 60], [4, 3], 32, 4, 2, 128, BF, granted=[0, 0], pad=1, mask=random_mask([4, 3], 1, 2), words=1)


def test_attention_skips_what_is_out_of_range():
    kc, vc, table = cache_of([40, 50, 60], [2, 2, 2], 16, 2, 64, BF, 0)
    good = check_attention([40, 50, 60], [2, 2, 2], 16, 4, 2, 64, BF, caches=(kc, vc, table))
    q = torch.randn(6, 4, 64, generator=torch.Generator().manual_seed(77)).to(BF).cuda()
    width = len(table[0])
    for lens, starts in (([40, -1, 60], [0, 2, 4, 6]), ([40, 16 * width, 60], [0, 2, 4, 6]),
                         ([40, 50, 60], [0, 2, 4, 7])):
        plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints(lens), starts=dev_ints(starts))
        out = torch.full((6, 4, 64), 7.0, dtype=BF, device="cuda")
        sa.sparse_attn_tree_fwd(q, kc.cuda(), vc.cuda(), plan, out=out)
        torch.cuda.synchronize()
        assert sa.sparse_attn_device_error() == 4
        skipped = [2, 3] if starts[-1] == 6 else [4, 5]
        rest = [i for i in range(6) if i not in skipped]
        assert torch.all(out[skipped] == 7.0)
        assert torch.equal(out[rest].cpu().double(), good[rest])
    for wrong in (-1, 1 << 20):                   # a page id that is not one: flagged, in bounds
        t2 = [list(row) for row in table]
        t2[1][1] = wrong
        plan = sa.CachePlan(table=dev_ints(t2), lens=dev_ints([40, 50, 60]), starts=dev_ints([0, 2, 4, 6]))
        out = sa.sparse_attn_tree_fwd(q, kc.cuda(), vc.cuda(), plan)
        torch.cuda.synchronize()
        assert sa.sparse_attn_device_error() == 2
        assert torch.equal(out[[0, 1, 4, 5]].cpu().double(), good[[0, 1, 4, 5]])


def test_attention_is_the_same_every_time():
    kc, vc, table = cache_of([3000, 100], [8, 8], 64, 4, 128, BF, 2)
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([3000, 100]), starts=dev_ints([0, 8, 16]), max_new=8)
    q = torch.randn(16, 8, 128).to(BF).cuda()
    kc, vc = kc.cuda(), vc.cuda()
    first = sa.sparse_attn_tree_fwd(q, kc, vc, plan)
    for _ in range(20):
        assert torch.equal(sa.sparse_attn_tree_fwd(q, kc, vc, plan), first)
    no_device_error()


def test_attention_of_many_requests():
    """More requests than threads in a block: the search for a piece runs in rounds."""
    rng = random.Random(1)
    ctx = [rng.randint(0, 90) for _ in range(500)]
    new = [rng.choice([0, 1, 1, 2]) for _ in range(500)]
    check_attention(ctx, new, 16, 2, 1, 64, BF, max_new=2)


# ------------------------------------------------------------------ accept

@pytest.mark.parametrize("layers,H,d,page,dtype,R,T", [
    (1, 1, 64, 16, BF, 1, 1), (3, 2, 128, 16, HF, 5, 40), (2, 5, 64, 64, BF, 9, 64), (1, 8, 128, 256, BF, 3, 100)])
def test_accept_moves_rows_to_their_places(layers, H, d, page, dtype, R, T):
    rng = random.Random(T)
    ctx = [rng.randint(0, 70) for _ in range(R)]
    need = [-(-(c + T) // page) for c in ctx]
    pages = sum(need) + 1
    ids = list(range(pages))
    rng.shuffle(ids)
    table = [[ids.pop() for _ in range(k)] + [-1] * (max(need) - k) for k in need]
    cols = min(T, 37)
    taken = [rng.randint(0, cols) for _ in range(R)]
    taken[0] = cols
    acc = [sorted(rng.sample(range(T), m)) + [-5] * (cols - m) for m in taken]
    shape = (layers, pages, page, H, d) if layers > 1 else (pages, page, H, d)
    kc, vc = torch.randn(shape).to(dtype), torch.randn(shape).to(dtype)
    want = [orc.accept(c, table, ctx, acc, taken) for c in (kc, vc)]
    kg, vg = kc.cuda(), vc.cuda()
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints(ctx), starts=dev_ints([T * r for r in range(R + 1)]))
    sa.sparse_attn_cache_accept(kg, vg, plan, dev_ints(acc), dev_ints(taken))
    no_device_error()
    assert torch.equal(kg.cpu(), want[0]) and torch.equal(vg.cpu(), want[1])


def test_accept_keeps_rows_of_requests_that_are_out_of_range():
    kc, vc, table = cache_of([20] * 6, [8] * 6, 16, 2, 64, BF, 4)
    acc = [[1, 3, 5], [1, 1, 5], [3, 2, 5], [0, 2, 8], [1, 2, 3], [2, 4, 6]]
    taken = [3, 3, 3, 3, 4, -1]                  # the first alone is right
    want = orc.accept(kc, table, [20], acc, [3])
    kg, vg = kc.cuda(), vc.cuda()
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([20] * 6), starts=dev_ints([8 * r for r in range(7)]))
    sa.sparse_attn_cache_accept(kg, vg, plan, dev_ints(acc), dev_ints(taken))
    torch.cuda.synchronize()
    assert sa.sparse_attn_device_error() == 4
    assert torch.equal(kg.cpu(), want) and torch.equal(vg.cpu(), orc.accept(vc, table, [20], acc, [3]))


# ------------------------------------------------------------------ together

def drafting_run(steps, graph, stream=None):
    """Prompts admitted, then drafted and accepted for some steps, in two layers; every
    attention is checked against the cache's own contents kept apart in plain lists."""
    R, page, Hq, Hkv, d, layers, T = 3, 16, 4, 2, 64, 2, 6
    pages, width = 60, 20
    g = torch.Generator().manual_seed(5)
    rng = random.Random(5)
    caches = [torch.full((layers, pages, page, Hkv, d), math.nan, dtype=BF, device="cuda") for _ in range(2)]
    free = dev_ints(torch.randperm(pages, generator=g).tolist())
    nfree, held = dev_ints([pages]), dev_ints([0] * R)
    table = dev_ints([[-1] * width] * R)
    lens = dev_ints([0] * R)
    past = [[[] for _ in range(R)] for _ in range(layers)]             # per layer and request: (k, v) of each token
    captured = {}

    def step(new, parents, words, cap):
        nonlocal held, nfree
        n = cap
        par = None if parents is None else parents + [-1] * (n - len(parents))
        q = torch.randn(layers, n, Hq, d, generator=g).to(BF)
        k, v = (torch.randn(layers, n, Hkv, d, generator=g).to(BF) for _ in range(2))
        key = (cap, words)
        if graph and key in captured:
            b = captured[key]
            for name, x in (("new", torch.tensor(new, dtype=torch.int32)), ("q", q), ("k", k), ("v", v),
                            ("held", held), ("nfree", nfree)):
                b[name].copy_(x)
            if par is not None:
                b["par"].copy_(torch.tensor(par, dtype=torch.int32))
            b["graph"].replay()
        else:
            b = dict(new=dev_ints(new), q=q.cuda(), k=k.cuda(), v=v.cuda(), held=held.clone(), nfree=nfree.clone(),
                     par=None if par is None else dev_ints(par))

            def work():
                p = sa.sparse_attn_cache_plan(lens, b["new"], table, b["held"], free, b["nfree"], n, page,
                                              parents=b["par"], mask_words=words)
                outs = []
                for layer in range(layers):
                    sa.sparse_attn_cache_write(b["k"][layer], b["v"][layer], p.slots, caches[0][layer],
                                               caches[1][layer])
                    outs.append(sa.sparse_attn_tree_fwd(b["q"][layer], caches[0][layer], caches[1][layer], p))
                return p, outs
            if graph:
                torch.cuda.synchronize()
                b["graph"] = torch.cuda.CUDAGraph()
                with torch.cuda.graph(b["graph"]):
                    b["out"] = work()
                captured[key] = b
                b["graph"].replay()
            else:
                b["out"] = work()
        p, outs = b["out"]
        torch.cuda.synchronize()
        held, nfree = p.held.clone(), p.nfree.clone()
        starts, slots = p.starts.tolist(), p.slots.tolist()
        mask = None if p.mask is None else p.mask.tolist()
        assert p.granted.tolist() == [max(t, 0) for t in new] and all(s == -1 for s in slots[starts[R]:])
        for layer in range(layers):
            for r in range(R):
                rows = list(range(starts[r], starts[r + 1]))
                fresh = [(k[layer, i], v[layer, i]) for i in rows]
                for t, i in enumerate(rows):
                    see = past[layer][r] + [fresh[j] for j, x in
                                            enumerate(orc.visible(None if mask is None else mask[i], t, len(rows))) if x]
                    kk = torch.stack([x[0] for x in see]).double().repeat_interleave(Hq // Hkv, 1)
                    vv = torch.stack([x[1] for x in see]).double().repeat_interleave(Hq // Hkv, 1)
                    s = torch.softmax(torch.einsum("hd,khd->hk", q[layer, i].double(), kk) * d ** -0.5, 1)
                    want = torch.einsum("hk,khd->hd", s, vv)
                    top = torch.einsum("hk,khd->hd", s, vv.abs())
                    # u a for P, u |o| for the result, and a twentieth of u a for all that is fp32
                    tol = 2.0 ** -8 * (1.05 * top + want.abs()) + 1e-6
                    assert torch.all((outs[layer][i].cpu().double() - want).abs() <= tol)
        return p, starts, k, v

    prompts = [20, 1, 45]
    p, starts, k, v = step(prompts, None, 0, 70)
    for layer in range(layers):
        for r in range(R):
            past[layer][r] += [(k[layer, i], v[layer, i]) for i in range(starts[r], starts[r + 1])]
    lens += p.granted
    for s in range(steps):
        new = [T if rng.random() < 0.8 else 1 for _ in range(R)]
        parents = [rng.randint(-1, i - 1) if i else -1 for t in new for i in range(t)]
        p, starts, k, v = step(new, parents, 1, R * T)
        acc, taken = [], []
        for r in range(R):
            node, path = rng.randrange(new[r]), []
            while node >= 0:
                path.append(node)
                node = parents[starts[r] + node]
            path.reverse()
            acc.append(path + [0] * (T - len(path)))
            taken.append(len(path))
            for layer in range(layers):
                past[layer][r] += [(k[layer, starts[r] + j], v[layer, starts[r] + j]) for j in path]
        sa.sparse_attn_cache_accept(caches[0], caches[1], p, dev_ints(acc), dev_ints(taken))
        lens += dev_ints(taken)
    used = int(held.sum())
    assert used + int(nfree) == pages
    ids = [x for r in range(R) for x in table[r, :int(held[r])].tolist()] + free[:int(nfree)].tolist()
    assert sorted(ids) == list(range(pages))              # every page is in one place
    no_device_error()


@pytest.mark.parametrize("graph", [False, True])
def test_drafting_steps_together(graph):
    drafting_run(7, graph)


def test_drafting_on_another_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        drafting_run(2, False)


def test_attention_calls_at_once_on_two_streams():
    """Each call has its own workspace, so two streams may run them together."""
    kc, vc, table = cache_of([2000, 1500], [4, 4], 64, 4, 128, BF, 3)
    kc, vc = kc.cuda(), vc.cuda()
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([2000, 1500]), starts=dev_ints([0, 4, 8]), max_new=4)
    qs = [torch.randn(8, 16, 128).to(BF).cuda() for _ in range(2)]
    want = [sa.sparse_attn_tree_fwd(q, kc, vc, plan) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    for _ in range(10):
        outs = []
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                outs.append(sa.sparse_attn_tree_fwd(q, kc, vc, plan))
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    no_device_error()


def test_cache_behind_a_block_sparse_prompt():
    """A prompt through the causal block-sparse forward (tau = 1: every block), its K and V
    into the cache; a chunk of the same prompt through the cache gives the same rows."""
    N, H, d, page, tail = 300, 2, 128, 64, 50
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(1, H, N, d, generator=g).to(BF).cuda() for _ in range(3))
    full = sa.sparse_attn_fwd(q, k, v, sa.sparse_attn_plan(q, k, 1.0, causal=True))
    pages = 8
    kc, vc = (torch.zeros(pages, page, H, d, dtype=BF, device="cuda") for _ in range(2))
    table, free = dev_ints([[0] * 6]), dev_ints([3, 7, 1, 0, 5, 2, 6, 4])
    p = sa.sparse_attn_cache_plan(dev_ints([0]), dev_ints([N]), table, dev_ints([0]), free, dev_ints([pages]), N, page)
    sa.sparse_attn_cache_write(k[0].transpose(0, 1), v[0].transpose(0, 1), p.slots, kc, vc)
    chunk = sa.CachePlan(table=table, lens=dev_ints([N - tail]), starts=dev_ints([0, tail]))
    got = sa.sparse_attn_tree_fwd(q[0].transpose(0, 1)[N - tail:], kc, vc, chunk)
    no_device_error()
    want = full[0].transpose(0, 1)[N - tail:]
    # both round P and O to bf16: 2 u each of values below 4
    assert (got.float() - want.float()).abs().max() <= 4 * 2.0 ** -8 * 4


# ------------------------------------------------------------------ refusals

def test_refusals():
    kc = torch.zeros(4, 16, 2, 64, dtype=BF, device="cuda")
    vc = kc.clone()
    plan = sa.CachePlan(table=dev_ints([[0, 1]]), lens=dev_ints([3]), starts=dev_ints([0, 2]))
    q = torch.zeros(2, 4, 64, dtype=BF, device="cuda")
    bad = [
        (q.to(HF), kc, vc, plan, {}),                                       # another type than the cache's
        (q[:, :3], kc, vc, plan, {}),                                       # heads not a multiple
        (q[..., :32], kc, vc, plan, {}),                                    # another d
        (q[:, :, ::2], kc, vc, plan, {}),                                   # d not contiguous
        (q.cpu(), kc, vc, plan, {}),
        (q[:1].expand(2, 4, 64), kc, vc, plan, {}),                         # a broadcast dimension
        (q, kc, vc[:, :, :1], plan, {}),
        (q, kc.float(), vc.float(), plan, {}),
        (q, kc, vc, sa.CachePlan(table=plan.table, lens=plan.lens.long(), starts=plan.starts), {}),
        (q, kc, vc, sa.CachePlan(table=plan.table, lens=plan.lens, starts=plan.starts[:1]), {}),
        (q, kc, vc, sa.CachePlan(table=plan.table, lens=plan.lens, starts=plan.starts, mask=dev_ints([[1]])), {}),
        (q, kc, vc, plan, dict(out=torch.zeros(2, 4, 32, dtype=BF, device="cuda"))),
        (q, kc, vc, plan, dict(lse=torch.zeros(2, 4, dtype=BF, device="cuda"))),
    ]
    for qq, k2, v2, p, kw in bad:
        with pytest.raises(ValueError):
            sa.sparse_attn_tree_fwd(qq, k2, v2, p, **kw)
    with pytest.raises(sa.SparseAttnError):                                 # a page of 24 tokens
        sa.sparse_attn_tree_fwd(q, torch.zeros(4, 24, 2, 64, dtype=BF, device="cuda"),
                                torch.zeros(4, 24, 2, 64, dtype=BF, device="cuda"), plan)
    with pytest.raises(sa.SparseAttnError):
        sa.sparse_attn_tree_fwd(q, kc, vc, plan, scale=math.nan)
    big = sa.CachePlan(table=dev_ints([[0] * 64]), lens=dev_ints([3]), starts=dev_ints([0, 2]))
    with pytest.raises(sa.SparseAttnError) as e:
        sa.sparse_attn_tree_fwd(q, kc, vc, big, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    with pytest.raises(ValueError):
        sa.sparse_attn_cache_write(q[:, :1], q[:, :1], dev_ints([0, 1]), kc, vc)
    with pytest.raises(ValueError):
        sa.sparse_attn_cache_write(q[:, :2], q[:, :2], dev_ints([0]), kc, vc)
    with pytest.raises(ValueError):
        sa.sparse_attn_cache_accept(kc, vc, plan, dev_ints([[0]]), dev_ints([0, 1]))
    one = dev_ints([1])
    with pytest.raises(ValueError):                                         # parents without masks
        sa.sparse_attn_cache_plan(one, one, dev_ints([[0]]), one, one, one, 1, 16, parents=one)
    with pytest.raises(sa.SparseAttnError):                                 # outputs on top of the inputs
        p = sa.sparse_attn_cache_plan(one, one, dev_ints([[0]]), one, one, one, 1, 16)
        sa.sparse_attn_cache_plan(one, one, dev_ints([[0]]), p.held, one, p.nfree, 1, 16, out=p)
    torch.cuda.synchronize()
    sa.sparse_attn_device_error()
