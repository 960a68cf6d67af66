"""Paged cache at the limits its calls state: probabilities far below a row's largest, sizes
and counts at the ends of their ranges, numbers out of range."""
import ctypes
import math
import random
import time

import pytest
import torch

from oracle import paged_cache_oracle as orc
from tests.test_gpu_cache import (BF, HF, cache_of, check_attention, check_plan, dev_ints, no_device_error, plan_case,
                                  random_mask, run_plan)

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import free_block_sparse_mean_b200 as sa


@pytest.mark.parametrize("R,T,ctx,peak", [(1, 1, 30000, 17001), (300, 1, 12000, 5), (300, 1, 12000, 11990),
                                          (300, 40, 3000, 1501), (150, 90, 3000, 64)])
@pytest.mark.parametrize("gap", [17.5, 19.0, 20.5])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_many_small_probabilities_behind_one_peak(R, T, ctx, peak, gap, dtype):
    """A key that takes nearly all of the softmax and has V = 0, `gap` nats above all others:
    what they hold together is the result. e^-20.5 is 2^-29.6 of the largest probability. R
    requests read one request's pages, so many that most rows are in one piece.

    Bound: u a for P, u |o| for the result (u half a step), as every row's (2^-22 for ex2 and
    (d + 3) 2^-23 of sum |q||k| for a score, twice; fp32 sums keys 2^-23). In fp16 also 2^-31 of
    the largest V for each key (P is rounded by 2^-25 at most below 2^-14, the row's sum is 2^6
    or more) and 2^-25 of a result below 2^-14."""
    d, page = 64, 64
    g = torch.Generator().manual_seed(T)
    kc, vc, table = cache_of([ctx], [T], page, 1, d, dtype, T, fill=0.0)
    q = torch.zeros(T, 1, d, dtype=dtype)
    q[:, :, 0] = 1.0
    flat = torch.zeros(ctx + T, 1, d, dtype=dtype)
    flat[:, :, 0] = (-gap + 0.25 * torch.rand(ctx + T, 1, generator=g)).to(dtype)
    flat[peak, :, 0] = 0.0
    val = (0.5 + torch.rand(ctx + T, 1, d, generator=g)).to(dtype)
    val[peak] = 0.0
    at = torch.arange(ctx + T)
    ids = torch.tensor(table[0])[at // page].long()
    kc[ids, at % page], vc[ids, at % page] = flat, val
    plan = sa.CachePlan(table=dev_ints(table * R), lens=dev_ints([ctx] * R),
                        starts=dev_ints([T * r for r in range(R + 1)]), max_new=T)
    lse = torch.empty(R * T, 1, device="cuda")
    got = sa.sparse_attn_tree_fwd(q.cuda().repeat(R, 1, 1), kc.cuda(), vc.cuda(), plan, 1.0, lse=lse).cpu().double()
    no_device_error()
    o, ref_lse, a, smax = orc.tree_attention(q, kc, vc, table, [ctx], [0, T], [T], None, 1.0)
    u = torch.finfo(dtype).eps / 2
    e = (d + 3) * 2.0 ** -23 * smax[..., None] + 2.0 ** -22
    keys = ctx + T
    tol = u * a * (1 + u) + u * (o.abs() + u * a) + 2 * e * a + keys * 2.0 ** -23 * a
    if dtype == HF:
        tol = tol + keys * 2.0 ** -31 * 1.5 + 2.0 ** -25
    err = (got.view(R, T, 1, d) - o).abs()
    assert torch.all(err <= tol), f"worst {float((err / tol).max()):.2f} of the bound"
    e = (d + 3) * 2.0 ** -23 * smax + (keys + 8) * 2.0 ** -23 + 2.0 ** -22 * ref_lse.abs()
    assert torch.all((lse.cpu().double().view(R, T, 1) - ref_lse).abs() <= e)


@pytest.mark.parametrize("size", [40.0, 3000.0, 10000.0])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_scores_of_any_size_stay_finite(size, dtype):
    """Scores whose steps in fp32 pass those of the exponent (up to 2e7): no infinity or NaN,
    and every row within the range of its values."""
    ctx, T, page, d = 700, 5, 32, 64
    kc, vc, table = cache_of([ctx], [T], page, 1, d, dtype, 3)
    kc = (kc.float() * 40).to(dtype)
    q = (torch.randn(T, 2, d, generator=torch.Generator().manual_seed(1)) * size).to(dtype)
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([ctx]), starts=dev_ints([0, T]), max_new=T)
    lse = torch.empty(T, 2, device="cuda")
    got = sa.sparse_attn_tree_fwd(q.cuda(), kc.cuda(), vc.cuda(), plan, 1.0, lse=lse)
    no_device_error()
    assert torch.isfinite(got).all() and torch.isfinite(lse).all()
    assert float(got.float().abs().max()) <= float(vc.float().abs().max()) * 1.01


@pytest.mark.parametrize("known", ["slots", "mask", None])
def test_accept_refuses_rows_that_are_not_the_steps(known):
    """Starts past the step's rows, negative or falling: the request keeps its rows and is
    flagged, as the attention does. (Without slots and mask the number of rows is not known.)"""
    n, R, T = 24, 3, 8
    kc, vc, table = cache_of([20] * R, [T] * R, 16, 2, 64, BF, 4)
    acc, taken = [[1, 3, 5]] * R, [3] * R
    extra = {} if known is None else {known: dev_ints([0] * n) if known == "slots" else dev_ints([[0]] * n)}
    for starts, moved, want in (([0, 8, 16, 24], [0, 1, 2], 0), ([0, 8, 16, 25], [0, 1] if known else [0, 1, 2], 4),
                                ([-8, 0, 8, 16], [1, 2], 4), ([0, 8, 4, 16], [0, 2], 4)):
        want = 0 if len(moved) == R else want
        kg, vg = kc.cuda(), vc.cuda()
        plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([20] * R), starts=dev_ints(starts), **extra)
        sa.sparse_attn_cache_accept(kg, vg, plan, dev_ints(acc), dev_ints(taken))
        torch.cuda.synchronize()
        assert sa.sparse_attn_device_error() == want, starts
        rows = [table[r] for r in moved]
        assert torch.equal(kg.cpu(), orc.accept(kc, rows, [20] * len(moved), acc, taken)), starts
        assert torch.equal(vg.cpu(), orc.accept(vc, rows, [20] * len(moved), acc, taken)), starts


def test_plan_returns_more_pages_than_ints_count():
    """Ended requests that claim R * width pages, nearly 2^31, behind a full list: their sum and
    the list's length pass 2^31. Nothing is written and the counts are flagged."""
    R, pages = 8192, 100000
    width = (2 ** 31 - 1) // R
    assert R * width < 2 ** 31 < R * width + pages
    table = torch.zeros(R, width, dtype=torch.int32, device="cuda")
    free = torch.arange(pages, dtype=torch.int32, device="cuda")
    guard = torch.full((R,), width, dtype=torch.int32, device="cuda")
    p = sa.sparse_attn_cache_plan(dev_ints([0] * R), dev_ints([-1] * R), table, guard, free, dev_ints([pages]), 4, 16)
    torch.cuda.synchronize()
    assert sa.sparse_attn_device_error() == 4
    assert torch.equal(free, torch.arange(pages, dtype=torch.int32, device="cuda")) and int(p.nfree) == pages
    # room for 7 more: the first request's pages fill the list
    table[0, :8] = dev_ints([41, 42, 43, 44, 45, 46, 47, 48])
    p = sa.sparse_attn_cache_plan(dev_ints([0] * R), dev_ints([-1] * R), table, guard, free, dev_ints([pages - 7]), 4, 16)
    torch.cuda.synchronize()
    assert sa.sparse_attn_device_error() == 4
    assert free[pages - 8:].tolist() == [pages - 8, 41, 42, 43, 44, 45, 46, 47] and int(p.nfree) == pages
    assert p.granted.count_nonzero() == 0 and p.held.count_nonzero() == 0


def test_a_workspace_that_is_a_view_of_less_memory_is_refused():
    """A broadcast tensor's nbytes count the same bytes again and again."""
    kc, vc, table = cache_of([100], [2], 16, 2, 64, BF, 4, fill=0.0)
    kc, vc = kc.cuda(), vc.cuda()
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([100]), starts=dev_ints([0, 2]))
    q = torch.zeros(2, 4, 64, dtype=BF, device="cuda")
    size = sa.sparse_attn_tree_workspace_size(q, kc, vc, plan)
    byte = torch.zeros(1, dtype=torch.uint8, device="cuda")
    for ws in (byte.expand(size), torch.zeros(size, 2, dtype=torch.uint8, device="cuda")[:, 0]):
        with pytest.raises(ValueError):
            sa.sparse_attn_tree_fwd(q, kc, vc, plan, workspace=ws)
    want = sa.sparse_attn_tree_fwd(q, kc, vc, plan)
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    assert torch.equal(sa.sparse_attn_tree_fwd(q, kc, vc, plan, workspace=ws), want)
    no_device_error()


def test_sizes_past_32_bits_are_refused():
    """The C calls' sizes are 32 bits wide; ctypes drops what is above them without a word."""
    one = dev_ints([1])
    call = lambda n=4, page=16, **kw: sa.sparse_attn_cache_plan(dev_ints([0]), one, dev_ints([[0]]), dev_ints([0]),
                                                                dev_ints([0]), one, n, page, **kw)
    p = call()
    # written again into buffers of 4 rows: a wide n must not be taken for its low bits
    for kw in (dict(n=2 ** 32 + 4), dict(page=2 ** 32 + 16), dict(max_new=2 ** 32 + 1), dict(mask_words=2 ** 32)):
        with pytest.raises(ValueError):
            call(out=p if "page" in kw else None, **kw)
    kc = torch.zeros(2, 16, 1, 64, dtype=BF, device="cuda")
    p = call()
    p.max_new = 2 ** 32 + 1
    with pytest.raises(ValueError):
        sa.sparse_attn_tree_fwd(torch.zeros(4, 1, 64, dtype=BF, device="cuda"), kc, kc.clone(), p)
    p.max_new = 1
    sa.sparse_attn_tree_fwd(torch.zeros(4, 1, 64, dtype=BF, device="cuda"), kc, kc.clone(), p)
    no_device_error()


def out_of_pool(kc):
    """Sets bit 1 through a write to a slot outside the pool."""
    row = torch.ones(1, kc.shape[2], kc.shape[3], dtype=kc.dtype, device="cuda")
    sa.sparse_attn_cache_write(row, row, dev_ints([kc.shape[0] * kc.shape[1]]), kc, kc.clone())


def test_the_error_word_gathers_every_code_once():
    """Codes of kernels of different translation units come back together and are cleared; one set
    on another stream while the word is read is not lost."""
    kc = torch.zeros(1, 16, 1, 64, dtype=BF, device="cuda")
    no_device_error()
    sa.sparse_attn_selftest_wait_timeout(1000)
    out_of_pool(kc)
    sa.sparse_attn_cache_plan(dev_ints([-1]), dev_ints([1]), dev_ints([[0]]), dev_ints([0]), dev_ints([0]), dev_ints([1]),
                              1, 16)
    assert sa.sparse_attn_device_error() == 7 and sa.sparse_attn_device_error() == 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(100):
        with torch.cuda.stream(side):
            out_of_pool(kc)
        seen, stop = 0, time.monotonic() + 10
        while not seen and time.monotonic() < stop:
            seen = sa.sparse_attn_device_error()
        assert seen == 2
        torch.cuda.synchronize()
        assert sa.sparse_attn_device_error() == 0


def test_reading_the_error_word_is_a_launch_and_a_copy():
    """sparse_attention reads the word in every call: 2.4 times the host time of a tensor's
    item(), one small copy that waits. A read, a clear and a wait for each of the library's three
    translation units were 5.5 times it."""
    x = torch.zeros(1, dtype=torch.int32, device="cuda")

    def least(call):
        best = math.inf
        for _ in range(500):
            t = time.perf_counter()
            call()
            best = min(best, time.perf_counter() - t)
        return best
    for call in (x.item, sa.sparse_attn_device_error):
        call()
    assert least(sa.sparse_attn_device_error) < 3.4 * least(x.item)


@pytest.mark.parametrize("R,Hkv,G,T,max_new,d", [
    (1, 1, 8, 5, 5, 128),       # 40, 64, 128 and 256 rows of one head: a tile in dozens of pieces
    (1, 1, 64, 1, 1, 64),
    (1, 1, 8, 16, 16, 128),
    (1, 1, 4, 64, 64, 64),
    (1, 4, 8, 9, 9, 128),
    (9, 1, 33, 1, 1, 64),       # as many tiles as are looked for, and one more
    (10, 1, 33, 1, 1, 64),
    (1, 1, 8, 61, 5, 128),      # more tokens than max_new: more cut tiles than blocks for them
    (2, 2, 5, 40, 3, 64),
    (1, 1, 4, 300, 65, 64)])
def test_tiles_in_many_pieces(R, Hkv, G, T, max_new, d):
    ctx = [6000 - 100 * r for r in range(R)]
    check_attention(ctx, [T] * R, 64, G * Hkv, Hkv, d, BF, max_new=max_new, seed=T)
    if max_new == T and R == 1:
        words = (T + 31) // 32
        check_attention(ctx, [T], 64, G * Hkv, Hkv, d, HF, max_new=max_new, words=words,
                        mask=random_mask([T], words, 7, "any"))


def test_a_row_more_than_a_warp_costs_no_other_join():
    """One head's tile over a long cache, in a piece for nearly every CTA: 40 rows take little more
    than 32 do (a join that reads a row's pieces one after another took 55 us for 33)."""
    ctx, page, d = 100000, 64, 128
    kc, vc = (torch.randn(ctx // page + 2, page, 1, d, dtype=BF, device="cuda") for _ in range(2))
    table = torch.arange(ctx // page + 1, dtype=torch.int32, device="cuda")[None].contiguous()
    took = {}
    for T in (4, 5):
        q = torch.randn(T, 8, d, dtype=BF, device="cuda")
        plan = sa.CachePlan(table=table, lens=dev_ints([ctx]), starts=dev_ints([0, T]), max_new=T)
        out = torch.empty_like(q)
        sa.sparse_attn_tree_fwd(q, kc, vc, plan, out=out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(20):
                sa.sparse_attn_tree_fwd(q, kc, vc, plan, out=out)
        took[T] = math.inf
        for _ in range(10):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            took[T] = min(took[T], a.elapsed_time(b))
    no_device_error()
    assert took[5] < 1.4 * took[4], took


def test_the_documented_loop_with_requests_that_end():
    """Prompts, drafts, ended requests, empty rows and new prompts in their place, lengths moved on
    as the README has it: no call flags anything and every page stays in one place."""
    R, page, Hkv, d, T, width, pages = 4, 16, 1, 64, 6, 12, 40
    g = torch.Generator().manual_seed(1)
    caches = [torch.zeros(pages, page, Hkv, d, dtype=BF, device="cuda") for _ in range(2)]
    lens, held, nfree = dev_ints([0] * R), dev_ints([0] * R), dev_ints([pages])
    table, free = dev_ints([[0] * width] * R), dev_ints(torch.randperm(pages, generator=g).tolist())
    want = [0] * R

    def step(new, drafts):
        nonlocal lens, held, nfree
        n = max(1, sum(max(t, 0) for t in new))
        fresh = dev_ints(new)
        p = sa.sparse_attn_cache_plan(lens, fresh, table, held, free, nfree, n, page, mask_words=1 if drafts else 0)
        k = torch.randn(n, Hkv, d, generator=g).to(BF).cuda()
        sa.sparse_attn_cache_write(k, k, p.slots, *caches)
        sa.sparse_attn_tree_fwd(k.repeat(1, 2, 1), *caches, p)
        if drafts:
            taken = [min(max(t, 0), 1 + r) for r, t in enumerate(new)]
            sa.sparse_attn_cache_accept(*caches, p, dev_ints([list(range(T))] * R), dev_ints(taken))
            lens += dev_ints(taken)
        else:
            taken = [max(t, 0) for t in new]
            lens += p.granted
        held, nfree = p.held, p.nfree
        lens.masked_fill_(fresh < 0, 0)
        no_device_error()
        for r, t in enumerate(new):
            want[r] = 0 if t < 0 else want[r] + taken[r]
        assert lens.tolist() == want
        ids = [x for r in range(R) for x in table[r, :int(held[r])].tolist()] + free[:int(nfree)].tolist()
        assert sorted(ids) == list(range(pages))
    step([50, 3, 17, 100], False)
    step([T, T, 1, 0], True)
    step([T, -1, T, T], True)
    step([1, -1, T, -1], True)       # an empty row may stay negative
    step([-1, 0, 2, 0], True)        # or count 0, its length being 0
    step([30, 40, 5, 0], False)
    step([T, T, T, -1], True)


@pytest.mark.parametrize("R,tree", [(3100, True), (8192, False)])
def test_plans_of_many_requests(R, tree):
    """Sums over all requests in more shared memory than a kernel has without asking (48 KB hold
    some 3,000), up to the most requests of a call."""
    rng = random.Random(R)
    c = plan_case(rng, R, 16, tree, R // 10, top_len=60, top_new=20)
    p = run_plan(c)
    no_device_error()
    check_plan(p, c)


def test_plan_flags_page_ids_outside_the_pool():
    """An id on the free list or in a held column that is no page: its tokens get no slot and bit 1
    is set, all else is as planned."""
    page, width, pages = 16, 4, 8
    for where in ("free", "held"):
        for wrong in (-1, pages, 1 << 30):
            table = [[0, -5, -5, -5], [1, -5, -5, -5]]
            free = [2, 3, 4, 5, 6, 7, 0, 0]
            if where == "free":
                free[5] = wrong                     # the first one taken
            else:
                table[0][0] = wrong
            t, f = dev_ints(table), dev_ints(free)
            p = sa.sparse_attn_cache_plan(dev_ints([10, 3]), dev_ints([20, 2]), t, dev_ints([1, 1]), f, dev_ints([6]),
                                          22, page)
            torch.cuda.synchronize()
            assert sa.sparse_attn_device_error() == 2
            ref = orc.plan([10, 3], [20, 2], [1, 1], 6, free, table, None, page, 22, 0)
            bad = set(range(6)) if where == "held" else set(range(6, 20))   # places 10..15, 16..29
            want = [-1 if i in bad else s for i, s in enumerate(ref["slots"])]
            assert p.slots.tolist() == want and p.granted.tolist() == [20, 2] and int(p.nfree) == ref["nfree"][0]
            assert p.positions.tolist() == ref["positions"] and p.table[1].tolist() == ref["table"][1]


@pytest.mark.parametrize("T,layout", [(257, "nhd"), (1024, "hnd")])
def test_accept_of_many_rows(T, layout):
    """More accepted rows than threads, the most of a call, some requests granted fewer, a cache
    by head."""
    rng = random.Random(T)
    page, H, d, R = 32, 2, 64, 3
    ctx, new, granted = [5, 31, 0], [T + 6] * R, [T + 6, T + 6, 40]
    kc, vc, table = cache_of(ctx, new, page, H, d, HF, T, layout)
    taken = [T, 300 if T > 300 else 256, 40]
    acc = [sorted(rng.sample(range(g), m)) + [0] * (T - m) for g, m in zip(granted, taken)]
    gpu = lambda x: x.transpose(1, 2).contiguous().cuda().transpose(1, 2) if layout == "hnd" else x.cuda()
    kg, vg = gpu(kc), gpu(vc)
    assert kg.stride() == vg.stride() and (layout == "nhd") == kg.is_contiguous()
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints(ctx), starts=dev_ints([(T + 6) * r for r in range(R + 1)]),
                        granted=dev_ints(granted))
    sa.sparse_attn_cache_accept(kg, vg, plan, dev_ints(acc), dev_ints(taken))
    no_device_error()
    assert torch.equal(kg.cpu(), orc.accept(kc, table, ctx, acc, taken))
    assert torch.equal(vg.cpu(), orc.accept(vc, table, ctx, acc, taken))
    # a row that was not granted is none to accept: the request keeps its rows
    kg, vg = gpu(kc), gpu(vc)
    acc[2][39] = 40
    sa.sparse_attn_cache_accept(kg, vg, plan, dev_ints(acc), dev_ints(taken))
    torch.cuda.synchronize()
    assert sa.sparse_attn_device_error() == 4
    assert torch.equal(kg.cpu(), orc.accept(kc, table[:2], ctx[:2], acc, taken))


def test_accept_flags_page_ids_outside_the_pool():
    """A page id that is none, where a row comes from or goes to: the request keeps all its rows,
    the others move."""
    ctx, new, page = [14, 14, 14], [40] * 3, 16
    kc, vc, table = cache_of(ctx, new, page, 2, 64, BF, 9)
    acc, taken = [[1, 2, 30]] * 3, [3] * 3
    for column in (0, 2):                           # places 14.. go to pages 0 and 1; 44 comes from page 2
        for wrong in (-1, kc.shape[0], 1 << 30):
            t2 = [list(row) for row in table]
            t2[1][column] = wrong
            kg, vg = kc.cuda(), vc.cuda()
            plan = sa.CachePlan(table=dev_ints(t2), lens=dev_ints(ctx), starts=dev_ints([0, 40, 80, 120]))
            sa.sparse_attn_cache_accept(kg, vg, plan, dev_ints(acc), dev_ints(taken))
            torch.cuda.synchronize()
            assert sa.sparse_attn_device_error() == 2
            rest = [table[0], table[2]]
            assert torch.equal(kg.cpu(), orc.accept(kc, rest, [14, 14], acc, taken))
            assert torch.equal(vg.cpu(), orc.accept(vc, rest, [14, 14], acc, taken))


def test_attention_of_the_most_requests():
    rng = random.Random(2)
    R = 8192
    ctx = [rng.randint(0, 40) for _ in range(R)]
    new = [rng.choice([0, 1, 1, 2]) for _ in range(R)]
    check_attention(ctx, new, 16, 2, 1, 64, BF, max_new=2)


def test_places_up_to_the_limit():
    """Requests of 2^31 - 1025 tokens, nearly all in one page that their tables name again and
    again; a key in another page (in the middle, and the new token's own) takes the whole softmax."""
    page, d = 16, 64
    width = (2 ** 31 - 1025) // page
    L = width * page - 1
    kc, vc = (torch.zeros(5, page, 1, d, dtype=BF, device="cuda") for _ in range(2))
    vc[0] = 1.0
    table = torch.zeros(2, width, dtype=torch.int32, device="cuda")
    table[0, width // 2 + 1] = 1                    # the peak of the first request
    kc[1, 5], vc[1, 5] = 8.0, 2.0
    table[:, width - 1] = dev_ints([2, 3])          # where the new tokens lie, the last place
    kc[3, 15], vc[2, 15], vc[3, 15] = 8.0, 5.0, 3.0
    q = torch.ones(2, 1, d, dtype=BF, device="cuda")
    plan = sa.CachePlan(table=table, lens=dev_ints([L, L]), starts=dev_ints([0, 1, 2]), max_new=1)
    lse = torch.empty(2, 1, device="cuda")
    o = sa.sparse_attn_tree_fwd(q, kc, vc, plan, 1.0, lse=lse)
    no_device_error()
    # the other scores are 0, the peak's 512: e^-512 is nothing
    assert torch.all(o[0] == 2.0) and torch.all(o[1] == 3.0)
    assert torch.all((lse - 512.0).abs() <= 512 * 2.0 ** -22)
    plan.lens = dev_ints([L + 1, L])                # one place more than the table holds
    o = sa.sparse_attn_tree_fwd(q, kc, vc, plan, 1.0)
    torch.cuda.synchronize()
    assert sa.sparse_attn_device_error() == 4 and torch.all(o[1] == 3.0)


def test_a_launch_that_fails_fails_no_later_call():
    """A capture that something else has spoilt: the attention's launch into it is refused, and the
    calls behind it on the stream, out of the capture again, are not."""
    rt = ctypes.CDLL("libcudart.so.12")
    kc, vc, table = cache_of([100], [2], 16, 2, 64, BF, 4, fill=0.0)
    kc, vc = kc.cuda(), vc.cuda()
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([100]), starts=dev_ints([0, 2]))
    q = torch.randn(2, 4, 64, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    want, out = sa.sparse_attn_tree_fwd(q, kc, vc, plan), torch.zeros_like(q)
    ws = torch.empty(sa.sparse_attn_tree_workspace_size(q, kc, vc, plan), dtype=torch.uint8, device="cuda")
    slot, row = dev_ints([0]), torch.zeros(1, 2, 64, dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    handle, graph = ctypes.c_void_p(side.cuda_stream), ctypes.c_void_p()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        assert rt.cudaStreamBeginCapture(handle, 2) == 0             # relaxed
        assert rt.cudaStreamSynchronize(handle) != 0                 # no wait in a capture: it is spoilt
        with pytest.raises(sa.SparseAttnError) as e:
            sa.sparse_attn_tree_fwd(q, kc, vc, plan, out=out, workspace=ws)
        assert e.value.status == 4
        with pytest.raises(sa.SparseAttnError):
            sa.sparse_attn_device_error()
        assert rt.cudaStreamEndCapture(handle, ctypes.byref(graph)) != 0
        rt.cudaGetLastError()
        sa.sparse_attn_cache_write(row, row, slot, kc.clone(), vc.clone())
        sa.sparse_attn_tree_fwd(q, kc, vc, plan, out=out, workspace=ws)
    no_device_error()
    assert torch.equal(out, want)
