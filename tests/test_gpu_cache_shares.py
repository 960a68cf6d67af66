"""Attention over the paged cache where a call's work is cut: tiles of two chains with and
without rows in the second, many short pieces, more requests than threads, pieces of
all sizes, outputs of other alignments, calls one after another on one stream."""
import math
import random
import threading

import pytest
import torch

from oracle import paged_cache_oracle as orc
from tests.test_gpu_cache import BF, HF, cache_of, check_attention, dev_ints, no_device_error, random_mask

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import free_block_sparse_mean_b200 as sa


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("kind", [None, "tree", "any"])
def test_two_chains_and_one_in_one_call(kind, d, dtype):
    """Tiles sized for 256 rows; requests with rows for one chain, for both, for parts of
    the second and for several tiles, and some without new tokens."""
    G, Hkv = 4, 2
    new = [70, 1, 0, 33, 64, 32, 5, 31, 0, 65, 100]
    ctx = [3, 200, 9, 0, 64, 127, 511, 63, 0, 1, 30]
    words = 4 if kind else 0
    check_attention(ctx, new, 32, G * Hkv, Hkv, d, dtype, mask=random_mask(new, words, 3, kind) if kind else None,
                    words=words, max_new=100, seed=d)


@pytest.mark.parametrize("max_new", [0, 1, 64])
def test_tiles_sized_for_other_numbers_of_tokens(max_new):
    """max_new only sizes the tiles: too small, too large or not given, the rows are the same."""
    check_attention([300, 10, 77], [40, 3, 17], 16, 8, 2, 128, BF, max_new=max_new)


@pytest.mark.parametrize("T,max_new", [(1, 1), (2, 40)])
def test_many_one_block_pieces(T, max_new):
    """Shares of dozens of one-block tiles: every ring wraps several times."""
    rng = random.Random(T)
    R = 260
    ctx = [rng.randint(0, 60) for _ in range(R)]
    new = [T] * R
    check_attention(ctx, new, 16, 12, 3, 64, HF, max_new=max_new)
    check_attention(ctx[:150], new[:150], 64, 8, 8, 128, BF, max_new=max_new)


@pytest.mark.parametrize("R,Hq,Hkv,max_new", [(257, 1, 1, 1), (700, 2, 1, 1), (1100, 4, 2, 70)])
def test_more_requests_than_threads(R, Hq, Hkv, max_new):
    """A thread places several requests on the line, most of them empty in one stretch."""
    rng = random.Random(R)
    ctx = [rng.randint(0, 200) for _ in range(R)]
    new = [rng.choice([0, 1, 1, 2]) if not R // 3 < r < R // 2 else 0 for r in range(R)]
    if max_new > 2:
        new[R - 2] = max_new
    check_attention(ctx, new, 32, Hq, Hkv, 64, BF, max_new=max_new)


@pytest.mark.parametrize("Hq,Hkv,T,max_new,ctx", [
    (1, 1, 1, 1, 30000),       # one row, a piece for nearly every CTA
    (16, 1, 1, 1, 9000),
    (5, 1, 7, 7, 9000),        # 35 rows: a warp joins a row alone
    (2, 2, 150, 150, 3000)])
def test_one_request_over_all_shares(Hq, Hkv, T, max_new, ctx):
    check_attention([ctx], [T], 64, Hq, Hkv, 128, BF, max_new=max_new, seed=T)


def test_nothing_to_do():
    """No new token at all, and no request granted any: nothing is written."""
    check_attention([5, 70], [0, 0], 16, 4, 2, 64, BF, pad=3)
    check_attention([5, 70], [2, 300], 16, 4, 2, 64, BF, granted=[0, 0], max_new=300)


def test_rows_that_are_16_byte_aligned_only():
    """Rows of O in a wider buffer, 16 bytes behind a 32-byte boundary."""
    kc, vc, table = cache_of([100, 3000], [3, 3], 64, 2, 128, BF, 1)
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([100, 3000]), starts=dev_ints([0, 3, 6]), max_new=3)
    q = torch.randn(6, 4, 128, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    want = sa.sparse_attn_tree_fwd(q, kc.cuda(), vc.cuda(), plan)
    wide = torch.full((6, 4, 144), 7.0, dtype=BF, device="cuda")
    got = sa.sparse_attn_tree_fwd(q, kc.cuda(), vc.cuda(), plan, out=wide[:, :, 8:136])
    assert torch.equal(got, want)
    assert torch.all(wide[:, :, :8] == 7.0) and torch.all(wide[:, :, 136:] == 7.0)
    no_device_error()


def test_requests_that_share_the_pages_of_a_prefix():
    page, shared = 16, 96
    kc, vc, table = cache_of([200, 200, 200], [2, 1, 4], page, 2, 64, HF, 5)
    for r in (1, 2):
        table[r][:shared // page] = table[0][:shared // page]
    check_attention([200, 200, 200], [2, 1, 4], page, 6, 2, 64, HF, caches=(kc, vc, table), max_new=4)


@pytest.mark.parametrize("T,max_new", [(1, 1), (20, 20), (90, 90)])
def test_values_that_are_not_finite_in_every_form(T, max_new):
    """One unseen infinite value in each request, in each of the kernel's forms and in pieces
    that begin and end in the tile: rows that do not see it are finite and right, rows
    that see it get it in its element alone."""
    ctx, R, page, Hkv, Hq, d = 700, 5, 16, 2, 8, 128
    rng = random.Random(T)
    kc, vc, table = cache_of([ctx] * R, [T + 1] * R, page, Hkv, d, BF, T)
    new = [T + 1] * R
    words = (T + 32) // 32
    # new token j sees itself and the earlier ones, but for `hole`, which half of them see
    hole = [rng.randrange(T + 1) for _ in range(R)]
    rows, sees = [], []
    for r in range(R):
        for t in range(T + 1):
            bits = (1 << (t + 1)) - 1
            if t % 2 == 0:
                bits &= ~(1 << hole[r])
            sees.append(bool(bits >> hole[r] & 1))
            rows.append([(bits >> (32 * w)) & 0xffffffff for w in range(words)])
    rows = [[x - (1 << 32) if x >> 31 else x for x in row] for row in rows]
    for r in range(R):
        at = ctx + hole[r]
        vc[table[r][at // page], at % page, 1, 3] = math.inf
    starts = [r * (T + 1) for r in range(R + 1)]
    q = torch.randn(starts[-1], Hq, d, generator=torch.Generator().manual_seed(T)).to(BF)
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([ctx] * R), starts=dev_ints(starts), mask=dev_ints(rows),
                        max_new=max_new + 1)
    o = sa.sparse_attn_tree_fwd(q.cuda(), kc.cuda(), vc.cuda(), plan).cpu()
    no_device_error()
    clean = vc.clone()
    clean[torch.isinf(clean)] = 0
    ref, _, a, _ = orc.tree_attention(q, kc, clean, table, [ctx] * R, starts, new, rows, d ** -0.5)
    hurt = torch.tensor(sees)[:, None, None] & (torch.arange(Hq) >= 4)[None, :, None] & (torch.arange(d) == 3)
    assert torch.all(o[hurt] == math.inf)
    # u a for P, u |o| for the result, a twentieth of u a for all that is fp32
    tol = 2.0 ** -8 * (1.05 * a + ref.abs()) + 1e-6
    assert torch.all(((o.double() - ref).abs() <= tol)[~hurt])


def test_calls_one_after_another_with_changing_inputs():
    """Inputs, lengths and a common workspace rewritten between calls on one stream, without a
    wait on the host: each call sees what was before it, and what is behind it waits."""
    kc, vc, table = cache_of([900, 400], [8, 8], 32, 2, 64, BF, 7, fill=0.0)
    kc, vc, table = kc.cuda(), vc.cuda(), dev_ints(table)
    g = torch.Generator().manual_seed(2)
    qs = [torch.randn(16, 8, 64, generator=g).to(BF).cuda() for _ in range(6)]
    lens = [dev_ints([900 - 50 * i, 400 - 60 * i]) for i in range(6)]
    forms = [dict(max_new=8), dict(max_new=1), dict(max_new=64)]

    def plan(now, form):
        return sa.CachePlan(table=table, lens=now, starts=dev_ints([0, 8, 16]), **form)
    want = []
    for q, now, form in zip(qs, lens, forms * 2):
        want.append(sa.sparse_attn_tree_fwd(q, kc, vc, plan(now, form)).clone())
        torch.cuda.synchronize()
    size = max(sa.sparse_attn_tree_workspace_size(qs[0], kc, vc, plan(lens[0], f)) for f in forms)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    q, now, out = torch.empty_like(qs[0]), torch.empty_like(lens[0]), torch.empty_like(qs[0])
    plans = [plan(now, f) for f in forms]
    for _ in range(5):
        got = []
        for i in range(6):
            q.copy_(qs[i])
            now.copy_(lens[i])
            sa.sparse_attn_tree_fwd(q, kc, vc, plans[i % 3], out=out, workspace=ws)
            q.fill_(math.nan)
            now.fill_(-1)
            ws.fill_(255)
            got.append(out.clone())
            out.fill_(7.0)
        for x, w in zip(got, want):
            assert torch.equal(x, w)
    no_device_error()


def test_a_captured_step_with_a_common_workspace():
    """Layers of one captured step share a workspace; replays with other lengths match calls."""
    kc, vc, table = cache_of([500, 60, 7], [4, 4, 4], 64, 2, 128, HF, 3, fill=0.0)
    kc, vc, table = kc.cuda(), vc.cuda(), dev_ints(table)
    g = torch.Generator().manual_seed(4)
    qs = [torch.randn(12, 8, 128, generator=g).to(HF).cuda() for _ in range(3)]
    lens = dev_ints([500, 60, 7])
    p = sa.CachePlan(table=table, lens=lens, starts=dev_ints([0, 4, 8, 12]), max_new=4)
    ws = torch.empty(sa.sparse_attn_tree_workspace_size(qs[0], kc, vc, p), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(q) for q in qs]

    def step():
        for q, o in zip(qs, outs):
            sa.sparse_attn_tree_fwd(q, kc, vc, p, out=o, workspace=ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for now in ([500, 60, 7], [1, 60, 0], [499, 0, 3]):
        lens.copy_(torch.tensor(now, dtype=torch.int32))
        want = [sa.sparse_attn_tree_fwd(q, kc, vc, p) for q in qs]
        for o in outs:
            o.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    no_device_error()


def test_write_and_accept_at_the_edges():
    """One token, one head; a step without rows; requests that accept all, none or the last."""
    kc = torch.zeros(2, 16, 1, 64, dtype=BF, device="cuda")
    vc = torch.zeros_like(kc)
    k = torch.randn(1, 1, 64).to(BF).cuda()
    sa.sparse_attn_cache_write(k, 2 * k, dev_ints([31]), kc, vc)
    assert torch.equal(kc[1, 15], k[0]) and torch.equal(vc[1, 15], 2 * k[0])
    assert kc.count_nonzero() == k.count_nonzero()
    sa.sparse_attn_cache_write(k[:0], k[:0], dev_ints([]), kc, vc)
    kc, vc, table = cache_of([15] * 4, [9] * 4, 16, 2, 64, HF, 6, fill=0.0)
    acc = [list(range(9)), [0] * 9, [8] + [0] * 8, [0, 8] + [0] * 7]
    taken = [9, 0, 1, 2]
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([15] * 4), starts=dev_ints([0, 9, 18, 27, 36]))
    kg, vg = kc.cuda(), vc.cuda()
    sa.sparse_attn_cache_accept(kg, vg, plan, dev_ints(acc), dev_ints(taken))
    no_device_error()
    assert torch.equal(kg.cpu(), orc.accept(kc, table, [15] * 4, acc, taken))
    assert torch.equal(vg.cpu(), orc.accept(vc, table, [15] * 4, acc, taken))


def test_offsets_behind_32_bits():
    """A pool of more than 2^31 elements: rows written, attended to and moved in its last pages
    give what they give in a small pool."""
    page, H, d, T = 16, 8, 128, 12
    pages = (1 << 31) // (page * H * d) + 40
    g = torch.Generator().manual_seed(9)
    k, v = (torch.randn(50 + T, H, d, generator=g).to(BF).cuda() for _ in range(2))
    q = torch.randn(T, 2 * H, d, generator=g).to(BF).cuda()
    acc, taken = dev_ints([[1, 4, 5, 11]]), dev_ints([4])
    results = []
    for pool, ids in ((8, [3, 1, 6, 0]), (pages, [pages - 1, pages - 7, pages // 2 + 1, pages - 2])):
        kc, vc = (torch.empty(pool, page, H, d, dtype=BF, device="cuda") for _ in range(2))
        slots = [ids[i // page] * page + i % page for i in range(50 + T)]
        sa.sparse_attn_cache_write(k, v, dev_ints(slots), kc, vc)
        plan = sa.CachePlan(table=dev_ints([ids]), lens=dev_ints([50]), starts=dev_ints([0, T]), max_new=T)
        o = sa.sparse_attn_tree_fwd(q, kc, vc, plan)
        sa.sparse_attn_cache_accept(kc, vc, plan, acc, taken)
        no_device_error()
        at = torch.tensor(slots[:54])
        results.append((o, kc.view(-1, H, d)[at.cuda()], vc.view(-1, H, d)[at.cuda()]))
        del kc, vc
    for x, y in zip(*results):
        assert torch.equal(x, y)
    moved = torch.cat([k[:50], k[50 + torch.tensor([1, 4, 5, 11])]])
    assert torch.equal(results[1][1], moved)


def test_captured_behind_copies_and_joined_streams():
    """A captured call whose inputs come from a copy on the same stream and from another stream
    that joins right before it, and whose output another stream reads."""
    kc, vc, table = cache_of([300, 9], [3, 3], 32, 2, 64, BF, 11, fill=0.0)
    kc, vc = kc.cuda(), vc.cuda()
    g = torch.Generator().manual_seed(5)
    qs = [torch.randn(6, 4, 64, generator=g).to(BF).cuda() for _ in range(2)]
    plan = sa.CachePlan(table=dev_ints(table), lens=dev_ints([300, 9]), starts=dev_ints([0, 3, 6]), max_new=3)
    want = [sa.sparse_attn_tree_fwd(q, kc, vc, plan) for q in qs]
    source, lens = torch.empty_like(qs[0]), dev_ints([300, 9])
    q = torch.zeros_like(source)
    plan.lens = torch.zeros_like(lens)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            plan.lens.copy_(lens)
        q.copy_(source)
        main.wait_stream(side)
        o = sa.sparse_attn_tree_fwd(q, kc, vc, plan)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            twice = o + o
        main.wait_stream(side)
        q.fill_(math.nan)
        plan.lens.fill_(-1)
    for i in (0, 1, 0):
        source.copy_(qs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[i]) and torch.equal(twice, want[i] + want[i])
    no_device_error()


def test_calls_from_two_threads():
    """Threads with streams of their own; the first calls of a form may come from both at once."""
    kc, vc, table = cache_of([600, 50], [5, 40], 16, 2, 128, HF, 12, fill=0.0)
    kc, vc, table = kc.cuda(), vc.cuda(), dev_ints(table)
    q = torch.randn(45, 4, 128, generator=torch.Generator().manual_seed(6)).to(HF).cuda()
    plans = [sa.CachePlan(table=table, lens=dev_ints([600, 50]), starts=dev_ints([0, 5, 45]), max_new=m) for m in (5, 64)]
    got = [[], []]
    torch.cuda.synchronize()

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got[i].append(sa.sparse_attn_tree_fwd(q, kc, vc, plans[i]))
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for i in range(2):
        want = sa.sparse_attn_tree_fwd(q, kc, vc, plans[i])
        assert len(got[i]) == 20 and all(torch.equal(o, want) for o in got[i])
    no_device_error()
