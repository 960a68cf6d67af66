"""Paged cache without a GPU: the C calls' checks of their arguments (none of these calls
gets past them) and the plain implementation's own invariants."""
import ctypes
import random

import pytest
import torch

import free_block_sparse_mean_b200 as sa
from free_block_sparse_mean_b200 import _lib
from oracle import paged_cache_oracle as orc

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
P = 1 << 20                                   # an aligned address that no call reads


def cache(**kw):
    f = dict(pages=4, page_size=16, Hkv=2, d=64, dtype=_lib.SA_BF16, page_stride=2048, token_stride=128, head_stride=64)
    f.update(kw)
    return _lib.SaCache(**f)


def step(**kw):
    f = dict(R=2, n=8, width=3, max_new=4, words=0, starts=P, lens=P, granted=None, table=P, mask=None)
    f.update(kw)
    return _lib.SaStep(**f)


def tree(c=None, s=None, **kw):
    a = dict(q=P, q_token=256, q_head=64, Hq=4, k=P, v=P, scale=0.1, o=P, o_token=256, o_head=64, lse=None, ws=P,
             ws_bytes=1 << 30)
    a.update(kw)
    return _lib.load().sparse_attn_tree_fwd(a["q"], a["q_token"], a["q_head"], a["Hq"], a["k"], a["v"], c or cache(),
                                            s or step(), a["scale"], a["o"], a["o_token"], a["o_head"], a["lse"], a["ws"],
                                            a["ws_bytes"], None)


@pytest.mark.parametrize("field,value,want", [
    ("pages", 0, INVALID), ("Hkv", 0, INVALID), ("page_size", 24, UNSUPPORTED), ("page_size", 8, UNSUPPORTED),
    ("page_size", 512, UNSUPPORTED), ("d", 96, UNSUPPORTED), ("d", 256, UNSUPPORTED), ("dtype", 2, UNSUPPORTED),
    ("Hkv", 65536, UNSUPPORTED), ("pages", 1 << 27, UNSUPPORTED), ("page_stride", 0, INVALID),
    ("page_stride", -2048, INVALID), ("token_stride", 124, INVALID), ("head_stride", 4, INVALID),
    ("page_stride", 1 << 38, INVALID)])
def test_caches_that_are_refused(field, value, want):
    lib, c = _lib.load(), cache(**{field: value})
    assert tree(c) == want
    assert lib.sparse_attn_cache_write(P, P, 128, 64, 8, P, P, P, c, None) == want
    assert lib.sparse_attn_cache_accept(P, P, c, 1, 0, step(), P, 4, P, None) == want
    assert lib.sparse_attn_tree_workspace_size(c, step(), 4) == 0


@pytest.mark.parametrize("field,value,want", [
    ("R", 0, INVALID), ("n", 0, INVALID), ("width", 0, INVALID), ("max_new", -1, INVALID), ("starts", None, INVALID),
    ("lens", None, INVALID), ("table", None, INVALID), ("starts", P + 2, INVALID), ("granted", P + 1, INVALID),
    ("words", 1, INVALID), ("R", 8193, UNSUPPORTED), ("width", 1 << 27, UNSUPPORTED), ("width", (1 << 27) - 64, UNSUPPORTED)])
def test_steps_that_are_refused(field, value, want):
    s = step(**{field: value})
    assert tree(s=s) == want
    assert _lib.load().sparse_attn_cache_accept(P, P, cache(), 1, 0, s, P, 4, P, None) == want


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(k=None), INVALID), (dict(q=P + 8), INVALID),
    (dict(o=P + 8), INVALID), (dict(lse=P + 2), INVALID), (dict(Hq=3), INVALID), (dict(Hq=0), INVALID),
    (dict(Hq=258), UNSUPPORTED), (dict(scale=0.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(q_token=0), INVALID), (dict(q_head=60), INVALID),
    (dict(o_token=-256), INVALID), (dict(ws=None), WORKSPACE), (dict(ws=P + 16), WORKSPACE), (dict(ws_bytes=64), WORKSPACE)])
def test_attention_calls_that_are_refused(kw, want):
    s = step(width=8)
    assert tree(s=s, **kw) == want


def test_masks_and_workspaces_that_do_not_fit():
    assert tree(s=step(mask=P, words=33)) == INVALID and tree(s=step(mask=P, words=0)) == INVALID
    lib = _lib.load()
    for new, hq in ((1, 2), (4, 4), (64, 8), (300, 64)):
        s = step(n=max(new, 8), max_new=new, width=100)
        size = lib.sparse_attn_tree_workspace_size(cache(), s, hq)
        # two pieces of a tile for each CTA that works: fp32 rows, their maximum and sum
        rows = min(new * hq // 2, (128 // (hq // 2)) * (hq // 2))
        chains = 2 if new * hq // 2 > rows else 1
        assert size >= 2 * (296 // chains) * chains * rows * (64 * 4 + 8)
        assert tree(s=s, Hq=hq, q_token=64 * hq, o_token=64 * hq, ws_bytes=size - 1) == WORKSPACE
    # without max_new the mean sizes the tiles, at least 32 rows; a mask's words bound them
    size = lambda **kw: lib.sparse_attn_tree_workspace_size(cache(), step(width=100, **kw), 8)      # 4 heads to a key head
    assert size(R=64, n=64, max_new=0) == size(R=64, n=64, max_new=8)
    assert size(R=4, n=200, max_new=0) == size(R=4, n=200, max_new=50)
    assert size(R=1, n=5, max_new=0) == size(R=1, n=5, max_new=5)
    assert size(R=1, n=64, max_new=0, mask=P, words=1) == size(R=1, n=64, max_new=32)
    # a request of one block is never cut
    assert lib.sparse_attn_tree_workspace_size(cache(), step(width=4), 4) == 256


def test_writes_plans_and_moves_that_are_refused():
    lib = _lib.load()
    w = lambda k=P, tok=128, head=64, n=8, slots=P: lib.sparse_attn_cache_write(k, P, tok, head, n, slots, P, P, cache(),
                                                                                None)
    assert w(k=None) == INVALID and w(k=P + 8) == INVALID and w(n=0) == INVALID and w(tok=0) == INVALID
    assert w(tok=100) == INVALID and w(head=4) == INVALID and w(slots=None) == INVALID and w(slots=P + 2) == INVALID
    a = lambda layers=1, stride=0, acc=P, cols=4, taken=P: lib.sparse_attn_cache_accept(
        P, P, cache(), layers, stride, step(), acc, cols, taken, None)
    assert a(layers=0) == INVALID and a(layers=2) == INVALID and a(layers=2, stride=100) == INVALID
    assert a(acc=None) == INVALID and a(cols=0) == INVALID and a(taken=P + 1) == INVALID and a(cols=1025) == UNSUPPORTED

    def plan(**kw):
        f = dict(lens=P, new=P, held=P, nfree=P, free=P, table=P, parents=None, R=2, pages=8, page=16, width=4, n=8,
                 words=0, held_out=P + 64, nfree_out=P + 64, starts=P, granted=P, slots=P, positions=P, mask=None)
        f.update(kw)
        return lib.sparse_attn_cache_plan(*f.values(), None)
    for kw, want in ((dict(lens=None), INVALID), (dict(slots=None), INVALID), (dict(held_out=P), INVALID),
                     (dict(nfree_out=P), INVALID), (dict(words=1), INVALID), (dict(parents=P), INVALID),
                     (dict(mask=P), INVALID), (dict(mask=P, words=33), INVALID), (dict(R=0), INVALID),
                     (dict(n=0), INVALID), (dict(table=P + 2), INVALID), (dict(page=48), UNSUPPORTED),
                     (dict(R=8193), UNSUPPORTED), (dict(width=1 << 30), UNSUPPORTED), (dict(pages=1 << 28), UNSUPPORTED)):
        assert plan(**kw) == want, kw


def test_tensors_on_the_cpu_are_refused():
    x = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    plan = sa.CachePlan(table=i[None], lens=i, starts=torch.zeros(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        sa.sparse_attn_tree_fwd(x[0, :1], x, x, plan)
    with pytest.raises(ValueError):
        sa.sparse_attn_cache_write(x[0, :1], x[0, :1], i, x, x)
    with pytest.raises(ValueError):
        sa.sparse_attn_cache_accept(x, x, plan, i[None], i)
    with pytest.raises(ValueError):
        sa.sparse_attn_cache_plan(i, i, i[None], i, i, i, 1, 16)


def test_the_plain_plan_keeps_every_page_in_one_place():
    rng = random.Random(3)
    R, page, width = 9, 16, 12
    pages = 60
    free, table, held, lens = list(range(pages)), [[-1] * width for _ in range(R)], [0] * R, [0] * R
    rng.shuffle(free)
    nfree = pages
    for _ in range(60):
        new = [rng.choice([-1, 0, 1, 7, 30]) for _ in range(R)]
        for r in range(R):
            if lens[r] + max(new[r], 0) > width * page:
                new[r] = -1
        n = max(1, sum(max(t, 0) for t in new))
        p = orc.plan(lens, new, held, nfree, free, table, None, page, n, 0)
        table, held, nfree, free = p["table"], p["held"], p["nfree"][0], p["free_pages"]
        for r in range(R):
            lens[r] = 0 if new[r] < 0 else lens[r] + p["granted"][r]
            assert held[r] * page >= lens[r]
        ids = [x for r in range(R) for x in table[r][:held[r]]] + free[:nfree]
        assert sorted(ids) == list(range(pages))
        live = [s for s in p["slots"] if s >= 0]
        assert len(set(live)) == len(live) == sum(p["granted"])
