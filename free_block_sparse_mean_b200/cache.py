"""Paged cache: decoding and drafting steps over cached keys and values.

Binding of the C calls of the same names (include/sparse_attn.h): tensors are checked
and marshalled, the kernels run on the tensors' device and the current torch stream.

    plan = sparse_attn_cache_plan(lens, new, table, held, free_pages, nfree, n, page_size,
                                  parents=parents, mask_words=2)
    for each layer:
        sparse_attn_cache_write(k, v, plan.slots, k_cache, v_cache)
        o = sparse_attn_tree_fwd(q, k_cache, v_cache, plan)
    sparse_attn_cache_accept(k_caches, v_caches, plan, accepted, taken)
    lens += taken                            # a step of prompts: lens += plan.granted, no accept
    held, nfree = plan.held, plan.nfree
    lens.masked_fill_(new < 0, 0)            # new < 0 ended a request: its row starts anew

A cache is a bf16 or fp16 CUDA tensor [pages, page_size, Hkv, d] (any strides with d
contiguous, so a transposed [pages, Hkv, page_size, d] fits), pages of 16, 32, 64,
128 or 256 tokens, d 64 or 128. Lengths, counts, tables and masks are int32 on the
same device. Nothing here waits for the GPU, so the calls can be captured into a
graph and replayed with other contents of the same buffers.
"""
from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import SaCache, SaStep, SparseAttnError

_DTYPES = {torch.bfloat16: _lib.SA_BF16, torch.float16: _lib.SA_F16}


@dataclass
class CachePlan:
    """A step over the cache: the output of sparse_attn_cache_plan, or put together by
    the caller (then table, lens and starts are needed).

    table      int32 [R, width]  page ids of each request
    lens       int32 [R]         tokens in the cache before the step's
    starts     int32 [R + 1]     request r's new tokens are rows starts[r]..starts[r+1]-1
    granted    int32 [R]         only the first granted[r] of them exist, or None: all
    mask       int32 [n, words]  bit j of a row: its token sees new token j of the request;
                                 None: it sees the request's new tokens up to itself
    slots      int32 [n]         slot of each new token, -1 for none
    positions  int32 [n]         place in the sequence (lens + depth in the tree)
    held       int32 [R]         pages in each table row, for the next step
    nfree      int32 [1]         ids on the free list, for the next step
    free_pages int32 [pages]     the free list
    max_new    int               the most new tokens of a request if known (0: not known, about
                                 the mean); only sizes the attention's tiles, so it is worth
                                 giving where requests differ much
    """
    table: torch.Tensor
    lens: torch.Tensor
    starts: torch.Tensor
    granted: Optional[torch.Tensor] = None
    mask: Optional[torch.Tensor] = None
    slots: Optional[torch.Tensor] = None
    positions: Optional[torch.Tensor] = None
    held: Optional[torch.Tensor] = None
    nfree: Optional[torch.Tensor] = None
    free_pages: Optional[torch.Tensor] = None
    max_new: int = 0


# The checks below are written for the host's time: a step of small requests costs its calls,
# not its kernels (a plan of 64 requests 4 us of 18), and a check that passes is one
# expression. What it refuses is looked at again for the message.
_I32 = torch.int32


def _launch(name: str, index: int, call, *args):
    """The C call on the GPU's current torch stream (no device switch if it is the current one).
    torch._C's functions spare the host what torch.cuda's wrap around them; a torch without CUDA
    does not have them, so they are looked up here and not at import."""
    c = torch._C
    if c._cuda_getDevice() == index:
        st = call(*args, c._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            st = call(*args, c._cuda_getCurrentRawStream(index))
    if st != _lib.SA_OK:
        raise SparseAttnError(name, st, _lib.load())


def _ints(name: str, t: torch.Tensor, shape, index: int):
    """t as a contiguous int32 tensor of the shape on the GPU; its address."""
    if not isinstance(t, torch.Tensor) or t.dtype is not _I32 or t.shape != shape or t.get_device() != index \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)} on cuda:{index}")
    return t.data_ptr()


def _rows(name: str, t: torch.Tensor, dtype, index: int):
    """t as rows [n, heads, d] of the type on the GPU; its address."""
    if t.dim() != 3 or t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be [n, heads, d] in the cache's type on its device")
    return _strides(name, t)


def _strides(name: str, t: torch.Tensor):
    """d contiguous, every other step a positive multiple of 8 elements, 16-byte base (the address returned)."""
    ptr, shape = t.data_ptr(), t.shape
    if ptr & 15 or not (t.is_contiguous() and shape[-1] & 7 == 0):
        st = t.stride()
        if ptr & 15 or st[-1] != 1 or any(x <= 0 or x & 7 for x, e in zip(st[:-1], shape) if e > 1):
            raise ValueError(f"{name} must have a contiguous last dimension, strides that are positive multiples of 8 "
                             "elements and a 16-byte aligned base")
    return ptr


def _sizes(any_of: int):
    """The C calls take sizes in 32 bits, and ctypes would drop the bits above: refuses the OR of
    sizes of which one needs more. (Rows of heads do not fit into memory before that.)"""
    if not -0x80000000 <= any_of <= 0x7fffffff:
        raise ValueError("a size is out of range (2^31 or more)")


def _same_layout(a: torch.Tensor, b: torch.Tensor) -> bool:
    x, y = a.stride(), b.stride()
    return x == y or all(i == j for i, j, e in zip(x, y, a.shape) if e > 1)


def _cache(k: torch.Tensor, v: torch.Tensor, dims: int = 4):
    """The caches' layout, their addresses and their GPU."""
    dtype, index, shape = _DTYPES.get(k.dtype), k.get_device(), k.shape
    if dtype is None or index < 0:
        raise ValueError("a cache must be a bf16 or fp16 CUDA tensor")
    if len(shape) != dims or v.shape != shape or v.dtype is not k.dtype or v.get_device() != index \
            or not _same_layout(k, v):
        raise ValueError("the caches must be [pages, page_size, Hkv, d] of one type, shape and layout")
    if 0 in shape:
        raise ValueError("the caches must not be empty")
    kp, vp = _strides("the cache", k), _strides("the cache", v)
    pages, page, heads, d = shape[-4:]
    ps, ts, hs, _ = k.stride()[-4:]
    return SaCache(pages, page, heads, d, dtype, ps if pages > 1 else page * heads * d, ts,
                   hs if heads > 1 else d), kp, vp, index


def _step(plan: CachePlan, n: int, index: int, masked: bool = True) -> SaStep:
    table, granted, mask, words = plan.table, plan.granted, None, 0
    if table.dim() != 2:
        raise ValueError("the plan's table must be [R, width]")
    R, width = shape = table.shape
    max_new = int(plan.max_new)
    _sizes(R | n | width | max_new)
    if granted is not None:
        granted = _ints("the plan's granted", granted, (R,), index)
    if masked and plan.mask is not None:
        words = plan.mask.shape[-1]
        mask = _ints("the plan's mask", plan.mask, (n, words), index)
    return SaStep(R, n, width, max_new, words, _ints("the plan's starts", plan.starts, (R + 1,), index),
                  _ints("the plan's lens", plan.lens, (R,), index), granted,
                  _ints("the plan's table", table, shape, index), mask)


def sparse_attn_cache_plan(lens: torch.Tensor, new_tokens: torch.Tensor, table: torch.Tensor, held: torch.Tensor,
                           free_pages: torch.Tensor, nfree: torch.Tensor, n: int, page_size: int, *,
                           parents: Optional[torch.Tensor] = None, mask_words: int = 0, max_new: int = 0,
                           out: Optional[CachePlan] = None) -> CachePlan:
    """Pages, block table, slots, positions and tree masks of a step, from the requests'
    lengths, in one launch.

    lens, new_tokens, held: int32 [R]; table: int32 [R, width] and free_pages: int32
    [pages], both updated in place; nfree: int32 [1]. A negative new_tokens[r] ends request
    r and returns its pages; the caller sets its lens to 0. n rows are planned (at least the
    new tokens' sum). mask_words > 0 (32 new tokens to a word, no request may have more) also
    makes the masks, from parents (int32 [n], each new token's parent among its request's,
    -1 for none) or for a chain.
    `out`, a plan of an earlier call of the same sizes, is written again (the plan's held
    and nfree must not be this call's inputs); the returned plan's table, lens and
    free_pages are the ones given."""
    lib = _lib.load()
    index = lens.get_device()
    if index < 0 or table.dim() != 2:
        raise ValueError("lens must be a CUDA tensor, table [R, width]")
    R, width = shape = table.shape
    vec = (R,)
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be [pages]")
    n, mask_words, page_size, max_new = int(n), int(mask_words), int(page_size), int(max_new)
    _sizes(R | width | free_pages.shape[0] | n | mask_words | page_size | max_new)
    if n < 1 or mask_words < 0:
        raise ValueError("n must be at least 1 and mask_words at least 0")
    ins = (_ints("lens", lens, vec, index), _ints("new_tokens", new_tokens, vec, index), _ints("held", held, vec, index),
           _ints("nfree", nfree, (1,), index), _ints("free_pages", free_pages, free_pages.shape, index),
           _ints("table", table, shape, index))
    tree = None                                  # (the tensor itself stays referred to)
    if parents is not None:
        if mask_words == 0:
            raise ValueError("parents needs mask_words")
        tree = _ints("parents", parents, (n,), index)
    if out is None:
        sizes = [R + 1, R, R, 1, n, n, n * mask_words]     # one buffer: an allocation costs more than a view
        starts, granted, held_out, nfree_out, slots, positions, mask = \
            lens.new_empty(sum(sizes)).split_with_sizes(sizes)
        out = CachePlan(table, lens, starts, granted, mask.view(n, mask_words) if mask_words else None, slots,
                        positions, held_out, nfree_out, free_pages, max_new)
    else:
        for name, t, want in (("starts", out.starts, (R + 1,)), ("granted", out.granted, vec), ("slots", out.slots, (n,)),
                              ("positions", out.positions, (n,)), ("held", out.held, vec),
                              ("nfree", out.nfree, (1,))):
            _ints(f"out.{name}", t, want, index)
        if mask_words:
            _ints("out.mask", out.mask, (n, mask_words), index)
        else:
            out.mask = None
        out.table, out.lens, out.free_pages, out.max_new = table, lens, free_pages, max_new
    _launch("sparse_attn_cache_plan", index, lib.sparse_attn_cache_plan, *ins, tree, R, free_pages.shape[0],
            page_size, width, n, mask_words, out.held.data_ptr(), out.nfree.data_ptr(), out.starts.data_ptr(),
            out.granted.data_ptr(), out.slots.data_ptr(), out.positions.data_ptr(),
            out.mask.data_ptr() if mask_words else None)
    return out


def sparse_attn_cache_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                            v_cache: torch.Tensor) -> None:
    """Writes rows k, v [n, Hkv, d] to their slots (int32 [n], -1 for none) of the caches.
    k and v may be strided with d contiguous (one layout for both), e.g. a transposed
    [Hkv, n, d] or a part of a fused projection. Slots other than -1 must differ."""
    lib = _lib.load()
    c, kc, vc, index = _cache(k_cache, v_cache)
    dtype, shape = k_cache.dtype, k.shape
    kp, vp = _rows("k", k, dtype, index), _rows("v", v, dtype, index)
    n = shape[0]
    if shape[1:] != k_cache.shape[2:] or v.shape != shape:
        raise ValueError(f"k and v must be [n, {c.Hkv}, {c.d}]")
    if not _same_layout(k, v):
        raise ValueError("k and v must have the same strides")
    at = _ints("slots", slots, (n,), index)
    if n == 0:
        return
    tok, head, _ = k.stride()
    _launch("sparse_attn_cache_write", index, lib.sparse_attn_cache_write, kp, vp, tok, head, n, at, kc, vc, c)


def sparse_attn_tree_workspace_size(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                    plan: CachePlan) -> int:
    """Bytes of workspace sparse_attn_tree_fwd needs for these tensors."""
    c, _, _, index = _cache(k_cache, v_cache)
    return int(_lib.load().sparse_attn_tree_workspace_size(c, _step(plan, q.shape[0], index), q.shape[1]))


def sparse_attn_tree_fwd(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, plan: CachePlan,
                         scale: Optional[float] = None, *, out: Optional[torch.Tensor] = None,
                         lse: Optional[torch.Tensor] = None,
                         workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of the step's new tokens q [n, Hq, d] over the cache: each request's cached
    tokens and the new ones its mask rows name (one token, a drafted tree, or a chunk of
    a prompt), whose keys and values are in the cache already.

    Hq is a multiple of Hkv (query head h reads key head h // (Hq / Hkv)). lse, if
    given (float32 [n, Hq]), receives the natural log of the softmax sums. out may be
    strided as q may. Rows of tokens that do not exist keep what `out` held (they are
    undefined in a new one); a row that sees nothing is 0."""
    lib = _lib.load()
    c, kc, vc, index = _cache(k_cache, v_cache)
    dtype, shape = k_cache.dtype, q.shape
    qp = _rows("q", q, dtype, index)
    n, Hq, d = shape
    if d != k_cache.shape[3] or Hq < 1 or Hq % k_cache.shape[2]:
        raise ValueError("q must be [n, Hq, d] with the cache's d and Hq a multiple of its heads")
    if out is None:
        out = q.new_empty(shape)
        op = out.data_ptr()
    else:
        op = _rows("out", out, dtype, index)
        if out.shape != shape:
            raise ValueError("out must have q's shape")
    if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (n, Hq) or lse.get_device() != index
                            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 tensor [n, Hq] on q's device")
    s = _step(plan, n, index)
    if n == 0:
        return out
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        workspace = q.new_empty(lib.sparse_attn_tree_workspace_size(c, s, Hq), dtype=torch.uint8)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on q's device")
    q_tok, q_head, _ = q.stride()
    o_tok, o_head, _ = out.stride()
    _launch("sparse_attn_tree_fwd", index, lib.sparse_attn_tree_fwd, qp, q_tok, q_head, Hq, kc, vc, c, s, float(scale), op,
            o_tok, o_head, None if lse is None else lse.data_ptr(), workspace.data_ptr(), workspace.nbytes)
    return out


def sparse_attn_cache_accept(k_cache: torch.Tensor, v_cache: torch.Tensor, plan: CachePlan, accepted: torch.Tensor,
                             taken: torch.Tensor) -> None:
    """Moves the accepted new tokens' rows to the places behind each request's cached ones:
    accepted int32 [R, cols] holds their indices among the request's new tokens in
    ascending order, taken int32 [R] how many there are. The caches are one layer's
    ([pages, page_size, Hkv, d]) or all layers' ([layers, ...]). The requests' lengths
    grow by `taken` (the caller adds it to lens)."""
    lib = _lib.load()
    layers, layer_stride, dims = 1, 0, 4
    if k_cache.dim() == 5:
        layers, layer_stride, dims = k_cache.shape[0], k_cache.stride(0), 5
    c, kc, vc, index = _cache(k_cache, v_cache, dims)
    # rows that a request claims past the step's buffers are refused as in the attention; a plan
    # put together without them has no number to check
    rows = plan.slots if plan.slots is not None else plan.mask
    s = _step(plan, 0x7fffffff if rows is None else rows.shape[0], index, masked=False)
    if accepted.dim() != 2 or accepted.shape[1] < 1:
        raise ValueError("accepted must be [R, cols]")
    R, cols = s.R, accepted.shape[1]
    _sizes(cols)
    _launch("sparse_attn_cache_accept", index, lib.sparse_attn_cache_accept, kc, vc, c, layers, layer_stride, s,
            _ints("accepted", accepted, (R, cols), index), cols, _ints("taken", taken, (R,), index))
