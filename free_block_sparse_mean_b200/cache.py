"""Paged cache: decoding and drafting steps over cached keys and values.

Binding of the C calls of the same names (include/sparse_attn.h): tensors are checked
and marshalled, the kernels run on the tensors' device and the current torch stream.

    plan = sparse_attn_cache_plan(lens, new, table, held, free_pages, nfree, n, page_size,
                                  parents=parents, mask_words=2)
    for each layer:
        sparse_attn_cache_write(k, v, plan.slots, k_cache, v_cache)
        o = sparse_attn_tree_fwd(q, k_cache, v_cache, plan)
    sparse_attn_cache_accept(k_caches, v_caches, plan, accepted, taken)

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
    max_new    int               the most new tokens of a request if known (0: not known);
                                 only sizes the attention's tiles
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


_get_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


def _launch(name: str, dev, call, *args):
    """The C call on the device's current torch stream. A step of small requests costs its
    calls, not its kernels (4 us of 37 for a plan of 64 requests), so nothing here is
    done that the case does not need: no device switch on the current device, no views."""
    if _get_device() == dev.index:
        st = call(*args, _raw_stream(dev.index))
    else:
        with torch.cuda.device(dev):
            st = call(*args, _raw_stream(dev.index))
    if st != _lib.SA_OK:
        raise SparseAttnError(name, st, _lib.load())


def _ints(name: str, t: torch.Tensor, shape, dev):
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.shape != shape or t.device != dev \
            or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)} on {dev}")


def _rows(name: str, t: torch.Tensor, dtype, dev):
    if t.dim() != 3 or t.dtype is not dtype or t.device != dev:
        raise ValueError(f"{name} must be [n, heads, d] in the cache's type on its device")
    _strides(name, t)


def _strides(name: str, t: torch.Tensor):
    """d contiguous, every other step a positive multiple of 8 elements, 16-byte base."""
    good = t.data_ptr() % 16 == 0
    if good and not (t.is_contiguous() and t.shape[-1] % 8 == 0):
        st = t.stride()
        good = st[-1] == 1 and all(s > 0 and s % 8 == 0 for s, e in zip(st[:-1], t.shape) if e > 1)
    if not good:
        raise ValueError(f"{name} must have a contiguous last dimension, strides that are positive multiples of 8 "
                         "elements and a 16-byte aligned base")


def _same_layout(a: torch.Tensor, b: torch.Tensor) -> bool:
    x, y = a.stride(), b.stride()
    return x == y or all(i == j for i, j, e in zip(x, y, a.shape) if e > 1)


def _cache(k: torch.Tensor, v: torch.Tensor, dims: int = 4) -> SaCache:
    dtype = _DTYPES.get(k.dtype)
    if dtype is None or not k.is_cuda:
        raise ValueError("a cache must be a bf16 or fp16 CUDA tensor")
    shape = k.shape
    if len(shape) != dims or v.shape != shape or v.dtype is not k.dtype or v.device != k.device \
            or not _same_layout(k, v):
        raise ValueError("the caches must be [pages, page_size, Hkv, d] of one type, shape and layout")
    if k.numel() == 0:
        raise ValueError("the caches must not be empty")
    _strides("the cache", k)
    _strides("the cache", v)
    pages, page, heads, d = shape[-4:]
    ps, ts, hs, _ = k.stride()[-4:]
    return SaCache(pages, page, heads, d, dtype, ps if pages > 1 else page * heads * d, ts, hs if heads > 1 else d)


def _step(plan: CachePlan, n: int, dev, masked: bool = True) -> SaStep:
    table, lens, starts, granted = plan.table, plan.lens, plan.starts, plan.granted
    if table.dim() != 2:
        raise ValueError("the plan's table must be [R, width]")
    R, width = shape = table.shape
    _ints("the plan's table", table, shape, dev)
    _ints("the plan's lens", lens, (R,), dev)
    _ints("the plan's starts", starts, (R + 1,), dev)
    if granted is not None:
        _ints("the plan's granted", granted, (R,), dev)
        granted = granted.data_ptr()
    words, mask = 0, None
    if masked and plan.mask is not None:
        words = plan.mask.shape[-1]
        _ints("the plan's mask", plan.mask, (n, words), dev)
        mask = plan.mask.data_ptr()
    return SaStep(R, n, width, int(plan.max_new), words, starts.data_ptr(), lens.data_ptr(), granted, table.data_ptr(),
                  mask)


def sparse_attn_cache_plan(lens: torch.Tensor, new_tokens: torch.Tensor, table: torch.Tensor, held: torch.Tensor,
                           free_pages: torch.Tensor, nfree: torch.Tensor, n: int, page_size: int, *,
                           parents: Optional[torch.Tensor] = None, mask_words: int = 0, max_new: int = 0,
                           out: Optional[CachePlan] = None) -> CachePlan:
    """Pages, block table, slots, positions and tree masks of a step, from the requests'
    lengths, in one launch.

    lens, new_tokens, held: int32 [R]; table: int32 [R, width] and free_pages: int32
    [pages], both updated in place; nfree: int32 [1]. A negative new_tokens[r] ends request
    r and returns its pages. n rows are planned (at least the new tokens' sum).
    mask_words > 0 (32 new tokens to a word) also makes the masks, from parents (int32 [n],
    each new token's parent among its request's, -1 for none) or for a chain.
    `out`, a plan of an earlier call of the same sizes, is written again (the plan's held
    and nfree must not be this call's inputs); the returned plan's table, lens and
    free_pages are the ones given."""
    lib = _lib.load()
    if not lens.is_cuda or table.dim() != 2:
        raise ValueError("lens must be a CUDA tensor, table [R, width]")
    dev = lens.device
    R, width = shape = table.shape
    _ints("table", table, shape, dev)
    for name, t in (("lens", lens), ("new_tokens", new_tokens), ("held", held)):
        _ints(name, t, (R,), dev)
    _ints("nfree", nfree, (1,), dev)
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be [pages]")
    _ints("free_pages", free_pages, free_pages.shape, dev)
    n, mask_words = int(n), int(mask_words)
    if n < 1 or mask_words < 0:
        raise ValueError("n must be at least 1 and mask_words at least 0")
    if parents is not None:
        if mask_words == 0:
            raise ValueError("parents needs mask_words")
        _ints("parents", parents, (n,), dev)
    if out is None:
        sizes = [R + 1, R, R, 1, n, n, n * mask_words]     # one buffer: an allocation costs more than a view
        starts, granted, held_out, nfree_out, slots, positions, mask = \
            torch.empty(sum(sizes), dtype=torch.int32, device=dev).split_with_sizes(sizes)
        out = CachePlan(table, lens, starts, granted, mask.view(n, mask_words) if mask_words else None, slots,
                        positions, held_out, nfree_out, free_pages, int(max_new))
    else:
        for name, t, shape in (("starts", out.starts, (R + 1,)), ("granted", out.granted, (R,)),
                               ("slots", out.slots, (n,)), ("positions", out.positions, (n,)),
                               ("held", out.held, (R,)), ("nfree", out.nfree, (1,))):
            _ints(f"out.{name}", t, shape, dev)
        if mask_words:
            _ints("out.mask", out.mask, (n, mask_words), dev)
        else:
            out.mask = None
        out.table, out.lens, out.free_pages, out.max_new = table, lens, free_pages, int(max_new)
    _launch("sparse_attn_cache_plan", dev, lib.sparse_attn_cache_plan, lens.data_ptr(), new_tokens.data_ptr(),
            held.data_ptr(), nfree.data_ptr(), free_pages.data_ptr(), table.data_ptr(),
            None if parents is None else parents.data_ptr(), R, free_pages.shape[0], int(page_size), width, n, mask_words,
            out.held.data_ptr(), out.nfree.data_ptr(), out.starts.data_ptr(), out.granted.data_ptr(),
            out.slots.data_ptr(), out.positions.data_ptr(), out.mask.data_ptr() if mask_words else None)
    return out


def sparse_attn_cache_write(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_cache: torch.Tensor,
                            v_cache: torch.Tensor) -> None:
    """Writes rows k, v [n, Hkv, d] to their slots (int32 [n], -1 for none) of the caches.
    k and v may be strided with d contiguous (one layout for both), e.g. a transposed
    [Hkv, n, d] or a part of a fused projection. Slots other than -1 must differ."""
    lib = _lib.load()
    c = _cache(k_cache, v_cache)
    dev = k_cache.device
    _rows("k", k, k_cache.dtype, dev)
    _rows("v", v, k_cache.dtype, dev)
    n = k.shape[0]
    if k.shape[1:] != (c.Hkv, c.d) or v.shape != k.shape:
        raise ValueError(f"k and v must be [n, {c.Hkv}, {c.d}]")
    if not _same_layout(k, v):
        raise ValueError("k and v must have the same strides")
    _ints("slots", slots, (n,), dev)
    if n == 0:
        return
    _launch("sparse_attn_cache_write", dev, lib.sparse_attn_cache_write, k.data_ptr(), v.data_ptr(), k.stride(0),
            k.stride(1), n, slots.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), c)


def sparse_attn_tree_workspace_size(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                    plan: CachePlan) -> int:
    """Bytes of workspace sparse_attn_tree_fwd needs for these tensors."""
    c = _cache(k_cache, v_cache)
    return int(_lib.load().sparse_attn_tree_workspace_size(c, _step(plan, q.shape[0], k_cache.device), q.shape[1]))


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
    c = _cache(k_cache, v_cache)
    dev = k_cache.device
    _rows("q", q, k_cache.dtype, dev)
    n, Hq, d = q.shape
    if d != c.d or Hq < 1 or Hq % c.Hkv:
        raise ValueError("q must be [n, Hq, d] with the cache's d and Hq a multiple of its heads")
    if out is None:
        out = torch.empty((n, Hq, d), dtype=q.dtype, device=dev)
    else:
        _rows("out", out, q.dtype, dev)
        if out.shape != q.shape:
            raise ValueError("out must have q's shape")
    if lse is not None and (lse.dtype != torch.float32 or tuple(lse.shape) != (n, Hq) or lse.device != dev
                            or not lse.is_contiguous()):
        raise ValueError("lse must be a contiguous float32 tensor [n, Hq] on q's device")
    s = _step(plan, n, dev)
    if n == 0:
        return out
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if workspace is None:
        workspace = torch.empty(int(lib.sparse_attn_tree_workspace_size(c, s, Hq)), dtype=torch.uint8, device=dev)
    elif workspace.device != dev:
        raise ValueError("workspace must be on q's device")
    _launch("sparse_attn_tree_fwd", dev, lib.sparse_attn_tree_fwd, q.data_ptr(), q.stride(0), q.stride(1), Hq,
            k_cache.data_ptr(), v_cache.data_ptr(), c, s, float(scale), out.data_ptr(), out.stride(0), out.stride(1),
            None if lse is None else lse.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size())
    return out


def sparse_attn_cache_accept(k_cache: torch.Tensor, v_cache: torch.Tensor, plan: CachePlan, accepted: torch.Tensor,
                             taken: torch.Tensor) -> None:
    """Moves the accepted new tokens' rows to the places behind each request's cached ones:
    accepted int32 [R, cols] holds their indices among the request's new tokens in
    ascending order, taken int32 [R] how many there are. The caches are one layer's
    ([pages, page_size, Hkv, d]) or all layers' ([layers, ...]). The requests' lengths
    grow by `taken` (the caller adds it to lens)."""
    lib = _lib.load()
    layers, layer_stride = 1, 0
    if k_cache.dim() == 5:
        layers, layer_stride = k_cache.shape[0], k_cache.stride(0)
    c = _cache(k_cache, v_cache, k_cache.dim() if k_cache.dim() == 5 else 4)
    dev = k_cache.device
    s = _step(plan, 1, dev, masked=False)        # the moves read no row of the step's buffers
    if accepted.dim() != 2 or accepted.shape[1] < 1:
        raise ValueError("accepted must be [R, cols]")
    _ints("accepted", accepted, (s.R, accepted.shape[1]), dev)
    _ints("taken", taken, (s.R,), dev)
    _launch("sparse_attn_cache_accept", dev, lib.sparse_attn_cache_accept, k_cache.data_ptr(), v_cache.data_ptr(), c,
            layers, layer_stride, s, accepted.data_ptr(), accepted.shape[1], taken.data_ptr())
