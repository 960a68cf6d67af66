// Kernels of the paged cache around the attention of new tokens: the plan of a step
// (block tables, slot map, positions, tree masks), the write of the new tokens'
// keys and values, and the move of the accepted drafts.
//
// A cache holds pages of `page` tokens; request r's token at place t lives in page
// table[r][t / page], slot page_id * page + t % page.
#pragma once

#include "sa_device.cuh"

namespace sa {

// ------------------------------------------------------------------ step plan
//
// Per request r with L cached, T new tokens and `held` pages in its table row:
//   T < 0   the request has ended: its held pages go back on the free list, in
//           request order, behind the nfree ids already there;
//   T >= 0  need = max(0, ceil((L + T) / page) - held) pages are taken from the
//           list's end, in request order, while they last: the request is served
//           when need = 0 or the running sum of the needs is at most the list's
//           length after the returns.
//
// One launch. What a token needs (its request, the request's place in the list) is
// a prefix sum over the requests, so every CTA sums over all of them itself, in
// shared memory, and then fills its own tokens and its own requests' rows: the
// bound is the latency of a few dependent reads, and a second launch would cost
// more than the repeated sum. No CTA reads what another writes: a page taken from
// the returned part of the list is looked up in the ended request's own row, not in
// the list, and the counts go to outputs apart from the inputs. Measured (one B200, in a
// captured graph): 64 requests of one token 4 us, 9 prompts of 75,000 tokens 6, 256
// requests of 48 drafts in chains 4.2, in trees 6.2 (a token walks up its tree in dependent
// reads, from L1), with 9 ended ones among them 8.8 and 10.1: one warp returns a request's pages
// (up to 942), 32 at a time, each a read of the table and then a write of the list.
struct CachePlanArgs {
  const int *lens, *fresh, *held, *nfree;
  int *free_pages, *table;
  const int* parents;       // or null: each new token follows the one before it
  int R, pages, page_shift, width, n, words;
  int *held_out, *nfree_out, *starts, *granted, *slots, *positions;
  unsigned* mask;           // [n][words] or null
};

constexpr int kCachePlanThreads = 256;
constexpr int kCacheMaxRequests = 8192;

// Exclusive prefix sums over the CTA of three values; the totals come back in tot.
__device__ __forceinline__ void block_scan3(long long (&v)[3], long long (&tot)[3], long long (*warp_sums)[3]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = kCachePlanThreads / 32;
  long long inc[3];
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    inc[c] = v[c];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, inc[c], o);
      if (lane >= o) inc[c] += x;
    }
  }
  __syncthreads();
  if (lane == 31) {
#pragma unroll
    for (int c = 0; c < 3; ++c) warp_sums[warp][c] = inc[c];
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < 3; ++c) {
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const long long s = warp_sums[w][c];
      if (w < warp) before += s;
      all += s;
    }
    v[c] = before + inc[c] - v[c];
    tot[c] = all;
  }
}

// The last index i in [0, n) with a[i] <= x, for a non-decreasing with a[0] <= x.
__device__ __forceinline__ int last_not_above(const int* a, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kCachePlanThreads) cache_plan_kernel(const CachePlanArgs a) {
  extern __shared__ int plan_smem[];
  __shared__ long long warp_sums[kCachePlanThreads / 32][3];
  int* s_start = plan_smem;                 // [R + 1] first token of each request
  int* s_need = s_start + a.R + 1;          // [R + 1] pages asked for by the requests before
  int* s_back = s_need + a.R + 1;           // [R + 1] pages returned by the requests before
  int* s_grant = s_back + a.R + 1;          // [R] tokens of the request if it is valid, else -1
  int nfree = *a.nfree;
  bool bad = nfree < 0 || nfree > a.pages;
  if (bad) nfree = 0;
  long long base[3] = {0, 0, 0};
  for (int r0 = 0; r0 < a.R; r0 += kCachePlanThreads) {
    const int r = r0 + threadIdx.x;
    long long v[3] = {0, 0, 0}, tot[3];
    int grant = -1;
    if (r < a.R) {
      const int T = a.fresh[r], L = a.lens[r], held = a.held[r];
      const bool held_ok = held >= 0 && held <= a.width;
      if (T < 0) {
        grant = 0;
        if (held_ok)
          v[2] = held;
        else
          bad = true;
      } else {
        v[0] = T;
        const long long want = (static_cast<long long>(L) + T + (1 << a.page_shift) - 1) >> a.page_shift;
        if (!held_ok || L < 0 || want > a.width || L > (static_cast<long long>(held) << a.page_shift) ||
            (a.mask && T > 32 * a.words)) {
          bad = true;
        } else {
          grant = T;
          v[1] = want > held ? want - held : 0;
        }
      }
    }
    const long long own[3] = {v[0], v[1], v[2]};
    block_scan3(v, tot, warp_sums);
    // a request whose tokens pass the step's n is not served and asks for no page:
    // the sums are taken again without its need
    const bool past = grant > 0 && base[0] + v[0] + own[0] > a.n;
    if (__syncthreads_or(past)) {
      if (past) {
        grant = -1;
        bad = true;
      }
      v[0] = own[0];
      v[1] = past ? 0 : own[1];
      v[2] = own[2];
      block_scan3(v, tot, warp_sums);
    }
    if (r < a.R) {
      s_start[r] = static_cast<int>(min(base[0] + v[0], static_cast<long long>(a.n)));
      s_need[r] = static_cast<int>(base[1] + v[1]);   // at most R * width, an int
      s_back[r] = static_cast<int>(base[2] + v[2]);
      s_grant[r] = grant;
    }
    for (int c = 0; c < 3; ++c) base[c] += tot[c];
  }
  if (threadIdx.x == 0) {
    s_start[a.R] = static_cast<int>(min(base[0], static_cast<long long>(a.n)));
    s_need[a.R] = static_cast<int>(base[1]);
    s_back[a.R] = static_cast<int>(base[2]);
  }
  __syncthreads();
  // the list after the returns; more pages than the pool has means a page in two rows
  int top = nfree + min(s_back[a.R], a.pages);
  if (top > a.pages || s_back[a.R] > a.pages) {
    bad = true;
    top = a.pages;
  }
  // the id at place m of the list after the returns
  auto list_at = [&](int m) {
    if (m < nfree) return a.free_pages[m];
    const int e = last_not_above(s_back, a.R, m - nfree);
    return a.table[static_cast<long long>(e) * a.width + (m - nfree - s_back[e])];
  };
  auto served = [&](int r) { return s_grant[r] >= 0 && (s_need[r + 1] == s_need[r] || s_need[r + 1] <= top); };

  // rows of the requests: one warp each
  const int lane = threadIdx.x & 31;
  const int nwarps = gridDim.x * (kCachePlanThreads / 32);
  for (int r = blockIdx.x * (kCachePlanThreads / 32) + (threadIdx.x >> 5); r < a.R; r += nwarps) {
    const int back = s_back[r + 1] - s_back[r], need = s_need[r + 1] - s_need[r];
    const bool ok = served(r);
    const int held = a.held[r];
    const long long row = static_cast<long long>(r) * a.width;
    if (back > 0) {
      // what the list has room for (nfree + s_back[r] may pass 2^31 where counts are wrong)
      const int fit = min(back, a.pages - nfree - min(s_back[r], a.pages - nfree));
      for (int j = lane; j < fit; j += 32) a.free_pages[nfree + s_back[r] + j] = a.table[row + j];
    } else if (ok && need > 0) {
      for (int j = lane; j < need; j += 32) a.table[row + held + j] = list_at(top - 1 - (s_need[r] + j));
    }
    if (lane == 0) {
      a.starts[r] = s_start[r];
      a.granted[r] = ok ? s_grant[r] : 0;
      a.held_out[r] = a.fresh[r] < 0 ? 0 : held + (ok ? need : 0);
    }
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    a.starts[a.R] = s_start[a.R];
    // the pages taken: the largest of the running sums that the list covers
    int lo = 0, hi = a.R + 1;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_need[mid] <= top)
        lo = mid;
      else
        hi = mid;
    }
    *a.nfree_out = top - s_need[lo];
  }

  // tokens: one thread each
  bool bad_page = false;
  const int live = s_start[a.R];
  for (long long i0 = static_cast<long long>(blockIdx.x) * kCachePlanThreads + threadIdx.x; i0 < a.n;
       i0 += static_cast<long long>(gridDim.x) * kCachePlanThreads) {
    const int i = static_cast<int>(i0);
    int slot = -1, position = 0;
    if (i < live) {
      const int r = last_not_above(s_start, a.R, i);
      const int t = i - s_start[r];
      const int L = a.lens[r];
      int depth = t;
      if (a.mask && s_grant[r] >= 0) {
        // up the tree from the token: parents come before their children, so the
        // words of its mask row are finished from the last to the first
        unsigned* out = a.mask + i0 * a.words;
        int node = t, w = a.words - 1;
        unsigned bits = 0;
        depth = -1;
        while (node >= 0) {
          for (; w > (node >> 5); --w) {
            out[w] = bits;
            bits = 0;
          }
          bits |= 1u << (node & 31);
          ++depth;
          const int up = a.parents ? a.parents[i - t + node] : node - 1;
          if (up >= node || up < -1) {
            bad = true;
            break;
          }
          node = up;
        }
        for (; w >= 0; --w) {
          out[w] = bits;
          bits = 0;
        }
      } else if (a.mask) {
        for (int w = 0; w < a.words; ++w) a.mask[i0 * a.words + w] = 0u;
      }
      position = L + depth;
      if (served(r)) {
        const int place = L + t, col = place >> a.page_shift;
        const int held = a.held[r];
        const int id = col < held ? a.table[static_cast<long long>(r) * a.width + col]
                                  : list_at(top - 1 - (s_need[r] + col - held));
        if (id >= 0 && id < a.pages)
          slot = (id << a.page_shift) + (place - (col << a.page_shift));
        else
          bad_page = true;
      }
    } else if (a.mask) {
      for (int w = 0; w < a.words; ++w) a.mask[i0 * a.words + w] = 0u;
    }
    a.slots[i] = slot;
    a.positions[i] = position;
  }
  if (bad) atomicOr(&g_dev_error, DEVERR_VALUE);
  if (bad_page) atomicOr(&g_dev_error, DEVERR_RANGE);
}

// ------------------------------------------------------------------ cache write
//
// cache[slot[i]] = row i, for K and V: 16-byte pieces, each thread four of them at
// a time so that four loads are in flight. Both caches in one launch (blockIdx.y). Bound
// by HBM: 29,601 rows of 24 heads of 128, given head by head, take 110 us (112 a Python call in a
// loop) for 727 MB, the rate of a copy. Loads and stores both stream: with stores that stay in L2 until their
// sector is pushed out the same rows took 151 us, and 113 without. Eight pieces a thread, or a tile of
// tokens with all heads for each CTA (longer runs of a source by head), change nothing.
struct CacheWriteArgs {
  const uint4* src[2];
  uint4* dst[2];
  const int* slots;
  long long src_token, src_head;                 // strides in 16-byte pieces
  long long dst_page, dst_token, dst_head;
  unsigned rows, H;                              // rows = tokens * heads
  int page_shift;
  long long slot_end;                            // pages * page
};

template <int kVecs>
__global__ void __launch_bounds__(256) cache_write_kernel(const CacheWriteArgs a) {
  constexpr int kUnroll = 4, kRowsPerPass = 256 / kVecs;
  const uint4* src = blockIdx.y ? a.src[1] : a.src[0];     // (an index would put the arguments in local memory)
  uint4* dst = blockIdx.y ? a.dst[1] : a.dst[0];
  const int vec = threadIdx.x % kVecs;
  const unsigned row0 = blockIdx.x * (kRowsPerPass * kUnroll) + threadIdx.x / kVecs;   // < 2^31 + 256
  uint4 val[kUnroll];
  long long to[kUnroll];
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kUnroll; ++u) {
    const unsigned row = row0 + u * kRowsPerPass;
    to[u] = -1;
    if (row < a.rows) {
      const unsigned tok = row / a.H, head = row - tok * a.H;
      const int slot = a.slots[tok];
      if (slot >= 0 && slot < a.slot_end) {
        val[u] = __ldcs(src + tok * a.src_token + head * a.src_head + vec);
        const int page = slot >> a.page_shift;
        to[u] = page * a.dst_page + (slot - (page << a.page_shift)) * a.dst_token + head * a.dst_head + vec;
      } else if (slot != -1) {
        bad = true;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < kUnroll; ++u)
    if (to[u] >= 0) __stcs(dst + to[u], val[u]);
  if (bad) atomicOr(&g_dev_error, DEVERR_RANGE);
}

// ------------------------------------------------------------------ accept
//
// Request r's new tokens lie at places L .. L + T - 1; its accepted ones, new
// tokens acc[0] < acc[1] < ... , move to L, L + 1, ... (acc[i] >= i, so no row is
// overwritten before it is read when the moves run in order of i). A thread owns
// one 16-byte column of a row (one of K and V, one head, one layer) for all the
// request's moves and takes them in order, eight loads at a time, so no two threads
// touch the same bytes and nothing has to wait. Rows that stay (acc[i] = i) are
// neither read nor written. 96 requests that accept up to 9 of 48 drafts in 32 layers of 4
// heads of 128 take 8 to 10 us for some 31 MB (a copy's time: 4.8): lengths, indices and page
// ids are three reads one after another before the first row, and of the 1,536 CTAs four fit
// on an SM (64 registers; 66 and three made it 9.4 for 8.1), so that is done in 2.6 rounds.
struct CacheAcceptArgs {
  uint4* cache[2];
  const int *lens, *starts, *granted, *table, *accepted, *taken;
  long long layer, page_stride, token, head;     // strides in 16-byte pieces
  int width, cols, pages, page_shift, vecs, H, layers, n;
};

constexpr int kAcceptMax = 1024;   // accepted tokens of one request

__global__ void __launch_bounds__(256, 4) cache_accept_kernel(const CacheAcceptArgs a) {
  __shared__ long long s_src[kAcceptMax], s_dst[kAcceptMax];
  const int r = blockIdx.x;
  const int m = a.taken[r];
  const int s0 = a.starts[r], s1 = a.starts[r + 1];
  const bool rows_ok = s0 >= 0 && s1 >= s0 && s1 <= a.n;
  const int T0 = rows_ok ? s1 - s0 : 0;
  const int T = a.granted ? min(T0, a.granted[r]) : T0;
  const int L = a.lens[r];
  const int page = 1 << a.page_shift;
  int err = 0;
  if (!rows_ok || m < 0 || m > a.cols || m > max(T, 0) || L < 0 ||
      static_cast<long long>(L) + max(T, 0) > static_cast<long long>(a.width) * page)
    err = DEVERR_VALUE;
  int first = 0x7fffffff;                        // the first token that moves
  if (!err) {
    const int* acc = a.accepted + static_cast<long long>(r) * a.cols;
    const int* row = a.table + static_cast<long long>(r) * a.width;
    for (int i = threadIdx.x; i < m; i += 256) {
      const int t = acc[i];
      if (t < i || t >= T || (i > 0 && acc[i - 1] >= t)) {
        err = DEVERR_VALUE;
        continue;
      }
      const int from = L + t, to = L + i;
      const int pf = row[from >> a.page_shift], pt = row[to >> a.page_shift];
      if (pf < 0 || pf >= a.pages || pt < 0 || pt >= a.pages) {
        err = DEVERR_RANGE;
        continue;
      }
      s_src[i] = pf * a.page_stride + (from & (page - 1)) * a.token;
      s_dst[i] = pt * a.page_stride + (to & (page - 1)) * a.token;
      if (t != i) first = min(first, i);
    }
  }
  const bool any = __syncthreads_or(err);
  if (any) {
    if (err) atomicOr(&g_dev_error, static_cast<unsigned>(err));
    return;
  }
  // first over the CTA: through shared memory that the moves do not need
  __shared__ int s_first;
  if (threadIdx.x == 0) s_first = 0x7fffffff;
  __syncthreads();
  if (first != 0x7fffffff) atomicMin(&s_first, first);
  __syncthreads();
  first = s_first;
  if (first >= m) return;
  const long long cols = 2LL * a.layers * a.H * a.vecs;
  for (long long c = static_cast<long long>(blockIdx.y) * 256 + threadIdx.x; c < cols;
       c += static_cast<long long>(gridDim.y) * 256) {
    const int vec = static_cast<int>(c % a.vecs);
    long long q = c / a.vecs;
    const int head = static_cast<int>(q % a.H);
    q /= a.H;
    const int layer = static_cast<int>(q >> 1);
    uint4* base = (q & 1 ? a.cache[1] : a.cache[0]) + layer * a.layer + head * a.head + vec;   // (as in the write)
    for (int i0 = first; i0 < m; i0 += 8) {
      uint4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u < m) v[u] = base[s_src[i0 + u]];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (i0 + u < m) base[s_dst[i0 + u]] = v[u];
    }
  }
}

}  // namespace sa
