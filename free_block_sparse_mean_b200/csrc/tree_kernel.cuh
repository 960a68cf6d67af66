// Attention of new tokens over a paged cache on sm_100a (tcgen05 + TMA + TMEM):
// one token, a tree of drafted tokens or a chunk of a prompt for each request.
//
//   o[t] = sum_j p[t,j] v_j / sum_j p[t,j],  p[t,j] = exp(scale q_t . k_j)
//
// over the L cached tokens of the request and the new tokens j that t sees (its row
// of mask bits, or all up to itself), in one pass with a running maximum and sum.
//
// Rows. The G query heads that share a key head read the same keys, so a tile is up
// to 128 rows of (new token, head of the group), token-major: TT = 128 / G tokens.
// One TMA box {64, G heads, TT tokens} per 128-byte column chunk brings them.
//
// Work. A tile's keys are cut into pieces of whole 64-key blocks; a CTA takes one
// piece of one tile. The lengths are on the GPU, so each CTA finds its piece there:
// all sum the requests' blocks (a scan over the requests), take the piece length
// from that total, so that about `target` pieces exist whatever the mix of lengths,
// and look up the piece of their own index. A tile of one piece is written to O by
// its CTA; the others leave (max, sum, unnormalised O) in fp32 for
// tree_combine_kernel.
//
// Keys. Per 64-key block the load warp reads the block's page ids and issues one TMA
// box (pages of 64 tokens and more) or one per page and column chunk (smaller
// pages). A page id is read only where the request has tokens; places behind the
// last token in its page are masked in S by column, and their V rows are set to zero
// in shared memory, since 0 * NaN is not 0. For the same reason V elements that are
// not finite are taken out of blocks that some row does not see whole; the rows that
// do see such a token get the element added at the end (see `special` below).
//
// Roles (224 threads): warp 0 loads, warp 1 owns TMEM and issues S = Q K^T, warp 2
// issues O += P V, warps 3..6 run the softmax (thread = row), the O correction and the
// epilogue; a softmax warp whose 32 rows are all empty leaves at once, so a
// single-token call pays the exponentials of one warp. TMEM (256 columns): S [0,64),
// P [64,96) and [96,128), O [128, 128 + D). Two CTAs fit on an SM.
//
// The barrier phases follow the block-sparse forward's argument: S(k+1) is issued only
// after every active softmax warp released S(k); P(k) goes to buffer k & 1 once
// P(k-2).V has finished; a K or V stage is refilled after the product that read it has
// completed. So no wait is ever more than one phase behind its barrier.
#pragma once

#include <cuda_fp16.h>

#include "sa_device.cuh"

namespace sa {

constexpr int kTreeThreads = 224;

// 16-bit element types of Q, K, V, P and O.
enum Elem16 : int { kElemBF16 = 0, kElemF16 = 1 };

// Instruction descriptor for kind::f16, A and B both bf16 (format 1) or both f16
// (format 0), fp32 D, A K-major.
__host__ __device__ constexpr uint32_t idesc_16_f32(int elem, int M, int N, bool b_mn_major) {
  return (1u << 4) | (elem == kElemBF16 ? (1u << 7) | (1u << 10) : 0u) | ((b_mn_major ? 1u : 0u) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

template <int kElem>
__device__ __forceinline__ uint32_t pack16x2(float lo, float hi) {
  if constexpr (kElem == kElemBF16) {
    return pack_bf16x2(lo, hi);
  } else {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// kSmallQ: the tile has at most 32 rows, so Q takes 32 rows of shared memory and the
// freed space a third stage of K and of V. The S product still reads 128 rows (rows
// behind Q are whatever lies there); a row's result touches no other row, and the
// rows that do not exist are never written out.
template <int D, bool kSmallQ>
struct TreeCfg {
  static constexpr int kChunks = D / 64;
  static constexpr int kQRows = kSmallQ ? 32 : 128;
  static constexpr int kQChunkBytes = kQRows * 128;
  static constexpr int kKVChunkBytes = kBlock * 128;
  static constexpr int kKVBytes = kChunks * kKVChunkBytes;
  static constexpr int ST = D == 64 ? (kSmallQ ? 6 : 5) : (kSmallQ ? 3 : 2);   // stages of K and of V
  static constexpr int oQ = 0;
  static constexpr int oK = oQ + kChunks * kQChunkBytes;
  static constexpr int oV = oK + ST * kKVBytes;
  static constexpr int oBar = oV + ST * kKVBytes;
  static constexpr int kNumBars = 4 * ST + 8;
  static constexpr int oMisc = oBar + kNumBars * 8;
  static constexpr int kSmemBytes = oMisc + 512 + 1024;
  static constexpr uint32_t kColS = 0, kColP0 = 64, kColP1 = 96, kColO = 128, kTmemCols = 256;
};

struct TreeArgs {
  const int *starts, *lens, *granted, *table;
  const uint32_t* mask;           // [n][words] or null
  int R, n, width, pages, page_shift, words;
  int Hkv, G, TT;                 // key heads, query heads each, tokens of a tile
  int target, min_blocks;         // pieces aimed at, smallest piece in blocks
  void* O;
  long long o_token, o_head;      // strides in elements
  float* lse;                     // [n][Hkv * G] or null
  float scale_log2;
  float* part_o;                  // [slot][tile rows][D]
  float2* part_ml;                // [slot][tile rows]
  int2* sched;                    // per request: pieces (0 or 1: nothing to combine), first slot
};

struct TreeReq {
  int T, L, nb, tiles;
};

// Request r as the kernels take it: T = 0 if it has nothing to compute or its
// numbers are out of range (then *bad is set).
__device__ __forceinline__ TreeReq tree_request(const TreeArgs& a, int r, bool* bad) {
  TreeReq q;
  const int s0 = a.starts[r], s1 = a.starts[r + 1];
  q.L = a.lens[r];
  q.T = s1 - s0;
  const bool ok = s0 >= 0 && s1 >= s0 && s1 <= a.n;
  if (a.granted) q.T = min(q.T, max(a.granted[r], 0));
  if (!ok || (q.T > 0 && (q.L < 0 || static_cast<long long>(q.L) + q.T >
                                         (static_cast<long long>(a.width) << a.page_shift) ||
                          (a.mask && q.T > 32 * a.words)))) {
    *bad = true;
    q.T = 0;
  }
  if (q.T == 0) q.L = 0;
  q.nb = q.T > 0 ? (q.L + q.T + kBlock - 1) / kBlock : 0;
  q.tiles = (q.T + a.TT - 1) / a.TT;
  return q;
}

// Key blocks that some row of the tile sees: all of them under a mask, up to its last
// token's place without one.
__device__ __forceinline__ int tree_tile_blocks(const TreeReq& q, int tile, int TT, bool masked) {
  return masked ? q.nb : (q.L + min(q.T, (tile + 1) * TT) + kBlock - 1) / kBlock;
}
// First block of piece p of `pieces` over nb blocks.
__device__ __forceinline__ int tree_piece_start(int nb, int p, int pieces) {
  return static_cast<int>(static_cast<long long>(nb) * p / pieces);
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, int v,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(smem_u32(bar))
      : "memory");
}

// 64 mask bits of one row from bit `off` on (bits past the row's words are 0).
__device__ __forceinline__ unsigned long long mask_bits64(const uint32_t* row, int words, int off) {
  const int w = off >> 5, s = off & 31;
  const uint32_t a = w < words ? row[w] : 0u;
  const uint32_t b = w + 1 < words ? row[w + 1] : 0u;
  const uint32_t c = w + 2 < words ? row[w + 2] : 0u;
  const uint32_t lo = __funnelshift_r(a, b, s), hi = __funnelshift_r(b, c, s);
  return (static_cast<unsigned long long>(hi) << 32) | lo;
}

__device__ __forceinline__ unsigned long long low_bits64(int n) {   // n may be out of 0..64
  return n >= 64 ? ~0ull : (n <= 0 ? 0ull : (1ull << n) - 1ull);
}

// The columns of key block kb .. kb + 63 that new token t of a request sees.
__device__ __forceinline__ unsigned long long tree_visible(const TreeArgs& a, int L, int T, int t, long long token,
                                                           int kb) {
  if (a.mask == nullptr) return low_bits64(L + t + 1 - kb);
  const int off = kb - L;
  unsigned long long v;
  const uint32_t* row = a.mask + token * a.words;
  if (off >= 0)
    v = mask_bits64(row, a.words, off);
  else if (off <= -64)
    return ~0ull;
  else
    v = low_bits64(-off) | (mask_bits64(row, a.words, 0) << (-off));
  return v & low_bits64(L + T - kb);
}

// True for a 16-bit element that is an infinity or NaN (as bits).
template <int kElem>
__device__ __forceinline__ bool not_finite16(uint32_t bits) {
  constexpr uint32_t e = kElem == kElemBF16 ? 0x7f80u : 0x7c00u;
  return (bits & e) == e;
}
template <int kElem>
__device__ __forceinline__ float to_float16(uint32_t bits) {
  if constexpr (kElem == kElemBF16)
    return __uint_as_float(bits << 16);
  else
    return __half2float(__ushort_as_half(static_cast<unsigned short>(bits)));
}

template <int D, int kElem, bool kSmallQ>
__global__ void __launch_bounds__(kTreeThreads, 2)
    tree_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TreeArgs a,
                    const uint16_t* __restrict__ Vraw, long long v_page, long long v_token, long long v_head) {
  using C = TreeCfg<D, kSmallQ>;
  constexpr uint32_t kIdescS = idesc_16_f32(kElem, 128, 64, false);
  constexpr uint32_t kIdescPV = idesc_16_f32(kElem, 128, D, true);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = base + C::oQ;
  uint8_t* sK = base + C::oK;
  uint8_t* sV = base + C::oV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::oBar);
  uint64_t* kfull = bars;                  // [ST] K stage loaded
  uint64_t* kempty = kfull + C::ST;        // [ST] K stage consumed by S MMA
  uint64_t* vfull = kempty + C::ST;        // [ST] V stage loaded
  uint64_t* vempty = vfull + C::ST;        // [ST] V stage consumed by P.V MMA
  uint64_t* q_full = vempty + C::ST;       // Q tile loaded
  uint64_t* s_full = q_full + 1;           // S(k) written by the MMA (phase k)
  uint64_t* s_free = q_full + 2;           // S(k) read by the active softmax warps (phase k)
  uint64_t* p_full = q_full + 3;           // [2] by k parity: P(k) in TMEM and O corrected
  uint64_t* pv_done = q_full + 5;          // [2] by k parity: P(k).V finished
  uint64_t* drain = q_full + 7;            // every MMA of the tile finished, `special` written
  int* misc = reinterpret_cast<int*>(base + C::oMisc);
  volatile int* abort_flag = misc + 0;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc + 1);
  volatile int* special = misc + 2;        // an element of V was taken out (not finite)
  int* found = misc + 4;                   // this CTA's piece: request, index in it, pieces, slot
  long long* wsum = reinterpret_cast<long long*>(misc + 16);   // [7 warps][2]

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned FULL = 0xffffffffu;

  // ------------------------------------------------------------ find this CTA's piece
  bool bad = false;
  TreeReq mine{0, 0, 0, 0};
  long long total = 0;
  for (int r = threadIdx.x; r < a.R; r += kTreeThreads) {
    mine = tree_request(a, r, &bad);
    total += static_cast<long long>(mine.tiles) * mine.nb;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(FULL, total, o);
  if (lane == 0) wsum[warp] = total;
  if (threadIdx.x == 0) {
    found[0] = -1;
    *abort_flag = 0;
    *special = 0;
  }
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kTreeThreads / 32; ++w) total += wsum[w];
  total *= a.Hkv;
  const int piece_blocks =
      static_cast<int>(max(static_cast<long long>(a.min_blocks), (total + a.target - 1) / a.target));
  __syncthreads();
  long long items_before = 0, slots_before = 0;
  for (int r0 = 0; r0 < a.R; r0 += kTreeThreads) {
    const int r = r0 + threadIdx.x;
    if (a.R > kTreeThreads) {
      bool again = false;
      mine = r < a.R ? tree_request(a, r, &again) : TreeReq{0, 0, 0, 0};
    }
    const int pieces = (mine.nb + piece_blocks - 1) / piece_blocks;
    const long long items = static_cast<long long>(mine.tiles) * pieces * a.Hkv;
    const long long slots = pieces > 1 ? items : 0;
    long long ii = items, ss = slots;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(FULL, ii, o), y = __shfl_up_sync(FULL, ss, o);
      if (lane >= o) {
        ii += x;
        ss += y;
      }
    }
    if (lane == 31) {
      wsum[2 * warp] = ii;
      wsum[2 * warp + 1] = ss;
    }
    __syncthreads();
    long long all_i = 0, all_s = 0;
#pragma unroll
    for (int w = 0; w < kTreeThreads / 32; ++w) {
      if (w == warp) {
        ii += items_before + all_i;
        ss += slots_before + all_s;
      }
      all_i += wsum[2 * w];
      all_s += wsum[2 * w + 1];
    }
    const long long first = ii - items, slot = ss - slots;
    if (items > 0 && blockIdx.x >= first && blockIdx.x < ii) {
      found[0] = r;
      found[1] = static_cast<int>(blockIdx.x - first);
      found[2] = pieces;
      found[3] = static_cast<int>(slot);
      found[4] = mine.T;
      found[5] = mine.L;
    }
    if (blockIdx.x == 0 && a.sched && r < a.R) a.sched[r] = make_int2(pieces, static_cast<int>(slot));
    items_before += all_i;
    slots_before += all_s;
    __syncthreads();
    if (found[0] >= 0 && blockIdx.x != 0) break;
  }
  if (blockIdx.x == 0 && bad) atomicOr(&g_dev_error, DEVERR_VALUE);
  if (found[0] < 0) return;
  const int req = found[0];
  const int pieces = found[2];
  TreeReq rq;
  rq.T = found[4];
  rq.L = found[5];
  rq.nb = (rq.L + rq.T + kBlock - 1) / kBlock;
  rq.tiles = (rq.T + a.TT - 1) / a.TT;
  // tiles change fastest, so that the CTAs that run together share the keys they read
  int rest = found[1];
  const int tile = rq.tiles - 1 - rest % rq.tiles;
  rest /= rq.tiles;
  const int piece = rest % pieces, head = rest / pieces;
  const bool masked = a.mask != nullptr;
  const int nbt = tree_tile_blocks(rq, tile, a.TT, masked);
  const int b0 = tree_piece_start(rq.nb, piece, pieces);
  const int b1 = min(nbt, tree_piece_start(rq.nb, piece + 1, pieces));
  const int n = b1 - b0;
  if (n <= 0) return;                                   // only past a tile's last key: nothing is combined from here
  const int t0 = tile * a.TT;
  const int rows = min(a.TT, rq.T - t0) * a.G;          // rows of the tile that exist
  const int nact = (rows + 31) >> 5;                    // softmax warps with rows
  const int keys = rq.L + rq.T;
  // every row sees the keys before `open`; from there on rows differ
  const int open = masked ? rq.L : rq.L + t0 + 1;
  const int* trow = a.table + static_cast<long long>(req) * a.width;
  const long long tok0 = static_cast<long long>(a.starts[req]) + t0;
  const int page = 1 << a.page_shift;

  if (threadIdx.x == 0) {
    for (int s = 0; s < C::ST; ++s) {
      mbar_init(&kfull[s], 1);
      mbar_init(&kempty[s], 1);
      mbar_init(&vfull[s], 1);
      mbar_init(&vempty[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(s_full, 1);
    mbar_init(s_free, nact);
    mbar_init(&p_full[0], nact);
    mbar_init(&p_full[1], nact);
    mbar_init(&pv_done[0], 1);
    mbar_init(&pv_done[1], 1);
    mbar_init(drain, 3);
    fence_mbar_init();
  }
  if (warp == 1) tmem_alloc(tmem_holder, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;

  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      tma_prefetch_desc(&tmV);
      mbar_expect_tx(q_full, C::kChunks * a.TT * a.G * 128);
#pragma unroll
      for (int c = 0; c < C::kChunks; ++c)
        tma_load_4d(sQ + c * C::kQChunkBytes, &tmQ, 0, head * a.G, static_cast<int>(tok0), c, q_full);
    }
    // a block is 64 / sub boxes of `sub` tokens; below 64 tokens a box holds one
    // 128-byte column chunk (lane = chunk * boxes + box), else the whole block
    const int sub_shift = min(a.page_shift, 6), sub = 1 << sub_shift;
    const int subs = kBlock >> sub_shift;
    const bool whole = subs == 1;
    const int my_sub = lane & (subs - 1), my_chunk = lane >> (6 - sub_shift);
    const bool loads = whole ? lane == 0 : my_chunk < C::kChunks;
    const int box_bytes = sub * 128 * (whole ? C::kChunks : 1);
    const int dst_off = my_chunk * C::kKVChunkBytes + my_sub * sub * 128;
    bool bad_page = false;
    auto page_of = [&](int k) {      // this lane's page of block k, -1 past the last token
      const int at = (b0 + k) * kBlock + my_sub * sub;
      if (k >= n || !loads || at >= keys) return -1;
      int id = trow[at >> a.page_shift];
      if (id < 0 || id >= a.pages) {
        bad_page = true;
        id = 0;                      // flagged; any page of the pool keeps the load in bounds
      }
      return id;
    };
    int id = page_of(0);
    bool ok = true;
    int k = 0;
    for (; k < n; ++k) {
      const int next_id = page_of(k + 1);
      const int s = k % C::ST;
      const uint32_t ph = static_cast<uint32_t>(k / C::ST - 1) & 1u;
      const int kb = (b0 + k) * kBlock;
      const int boxes = (min(keys - kb, kBlock) + sub - 1) >> sub_shift;
      const uint32_t bytes = static_cast<uint32_t>(boxes) * sub * 128 * C::kChunks;
      const int y = (kb + my_sub * sub) & (page - 1);
      if (k >= C::ST) ok = warp_wait(&kempty[s], ph, abort_flag);
      if (!ok) break;
      if (lane == 0) mbar_expect_tx(&kfull[s], bytes);
      __syncwarp();
      if (id >= 0) tma_load_5d(sK + s * C::kKVBytes + dst_off, &tmK, 0, y, my_chunk, head, id, &kfull[s]);
      if (k >= C::ST) ok = warp_wait(&vempty[s], ph, abort_flag);
      if (!ok) break;
      if (lane == 0) mbar_expect_tx(&vfull[s], bytes);
      __syncwarp();
      if (id >= 0) tma_load_5d(sV + s * C::kKVBytes + dst_off, &tmV, 0, y, my_chunk, head, id, &vfull[s]);
      id = next_id;
    }
    if (bad_page) atomicOr(&g_dev_error, DEVERR_RANGE);
    (void)box_bytes;
    // every load that was issued has landed before the CTA leaves (bounded)
    if (lane == 0) {
      mbar_wait_drain(q_full, 0u);
      for (int kk = max(0, k - C::ST); kk < k; ++kk) {
        mbar_wait_drain(&kfull[kk % C::ST], static_cast<uint32_t>(kk / C::ST) & 1u);
        mbar_wait_drain(&vfull[kk % C::ST], static_cast<uint32_t>(kk / C::ST) & 1u);
      }
      // K(k) may have been issued without V(k)
      if (!ok && k < n) {
        const int s = k % C::ST;
        mbar_wait_drain(&kfull[s], static_cast<uint32_t>(k / C::ST) & 1u);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ S issuer
    if (lane == 0) {
      const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK);
      bool ok = mbar_wait(q_full, 0u, abort_flag);
      for (int k = 0; ok && k < n; ++k) {
        if (k > 0 && !mbar_wait(s_free, static_cast<uint32_t>(k - 1) & 1u, abort_flag)) break;
        const int s = k % C::ST;
        if (!mbar_wait(&kfull[s], static_cast<uint32_t>(k / C::ST) & 1u, abort_flag)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk & 3) * 32;
          const uint64_t ad = sdesc_sw128(sQa + (kk >> 2) * C::kQChunkBytes + off, 16, 1024);
          const uint64_t bd = sdesc_sw128(sKa + s * C::kKVBytes + (kk >> 2) * C::kKVChunkBytes + off, 16, 1024);
          tc_mma_ss(tmem_base + C::kColS, ad, bd, kIdescS, kk > 0 ? 1u : 0u);
        }
        tc_commit(s_full);
        tc_commit(&kempty[s]);
      }
      tc_commit(drain);
      mbar_wait_drain(drain, 0u);
    }
  } else if (warp == 2) {
    // ------------------------------------------------------------ P.V issuer
    const uint32_t sVa = smem_u32(sV);
    bool taken_out = false;
    for (int k = 0; k < n; ++k) {
      const int s = k % C::ST;
      if (!warp_wait(&vfull[s], static_cast<uint32_t>(k / C::ST) & 1u, abort_flag)) break;
      const int kb = (b0 + k) * kBlock;
      if (kb + kBlock > open || kb + kBlock > keys) {
        // rows behind the last token to zero; elements that are not finite out of
        // the rows that not every query sees
        const int live = min(kBlock, keys - kb), seen = max(0, min(open - kb, live));
        uint8_t* v = sV + s * C::kKVBytes;
        for (int c = 0; c < C::kChunks; ++c) {
          for (int x = seen * 8 + lane; x < kBlock * 8; x += 32) {     // 16-byte pieces, 8 a row
            uint4* at = reinterpret_cast<uint4*>(v + c * C::kKVChunkBytes + x * 16);
            if (x >= live * 8) {
              *at = make_uint4(0u, 0u, 0u, 0u);
            } else {
              uint4 w = *at;
              uint32_t* e = reinterpret_cast<uint32_t*>(&w);
              bool any = false;
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const bool lo = not_finite16<kElem>(e[u]), hi = not_finite16<kElem>(e[u] >> 16);
                if (lo) e[u] &= 0xffff0000u;
                if (hi) e[u] &= 0x0000ffffu;
                any |= lo | hi;
              }
              if (any) {
                *at = w;
                taken_out = true;
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      if (!warp_wait(&p_full[k & 1], static_cast<uint32_t>(k >> 1) & 1u, abort_flag)) break;
      tc_fence_after();
      if (lane == 0) {
        const uint32_t aP = tmem_base + ((k & 1) ? C::kColP1 : C::kColP0);
#pragma unroll
        for (int kk = 0; kk < kBlock / 16; ++kk) {
          const uint64_t bd = sdesc_sw128(sVa + s * C::kKVBytes + kk * 16 * 128, C::kKVChunkBytes, 1024);
          tc_mma_ts(tmem_base + C::kColO, aP + kk * 8, bd, kIdescPV, (k > 0 || kk > 0) ? 1u : 0u);
        }
        tc_commit(&pv_done[k & 1]);
        tc_commit(&vempty[s]);
      }
      __syncwarp();
    }
    if (__any_sync(FULL, taken_out) && lane == 0) *special = 1;
    if (lane == 0) {
      mbar_arrive(drain);              // `special` is written
      tc_commit(drain);
      mbar_wait_drain(drain, 0u);
    }
  } else {
    // ------------------------------------------------------------ softmax warps
    const int wq = warp & 3;                       // TMEM lane quadrant: rows 32*wq ..
    if (wq < nact) {
      const int row = wq * 32 + lane;
      const bool valid = row < rows;
      const int tl = valid ? row / a.G : 0;         // token of the tile, head of the group
      const int g = valid ? row - tl * a.G : 0;
      const int t = t0 + tl;
      const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
      const uint32_t s_addr = tmem_base + lane_bits + C::kColS;
      const uint32_t o_addr = tmem_base + lane_bits + C::kColO;
      float m_ref = -INFINITY, l = 0.f;
      bool alive = true;
      float s[64];
      if (warp_wait(s_full, 0u, abort_flag)) {
        tc_fence_after();
        tmem_ld32(s_addr, *reinterpret_cast<float(*)[32]>(&s[0]));
        tmem_ld32(s_addr + 32, *reinterpret_cast<float(*)[32]>(&s[32]));
      } else {
        alive = false;
      }
      for (int k = 0; alive && k < n; ++k) {
        const int kb = (b0 + k) * kBlock;
        unsigned long long vis = ~0ull;
        const bool part = kb + kBlock > open;       // some row does not see the whole block
        if (part) vis = valid ? tree_visible(a, rq.L, rq.T, t, tok0 + tl, kb) : 0ull;
        tmem_wait_ld();
        pin32(*reinterpret_cast<float(*)[32]>(&s[0]));
        pin32(*reinterpret_cast<float(*)[32]>(&s[32]));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s_free);
        if (part) {
          const uint32_t vlo = static_cast<uint32_t>(vis), vhi = static_cast<uint32_t>(vis >> 32);
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            s[c] = (vlo >> c) & 1u ? s[c] : -INFINITY;
            s[c + 32] = (vhi >> c) & 1u ? s[c + 32] : -INFINITY;
          }
        }
        float mx[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) mx[u] = fmax3(s[u], s[u + 8], s[u + 16]);
#pragma unroll
        for (int c = 24; c < 56; c += 16) {
#pragma unroll
          for (int u = 0; u < 8; ++u) mx[u] = fmax3(mx[u], s[c + u], s[c + 8 + u]);
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) mx[u] = fmaxf(mx[u], s[56 + u]);
        const float rmax = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) *
                           a.scale_log2;
        // the reference maximum is raised only when a row's maximum grows by more
        // than 2^8: P stays below 2^8 (in range of both types), O and l unchanged
        const bool raise = rmax > m_ref + 8.f;
        float alpha = 1.f;
        if (raise) {
          alpha = ex2(m_ref - rmax);
          m_ref = rmax;
        }
        const bool any_raise = __any_sync(FULL, raise);
        const float mref = (m_ref == -INFINITY) ? 0.f : m_ref;
        uint32_t pk[32];
        uint64_t acc0 = f2pack(0.f, 0.f), acc1 = acc0;
        const uint64_t sc2 = f2pack(a.scale_log2, a.scale_log2), nm2 = f2pack(-mref, -mref);
#pragma unroll
        for (int c = 0; c < 64; c += 2) {
          float x0, x1;
          f2unpack(ffma2(f2pack(s[c], s[c + 1]), sc2, nm2), x0, x1);
          const float p0 = ex2(x0), p1 = ex2(x1);
          if ((c >> 1) & 1)
            acc1 = fadd2(acc1, f2pack(p0, p1));
          else
            acc0 = fadd2(acc0, f2pack(p0, p1));
          pk[c >> 1] = pack16x2<kElem>(p0, p1);
        }
        float r0, r1, r2, r3;
        f2unpack(acc0, r0, r1);
        f2unpack(acc1, r2, r3);
        l = l * alpha + ((r0 + r1) + (r2 + r3));
        // P(k) into buffer k & 1 once its previous reader, P(k-2).V, has finished
        if (k >= 2) {
          if (!warp_wait(&pv_done[k & 1], static_cast<uint32_t>((k - 2) >> 1) & 1u, abort_flag)) {
            alive = false;
            break;
          }
          tc_fence_after();
        }
        tmem_st32u(tmem_base + lane_bits + ((k & 1) ? C::kColP1 : C::kColP0), pk);
        if (k > 0 && any_raise) {
          if (!warp_wait(&pv_done[(k - 1) & 1], static_cast<uint32_t>((k - 1) >> 1) & 1u, abort_flag)) {
            alive = false;
            break;
          }
          tc_fence_after();
#pragma unroll 1
          for (int cc = 0; cc < D; cc += 32) {
            float o[32];
            tmem_ld32(o_addr + cc, o);
            tmem_wait_ld();
            pin32(o);
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] *= alpha;
            tmem_st32(o_addr + cc, o);
          }
        }
        if (k + 1 < n) {
          if (!warp_wait(s_full, static_cast<uint32_t>(k + 1) & 1u, abort_flag)) {
            alive = false;
            break;
          }
          tc_fence_after();
          tmem_ld32(s_addr, *reinterpret_cast<float(*)[32]>(&s[0]));
          tmem_ld32(s_addr + 32, *reinterpret_cast<float(*)[32]>(&s[32]));
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[k & 1]);
      }
      tmem_wait_ld();
      // ------------------------------------------------------------ epilogue
      if (alive && warp_wait(drain, 0u, abort_flag)) {
        tc_fence_after();
        const bool whole_row = pieces == 1;
        const float mul = whole_row ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;   // a NaN sum stays one
        const bool fix = *special != 0;
        const long long token = tok0 + tl;
        const int hq = head * a.G + g;
        const long long prow = (static_cast<long long>(found[3]) + found[1]) * (a.TT * a.G) + row;
        uint16_t* orow = static_cast<uint16_t*>(a.O) + token * a.o_token + hq * a.o_head;
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          float o[32];
          tmem_ld32(o_addr + cc, o);
          tmem_wait_ld();
          pin32(o);
          if (!valid) continue;
          if (l == 0.f) {
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = 0.f;
          }
          if (fix) {
            // the elements taken out of V, for the rows that see their token
            for (int kb = b0 * kBlock; kb < b1 * kBlock; kb += kBlock) {
              if (kb + kBlock <= open) continue;
              unsigned long long vis = tree_visible(a, rq.L, rq.T, t, token, kb);
              if (open > kb) vis &= ~low_bits64(open - kb);
              for (; vis; vis &= vis - 1) {
                const int at = kb + __ffsll(static_cast<long long>(vis)) - 1;
                const int id = trow[at >> a.page_shift];
                if (id < 0 || id >= a.pages) continue;
                const uint16_t* v = Vraw + id * v_page + (at & (page - 1)) * v_token + head * v_head + cc;
#pragma unroll
                for (int x = 0; x < 32; ++x) {
                  const uint32_t e = v[x];
                  if (not_finite16<kElem>(e)) o[x] += to_float16<kElem>(e);
                }
              }
            }
          }
          if (whole_row) {
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
              uint4 w;
              w.x = pack16x2<kElem>(o[x + 0] * mul, o[x + 1] * mul);
              w.y = pack16x2<kElem>(o[x + 2] * mul, o[x + 3] * mul);
              w.z = pack16x2<kElem>(o[x + 4] * mul, o[x + 5] * mul);
              w.w = pack16x2<kElem>(o[x + 6] * mul, o[x + 7] * mul);
              *reinterpret_cast<uint4*>(orow + cc + x) = w;
            }
          } else {
            float4* to = reinterpret_cast<float4*>(a.part_o + prow * D + cc);
#pragma unroll
            for (int x = 0; x < 8; ++x) to[x] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          }
        }
        if (valid) {
          if (!whole_row)
            a.part_ml[prow] = make_float2(m_ref, l);
          else if (a.lse)
            a.lse[token * (a.Hkv * a.G) + hq] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * 0.6931471805599453f;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

// Joins the pieces of the tiles that have more than one: for each row the largest of
// the pieces' maxima, then O = sum w_p O_p / sum w_p l_p, w_p = 2^(m_p - m). One warp
// for each (token, query head), pieces in ascending order.
template <int D, int kElem>
__global__ void __launch_bounds__(128) tree_combine_kernel(const __grid_constant__ TreeArgs a) {
  const int lane = threadIdx.x & 31;
  const int Hq = a.Hkv * a.G;
  const long long wid = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (wid >= static_cast<long long>(a.n) * Hq) return;
  const int token = static_cast<int>(wid / Hq), hq = static_cast<int>(wid - static_cast<long long>(token) * Hq);
  // the request of the token
  int lo = 0, hi = a.R;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.starts[mid] <= token)
      lo = mid;
    else
      hi = mid;
  }
  const int2 sc = a.sched[lo];
  const int pieces = sc.x;
  if (pieces <= 1) return;
  bool bad = false;
  const TreeReq q = tree_request(a, lo, &bad);
  const int t = token - a.starts[lo];
  if (t < 0 || t >= q.T) return;
  const int tile = t / a.TT, head = hq / a.G;
  const int row = (t - tile * a.TT) * a.G + (hq - head * a.G);
  const int nbt = tree_tile_blocks(q, tile, a.TT, a.mask != nullptr);
  // pieces that hold a block of this tile: those that start before its last one
  int np = pieces;
  while (np > 1 && tree_piece_start(q.nb, np - 1, pieces) >= nbt) --np;
  const int rows = a.TT * a.G;
  const int rtile = q.tiles - 1 - tile;
  const long long slot0 = sc.y + static_cast<long long>(head) * pieces * q.tiles + rtile;
  auto prow = [&](int p) { return (slot0 + static_cast<long long>(p) * q.tiles) * rows + row; };
  float m = -INFINITY;
  for (int p = lane; p < np; p += 32) m = fmaxf(m, a.part_ml[prow(p)].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float mref = m == -INFINITY ? 0.f : m;
  constexpr int kPer = D / 32;                      // elements of a lane
  float acc[kPer] = {}, l = 0.f;
#pragma unroll 4
  for (int p = 0; p < np; ++p) {
    const long long at = prow(p);
    const float2 ml = a.part_ml[at];
    const float w = ex2(ml.x - mref);
    float v[kPer];
    if constexpr (kPer == 4) {
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(a.part_o + at * D + lane * 4);
    } else {
      *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(a.part_o + at * D + lane * 2);
    }
    l += w * ml.y;
#pragma unroll
    for (int x = 0; x < kPer; ++x) acc[x] += w * v[x];
  }
  const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
  uint16_t* orow = static_cast<uint16_t*>(a.O) + token * a.o_token + hq * a.o_head;
  if constexpr (kPer == 4) {
    uint2 w;
    w.x = pack16x2<kElem>(acc[0] * inv, acc[1] * inv);
    w.y = pack16x2<kElem>(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2*>(orow + lane * 4) = w;
  } else {
    *reinterpret_cast<uint32_t*>(orow + lane * 2) = pack16x2<kElem>(acc[0] * inv, acc[1] * inv);
  }
  if (a.lse && lane == 0) a.lse[wid] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace sa
