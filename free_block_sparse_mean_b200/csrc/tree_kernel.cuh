// Attention of new tokens over a paged cache on sm_100a (tcgen05 + TMA + TMEM):
// one token, a tree of drafted tokens or a chunk of a prompt for each request.
//
//   o[t] = sum_j p[t,j] v_j / sum_j p[t,j],  p[t,j] = exp(scale q_t . k_j)
//
// over the L cached tokens of the request and the new tokens j that t sees (its row
// of mask bits, or all up to itself), in one pass with a running maximum and sum.
//
// Rows. The G query heads that share a key head read the same keys, so a chain of
// products is up to 128 rows of (new token, head of the group), token-major: TC = 128 / G
// tokens. One TMA box {64, G heads, TC tokens} per 128-byte column chunk brings them. A
// request with more rows than that has tiles of two chains (256 rows) on one ring of
// keys and values, so that each block is read once for both: one CTA on an SM, else two.
//
// Work. The lengths are on the GPU and ragged, so a call's work is one line of key
// blocks: request by request, key head by key head, tile by tile, each tile's blocks in
// order and a fixed cost behind them. `ctas` CTAs take equal shares of the line, whatever
// tiles they run through: every CTA finds its share itself, from a scan over the requests.
// A tile that one CTA runs from end to end is written to O; of a tile cut by the border
// between shares each CTA leaves (max, sum, unnormalised O) in fp32 for
// tree_combine_kernel. A CTA cuts at most two tiles, one at each end of its share, so
// 2 * ctas such pieces are all there can be. (One CTA for each tile or for a fixed number
// of blocks, the first form: 425 us for 64 ragged requests, 385 with four times as many
// and smaller pieces, which then cost the short calls; the line: 363.)
//
// Keys. Per 64-key block a warp issues one TMA box (pages of 64 tokens and more) or one
// per page and column chunk (smaller pages). A page id is read only where the request has
// tokens; places behind the last token in its page are masked in S by column, and their V
// rows are set to zero in shared memory, since 0 * NaN is not 0. For the same reason V
// elements that are not finite are taken out of blocks that some row does not see whole;
// the rows that do see such a token get the element added at the end (`special`).
//
// Roles. Of 4 NC warps that issue, 0 walks the share, writes a descriptor of each piece
// for the others and loads K (and V, with one chain), 1 loads Q and deals with unseen V
// rows, then one a chain issues S = Q K^T and one O += P V; with two chains one more
// loads V. 4 NC warps run the softmax (thread = row), the O correction and the epilogue; one
// whose rows do not exist only keeps the barriers' counts. TMEM, 256 columns a chain: S(k)
// in [0,64) or [64,128) by k's parity, P(k) over its first half, O [128, 128 + D).
// What a warp that issues does beside its products, its chain waits for: with the loads in
// the warps of the products, a read of a page id a block, a wait for every V block or
// descriptors of the MMAs built a thread, the 64-key block of two chains took 2,374 cycles;
// now 1,750 (D = 128; 1,024 are the exponential unit's, 1,264 the tensor cores').
//
// Blocks are counted through the CTA's whole share, pieces included, and so are the
// barrier phases: block k uses ring stage k % ST. S(k+2) is issued once P(k).V has
// finished, which needs P(k) of every softmax warp, so each has read S(k) and waited for
// it; the softmax of k+1 runs meanwhile on an S that is there when it begins. P(k) goes
// over S(k): a warp stores its own rows after it has loaded them. A stage is refilled
// after the products that read it have completed. A piece's first P.V overwrites O: its P
// is published only after the softmax warps have read the piece before out of TMEM. The
// softmax waits for P(k-1).V only to correct O. So no wait is ever more than one phase
// behind its barrier.
//
// Measured (B200s, bf16 unless said, in replayed graphs from a cool start; in brackets a long
// loop of calls, where all but the second case may run at the power limit's clock): 64 requests of
// 1..16,384 cached tokens, 32 / 8 heads of 128, one token each, fp16: 336 us (341 to 375),
// 2.2 GB, the rate of a copy; one request of 4,096, 24 heads: 16 us (21, the host's) for 50 MB,
// bound by its chain of set-up, load, softmax, join; 16 requests x 64 drafted tokens: 156 to 171
// us (180 to 187), 586 MB and 145 GFLOP; two chunks of 2,048 tokens behind 30,000 and 7,080:
// 1,235 to 1,250 us (1,255), 1,050 TFLOP/s, bound by the chain of a block's softmax and products;
// with heads of 64 944 us, of which the exponentials are 570. Tried on the chunks and slower or no
// different, each against the build of its time: chains taking turns at the exponentials
// (1,238 -> 1,404), a part of them as polynomials on the FMA pipe (1,406 to 1,469 for one in eight
// to one in two against 1,410 to 1,429, when other things bounded the kernel), exponentials ahead
// of the block's maximum (1,322 -> 1,441), registers split by setmaxnreg (spills).
#pragma once

#include <cuda_fp16.h>

#include "sa_device.cuh"

namespace sa {

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

// NC: chains of a CTA, 128 rows each. Two chains (one CTA on an SM) read every K and V
// block once for 256 rows; a tile of at most 128 rows has one chain, two CTAs on an SM.
// kSmallQ: the tile has at most 32 rows, so Q takes 32 rows of shared memory (twice, so
// that the next tile's is there early) and the freed space a third stage of K and of V.
// The S product reads 64 rows (those behind Q are whatever lies there); a row's
// result touches no other row, and the rows that do not exist are never written out.
template <int D, int NC, bool kSmallQ>
struct TreeCfg {
  static_assert(!(kSmallQ && NC > 1), "a small tile is one chain");
  static constexpr int kThreads = 256 * NC;                // 4 NC warps that issue, 4 NC softmax warps
  static constexpr int kCtas = NC == 1 ? 2 : 1;            // on an SM
  static constexpr int kChunks = D / 64;
  static constexpr int kM = kSmallQ ? 64 : 128;            // rows of the products
  static constexpr int kWarpRows = kM / 4;                 // in each TMEM lane quadrant, in its first lanes
  static constexpr int kQRows = kSmallQ ? 32 : 128;
  static constexpr int kQBufs = kSmallQ ? 2 : 1;
  static constexpr int kQChunkBytes = kQRows * 128;
  static constexpr int kQBytes = kChunks * kQChunkBytes;   // one chain's
  static constexpr int kKVChunkBytes = kBlock * 128;
  static constexpr int kKVBytes = kChunks * kKVChunkBytes;
  static constexpr int ST =                                // stages of K and of V
      NC == 2 ? (D == 64 ? 10 : 5) : (D == 64 ? (kSmallQ ? 6 : 5) : (kSmallQ ? 3 : 2));
  static constexpr int kPieces = 8;                        // ring of piece descriptors, see TreePiece
  static constexpr int oQ = 0;
  static constexpr int oK = oQ + NC * kQBufs * kQBytes;
  static constexpr int oV = oK + ST * kKVBytes;
  static constexpr int oBar = oV + ST * kKVBytes;
  static constexpr int kNumBars = 6 * ST + 2 * kPieces + NC * (2 * kQBufs + 6) + 1;
  static constexpr int oMisc = oBar + kNumBars * 8;
  static constexpr int oPieces = oMisc + 16 * 4 + kThreads / 32 * 8;
  static constexpr int kSmemBytes = oPieces + kPieces * 48;
  static constexpr uint32_t kColS = 0, kColO = 128, kChainCols = 256;   // S(k), then P(k): kColS + 64 (k & 1)
  static_assert(kCtas * (kSmemBytes + 1024) <= 228 * 1024, "shared memory of an SM");
};

struct TreeArgs {
  const int *starts, *lens, *granted, *table;
  const uint32_t* mask;           // [n][words] or null
  int R, n, width, pages, page_shift, words;
  int Hkv, G, TT, TC;             // key heads, query heads each, tokens of a tile, of a chain's part of it
  int tile_cost;                  // what a tile costs beside its blocks, in blocks
  int min_cost;                   // smallest share of a CTA
  void* O;
  long long o_token, o_head;      // strides in elements
  int o_wide;                     // rows of O are 32-byte aligned
  float* lse;                     // [n][Hkv * G] or null
  float scale_log2;
  float* part_o;                  // [2 * CTA + (0: the piece ends its tile, or 1: begins it)][TT * G][D]
  float2* part_ml;                // [as part_o][tile rows]
  int4* cut;                      // [CTA]: first token, rows (0: none) and key head of a tile that it begins and
                                  // does not end, and the CTA that ends it
};

struct TreeReq {
  int T, L, nb, tiles, tok0;      // new and cached tokens, key blocks, tiles, first row of the step
};

// Request r as the kernels take it: T = 0 if it has nothing to compute or its
// numbers are out of range (then *bad is set).
__device__ __forceinline__ TreeReq tree_request(const TreeArgs& a, int r, bool* bad) {
  TreeReq q;
  const int s0 = a.starts[r], s1 = a.starts[r + 1];
  q.L = a.lens[r];
  q.T = s1 - s0;
  q.tok0 = s0;
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

// a / b for a >= 0, b > 0: 64-bit division is a long subroutine, and hardly ever needed.
__device__ __forceinline__ long long div64(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// sum of floor((a i + b) / 64) over i = 0 .. n-1 (a, b >= 0), by the Euclidean reduction:
// take whole parts out of a and b, then count the lattice points the other way. Tiles of
// whole blocks (a a multiple of 64) are done after the first step, which needs no division.
__device__ __forceinline__ long long floor_sum64(long long n, int a0, int b0) {
  static_assert(kBlock == 64, "shifts below");
  long long sum = (n - 1) * n / 2 * (a0 >> 6) + n * (b0 >> 6);
  long long a = a0 & 63, b = b0 & 63, m = 64, y = a * n + b;
  while (y >= m) {
    n = div64(y, m);
    b = y - n * m;
    const long long t = m;
    m = a;
    a = t;
    const long long qa = div64(a, m), qb = div64(b, m);
    sum += (n - 1) * n / 2 * qa + n * qb;
    a -= qa * m;
    b -= qb * m;
    y = a * n + b;
  }
  return sum;
}

// Cost of a key head's first `tiles` tiles of a request: their blocks and tile_cost each.
__device__ __forceinline__ long long tree_cost_before(const TreeReq& q, int tiles, const TreeArgs& a) {
  if (tiles <= 0) return 0;
  const long long own = static_cast<long long>(tiles) * a.tile_cost;
  if (a.mask != nullptr) return static_cast<long long>(tiles) * q.nb + own;
  const int full = min(tiles, q.tiles - 1);            // the last tile may hold fewer tokens
  const long long s = full > 0 ? floor_sum64(full, a.TT, q.L + a.TT + kBlock - 1) : 0;
  return (tiles == q.tiles ? s + q.nb : s) + own;
}

// The share of the line that CTA c of `ctas` takes begins here: floor(total * c / ctas).
__device__ __forceinline__ long long tree_share(long long total, int c, int ctas) {
  const long long q = div64(total, ctas);
  const int rest = static_cast<int>(total - q * ctas);
  return q * c + rest * c / ctas;
}
// The CTA whose share holds place x of the line.
__device__ __forceinline__ int tree_owner(long long total, long long x, int ctas) {
  return static_cast<int>(div64((x + 1) * ctas + total - 1, total)) - 1;
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, int v,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(v), "r"(smem_u32(bar))
      : "memory");
}

// True if the phase with the given parity has completed; does not wait.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// 32 bytes, a whole sector, to a 32-byte aligned address.
__device__ __forceinline__ void st_global_32(void* p, const uint32_t* v) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// True in one thread of the warp, the same one every time. The compiler keeps what is
// uniform in such a branch in uniform registers, where an MMA takes its operands from.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(p));
  return p != 0;
}

// tcgen05.st of 16 packed 32-bit values to this warp's lanes.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
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

// p = 2^(s * sc + nm) for 32 columns of a row: P as 16-bit pairs, the sums of the p on
// two pairs of accumulators. 334 cycles for a warp alone, 268 each for two on a scheduler
// (the exponential unit's own bound is 256; with the multiply-add on pairs 388 and 280).
template <int kElem>
__device__ __forceinline__ void tree_exp32(const float (&s)[32], float sc, float nm, uint64_t& acc0, uint64_t& acc1,
                                           uint32_t* pk) {
#pragma unroll
  for (int c = 0; c < 32; c += 2) {
    const float p0 = ex2(fmaf(s[c], sc, nm)), p1 = ex2(fmaf(s[c + 1], sc, nm));
    if ((c >> 1) & 1)
      acc1 = fadd2(acc1, f2pack(p0, p1));
    else
      acc0 = fadd2(acc0, f2pack(p0, p1));
    pk[c >> 1] = pack16x2<kElem>(p0, p1);
  }
}

// A walk along a CTA's share of the line, tile by tile: the piece of the current tile
// is its blocks [b0, b0 + n). A piece that begins inside its tile is kept for the end, so
// that every CTA begins with block 0 of some tile: the CTAs on one key head then read the
// same keys at about the same time, from L2. In the line's order a prompt's chunk (2 x
// 2,048 tokens behind 30,000, 8 key heads) took 1,622 us, DRAM bound at 9 GB a call,
// against 1,410 (the kernel's first form).
struct TreeWalk {
  int r, head, tile, b0, n, nbt;
  TreeReq q;
  long long left;                 // the share's cost from this piece on, the kept piece aside
  int kr, khead, ktile, kb0;      // the kept piece (kr = -1: none)

  __device__ __forceinline__ void cut(const TreeArgs& a) {
    nbt = tree_tile_blocks(q, tile, a.TT, a.mask != nullptr);
    n = static_cast<int>(min(left, static_cast<long long>(nbt - b0)));
  }
  __device__ __forceinline__ long long after(const TreeArgs& a) const {
    return left - n - (b0 + n == nbt ? a.tile_cost : 0);
  }
  __device__ __forceinline__ bool last(const TreeArgs& a) const { return after(a) <= 0 && kr < 0; }
  // The first piece, from the share's first place: `at` in its tile (r, head, tile, q and
  // left set). False if the share holds no block.
  __device__ __forceinline__ bool begin(const TreeArgs& a, int at) {
    kr = -1;
    nbt = tree_tile_blocks(q, tile, a.TT, a.mask != nullptr);
    if (at >= nbt) {                        // the share begins in what the tile costs beside its blocks
      b0 = nbt;
      n = 0;
      left += at - nbt;
      return next(a);
    }
    b0 = at;
    cut(a);
    if (b0 > 0 && after(a) > 0) {
      const int first = r;
      khead = head;
      ktile = tile;
      kb0 = b0;
      next(a);
      kr = first;
    }
    return true;
  }
  // To the next piece of the share; false at its end.
  __device__ __forceinline__ bool next(const TreeArgs& a) {
    left = after(a);
    bool bad;
    if (left <= 0) {
      if (kr < 0) return false;
      r = kr;
      head = khead;
      tile = ktile;
      b0 = kb0;
      q = tree_request(a, r, &bad);
      nbt = tree_tile_blocks(q, tile, a.TT, a.mask != nullptr);
      n = nbt - b0;
      left = n;
      kr = -1;
      return true;
    }
    b0 = 0;
    if (++tile == q.tiles) {
      tile = 0;
      if (++head == a.Hkv) {
        head = 0;
        do {
          if (++r >= a.R) return false;       // (not reached while the lengths stay as they were)
          q = tree_request(a, r, &bad);
        } while (q.T == 0);
      }
    }
    cut(a);
    return true;
  }
};

// What the other warps need to know of a piece, from the load warp in a ring of kPieces.
struct TreePiece {
  int r, tok0, L, T;              // request, its first row of the step, cached and new tokens
  int head, tile, b0, n, nbt;     // key head, tile, first block, blocks of the piece and of the whole tile
  int last;                       // 1: the share's last piece
  int special;                    // 1: an element of V was taken out
  int pad;
};

// The page ids of a request, for the loads: the lanes hold those of the 32 pages from
// `base` on, and of the 32 behind them, read a window ahead of their use (a read of one id a
// block cost its warp 700 cycles a block). A block's pages never lie in two windows.
struct TreePages {
  const int* row;
  int base, pages, ids, ahead;
  __device__ __forceinline__ int read(int p) const { return p < pages ? row[p] : 0; }
  __device__ __forceinline__ void open(const TreeArgs& a, int r, int keys, int b0, int lane) {
    row = a.table + static_cast<long long>(r) * a.width;
    pages = (keys + (1 << a.page_shift) - 1) >> a.page_shift;
    base = (b0 * kBlock) >> a.page_shift;
    ids = read(base + lane);
    ahead = read(base + 32 + lane);
  }
  __device__ __forceinline__ void advance(const TreeArgs& a, int block, int lane) {
    if ((block * kBlock >> a.page_shift) >= base + 32) {
      base += 32;
      ids = ahead;
      ahead = read(base + 32 + lane);
    }
  }
};

template <int D, int kElem, int NC, bool kSmallQ>
__global__ void __launch_bounds__(TreeCfg<D, NC, kSmallQ>::kThreads, TreeCfg<D, NC, kSmallQ>::kCtas)
    tree_fwd_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                    const __grid_constant__ CUtensorMap tmV, const __grid_constant__ TreeArgs a,
                    const uint16_t* __restrict__ Vraw, long long v_page, long long v_token, long long v_head) {
  using C = TreeCfg<D, NC, kSmallQ>;
  constexpr uint32_t kIdescS = idesc_16_f32(kElem, C::kM, 64, false);
  constexpr uint32_t kIdescPV = idesc_16_f32(kElem, C::kM, D, true);
  constexpr int kWarps = C::kThreads / 32;
  extern __shared__ __align__(1024) uint8_t tree_smem[];
  uint8_t* base = tree_smem;
  if (smem_u32(base) & 1023u) {               // the swizzled tiles need it; the kernel has no static shared memory
    if (threadIdx.x == 0) atomicOr(&g_dev_error, DEVERR_VALUE);
    return;
  }
  uint8_t* sQ = base + C::oQ;
  uint8_t* sK = base + C::oK;
  uint8_t* sV = base + C::oV;
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + C::oBar);
  uint64_t* kfull = bars;                  // [ST] K stage loaded
  uint64_t* kempty = kfull + C::ST;        // [ST] K stage consumed by every chain's S MMA
  uint64_t* vfull = kempty + C::ST;        // [ST] V stage loaded
  uint64_t* vempty = vfull + C::ST;        // [ST] V stage consumed by every chain's P.V MMA
  uint64_t* vready = vempty + C::ST;       // [ST] by number of such a block: what its V holds unseen is dealt with
  uint64_t* vpart = vready + C::ST;        // [ST] by the same number: its V load was issued
  uint64_t* piece_full = vpart + C::ST;   // [kPieces] piece written
  uint64_t* piece_empty = piece_full + C::kPieces;  // [kPieces] piece read by every other warp with a part in it
  uint64_t* q_full = piece_empty + C::kPieces;   // [NC][kQBufs] Q of a tile loaded
  uint64_t* q_empty = q_full + NC * C::kQBufs;  // [NC][kQBufs] the S MMAs of the Q's piece finished
  uint64_t* s_full = q_empty + NC * C::kQBufs;  // [NC][2] by block parity: S(k) written by the MMA
  uint64_t* p_full = s_full + 2 * NC;      // [NC][2] by block parity: P(k) in TMEM and O corrected
  uint64_t* pv_done = p_full + 2 * NC;     // [NC][2] by block parity: P(k).V finished (the MMA and `special`)
  uint64_t* drain = pv_done + 2 * NC;      // every MMA of the CTA finished
  int* misc = reinterpret_cast<int*>(base + C::oMisc);
  volatile int* abort_flag = misc + 0;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(misc + 1);
  int* found = misc + 2;                   // the share's first request, its T, L and first row
  long long* found_at = reinterpret_cast<long long*>(misc + 8);   // the share's start in it, the cost of a key head
  long long* wsum = reinterpret_cast<long long*>(misc + 16);      // [kWarps]
  TreePiece* pieces = reinterpret_cast<TreePiece*>(base + C::oPieces);

  const unsigned FULL = 0xffffffffu;
  const int warp = __shfl_sync(FULL, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;

  // ------------------------------------------------------------ set up, find this CTA's share
  if (threadIdx.x < C::kNumBars) {
    uint64_t* bar = bars + threadIdx.x;
    int count = 1;
    if ((bar >= kempty && bar < vfull) || (bar >= vempty && bar < vready)) count = NC;
    if (bar >= piece_empty && bar < q_full) count = NC + 6 * NC;      // V's loads of two chains read pieces too
    if (bar >= p_full && bar < pv_done) count = 4;
    if (bar >= pv_done && bar < drain) count = 2;
    if (bar == drain) count = 2 * NC;
    mbar_init(bar, count);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) {
    *abort_flag = 0;
    found[0] = -1;
  }
  // what is before in the stream has finished; what is behind may set itself up
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int cta = static_cast<int>(blockIdx.x);
  bool bad = false;
  const bool masked = a.mask != nullptr;
  // a thread takes `per` requests in a row; one scan over the CTA places them on the line
  TreeReq mine{};
  long long per_head = 0, cost = 0;           // of the thread's last request's key heads, of its requests
  const int per = (a.R + C::kThreads - 1) / C::kThreads, r0 = static_cast<int>(threadIdx.x) * per;
  for (int r = r0; r < min(r0 + per, a.R); ++r) {
    mine = tree_request(a, r, &bad);
    per_head = tree_cost_before(mine, mine.tiles, a);
    cost += per_head * a.Hkv;
  }
  long long upto = cost, all = 0;             // of the requests up to the thread's last, of all
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(FULL, upto, o);
    if (lane >= o) upto += x;
  }
  if (lane == 31) wsum[warp] = upto;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) upto += wsum[w];
    all += wsum[w];
  }
  const int ctas = static_cast<int>(min(static_cast<long long>(gridDim.x), div64(all + a.min_cost - 1, a.min_cost)));
  if (threadIdx.x == 0 && a.cut) a.cut[cta] = make_int4(0, 0, 0, 0);
  if (cta == 0 && bad) atomicOr(&g_dev_error, DEVERR_VALUE);
  if (cta >= ctas) return;
  const long long share0 = tree_share(all, cta, ctas), share1 = tree_share(all, cta + 1, ctas);
  if (warp == 1) tmem_alloc(tmem_holder, NC * C::kChainCols);
  if (share0 >= upto - cost && share0 < upto) {       // the share's first place lies in the thread's requests
    int r = r0;
    long long at = upto - cost;
    if (per > 1) {
      for (;; ++r) {
        mine = tree_request(a, r, &bad);
        per_head = tree_cost_before(mine, mine.tiles, a);
        if (share0 < at + per_head * a.Hkv || r + 1 >= min(r0 + per, a.R)) break;
        at += per_head * a.Hkv;
      }
    }
    found[0] = r;
    found[1] = mine.T;
    found[2] = mine.L;
    found[3] = mine.tok0;
    found_at[0] = share0 - at;
    found_at[1] = per_head;
  }
  const int page = 1 << a.page_shift;
  // a block is 64 / sub boxes of `sub` tokens; below 64 tokens a box holds one
  // 128-byte column chunk (lane = chunk * boxes + box), else the whole block
  const int sub_shift = min(a.page_shift, 6), sub = 1 << sub_shift;
  const int subs = kBlock >> sub_shift;
  const int my_sub = lane & (subs - 1), my_chunk = lane >> (6 - sub_shift);
  const bool loads = subs == 1 ? lane == 0 : my_chunk < C::kChunks;
  const int sub_off = my_sub * sub, dst_off = my_chunk * C::kKVChunkBytes + sub_off * 128;

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // piece `item` of the share, once the load warp has written it; null if a wait was given up
  auto piece = [&](int item) -> TreePiece* {
    if (!warp_wait(&piece_full[item % C::kPieces], static_cast<uint32_t>(item / C::kPieces) & 1u, abort_flag))
      return nullptr;
    return &pieces[item % C::kPieces];
  };
  auto release = [&](int item) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&piece_empty[item % C::kPieces]);
  };
  // the first block of a piece from b0 on that reaches place `open`
  auto first_part = [](int open, int b0) { return max(open / kBlock - b0, 0); };
  // the chain has rows in the piece
  auto active = [&](const TreePiece* p, int c) { return p->tile * a.TT + c * a.TC < p->T; };

  // One block of K or V into a stage of its ring: each lane's page and box of it.
  bool bad_page = false;
  auto load_block = [&](const TreePages& pg, uint8_t* dst, const CUtensorMap* map, uint64_t* full, int block, int keys,
                        int head) {
    const int at = block * kBlock + sub_off;
    const int boxes = (min(keys - block * kBlock, kBlock) + sub - 1) >> sub_shift;
    int id = __shfl_sync(FULL, pg.ids, (at >> a.page_shift) - pg.base);
    if (lane == 0) mbar_expect_tx(full, static_cast<uint32_t>(boxes) * sub * 128 * C::kChunks);
    __syncwarp();
    if (loads && at < keys) {
      if (id < 0 || id >= a.pages) {
        bad_page = true;
        id = 0;                                   // flagged; any page of the pool keeps the load in bounds
      }
      tma_load_5d(dst + dst_off, map, 0, at & (page - 1), my_chunk, head, id, full);
    }
  };
  // every load that was issued has landed before the CTA leaves (bounded)
  auto drain_loads = [&](uint64_t* full, int issued) {
    if (lane == 0) {
      for (int b = max(0, issued - C::ST); b < issued; ++b)
        mbar_wait_drain(&full[b % C::ST], static_cast<uint32_t>(b / C::ST) & 1u);
    }
  };
  // what a wait for the stage's previous block waits for
  auto before = [](int n) { return static_cast<uint32_t>(n / C::ST - 1) & 1u; };

  if (warp == 0) {
    // ------------------------------------------------------------ pieces, K loads (one chain: V loads too)
    // stage k % ST holds block k of the share, loaded when the products that read block
    // k - ST have completed
    if (lane == 0) {
      tma_prefetch_desc(&tmK);
      if (NC == 1) tma_prefetch_desc(&tmV);
    }
    TreeWalk w;
    w.r = found[0];
    w.q.T = found[1];
    w.q.L = found[2];
    w.q.tok0 = found[3];
    w.q.nb = (w.q.L + w.q.T + kBlock - 1) / kBlock;
    w.q.tiles = (w.q.T + a.TT - 1) / a.TT;
    w.left = share1 - share0;
    const long long head_cost = max(found_at[1], 1LL);
    long long x = found_at[0], at_tile = 0;
    w.head = static_cast<int>(div64(x, head_cost));
    x -= w.head * head_cost;
    int lo = 0, hi = w.q.tiles;                   // the last tile that begins at or before x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      const long long v = tree_cost_before(w.q, mid, a);
      if (v <= x) {
        lo = mid;
        at_tile = v;
      } else {
        hi = mid;
      }
    }
    w.tile = lo;
    // (every share begins in some request while the lengths stay as they were)
    bool more = found[0] >= 0 && w.begin(a, static_cast<int>(x - at_tile));
    if (!more && lane == 0) {                     // no block at all: an empty piece for the others
      pieces[0] = TreePiece{};
      pieces[0].last = 1;
      mbar_arrive(&piece_full[0]);
    }
    int k = 0, nk = 0, nw = 0;                    // blocks of the share, K loads, blocks seen in part
    for (int item = 0; more; ++item) {
      if (item >= C::kPieces &&
          !warp_wait(&piece_empty[item % C::kPieces], static_cast<uint32_t>(item / C::kPieces - 1) & 1u, abort_flag))
        break;
      const int keys = w.q.L + w.q.T;
      TreePages pg;
      pg.open(a, w.r, keys, w.b0, lane);
      if (lane == 0) {
        TreePiece* p = &pieces[item % C::kPieces];
        p->r = w.r;
        p->tok0 = w.q.tok0;
        p->L = w.q.L;
        p->T = w.q.T;
        p->head = w.head;
        p->tile = w.tile;
        p->b0 = w.b0;
        p->n = w.n;
        p->nbt = w.nbt;
        p->last = w.last(a);
        p->special = 0;
        if (w.b0 == 0 && w.n < w.nbt)             // (its blocks are the share's last)
          a.cut[cta] = make_int4(p->tok0 + p->tile * a.TT, min(a.TT, p->T - p->tile * a.TT) * a.G, p->head,
                                 tree_owner(all, share1 - p->n + p->nbt - 1, ctas));
        mbar_arrive(&piece_full[item % C::kPieces]);
      }
      __syncwarp();
      const int part = first_part(masked ? w.q.L : w.q.L + w.tile * a.TT + 1, w.b0);
      int i = 0;
      for (; i < w.n; ++i, ++k) {
        const int s = k % C::ST;
        pg.advance(a, w.b0 + i, lane);
        if (k >= C::ST && !warp_wait(&kempty[s], before(k), abort_flag)) break;
        load_block(pg, sK + s * C::kKVBytes, &tmK, &kfull[s], w.b0 + i, keys, w.head);
        nk = k + 1;
        if (NC == 1) {
          if (k >= C::ST && !warp_wait(&vempty[s], before(k), abort_flag)) break;
          load_block(pg, sV + s * C::kKVBytes, &tmV, &vfull[s], w.b0 + i, keys, w.head);
          if (i >= part) {
            if (lane == 0) mbar_arrive(&vpart[nw % C::ST]);
            ++nw;
          }
        }
      }
      if (i < w.n) break;
      more = w.next(a);
    }
    drain_loads(kfull, nk);
    if (NC == 1) drain_loads(vfull, k);
  } else if (NC == 2 && warp == 2 + 2 * NC) {
    // ------------------------------------------------------------ V loads
    if (lane == 0) tma_prefetch_desc(&tmV);
    int k = 0, nw = 0;
    for (int item = 0;; ++item) {
      const TreePiece* p = piece(item);
      if (!p) break;
      const int keys = p->L + p->T, n = p->n, b0 = p->b0, head = p->head, last = p->last;
      const int part = first_part(masked ? p->L : p->L + p->tile * a.TT + 1, b0);
      TreePages pg;
      pg.open(a, p->r, keys, b0, lane);
      release(item);
      int i = 0;
      for (; i < n; ++i, ++k) {
        const int s = k % C::ST;
        pg.advance(a, b0 + i, lane);
        if (k >= C::ST && !warp_wait(&vempty[s], before(k), abort_flag)) break;
        load_block(pg, sV + s * C::kKVBytes, &tmV, &vfull[s], b0 + i, keys, head);
        if (i >= part) {
          if (lane == 0) mbar_arrive(&vpart[nw % C::ST]);
          ++nw;
        }
      }
      if (i < n || last) break;
    }
    drain_loads(vfull, k);
  } else if (warp == 1) {
    // ------------------------------------------------------------ Q loads, what a V block holds unseen
    if (lane == 0) tma_prefetch_desc(&tmQ);
    // Only blocks that some row does not see whole are waited for: a warp that waited for
    // every V block as it came in slowed the softmax warps on its scheduler by a third.
    int k = 0, nw = 0, nq[NC] = {};               // blocks of the share, of them seen in part, Q tiles of each chain
    bool ok = true;
    for (int item = 0; ok; ++item) {
      TreePiece* p = piece(item);
      if (!p) break;
#pragma unroll
      for (int c = 0; c < NC; ++c) {
        if (!ok || !active(p, c)) continue;
        const int buf = c * C::kQBufs + nq[c] % C::kQBufs;
        if (nq[c] >= C::kQBufs &&
            !warp_wait(&q_empty[buf], static_cast<uint32_t>(nq[c] / C::kQBufs - 1) & 1u, abort_flag)) {
          ok = false;
          continue;
        }
        if (lane == 0) {
          mbar_expect_tx(&q_full[buf], C::kChunks * a.TC * a.G * 128);
#pragma unroll
          for (int x = 0; x < C::kChunks; ++x)
            tma_load_4d(sQ + buf * C::kQBytes + x * C::kQChunkBytes, &tmQ, 0, p->head * a.G,
                        p->tok0 + p->tile * a.TT + c * a.TC, x, &q_full[buf]);
        }
        __syncwarp();
        ++nq[c];
      }
      const int keys = p->L + p->T, n = p->n, b0 = p->b0, last = p->last;
      // every row of the tile sees the keys before `open`; from there on rows differ
      const int open = masked ? p->L : p->L + p->tile * a.TT + 1;
      for (int i = first_part(open, b0); ok && i < n; ++i, ++nw) {
        const int s = (k + i) % C::ST;
        // (vpart first: the block's phase of vfull has begun)
        if (!warp_wait(&vpart[nw % C::ST], static_cast<uint32_t>(nw / C::ST) & 1u, abort_flag) ||
            !warp_wait(&vfull[s], static_cast<uint32_t>((k + i) / C::ST) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        const int kb = (b0 + i) * kBlock;
        // rows behind the last token to zero; elements that are not finite out of
        // the rows that not every query sees
        const int live = min(kBlock, keys - kb), seen = max(0, min(open - kb, live));
        bool taken_out = false;
        uint8_t* v = sV + s * C::kKVBytes;
        for (int h = 0; h < C::kChunks; ++h) {
          for (int x = seen * 8 + lane; x < kBlock * 8; x += 32) {     // 16-byte pieces, 8 a row
            uint4* at = reinterpret_cast<uint4*>(v + h * C::kKVChunkBytes + x * 16);
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
        if (__any_sync(FULL, taken_out) && lane == 0) p->special = 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(&vready[nw % C::ST]);
      }
      k += n;
      release(item);
      if (last) break;
    }
    if (lane == 0) {                              // (bounded; complete unless aborted)
      for (int c = 0; c < NC; ++c)
        for (int b = max(0, nq[c] - C::kQBufs); b < nq[c]; ++b)
          mbar_wait_drain(&q_full[c * C::kQBufs + b % C::kQBufs], static_cast<uint32_t>(b / C::kQBufs) & 1u);
    }
  } else if (warp < 2 + NC) {
    // ------------------------------------------------------------ S = Q K^T of chain c
    const int c = warp - 2;
    const uint32_t tS = tmem_base + c * C::kChainCols + C::kColS;
    const uint64_t dK = sdesc_sw128(smem_u32(sK), 16, 1024);
    const uint64_t dQ = sdesc_sw128(smem_u32(sQ) + c * C::kQBufs * C::kQBytes, 16, 1024);
    int k = 0, kc = 0, nq = 0;                    // blocks of the share, of the chain, tiles of the chain
    bool ok = true;
    for (int item = 0; ok; ++item) {
      const TreePiece* p = piece(item);
      if (!p) break;
      const bool act = active(p, c);
      const int n = p->n, last = p->last, buf = nq % C::kQBufs;
      const uint64_t dq = dQ + buf * (C::kQBytes >> 4);
      release(item);
      if (act && !warp_wait(&q_full[c * C::kQBufs + buf], static_cast<uint32_t>(nq / C::kQBufs) & 1u, abort_flag))
        break;
      for (int i = 0; i < n; ++i, ++k) {
        const int s = k % C::ST;
        if ((act && kc > 1 &&
             !warp_wait(&pv_done[2 * c + (kc & 1)], static_cast<uint32_t>((kc - 2) >> 1) & 1u, abort_flag)) ||
            !warp_wait(&kfull[s], static_cast<uint32_t>(k / C::ST) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        if (!act) {
          if (lane == 0) mbar_arrive(&kempty[s]);
          continue;
        }
        tc_fence_after();
        const uint64_t dk = dK + s * (C::kKVBytes >> 4);
        const uint32_t tD = tS + (kc & 1) * 64;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk & 3) * 2;            // 16 columns, in 16-byte steps
            tc_mma_ss(tD, dq + (kk >> 2) * (C::kQChunkBytes >> 4) + off, dk + (kk >> 2) * (C::kKVChunkBytes >> 4) + off,
                      kIdescS, kk > 0 ? 1u : 0u);
          }
          tc_commit(&s_full[2 * c + (kc & 1)]);
          tc_commit(&kempty[s]);
          if (i + 1 == n) tc_commit(&q_empty[c * C::kQBufs + buf]);
        }
        __syncwarp();
        ++kc;
      }
      if (act) ++nq;
      if (last) break;
    }
    if (elect_one()) {                            // (bounded)
      tc_commit(drain);
      mbar_wait_drain(drain, 0u);
    }
  } else if (warp < 2 + 2 * NC) {
    // ------------------------------------------------------------ O += P V of chain c
    const int c = warp - 2 - NC;
    const uint32_t tP = tmem_base + c * C::kChainCols + C::kColS, tO = tmem_base + c * C::kChainCols + C::kColO;
    const uint64_t dV = sdesc_sw128(smem_u32(sV), C::kKVChunkBytes, 1024);
    int k = 0, kc = 0, nw = 0;                    // blocks of the share, of the chain, of those seen in part
    bool ok = true;
    for (int item = 0; ok; ++item) {
      const TreePiece* p = piece(item);
      if (!p) break;
      const bool act = active(p, c);
      const int n = p->n, last = p->last;
      const int part = first_part(masked ? p->L : p->L + p->tile * a.TT + 1, p->b0);
      release(item);
      for (int i = 0; i < n; ++i, ++k) {
        const int s = k % C::ST;
        bool ready = warp_wait(&vfull[s], static_cast<uint32_t>(k / C::ST) & 1u, abort_flag);
        if (ready && i >= part) {
          ready = warp_wait(&vready[nw % C::ST], static_cast<uint32_t>(nw / C::ST) & 1u, abort_flag);
          ++nw;
        }
        if (!ready ||
            (act && !warp_wait(&p_full[2 * c + (kc & 1)], static_cast<uint32_t>(kc >> 1) & 1u, abort_flag))) {
          ok = false;
          break;
        }
        if (!act) {
          if (lane == 0) mbar_arrive(&vempty[s]);
          continue;
        }
        tc_fence_after();
        const uint64_t dv = dV + s * (C::kKVBytes >> 4);
        const uint32_t tA = tP + (kc & 1) * 64, more = i > 0 ? 1u : 0u;
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < kBlock / 16; ++kk)
            tc_mma_ts(tO, tA + kk * 8, dv + kk * (16 * 128 >> 4), kIdescPV, kk > 0 ? 1u : more);
          tc_commit(&pv_done[2 * c + (kc & 1)]);
          tc_commit(&vempty[s]);
          mbar_arrive(&pv_done[2 * c + (kc & 1)]);      // passes on the piece's `special`, seen through vready
        }
        __syncwarp();
        ++kc;
      }
      if (last) break;
    }
    if (elect_one()) {                            // (bounded)
      tc_commit(drain);
      mbar_wait_drain(drain, 0u);
    }
  } else if (warp >= 4 * NC) {
    // ------------------------------------------------------------ softmax warps
    const int c = (warp - 4 * NC) >> 2;            // the chain
    const int wq = warp & 3;                       // TMEM lane quadrant: rows 32*wq ..
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t s_addr = tmem_base + lane_bits + c * C::kChainCols + C::kColS;
    const uint32_t o_addr = tmem_base + lane_bits + c * C::kChainCols + C::kColO;
    s_full += 2 * c;
    p_full += 2 * c;
    pv_done += 2 * c;
    const int row = wq * C::kWarpRows + lane;
    // P = 2^(s - m_ref) is rounded to the type: that is what the tensor cores multiply V with
    // (two products, of P's head and rest, would be half as many again). bf16 has fp32's range.
    // fp16 holds 2^-24 to 2^16: its reference is 2^6 below the maximum it was taken from, so
    // that P stays below 2^12 (2^14 with scores up to 2^26, whose own steps are 4) and a key is
    // only lost below 2^-31 of the row's largest probability. With the maximum itself as reference
    // that was 2^-25: 100,000 such keys behind one peak weigh 3e-3, six roundings of the result.
    constexpr float kRefBelow = kElem == kElemF16 ? 6.f : 0.f, kRefGrowth = kElem == kElemF16 ? 12.f : 8.f;
    bool alive = true;
    int k = 0;                                     // blocks of the chain
    for (int item = 0; alive; ++item) {
      const TreePiece* p = piece(item);
      if (!p) break;
      const int n = p->n, last = p->last;
      const int t0 = p->tile * a.TT + c * a.TC;
      const int rows = min(a.TC, p->T - t0) * a.G;            // rows of the chain that exist
      if (wq * C::kWarpRows >= rows) {
        for (int i = 0; rows > 0 && i < n; ++i, ++k) {
          if (!warp_wait(&s_full[k & 1], static_cast<uint32_t>(k >> 1) & 1u, abort_flag)) {
            alive = false;
            break;
          }
          if (lane == 0) mbar_arrive(&p_full[k & 1]);
        }
        release(item);
        if (last) break;
        continue;
      }
      const bool valid = row < rows && lane < C::kWarpRows;
      const int b0 = p->b0;
      const int open = masked ? p->L : p->L + t0 + 1;         // every row of the chain sees the keys before it
      float m_ref = -INFINITY, l = 0.f;
      float s0[32], s1[32];                        // S(k) of the row: columns 0..31 and 32..63
      if (warp_wait(&s_full[k & 1], static_cast<uint32_t>(k >> 1) & 1u, abort_flag)) {
        tc_fence_after();
        tmem_ld32(s_addr + (k & 1) * 64, s0);
        tmem_ld32(s_addr + (k & 1) * 64 + 32, s1);
      } else {
        alive = false;
      }
      for (int i = 0; alive && i < n; ++i, ++k) {
        const int kb = (b0 + i) * kBlock;
        unsigned long long vis = ~0ull;
        const bool part = kb + kBlock > open;       // some row does not see the whole block
        if (part) {
          const int t = t0 + row / a.G;
          vis = valid ? tree_visible(a, p->L, p->T, t, static_cast<long long>(p->tok0) + t, kb) : 0ull;
        }
        tmem_wait_ld();
        pin32(s0);
        pin32(s1);
        if (part) {
          const uint32_t vlo = static_cast<uint32_t>(vis), vhi = static_cast<uint32_t>(vis >> 32);
#pragma unroll
          for (int x = 0; x < 32; ++x) {
            s0[x] = (vlo >> x) & 1u ? s0[x] : -INFINITY;
            s1[x] = (vhi >> x) & 1u ? s1[x] : -INFINITY;
          }
        }
        float mx[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) mx[u] = fmax3(s0[u], s0[u + 8], s0[u + 16]);
#pragma unroll
        for (int u = 0; u < 8; ++u) mx[u] = fmax3(mx[u], s0[u + 24], s1[u]);
#pragma unroll
        for (int u = 0; u < 8; ++u) mx[u] = fmax3(mx[u], s1[u + 8], s1[u + 16]);
#pragma unroll
        for (int u = 0; u < 8; ++u) mx[u] = fmaxf(mx[u], s1[u + 24]);
        const float rmax = fmax3(fmax3(mx[0], mx[1], mx[2]), fmax3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) *
                           a.scale_log2;
        // the reference is raised only when a row's maximum has grown by more than
        // 2^8 (fp16: 2^6), so that O and l are seldom corrected; see kRefBelow
        const bool raise = rmax > m_ref + kRefGrowth;
        float alpha = 1.f;
        if (raise) {
          const float m_new = rmax - kRefBelow;
          alpha = ex2(m_ref - m_new);
          m_ref = m_new;
        }
        const bool any_raise = __any_sync(FULL, raise);
        const float mref = (m_ref == -INFINITY) ? 0.f : m_ref;
        uint64_t acc0 = f2pack(0.f, 0.f), acc1 = acc0;
        uint32_t pk[16];
        tree_exp32<kElem>(s0, a.scale_log2, -mref, acc0, acc1, pk);
        tmem_st16u(s_addr + (k & 1) * 64, pk);
        // S(k+1), if it is there already, comes in under the second half
        const uint32_t s_next = s_addr + ((k + 1) & 1) * 64;
        const bool early = NC == 2 && i + 1 < n &&
                           __all_sync(FULL, mbar_test(&s_full[(k + 1) & 1], static_cast<uint32_t>((k + 1) >> 1) & 1u));
        if (early) {
          tc_fence_after();
          tmem_ld32(s_next, s0);
        }
        tree_exp32<kElem>(s1, a.scale_log2, -mref, acc0, acc1, pk);
        tmem_st16u(s_addr + (k & 1) * 64 + 16, pk);
        if (early) tmem_ld32(s_next + 32, s1);
        float r0, r1, r2, r3;
        f2unpack(acc0, r0, r1);
        f2unpack(acc1, r2, r3);
        l = l * alpha + ((r0 + r1) + (r2 + r3));
        if (i > 0 && any_raise) {
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
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[k & 1]);
        if (i + 1 < n && !early) {
          if (!warp_wait(&s_full[(k + 1) & 1], static_cast<uint32_t>((k + 1) >> 1) & 1u, abort_flag)) {
            alive = false;
            break;
          }
          tc_fence_after();
          tmem_ld32(s_next, s0);
          tmem_ld32(s_next + 32, s1);
        }
      }
      tmem_wait_ld();
      // ------------------------------------------------------------ epilogue of the piece
      if (!alive || !warp_wait(&pv_done[(k - 1) & 1], static_cast<uint32_t>((k - 1) >> 1) & 1u, abort_flag)) break;
      tc_fence_after();
      const bool whole_row = b0 == 0 && n == p->nbt;
      const float mul = whole_row ? (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l)) : 1.f;   // a NaN sum stays one
      const bool fix = *reinterpret_cast<volatile const int*>(&p->special) != 0;
      const int row_t = row / a.G, t = t0 + row_t;
      const int hq = p->head * a.G + row - row_t * a.G;
      const long long token = static_cast<long long>(p->tok0) + t;
      const long long prow = (2LL * cta + (b0 == 0 ? 1 : 0)) * (a.TT * a.G) + c * a.TC * a.G + row;
      uint16_t* orow = static_cast<uint16_t*>(a.O) + token * a.o_token + hq * a.o_head;
      if (__builtin_expect(fix, 0)) {
        // The elements taken out of V (from the tile's `open` on) are added to O, for the
        // rows that see their token. Apart from the pass below: in it, this code cost every
        // piece its instruction fetches (500 requests of up to 500 tokens: 152 us for 125).
        const int out0 = masked ? p->L : p->L + p->tile * a.TT + 1;
        const int* trow = a.table + static_cast<long long>(p->r) * a.width;
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          float o[32];
          tmem_ld32(o_addr + cc, o);
          tmem_wait_ld();
          pin32(o);
          for (int kb = b0 * kBlock; valid && kb < (b0 + n) * kBlock; kb += kBlock) {
            if (kb + kBlock <= out0) continue;
            unsigned long long vis = tree_visible(a, p->L, p->T, t, token, kb);
            if (out0 > kb) vis &= ~low_bits64(out0 - kb);
            for (; vis; vis &= vis - 1) {
              const int at = kb + __ffsll(static_cast<long long>(vis)) - 1;
              const int id = trow[at >> a.page_shift];
              if (id < 0 || id >= a.pages) continue;
              const uint16_t* v = Vraw + id * v_page + (at & (page - 1)) * v_token + p->head * v_head + cc;
#pragma unroll
              for (int x = 0; x < 32; ++x) {
                const uint32_t e = v[x];
                if (not_finite16<kElem>(e)) o[x] += to_float16<kElem>(e);
              }
            }
          }
          __syncwarp();
          tmem_st32(o_addr + cc, o);
        }
        tmem_wait_st();
      }
#pragma unroll 1
      for (int cc = 0; cc < D; cc += 64) {
        tmem_ld32(o_addr + cc, s0);
        tmem_ld32(o_addr + cc + 32, s1);
        tmem_wait_ld();
        pin32(s0);
        pin32(s1);
        if (valid) {
          if (l == 0.f) {                             // nothing was seen: 0 whatever the products were
#pragma unroll
            for (int x = 0; x < 32; ++x) s0[x] = s1[x] = 0.f;
          }
          if (whole_row) {
            uint32_t w[32];
#pragma unroll
            for (int x = 0; x < 16; ++x) {
              w[x] = pack16x2<kElem>(s0[2 * x] * mul, s0[2 * x + 1] * mul);
              w[x + 16] = pack16x2<kElem>(s1[2 * x] * mul, s1[2 * x + 1] * mul);
            }
            if (a.o_wide) {
#pragma unroll
              for (int x = 0; x < 32; x += 8) st_global_32(orow + cc + 2 * x, w + x);
            } else {
#pragma unroll
              for (int x = 0; x < 32; x += 4)
                *reinterpret_cast<uint4*>(orow + cc + 2 * x) = make_uint4(w[x], w[x + 1], w[x + 2], w[x + 3]);
            }
          } else {
            float* to = a.part_o + prow * D + cc;
#pragma unroll
            for (int x = 0; x < 32; x += 8) {
              st_global_32(to + x, reinterpret_cast<const uint32_t*>(s0) + x);
              st_global_32(to + 32 + x, reinterpret_cast<const uint32_t*>(s1) + x);
            }
          }
        }
        __syncwarp();
      }
      if (valid) {
        if (!whole_row)
          a.part_ml[prow] = make_float2(m_ref, l);
        else if (a.lse)
          a.lse[token * (a.Hkv * a.G) + hq] = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * 0.6931471805599453f;
      }
      tc_fence_before();                            // O is read before the next piece's P is published
      release(item);
      if (last) break;
    }
  }
  if (bad_page) atomicOr(&g_dev_error, DEVERR_RANGE);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, NC * C::kChainCols);
  }
}

// Joins the pieces of the tiles that the shares' borders cut: for each row the largest
// of the pieces' maxima, then O = sum w_p O_p / sum w_p l_p, w_p = 2^(m_p - m), summed in a
// fixed order. The tile that CTA c began and did not end is in entry c of `cut`. (Looking for
// cut tiles from every (token, head) took 89 us for a prompt's chunk of 4,096 x 32 rows of which
// 148 x 256 are cut; this takes 9.)
// Forms, by what the host expects:
// kJoinWide: block x looks at entry x, blocks y share its rows, a warp to each. Many tiles, each
// in few pieces; most blocks find nothing to do.
// kJoinEach: block (x, y) takes row y of entry x, all warps together, each every eighth piece.
// Tiles of one to four rows.
// kJoinFew: as kJoinEach, but blocks x share the cut tiles, looked for through all entries, so
// that no more blocks are launched than there are rows. Few tiles, each in dozens of pieces.
// kBatch: pieces that a warp reads at once. Tiles of two chains have many rows in two or three
// pieces: two, in the registers that let an SM hold all its warps (3 x 500 new tokens behind
// 1,000, the whole call: 54 us for four, 50 for two). Others four (7 x 13 drafts 18.2 us, for two
// 20.3).
constexpr int kCombineWarps = 8;
constexpr int kCombineRows = 8;      // of a block, kJoinWide
constexpr int kCutWords = 10;        // 32 entries of `cut` each

enum JoinForm : int { kJoinWide, kJoinEach, kJoinFew };

template <int D, int kElem, int kBatch, int kForm>
__global__ void __launch_bounds__(32 * kCombineWarps, kBatch == 2 ? 8 : 4)
    tree_combine_kernel(const __grid_constant__ TreeArgs a, int ctas) {
  constexpr int kPer = D / 32;                      // elements of a lane
  constexpr bool kTogether = kForm != kJoinWide;    // all warps at one row
  constexpr int kStep = kTogether ? kCombineWarps : 1;
  __shared__ float s_o[kTogether ? kCombineWarps : 1][D];
  __shared__ float2 s_ml[kTogether ? kCombineWarps : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  auto join = [&](const int4& tile, int c0, int row) {
    const int np = tile.w - c0 + 1;
    auto at = [&](int p) { return (2LL * (c0 + p) + (p == 0 ? 1 : 0)) * (a.TT * a.G) + row; };
    float m = -INFINITY, l = 0.f, acc[kPer] = {};
    auto add = [&](float m1, float l1, const float (&v)[kPer]) {   // one more piece
      const float top = fmaxf(m, m1), ref = top == -INFINITY ? 0.f : top;
      const float w0 = ex2(m - ref), w1 = ex2(m1 - ref);
      m = top;
      l = l * w0 + l1 * w1;
#pragma unroll
      for (int x = 0; x < kPer; ++x) acc[x] = acc[x] * w0 + v[x] * w1;
    };
    for (int p0 = kTogether ? warp : 0; p0 < np; p0 += kBatch * kStep) {
      float2 ml[kBatch];
      float v[kBatch][kPer];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const int p = p0 + u * kStep;
        if (p < np) {
          ml[u] = a.part_ml[at(p)];
          if constexpr (kPer == 4) {
            *reinterpret_cast<float4*>(v[u]) = *reinterpret_cast<const float4*>(a.part_o + at(p) * D + lane * 4);
          } else {
            *reinterpret_cast<float2*>(v[u]) = *reinterpret_cast<const float2*>(a.part_o + at(p) * D + lane * 2);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (p0 + u * kStep < np) add(ml[u].x, ml[u].y, v[u]);
    }
    if constexpr (kTogether) {
#pragma unroll
      for (int x = 0; x < kPer; ++x) s_o[warp][lane * kPer + x] = acc[x];
      if (lane == 0) s_ml[warp] = make_float2(m, l);
      __syncthreads();
      if (warp == 0) {
        const int used = min(kCombineWarps, np);
        for (int w = 1; w < used; ++w) {
          float v[kPer];
#pragma unroll
          for (int x = 0; x < kPer; ++x) v[x] = s_o[w][lane * kPer + x];
          add(s_ml[w].x, s_ml[w].y, v);
        }
      }
    }
    if (!kTogether || warp == 0) {
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      const long long token = static_cast<long long>(tile.x) + row / a.G;
      const int hq = tile.z * a.G + row % a.G;
      uint16_t* orow = static_cast<uint16_t*>(a.O) + token * a.o_token + hq * a.o_head;
      if constexpr (kPer == 4) {
        uint2 w;
        w.x = pack16x2<kElem>(acc[0] * inv, acc[1] * inv);
        w.y = pack16x2<kElem>(acc[2] * inv, acc[3] * inv);
        *reinterpret_cast<uint2*>(orow + lane * 4) = w;
      } else {
        *reinterpret_cast<uint32_t*>(orow + lane * 2) = pack16x2<kElem>(acc[0] * inv, acc[1] * inv);
      }
      if (a.lse && lane == 0)
        a.lse[token * (a.Hkv * a.G) + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
    }
    if constexpr (kForm == kJoinFew) __syncthreads();
  };
  const int x = static_cast<int>(blockIdx.x), y = static_cast<int>(blockIdx.y);
  if constexpr (kForm == kJoinWide) {
    const int4 tile = a.cut[x];
    const int row0 = y * kCombineRows;
    for (int row = row0 + warp; row < min(row0 + kCombineRows, tile.y); row += kCombineWarps) join(tile, x, row);
  } else if constexpr (kForm == kJoinEach) {
    const int4 tile = a.cut[x];
    if (y < tile.y) join(tile, x, y);
  } else {
    unsigned has[kCutWords];                        // the entries whose tile has row y
#pragma unroll
    for (int w = 0; w < kCutWords; ++w) {
      const int c = w * 32 + lane;
      has[w] = __ballot_sync(0xffffffffu, c < ctas && a.cut[c].y > y);
    }
    for (int k = x;; k += static_cast<int>(gridDim.x)) {
      int before = 0, c0 = -1;                      // the k-th of them
#pragma unroll
      for (int w = 0; w < kCutWords; ++w) {
        const int n = __popc(has[w]);
        if (k >= before && k < before + n) {
          unsigned rest = has[w];
          for (int i = before; i < k; ++i) rest &= rest - 1;
          c0 = w * 32 + __ffs(static_cast<int>(rest)) - 1;
        }
        before += n;
      }
      if (c0 < 0) return;
      join(a.cut[c0], c0, y);
    }
  }
}

}  // namespace sa
