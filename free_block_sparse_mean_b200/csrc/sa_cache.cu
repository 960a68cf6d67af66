// C ABI of the paged cache: argument checks, TMA descriptors, workspace layout and
// launches of the step plan, the cache write, the attention of new tokens and the
// move of accepted drafts (kernels: cache_kernels.cuh, tree_kernel.cuh). The
// library's third translation unit, with a device error word of its own that
// sparse_attn_device_error reads with the others.
#include <cudaTypedefs.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/sparse_attn.h"
#include "cache_kernels.cuh"
#include "plan_launch.cuh"
#include "tree_kernel.cuh"

namespace {

constexpr int kSMs = 148;                       // B200
constexpr int64_t kMaxPlaces = 0x7fffffff - 1024;   // places of a request: the sums of one and a block stay ints
// What a tile of one or two chains costs its CTA beside its blocks, in blocks: Q's load, the pass
// of O out of TMEM (256 rows: 4 us). 64 ragged requests of up to 1,000 tokens, us: 51 for 0, 35.6
// for 2, 35.1 for 3, 35.4 for 4; a prompt of 2,048 tokens: 84 for 2, 74 for 4, 70 for 6, 69 for 9;
// 16 x 64 drafts: 193, 181, 176, 177.
constexpr int kTileCost1 = 3, kTileCost2 = 6;
// The join's forms (tree_kernel.cuh), by the tiles that the host expects: a block for each row and
// border at tiles of up to kEachRows rows while there are fewer than kEachTiles; where a tile may be
// in kFewPieces pieces or more, a block for each row of each tile; else eight rows to a block. The
// whole call in us, "each", "few" and "wide", bf16, heads of 128, cached tokens behind the @:
//   1 row, 1 tile @20,000    12.8 14.2 18.4    32 rows, 1 tile @20,000    21.8 14.8 22.0
//   1 row, 24 tiles @4,000   15.8 17.3 16.8    32 rows, 8 tiles @4,000    20.9 14.3 14.6
//   4 rows, 1 tile @20,000   13.8 14.8 19.5    32 rows, 10 tiles @1,000   20.3 13.5 12.4
//   4 rows, 40 tiles @4,000  18.6 20.2 18.9    64 rows, 1 tile @20,000    32.1 15.4 23.5
//   4 rows, 96 tiles @1,000  20.0 22.1 19.3    128 rows, 9 tiles @20,000  67.8 35.7 37.8
//   8 rows, 1 tile @20,000   16.3 16.1 21.7    128 rows, 10 tiles @4,000  54.8 23.4 22.7
//   8 rows, 24 tiles @1,000  14.1 14.1 12.8    two chains, 4 and 5 tiles @4,000: few 23.9, 25.5; wide 24.5, 24.9
// Over 100,000 tokens tiles of 32, 40, 64 and 128 rows of one head: few 24, 25, 26, 31; wide 51, 52, 54, 59.
constexpr int kEachRows = 4, kEachTiles = 64, kFewPieces = 32;
static_assert(2 * kSMs <= 32 * sa::kCutWords, "entries of `cut`");

// A failed call of the runtime stays its last error, and would fail the next call's check of
// its launch, until it is read.
sa_status cuda_failed() {
  (void)cudaGetLastError();
  return SA_ERR_CUDA;
}

bool aligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// A stride of a dimension that is stepped over, in elements: positive, 16-byte steps.
bool good_stride(int64_t s) { return s > 0 && s % 8 == 0 && s < (int64_t{1} << 38); }

int log2_exact(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

sa_status check_cache(const sa_cache& c) {
  if (c.pages < 1 || c.Hkv < 1) return SA_ERR_INVALID_ARG;
  if (c.page_size != 16 && c.page_size != 32 && c.page_size != 64 && c.page_size != 128 && c.page_size != 256)
    return SA_ERR_UNSUPPORTED;
  if (c.d != 64 && c.d != 128) return SA_ERR_UNSUPPORTED;
  if (c.dtype != SA_BF16 && c.dtype != SA_F16) return SA_ERR_UNSUPPORTED;
  if (c.Hkv > 65535) return SA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c.pages) * c.page_size > 0x7fffffff) return SA_ERR_UNSUPPORTED;
  if (!good_stride(c.page_stride) || !good_stride(c.token_stride) || (c.Hkv > 1 && !good_stride(c.head_stride)))
    return SA_ERR_INVALID_ARG;
  return SA_OK;
}

sa_status check_step(const sa_step& s, int page_size) {
  if (s.R < 1 || s.n < 1 || s.width < 1 || s.max_new < 0) return SA_ERR_INVALID_ARG;
  if (!s.starts || !s.lens || !s.table) return SA_ERR_INVALID_ARG;
  if (!aligned(s.starts, 4) || !aligned(s.lens, 4) || !aligned(s.table, 4) || !aligned(s.granted, 4) ||
      !aligned(s.mask, 4))
    return SA_ERR_INVALID_ARG;
  if (s.R > sa::kCacheMaxRequests) return SA_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(s.R) * s.width > 0x7fffffff ||
      static_cast<int64_t>(s.width) * page_size > kMaxPlaces)
    return SA_ERR_UNSUPPORTED;
  if (s.mask ? (s.words < 1 || s.words > 32) : s.words != 0) return SA_ERR_INVALID_ARG;
  return SA_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

bool encode(CUtensorMap* map, const void* ptr, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
            const cuuint32_t* box) {
  auto enc = get_encode();
  if (!enc) return false;
  const cuuint32_t estr[5] = {1u, 1u, 1u, 1u, 1u};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(ptr), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries [n][Hq][d] with their strides as {64 elements, Hq, n, d/64 chunks}: the box
// {64, G, TT, 1} is one column chunk of a tile's rows, token-major.
bool make_q_map(CUtensorMap* map, const void* ptr, int64_t tok, int64_t head, int n, int Hq, int d, int G, int TT) {
  const cuuint64_t dims[4] = {64u, static_cast<cuuint64_t>(Hq), static_cast<cuuint64_t>(n),
                              static_cast<cuuint64_t>(d / 64)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(Hq > 1 ? head : d) * 2,
                                 static_cast<cuuint64_t>(n > 1 ? tok : static_cast<int64_t>(Hq) * d) * 2, 128u};
  const cuuint32_t box[4] = {64u, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(TT), 1u};
  return encode(map, ptr, 4, dims, strides, box);
}

// A cache as {64 elements, page tokens, d/64 chunks, Hkv, pages}. Pages of 64 tokens
// and more: one box {64, 64, d/64, 1, 1} is a whole 64-key block, landing as
// [chunk][token][128 B]; smaller pages: {64, page, 1, 1, 1}, one column chunk of a page.
bool make_cache_map(CUtensorMap* map, const void* ptr, const sa_cache& c) {
  const cuuint64_t dims[5] = {64u, static_cast<cuuint64_t>(c.page_size), static_cast<cuuint64_t>(c.d / 64),
                              static_cast<cuuint64_t>(c.Hkv), static_cast<cuuint64_t>(c.pages)};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(c.token_stride) * 2, 128u,
                                 static_cast<cuuint64_t>(c.Hkv > 1 ? c.head_stride : c.d) * 2,
                                 static_cast<cuuint64_t>(c.page_stride) * 2};
  const bool whole = c.page_size >= 64;
  const cuuint32_t box[5] = {64u, static_cast<cuuint32_t>(whole ? 64 : c.page_size),
                             static_cast<cuuint32_t>(whole ? c.d / 64 : 1), 1u, 1u};
  return encode(map, ptr, 5, dims, strides, box);
}

// The tiling and workspace of sparse_attn_tree_fwd, from what the host knows.
struct TreeLayout {
  int G, TC, chains;          // query heads of a key head, tokens of a chain, chains of a CTA
  int ctas;                   // CTAs that share the call's key blocks
  bool split;                 // the border between two CTAs' shares may cut a tile
  int64_t tiles;              // of the call, if no request has more new tokens than expected
  size_t part_o, part_ml, cut, total;
};
TreeLayout tree_layout(const sa_cache& c, const sa_step& s, int Hq) {
  auto al = [](size_t x) { return (x + 255) / 256 * 256; };
  TreeLayout L{};
  L.G = Hq / c.Hkv;
  // new tokens of a request: the most as given, else their mean, but a full tile of the smallest form
  int most = s.max_new > 0 ? s.max_new : std::max((s.n - 1) / s.R + 1, 32 / L.G);
  if (s.mask) most = std::min(most, 32 * s.words);
  most = std::min(most, s.n);
  L.TC = std::min(128 / L.G, most);
  L.chains = most > L.TC ? 2 : 1;
  L.ctas = L.chains == 2 ? kSMs : 2 * kSMs;
  L.tiles = static_cast<int64_t>(s.R) * c.Hkv * ((most - 1) / (L.chains * L.TC) + 1);
  L.split = static_cast<int64_t>(s.width) * c.page_size > sa::kBlock;
  const size_t rows = L.split ? size_t{2} * L.ctas * L.chains * L.TC * L.G : 0;
  size_t o = 0;
  L.part_o = o; o += al(rows * c.d * sizeof(float));
  L.part_ml = o; o += al(rows * sizeof(float2));
  L.cut = o; o += L.split ? al(L.ctas * sizeof(int4)) : 0;
  L.total = o;
  return L;
}

template <int D, int kElem, int NC, bool kSmallQ>
sa_status launch_tree(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const sa::TreeArgs& a,
                      const void* V, const sa_cache& c, const TreeLayout& L, cudaStream_t st) {
  using Cfg = sa::TreeCfg<D, NC, kSmallQ>;
  auto kern = sa::tree_fwd_kernel<D, kElem, NC, kSmallQ>;
  if (sa::set_smem(kern, Cfg::kSmemBytes) != SA_OK) return cuda_failed();
  // each kernel sets itself up while the one before it in the stream ends, and waits for that itself
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(L.ctas);
  cfg.blockDim = dim3(Cfg::kThreads);
  cfg.dynamicSmemBytes = Cfg::kSmemBytes;
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, mq, mk, mv, a, static_cast<const uint16_t*>(V),
                         static_cast<long long>(c.page_stride), static_cast<long long>(c.token_stride),
                         static_cast<long long>(c.head_stride)) != cudaSuccess)
    return cuda_failed();
  if (L.split) {
    const int rows = a.TT * a.G;
    const int form = rows <= kEachRows && L.tiles < kEachTiles ? sa::kJoinEach
                     : L.tiles * kFewPieces <= L.ctas          ? sa::kJoinFew
                                                               : sa::kJoinWide;
    const auto join = form == sa::kJoinEach  ? sa::tree_combine_kernel<D, kElem, 4, sa::kJoinEach>
                      : form == sa::kJoinFew ? sa::tree_combine_kernel<D, kElem, 4, sa::kJoinFew>
                                             : sa::tree_combine_kernel<D, kElem, NC == 2 ? 2 : 4, sa::kJoinWide>;
    cfg.gridDim = dim3(form == sa::kJoinFew ? static_cast<unsigned>(L.tiles) : L.ctas,
                       form == sa::kJoinWide ? (rows + sa::kCombineRows - 1) / sa::kCombineRows : rows);
    cfg.blockDim = dim3(32 * sa::kCombineWarps);
    cfg.dynamicSmemBytes = 0;
    if (cudaLaunchKernelEx(&cfg, join, a, L.ctas) != cudaSuccess) return cuda_failed();
  }
  return SA_OK;
}

}  // namespace

namespace sa {
// The current GPU's copy of this translation unit's device error word.
cudaError_t cache_device_error_word(void** word) { return cudaGetSymbolAddress(word, g_dev_error); }
}  // namespace sa

extern "C" {

sa_status sparse_attn_cache_plan(const int32_t* lens, const int32_t* new_tokens, const int32_t* held,
                                 const int32_t* nfree, int32_t* free_pages, int32_t* table, const int32_t* parents,
                                 int32_t R, int32_t pages, int32_t page_size, int32_t width, int32_t n,
                                 int32_t words, int32_t* held_out, int32_t* nfree_out, int32_t* starts,
                                 int32_t* granted, int32_t* slots, int32_t* positions, uint32_t* mask,
                                 void* stream) {
  if (!lens || !new_tokens || !held || !nfree || !free_pages || !table || !held_out || !nfree_out || !starts ||
      !granted || !slots || !positions)
    return SA_ERR_INVALID_ARG;
  if (held_out == held || nfree_out == nfree) return SA_ERR_INVALID_ARG;
  if (mask ? (words < 1 || words > 32) : (words != 0 || parents != nullptr)) return SA_ERR_INVALID_ARG;
  if (R < 1 || pages < 1 || width < 1 || n < 1) return SA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(lens), static_cast<const void*>(new_tokens),
                        static_cast<const void*>(held), static_cast<const void*>(nfree),
                        static_cast<const void*>(free_pages), static_cast<const void*>(table),
                        static_cast<const void*>(parents), static_cast<const void*>(held_out),
                        static_cast<const void*>(nfree_out), static_cast<const void*>(starts),
                        static_cast<const void*>(granted), static_cast<const void*>(slots),
                        static_cast<const void*>(positions), static_cast<const void*>(mask)})
    if (!aligned(p, 4)) return SA_ERR_INVALID_ARG;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128 && page_size != 256)
    return SA_ERR_UNSUPPORTED;
  if (R > sa::kCacheMaxRequests || static_cast<int64_t>(pages) * page_size > 0x7fffffff ||
      static_cast<int64_t>(R) * width > 0x7fffffff || static_cast<int64_t>(width) * page_size > kMaxPlaces)
    return SA_ERR_UNSUPPORTED;
  const int bytes = (4 * R + 3) * static_cast<int>(sizeof(int));
  if (sa::set_smem(sa::cache_plan_kernel, (4 * sa::kCacheMaxRequests + 3) * static_cast<int>(sizeof(int))) != SA_OK)
    return cuda_failed();
  sa::CachePlanArgs a{};
  a.lens = lens;
  a.fresh = new_tokens;
  a.held = held;
  a.nfree = nfree;
  a.free_pages = free_pages;
  a.table = table;
  a.parents = parents;
  a.R = R;
  a.pages = pages;
  a.page_shift = log2_exact(page_size);
  a.width = width;
  a.n = n;
  a.words = words;
  a.held_out = held_out;
  a.nfree_out = nfree_out;
  a.starts = starts;
  a.granted = granted;
  a.slots = slots;
  a.positions = positions;
  a.mask = mask;
  // a thread for each token and a warp for each request, within two CTAs on an SM
  const int64_t want = std::max<int64_t>((static_cast<int64_t>(n) + sa::kCachePlanThreads - 1) / sa::kCachePlanThreads,
                                         (R + 7) / 8);
  sa::cache_plan_kernel<<<static_cast<unsigned>(std::min<int64_t>(want, 2 * kSMs)), sa::kCachePlanThreads, bytes,
                          static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

sa_status sparse_attn_cache_write(const void* K, const void* V, int64_t token_stride, int64_t head_stride, int32_t n,
                                  const int32_t* slots, void* K_cache, void* V_cache, sa_cache c, void* stream) {
  if (!K || !V || !slots || !K_cache || !V_cache || n < 1) return SA_ERR_INVALID_ARG;
  const sa_status cs = check_cache(c);
  if (cs != SA_OK) return cs;
  if ((n > 1 && !good_stride(token_stride)) || (c.Hkv > 1 && !good_stride(head_stride))) return SA_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(K_cache, 16) || !aligned(V_cache, 16) || !aligned(slots, 4))
    return SA_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(n) * c.Hkv;
  if (rows > 0x7fffffff) return SA_ERR_UNSUPPORTED;
  sa::CacheWriteArgs a{};
  a.src[0] = static_cast<const uint4*>(K);
  a.src[1] = static_cast<const uint4*>(V);
  a.dst[0] = static_cast<uint4*>(K_cache);
  a.dst[1] = static_cast<uint4*>(V_cache);
  a.slots = slots;
  a.src_token = n > 1 ? token_stride / 8 : 0;
  a.src_head = c.Hkv > 1 ? head_stride / 8 : 0;
  a.dst_page = c.page_stride / 8;
  a.dst_token = c.token_stride / 8;
  a.dst_head = c.Hkv > 1 ? c.head_stride / 8 : 0;
  a.rows = static_cast<unsigned>(rows);
  a.H = static_cast<unsigned>(c.Hkv);
  a.page_shift = log2_exact(c.page_size);
  a.slot_end = static_cast<long long>(c.pages) * c.page_size;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int per = (256 / (c.d / 8)) * 4;             // rows of a CTA
  const dim3 grid(static_cast<unsigned>((rows + per - 1) / per), 2);
  if (c.d == 64)
    sa::cache_write_kernel<8><<<grid, 256, 0, st>>>(a);
  else
    sa::cache_write_kernel<16><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

size_t sparse_attn_tree_workspace_size(sa_cache c, sa_step s, int32_t Hq) {
  if (check_cache(c) != SA_OK || Hq < 1 || Hq % c.Hkv != 0 || Hq / c.Hkv > 128) return 0;
  if (s.R < 1 || s.n < 1 || s.width < 1 || s.max_new < 0 || s.R > sa::kCacheMaxRequests) return 0;
  return std::max<size_t>(tree_layout(c, s, Hq).total, 256);
}

sa_status sparse_attn_tree_fwd(const void* Q, int64_t q_token, int64_t q_head, int32_t Hq, const void* K_cache,
                               const void* V_cache, sa_cache c, sa_step s, float scale, void* O, int64_t o_token,
                               int64_t o_head, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  if (!Q || !K_cache || !V_cache || !O) return SA_ERR_INVALID_ARG;
  const sa_status cs = check_cache(c);
  if (cs != SA_OK) return cs;
  const sa_status ss = check_step(s, c.page_size);
  if (ss != SA_OK) return ss;
  if (Hq < 1 || Hq % c.Hkv != 0) return SA_ERR_INVALID_ARG;
  if (Hq / c.Hkv > 128) return SA_ERR_UNSUPPORTED;
  const float scale_log2 = scale * 1.4426950408889634f;
  if (!(std::isfinite(scale_log2) && scale > 0.f)) return SA_ERR_INVALID_ARG;
  if ((s.n > 1 && (!good_stride(q_token) || !good_stride(o_token))) ||
      (Hq > 1 && (!good_stride(q_head) || !good_stride(o_head))))
    return SA_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(K_cache, 16) || !aligned(V_cache, 16) || !aligned(O, 16) || !aligned(lse, 4))
    return SA_ERR_INVALID_ARG;
  const TreeLayout L = tree_layout(c, s, Hq);
  if (L.total > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < L.total)) return SA_ERR_WORKSPACE;
  CUtensorMap mq, mk, mv;
  if (!make_q_map(&mq, Q, q_token, q_head, s.n, Hq, c.d, L.G, L.TC) || !make_cache_map(&mk, K_cache, c) ||
      !make_cache_map(&mv, V_cache, c))
    return SA_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  sa::TreeArgs a{};
  a.starts = s.starts;
  a.lens = s.lens;
  a.granted = s.granted;
  a.table = s.table;
  a.mask = s.mask;
  a.R = s.R;
  a.n = s.n;
  a.width = s.width;
  a.pages = c.pages;
  a.page_shift = log2_exact(c.page_size);
  a.words = s.words;
  a.Hkv = c.Hkv;
  a.G = L.G;
  a.TT = L.chains * L.TC;
  a.TC = L.TC;
  a.tile_cost = L.chains == 2 ? kTileCost2 : kTileCost1;
  a.min_cost = a.tile_cost + 1;
  a.O = O;
  a.o_token = s.n > 1 ? o_token : 0;
  a.o_head = Hq > 1 ? o_head : 0;
  a.o_wide = aligned(O, 32) && a.o_token % 16 == 0 && a.o_head % 16 == 0;
  a.lse = lse;
  a.scale_log2 = scale_log2;
  if (L.split) {
    a.part_o = reinterpret_cast<float*>(ws + L.part_o);
    a.part_ml = reinterpret_cast<float2*>(ws + L.part_ml);
    a.cut = reinterpret_cast<int4*>(ws + L.cut);
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool small = L.TC * L.G <= 32, f16 = c.dtype == SA_F16;
#define SA_TREE(D, E)                                                                \
  (L.chains == 2 ? launch_tree<D, E, 2, false>(mq, mk, mv, a, V_cache, c, L, st)     \
   : small       ? launch_tree<D, E, 1, true>(mq, mk, mv, a, V_cache, c, L, st)      \
                 : launch_tree<D, E, 1, false>(mq, mk, mv, a, V_cache, c, L, st))
  if (c.d == 64) return f16 ? SA_TREE(64, sa::kElemF16) : SA_TREE(64, sa::kElemBF16);
  return f16 ? SA_TREE(128, sa::kElemF16) : SA_TREE(128, sa::kElemBF16);
#undef SA_TREE
}

sa_status sparse_attn_cache_accept(void* K_cache, void* V_cache, sa_cache c, int32_t layers, int64_t layer_stride,
                                   sa_step s, const int32_t* accepted, int32_t cols, const int32_t* taken,
                                   void* stream) {
  if (!K_cache || !V_cache || !accepted || !taken || layers < 1 || cols < 1) return SA_ERR_INVALID_ARG;
  const sa_status cs = check_cache(c);
  if (cs != SA_OK) return cs;
  const sa_status ss = check_step(s, c.page_size);
  if (ss != SA_OK) return ss;
  if (layers > 1 && !good_stride(layer_stride)) return SA_ERR_INVALID_ARG;
  if (!aligned(K_cache, 16) || !aligned(V_cache, 16) || !aligned(accepted, 4) || !aligned(taken, 4))
    return SA_ERR_INVALID_ARG;
  if (cols > sa::kAcceptMax) return SA_ERR_UNSUPPORTED;
  if (K_cache == V_cache) return SA_ERR_INVALID_ARG;   // two threads would move the same rows, each at its own pace
  sa::CacheAcceptArgs a{};
  a.cache[0] = static_cast<uint4*>(K_cache);
  a.cache[1] = static_cast<uint4*>(V_cache);
  a.lens = s.lens;
  a.starts = s.starts;
  a.granted = s.granted;
  a.table = s.table;
  a.accepted = accepted;
  a.taken = taken;
  a.layer = layers > 1 ? layer_stride / 8 : 0;
  a.page_stride = c.page_stride / 8;
  a.token = c.token_stride / 8;
  a.head = c.Hkv > 1 ? c.head_stride / 8 : 0;
  a.n = s.n;
  a.width = s.width;
  a.cols = cols;
  a.pages = c.pages;
  a.page_shift = log2_exact(c.page_size);
  a.vecs = c.d / 8;
  a.H = c.Hkv;
  a.layers = layers;
  const int64_t columns = int64_t{2} * layers * c.Hkv * a.vecs;
  const dim3 grid(static_cast<unsigned>(s.R), static_cast<unsigned>(std::min<int64_t>((columns + 255) / 256, 65535)));
  sa::cache_accept_kernel<<<grid, 256, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // extern "C"
