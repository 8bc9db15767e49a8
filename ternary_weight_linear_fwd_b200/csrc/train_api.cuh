// train_api.cuh -- the C entry points of BitLinear's training side
// (include/bitlinear.h, section "Training"): argument checks, launch shapes and
// launches.  Part of the library's one translation unit.
#pragma once
#include "train_few.cuh"

namespace bl {
namespace {

// Most 8-wide chunks of a row that a lane of the row kernels keeps in registers.
constexpr int kLnMaxChunks = 10;
constexpr int kGluMaxChunks = 6;

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline bool aligned2(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 1u) == 0; }

bitlinear_status check_rows(int M, int K) {
  return M < 1 || M > BITLINEAR_MAX_M || K < 1 || K > BITLINEAR_MAX_K ? BITLINEAR_ERR_SHAPE : BITLINEAR_OK;
}

// Threads a row for the element-wise kernels of 16 values a thread and step: at most `steps` steps, since each
// step's loads are independent of the last one's and rows seldom divide into many threads evenly (4096 x 2560:
// the restored activation 8.8 us with eight steps, 9.6 with four; the gate's gradients 17.8 and 16.8).
int row_lanes(int M, int K, int steps, int sm_count) {
  int lanes = 32;
  while (lanes < 256 && 16 * lanes < K &&
         (steps * 16 * lanes < K || static_cast<int64_t>(M) * lanes * steps < 4096ll * sm_count))
    lanes *= 2;
  return lanes;
}

// Warps a row: the fewest that keep it in registers (at most G 8-wide chunks a lane), more while the rows are few.
int row_warps(int M, int K, int G, int sm_count) {
  const int chunks = (K + 7) / 8;
  int wpr = 1;
  while (wpr < kQuantWarps && (chunks > G * 32 * wpr ||
                               (static_cast<int64_t>(M) * wpr < 12ll * sm_count && chunks > 32 * wpr)))
    wpr *= 2;
  return wpr;
}
int log2i(int v) { return v <= 1 ? 0 : 1 + log2i(v / 2); }
int row_chunks(int K, int wpr) { return ((K + 7) / 8 + 32 * wpr - 1) / (32 * wpr); }

// Rows of K bf16, ld apart, that 16-byte accesses can take.
bool rows16(const void* p, int64_t ld, int K) { return K % 8 == 0 && ld % 8 == 0 && aligned16(p); }
inline bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }
inline bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

template <bool kCodes>
bitlinear_status layernorm_launch(LnArgs a, cudaStream_t s, int sm_count) {
  const int wpr = row_warps(a.M, a.K, kLnMaxChunks, sm_count);
  a.lw = log2i(wpr);
  a.dk = a.K;
  a.inv_k = 1.0 / a.K;
  const bool fast = rows16(a.x, a.ldx, a.K) && aligned32(a.w) && aligned32(a.b) && aligned16(a.y) && aligned8(a.q);
  const int need = row_chunks(a.K, wpr);
  const int rpc = kQuantWarps / wpr;
  const dim3 grid((a.M + rpc - 1) / rpc), block(32 * kQuantWarps);
  auto go = [&](auto kern) { return launch(kern, grid, block, 0, s, false, a); };
  if (need > kLnMaxChunks)
    return fast ? go(layernorm_kernel<kCodes, false, 0>) : go(layernorm_kernel<kCodes, true, 0>);
  if (fast) {
    if (need <= 1) return go(layernorm_kernel<kCodes, false, 1>);
    if (need <= 2) return go(layernorm_kernel<kCodes, false, 2>);
    if (need <= 3) return go(layernorm_kernel<kCodes, false, 3>);
    if (need <= 4) return go(layernorm_kernel<kCodes, false, 4>);
    if (need <= 5) return go(layernorm_kernel<kCodes, false, 5>);
    if (need <= 6) return go(layernorm_kernel<kCodes, false, 6>);
    if (need <= 8) return go(layernorm_kernel<kCodes, false, 8>);
    return go(layernorm_kernel<kCodes, false, kLnMaxChunks>);
  }
  if (need <= 1) return go(layernorm_kernel<kCodes, true, 1>);
  if (need <= 2) return go(layernorm_kernel<kCodes, true, 2>);
  if (need <= 4) return go(layernorm_kernel<kCodes, true, 4>);
  if (need <= 6) return go(layernorm_kernel<kCodes, true, 6>);
  return go(layernorm_kernel<kCodes, true, kLnMaxChunks>);
}

bitlinear_status check_layernorm(const LnArgs& a) {
  const bitlinear_status st = check_rows(a.M, a.K);
  if (st != BITLINEAR_OK) return st;
  if (a.ldx < a.K || !(a.eps >= 0.0f) || a.eps > 1.0f) return BITLINEAR_ERR_SHAPE;
  if (!aligned2(a.x) || !aligned4(a.w) || !aligned4(a.b) || !aligned4(a.mean) || !aligned4(a.rstd))
    return BITLINEAR_ERR_ALIGN;
  return BITLINEAR_OK;
}

// Launch shape of the norm gradients: G chunks of 8 columns a thread, T threads
// a row group, rg groups a CTA, `ctas` CTAs (partial rows of the column sums).
// Longer rows than kNbMaxK: T = 0, `ctas` slabs of rows.
struct NbPlan {
  int G, T, rg, ctas;
};

// Two chunks a thread, four where rows are too long for that; one where the rows are few (a short chain counts) or
// would leave more than a sixth of two-chunk threads idle.
NbPlan nb_plan(int M, int K, int sm_count) {
  NbPlan p;
  const int chunks = (K + 7) / 8;
  if (K > kNbMaxK) {
    p.G = p.T = p.rg = 0;
    p.ctas = std::min(M, 64);
    return p;
  }
  auto threads = [&](int G) { return ((chunks + G - 1) / G + 31) / 32 * 32; };
  p.G = threads(2) <= nb_max_threads(2) ? 2 : 4;
  if (threads(1) <= nb_max_threads(1) && (M <= 4 * sm_count || 5 * 2 * threads(2) > 6 * threads(1))) p.G = 1;
  p.T = threads(p.G);  // (G - 1) T < chunks: with G = 2 since more than 32 chunks, with G = 4 since more than 1024
  p.rg = std::max(1, std::min({kNbMaxGroups, nb_max_threads(p.G) / p.T, (M + sm_count - 1) / sm_count}));
  p.ctas = std::min(sm_count, (M + p.rg - 1) / p.rg);
  return p;
}

size_t nb_part_bytes(const NbPlan& p, int K) { return align256(static_cast<size_t>(p.ctas) * 2 * K * 4); }

template <bool kLayer>
bitlinear_status norm_backward(NbArgs a, float* dw, float* db, void* ws, size_t ws_bytes, cudaStream_t s,
                               DeviceState* dev) {
  const NbPlan p = nb_plan(a.M, a.K, dev->sm_count);
  const size_t part = nb_part_bytes(p, a.K);
  if (!ws || !aligned16(ws) || ws_bytes < part + (p.T ? 0 : align256(4 * static_cast<size_t>(a.M))))
    return BITLINEAR_ERR_WORKSPACE;
  a.part = static_cast<float*>(ws);
  a.T = p.T;
  a.rg = p.rg;
  bitlinear_status st;
  if (p.T) {
    const size_t smem = static_cast<size_t>(32) * p.G * nb_max_threads(p.G) * (p.rg > 1 ? 2 : 1);
    auto go = [&](auto kern) { return launch(kern, dim3(p.ctas), dim3(p.T * p.rg), smem, s, false, a); };
    const bool fast = rows16(a.x, a.ldx, a.K) && rows16(a.dy, a.lddy, a.K) && aligned16(a.dx);
    st = p.G == 1   ? go(fast ? norm_backward_kernel<kLayer, true, 1> : norm_backward_kernel<kLayer, false, 1>)
         : p.G == 2 ? go(fast ? norm_backward_kernel<kLayer, true, 2> : norm_backward_kernel<kLayer, false, 2>)
                    : go(fast ? norm_backward_kernel<kLayer, true, 4> : norm_backward_kernel<kLayer, false, 4>);
  } else {
    float* r = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + part);
    st = launch(norm_backward_long_kernel<kLayer>, dim3(a.M), dim3(1024), 0, s, false, a, r);
    if (st != BITLINEAR_OK) return st;
    st = launch(norm_columns_kernel<kLayer>, dim3((a.K + 255) / 256, p.ctas), dim3(256), 0, s, false, a,
                kLayer ? a.rstd : static_cast<const float*>(r));
  }
  if (st != BITLINEAR_OK) return st;
  const int64_t cols = static_cast<int64_t>(a.K) * (kLayer ? 2 : 1);
  return launch(norm_reduce_kernel, dim3(static_cast<unsigned>((cols + 31) / 32)), dim3(1024), 0, s, true,
                static_cast<const float*>(a.part), p.ctas, cols, static_cast<int64_t>(a.K), dw, db);
}

bitlinear_status check_norm_backward(const NbArgs& a, const float* dw, const float* db) {
  const bitlinear_status st = check_rows(a.M, a.K);
  if (st != BITLINEAR_OK) return st;
  if (a.ldx < a.K || a.lddy < a.K) return BITLINEAR_ERR_SHAPE;
  if (!aligned2(a.x) || !aligned2(a.dy) || !aligned2(a.dx) || !aligned4(a.w) || !aligned4(a.mean) ||
      !aligned4(a.rstd) || !aligned4(dw) || !aligned4(db))
    return BITLINEAR_ERR_ALIGN;
  return BITLINEAR_OK;
}

// Elements of a contiguous M x K matrix for the flat kernels (32-bit counts), 0 where they do not apply.
uint32_t flat_count(int M, int K) {
  const int64_t n = static_cast<int64_t>(M) * K;
  return K >= 16 && n < (1ll << 32) - 65536 ? static_cast<uint32_t>(n) : 0u;
}

bitlinear_status dequant_launch(const int8_t* q, int64_t ldq, const float* gamma, int M, int K, uint16_t* y,
                                int64_t ldy, cudaStream_t s, bool pdl, int sm_count) {
  const uint32_t count = flat_count(M, K), per = 16 * 256 * kFlatChunks;
  if (count > 0 && ldq == K && ldy == K && aligned16(q) && aligned32(y))
    return launch(dequant_flat_kernel, dim3((count / 16 * 16 + per - 1) / per), dim3(256), 0, s, pdl, q, gamma,
                  static_cast<uint32_t>(K), count, y);
  const int lanes = row_lanes(M, K, 8, sm_count), rpc = 256 / lanes;
  return launch(dequant_act_kernel, dim3((M + rpc - 1) / rpc), dim3(256), 0, s, pdl, q, ldq, gamma, M, K, y, ldy, lanes);
}

// ---------------------------------------------------------------- gradient products
// How a product's 256 x 256 tiles are given to the pairs: whole rounds of
// tiles over their whole reduction, the tiles left over cut into `split` parts.
struct GgPlan {
  int row_tiles, col_tiles, kblocks, full, split, per, units, pairs;
};

// Parts of the tiles left over, by the time of their rounds: kb us a k-block (0.43 with 2-bit rows, 0.53 with 8-bit
// codes), 0.3 a round, and once they are split 3 for the last launch and 0.04 for each part's way through memory.
// Measured with s parts (us): dx 777 x 2560 x 640, 12 tiles of 40 k-blocks: 20.3 (s = 1), 15.4 (2), 12.5 (4, 6), 14.1
// (8); dx 128 x 2560 x 6912, 27 of 40: 20.9, 16.2 (2), 17.8 (4); dW 2048 x 640 x 2560, 30 of 32: 23.1, 18.8 (2), 20.7 (4).
GgPlan gg_plan(int64_t rows, int cols, int red, double kb, int sm_count) {
  GgPlan p;
  p.pairs = sm_count / 2;
  p.row_tiles = static_cast<int>((rows + kGgRows - 1) / kGgRows);
  p.col_tiles = (cols + kGgCols - 1) / kGgCols;
  p.kblocks = (red + kGgRed - 1) / kGgRed;
  const int tiles = p.row_tiles * p.col_tiles;  // at most 2^16 * 2^8
  const int left = tiles % p.pairs;
  p.full = tiles - left;
  p.split = 1;
  p.per = p.kblocks;
  if (left > 0) {
    double best = p.kblocks * kb + 0.3;
    for (int s = 2; s <= 32 && 2 * s <= p.kblocks; ++s) {
      const int per = (p.kblocks + s - 1) / s;
      const int parts = (p.kblocks + per - 1) / per;
      const int64_t rounds = (static_cast<int64_t>(left) * parts + p.pairs - 1) / p.pairs;
      const double cost = static_cast<double>(rounds) * (per * kb + 0.3) + 3.0 + 0.04 * left * parts;
      if (cost < best) {
        best = cost;
        p.split = parts;
        p.per = per;
      }
    }
  }
  if (p.split == 1) p.full = tiles;
  p.units = p.full + (tiles - p.full) * p.split;
  p.pairs = std::min(p.pairs, p.units);
  return p;
}

// dW: 0.53 us a k-block with expansion; long reductions run without (bw_dense), 0.38.
GgPlan bw_plan(int N, int K, int M, int sm_count) {
  return gg_plan(N, K, M, M > kGgOneSum * kGgRed ? 0.38 : 0.53, sm_count);
}

size_t gg_slab_bytes(const GgPlan& p) { return static_cast<size_t>(p.units - p.full) * kGgSlab * 4; }
size_t gg_done_bytes(const GgPlan& p) { return static_cast<size_t>(p.units - p.full) * 2 * kGgStoring * 4; }

// Whether a product restores its compressed operand (`elems` elements) to bf16 before it starts: where what its
// k-blocks save (us each, against expanding in place) exceeds the extra pass, a launch and `bytes` of traffic an
// element at 6 TB/s.
bool gg_dense(const GgPlan& p, double save_us, int64_t elems, double bytes) {
  const int64_t rounds = (p.full + p.pairs - 1) / p.pairs;
  const int64_t left = p.units - p.full;
  const double kblocks = static_cast<double>(rounds) * p.kblocks + static_cast<double>((left + p.pairs - 1) / p.pairs) * p.per;
  return kblocks * save_us > 2.5 + static_cast<double>(elems) * bytes / 6e6;
}

// Few-token products take train_few.cuh: up to 32 tokens, or while its CTAs, one for 16 tokens and half a span of
// columns, fit the SMs once.  Measured (us, few / pair GEMM): 16 tokens, N = 2560, K = 6912: 7.8 / 18.0; 32: 14.1 /
// 19.3; 64: 20.7 / 19.9.  N = 11008, K = 2048, 64 tokens (128 CTAs): 21.5 / 25.6; 96: 40 / 26.
bool few_tokens(int M, int K, int sm_count) {
  const int64_t groups = 2 * ((K + kFewSpan - 1) / kFewSpan);
  return M <= 32 || groups * ((M + 15) / 16) <= sm_count;
}

bitlinear_status few_launch(FewArgs a, cudaStream_t s, int sm_count) {
  const int groups = 2 * ((a.K + kFewSpan - 1) / kFewSpan), mt = (a.M + 15) / 16;
  a.chunks = (a.N + kFewRed - 1) / kFewRed;
  // parts of N: while the CTAs fit the SMs and each warp keeps a piece of its own
  a.cs = 1;
  while (a.cs < 8 && 2 * a.cs * groups * mt <= sm_count && 2 * a.cs * kFewWarps <= a.chunks) a.cs *= 2;
  a.per = (a.chunks + a.cs - 1) / a.cs;
  return launch_ex(few_input_kernel, dim3(groups * a.cs, mt), dim3(32 * kFewWarps), kFewSmem, s, true, a.cs, a);
}

// Workspace: slabs and their marks | dy with padded rows | B: codes with padded rows, expanded N:M codes, or bf16 values.
struct GgLayout {
  size_t dy, b, total;  // offsets of the second and third part, whole size
  int64_t lddy;         // row stride of dy that TMA reads, in elements
};
GgLayout gg_layout(const GgPlan& p, int64_t M, int64_t N, int64_t lddy, size_t b_bytes) {
  GgLayout l;
  l.dy = align256(gg_slab_bytes(p) + gg_done_bytes(p));
  const bool pad = lddy % 8 != 0;
  l.lddy = pad ? (N + 7) / 8 * 8 : lddy;
  l.b = l.dy + (pad ? align256(static_cast<size_t>(M) * l.lddy * 2) : 0);
  l.total = l.b + align256(b_bytes);
  return l;
}

// dW also where a part is longer than one sum in TMEM may be: only the kernel without expansion has registers to add up
// several.
bool bw_dense(const GgPlan& p, int64_t M, int K) {
  return (p.full ? p.kblocks : p.per) > kGgOneSum || gg_dense(p, 0.14, M * K, 3.0);
}
bool bi_dense(const GgPlan& p, int64_t N, int K) { return gg_dense(p, 0.06, N * K, 2.25); }
size_t bw_b_bytes(const GgPlan& p, int64_t M, int K, int64_t ldq) {
  return bw_dense(p, M, K) ? static_cast<size_t>(M) * k16(K) * 2 : ldq % 16 ? static_cast<size_t>(M) * k16(K) : 0;
}
size_t bi_few_bytes(int N, int K, int nm_m) { return nm_m ? static_cast<size_t>(N) * dense_ld(K) : 0; }
size_t bi_b_bytes(const GgPlan& p, int N, int K, int nm_m) {
  return bi_dense(p, N, K) ? static_cast<size_t>(N) * k16(K) * 2 : nm_m ? static_cast<size_t>(N) * dense_ld(K) : 0;
}

// Puts the rows of dy (l.lddy is another stride) and of the codes (q_out) where TMA can step them, if they are not.
bitlinear_status gg_pad(const uint16_t** dy, int64_t lddy, const int8_t* q, int64_t ldq, int8_t* q_out, int M, int N,
                        int K, uint8_t* ws, const GgLayout& l, cudaStream_t s) {
  const bool pad = l.lddy != lddy;
  if (!pad && !q_out) return BITLINEAR_OK;
  PadArgs a;
  std::memset(&a, 0, sizeof a);
  a.M = M;
  a.N = N;
  a.K = K;
  auto blocks = [&](int64_t chunks) { return static_cast<unsigned>((static_cast<int64_t>(M) * chunks + 255) / 256); };
  unsigned grid = 0;
  if (pad) {
    a.dy = *dy;
    a.lddy = lddy;
    a.ldd = l.lddy;
    a.dy_out = reinterpret_cast<uint16_t*>(ws + l.dy);
    *dy = a.dy_out;
    grid = a.dy_blocks = blocks(l.lddy / 8);
  }
  if (q_out) {
    a.q = q;
    a.ldq = ldq;
    a.ldqd = k16(K);
    a.q_out = q_out;
    grid += blocks(k16(K) / 16);
  }
  return launch(pad_rows_kernel, dim3(grid), dim3(256), 0, s, false, a);
}

template <bool kWeight>
bitlinear_status gg_launch(const CUtensorMap& mA, const CUtensorMap& mB, const CUtensorMap& mC, const GradArgs& a,
                           const GgPlan& p, bool dense, cudaStream_t s) {
  auto go = [&](auto kern, int threads, size_t smem) {
    return launch_ex(kern, dim3(2 * p.pairs), dim3(threads), smem, s, true, 2, mA, mB, mC, a);
  };
  bitlinear_status st = dense ? go(grad_gemm_kernel<kWeight, true>, GG<kWeight, true>::THREADS, GG<kWeight, true>::SMEM)
                              : go(grad_gemm_kernel<kWeight, false>, GG<kWeight, false>::THREADS,
                                   GG<kWeight, false>::SMEM);
  if (st != BITLINEAR_OK || p.units == p.full) return st;
  const int tiles = p.row_tiles * p.col_tiles - p.full;
  return launch(grad_reduce_kernel<kWeight>, dim3(kGgReduceCtas * tiles), dim3(256), 0, s, true, a);
}

// The packed rows as dense codes, or as bf16 values, in `out`.
bitlinear_status bi_expand(const bitlinear_weights* w, uint8_t* out, bool bf16, bool pdl, cudaStream_t s) {
  ExpandArgs e;
  e.codes = w->codes;
  e.meta = w->meta;
  const bitlinear_status st = bitlinear_packed_layout(w->N, w->K, w->nm_n, w->nm_m, &e.ldc, &e.ldm, nullptr, nullptr);
  if (st != BITLINEAR_OK) return st;
  e.ldd = bf16 ? k16(w->K) : dense_ld(w->K);
  e.N = w->N;
  e.K = w->K;
  e.nm_n = w->nm_n;
  e.nm_m = w->nm_m;
  e.out = reinterpret_cast<uint32_t*>(out);
  const int64_t words = static_cast<int64_t>(w->N) * (e.ldd / (bf16 ? 16 : 4));
  const dim3 grid(static_cast<unsigned>((words + 255) / 256));
  return bf16 ? launch(ternary_bf16_kernel, grid, dim3(256), 0, s, pdl, e)
              : launch(nm_expand_kernel, grid, dim3(256), 0, s, pdl, e);
}

void gg_args(GradArgs* a, const GgPlan& p, int rows, int cols, int red, void* ws, DeviceState* dev) {
  std::memset(a, 0, sizeof *a);
  a->rows = rows;
  a->cols = cols;
  a->red = red;
  a->col_tiles = p.col_tiles;
  a->kblocks = p.kblocks;
  a->full = p.full;
  a->units = p.units;
  a->split = p.split;
  a->per = p.per;
  a->slab = static_cast<float*>(ws);
  a->done = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) + gg_slab_bytes(p));
  a->status = dev->status;
}

}  // namespace
}  // namespace bl

using namespace bl;

extern "C" {

bitlinear_status bitlinear_layernorm(const uint16_t* x, int64_t ldx, int32_t M, int32_t K, const float* w,
                                     const float* b, float eps, uint16_t* y, float* mean, float* rstd, void* stream) {
  if (!x || !w || !y) return BITLINEAR_ERR_NULL;
  LnArgs a;
  std::memset(&a, 0, sizeof a);
  a.x = x;
  a.ldx = ldx;
  a.M = M;
  a.K = K;
  a.w = w;
  a.b = b;
  a.eps = eps;
  a.y = y;
  a.mean = mean;
  a.rstd = rstd;
  bitlinear_status st = check_layernorm(a);
  if (st != BITLINEAR_OK) return st;
  if (!aligned2(y)) return BITLINEAR_ERR_ALIGN;
  DeviceState* dev = nullptr;
  st = current_device(&dev);
  if (st != BITLINEAR_OK) return st;
  st = layernorm_launch<false>(a, static_cast<cudaStream_t>(stream), dev->sm_count);
  if (st == BITLINEAR_OK) t_last_kernel = "layernorm";
  return st;
}

bitlinear_status bitlinear_layernorm_quant_act(const uint16_t* x, int64_t ldx, int32_t M, int32_t K, const float* w,
                                               const float* b, float eps, int8_t* q, float* gamma, int32_t* rowsum,
                                               float* mean, float* rstd, void* stream) {
  if (!x || !w || !q || !gamma) return BITLINEAR_ERR_NULL;
  LnArgs a;
  std::memset(&a, 0, sizeof a);
  a.x = x;
  a.ldx = ldx;
  a.M = M;
  a.K = K;
  a.w = w;
  a.b = b;
  a.eps = eps;
  a.q = q;
  a.gamma = gamma;
  a.rowsum = rowsum;
  a.mean = mean;
  a.rstd = rstd;
  bitlinear_status st = check_layernorm(a);
  if (st != BITLINEAR_OK) return st;
  if (!aligned4(gamma) || !aligned4(rowsum)) return BITLINEAR_ERR_ALIGN;
  DeviceState* dev = nullptr;
  st = current_device(&dev);
  if (st != BITLINEAR_OK) return st;
  st = layernorm_launch<true>(a, static_cast<cudaStream_t>(stream), dev->sm_count);
  if (st == BITLINEAR_OK) t_last_kernel = "layernorm_quant_act";
  return st;
}

size_t bitlinear_norm_backward_workspace_bytes(int32_t M, int32_t K) {
  if (check_rows(M, K) != BITLINEAR_OK) return 0;
  const NbPlan p = nb_plan(M, K, plan_sm_count());
  return nb_part_bytes(p, K) + (p.T ? 0 : align256(4 * static_cast<size_t>(M)));
}

bitlinear_status bitlinear_layernorm_backward(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx,
                                              int32_t M, int32_t K, const float* w, const float* mean,
                                              const float* rstd, uint16_t* dx, float* dw, float* db, void* workspace,
                                              size_t workspace_bytes, void* stream) {
  if (!dy || !x || !w || !mean || !rstd || !dx || !dw) return BITLINEAR_ERR_NULL;
  NbArgs a;
  std::memset(&a, 0, sizeof a);
  a.dy = dy;
  a.lddy = lddy;
  a.x = x;
  a.ldx = ldx;
  a.M = M;
  a.K = K;
  a.w = w;
  a.mean = mean;
  a.rstd = rstd;
  a.dx = dx;
  bitlinear_status st = check_norm_backward(a, dw, db);
  if (st != BITLINEAR_OK) return st;
  DeviceState* dev = nullptr;
  st = current_device(&dev);
  if (st != BITLINEAR_OK) return st;
  st = norm_backward<true>(a, dw, db, workspace, workspace_bytes, static_cast<cudaStream_t>(stream), dev);
  if (st == BITLINEAR_OK) t_last_kernel = "layernorm_backward";
  return st;
}

bitlinear_status bitlinear_rmsnorm_backward(const uint16_t* dy, int64_t lddy, const uint16_t* x, int64_t ldx,
                                            int32_t M, int32_t K, const float* g, float eps, uint16_t* dx, float* dg,
                                            void* workspace, size_t workspace_bytes, void* stream) {
  if (!dy || !x || !g || !dx || !dg) return BITLINEAR_ERR_NULL;
  NbArgs a;
  std::memset(&a, 0, sizeof a);
  a.dy = dy;
  a.lddy = lddy;
  a.x = x;
  a.ldx = ldx;
  a.M = M;
  a.K = K;
  a.w = g;
  a.eps = eps;
  a.dx = dx;
  bitlinear_status st = check_norm_backward(a, dg, nullptr);
  if (st != BITLINEAR_OK) return st;
  if (!(eps >= 0.0f) || eps > 1.0f) return BITLINEAR_ERR_SHAPE;
  DeviceState* dev = nullptr;
  st = current_device(&dev);
  if (st != BITLINEAR_OK) return st;
  st = norm_backward<false>(a, dg, nullptr, workspace, workspace_bytes, static_cast<cudaStream_t>(stream), dev);
  if (st == BITLINEAR_OK) t_last_kernel = "rmsnorm_backward";
  return st;
}

bitlinear_status bitlinear_dequant_act(const int8_t* q, int64_t ldq, const float* gamma, int32_t M, int32_t K,
                                       uint16_t* y, void* stream) {
  if (!q || !gamma || !y) return BITLINEAR_ERR_NULL;
  bitlinear_status st = check_rows(M, K);
  if (st != BITLINEAR_OK) return st;
  if (ldq < K) return BITLINEAR_ERR_SHAPE;
  if (!aligned4(gamma) || !aligned2(y)) return BITLINEAR_ERR_ALIGN;
  DeviceState* dev = nullptr;
  st = current_device(&dev);
  if (st != BITLINEAR_OK) return st;
  st = dequant_launch(q, ldq, gamma, M, K, y, K, static_cast<cudaStream_t>(stream), false, dev->sm_count);
  if (st == BITLINEAR_OK) t_last_kernel = "dequant_act";
  return st;
}

bitlinear_status bitlinear_relu2_glu_quant_act(const uint16_t* g, int64_t ldg, const uint16_t* u, int64_t ldu,
                                               int32_t M, int32_t N, int8_t* q_g, float* gamma_g, int8_t* q_u,
                                               float* gamma_u, int8_t* q_h, float* gamma_h, int32_t* rowsum_h,
                                               void* stream) {
  if (!g || !u || !q_g || !gamma_g || !q_u || !gamma_u || !q_h || !gamma_h) return BITLINEAR_ERR_NULL;
  bitlinear_status st = check_rows(M, N);
  if (st != BITLINEAR_OK) return st;
  if (ldg < N || ldu < N) return BITLINEAR_ERR_SHAPE;
  if (!aligned2(g) || !aligned2(u) || !aligned4(gamma_g) || !aligned4(gamma_u) || !aligned4(gamma_h) ||
      !aligned4(rowsum_h))
    return BITLINEAR_ERR_ALIGN;
  DeviceState* dev = nullptr;
  st = current_device(&dev);
  if (st != BITLINEAR_OK) return st;
  GluSaveArgs a;
  a.g = g;
  a.ldg = ldg;
  a.u = u;
  a.ldu = ldu;
  a.M = M;
  a.N = N;
  a.qg = q_g;
  a.qu = q_u;
  a.qh = q_h;
  a.gg = gamma_g;
  a.gu = gamma_u;
  a.gh = gamma_h;
  a.rowsum = rowsum_h;
  const int wpr = row_warps(M, N, kGluMaxChunks, dev->sm_count);
  a.lw = log2i(wpr);
  const bool fast = rows16(g, ldg, N) && rows16(u, ldu, N) && aligned8(q_g) && aligned8(q_u) && aligned8(q_h);
  const int need = row_chunks(N, wpr);
  const int rpc = kQuantWarps / wpr;
  auto go = [&](auto kern) {
    return launch(kern, dim3((M + rpc - 1) / rpc), dim3(32 * kQuantWarps), 0, static_cast<cudaStream_t>(stream), false,
                  a);
  };
  if (need > kGluMaxChunks)
    st = fast ? go(relu2_glu_quant_kernel<false, 0>) : go(relu2_glu_quant_kernel<true, 0>);
  else if (fast)
    st = need <= 1   ? go(relu2_glu_quant_kernel<false, 1>)
         : need <= 2 ? go(relu2_glu_quant_kernel<false, 2>)
         : need <= 3 ? go(relu2_glu_quant_kernel<false, 3>)
         : need <= 4 ? go(relu2_glu_quant_kernel<false, 4>)
         : need <= 5 ? go(relu2_glu_quant_kernel<false, 5>)
                     : go(relu2_glu_quant_kernel<false, kGluMaxChunks>);
  else
    st = need <= 1   ? go(relu2_glu_quant_kernel<true, 1>)
         : need <= 2 ? go(relu2_glu_quant_kernel<true, 2>)
         : need <= 4 ? go(relu2_glu_quant_kernel<true, 4>)
                     : go(relu2_glu_quant_kernel<true, kGluMaxChunks>);
  if (st == BITLINEAR_OK) t_last_kernel = "relu2_glu_quant_act";
  return st;
}

bitlinear_status bitlinear_relu2_glu_backward(const uint16_t* dh, int64_t lddh, const int8_t* q_g,
                                              const float* gamma_g, const int8_t* q_u, const float* gamma_u, int32_t M,
                                              int32_t N, uint16_t* dg, uint16_t* du, void* stream) {
  if (!dh || !q_g || !gamma_g || !q_u || !gamma_u || !dg || !du) return BITLINEAR_ERR_NULL;
  bitlinear_status st = check_rows(M, N);
  if (st != BITLINEAR_OK) return st;
  if (lddh < N) return BITLINEAR_ERR_SHAPE;
  if (!aligned2(dh) || !aligned2(dg) || !aligned2(du) || !aligned4(gamma_g) || !aligned4(gamma_u))
    return BITLINEAR_ERR_ALIGN;
  DeviceState* dev = nullptr;
  st = current_device(&dev);
  if (st != BITLINEAR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const uint32_t count = flat_count(M, N);
  if (count > 0 && lddh == N && aligned32(dh) && aligned16(q_g) && aligned16(q_u) && aligned32(dg) && aligned32(du)) {
    st = launch(N % 16 ? relu2_glu_backward_flat_kernel<true> : relu2_glu_backward_flat_kernel<false>,
                dim3((count / 16 + 511) / 512), dim3(256), 0, s, false, dh, q_g, gamma_g, q_u, gamma_u,
                static_cast<uint32_t>(N), count, dg, du);
  } else {
    const int lanes = row_lanes(M, N, 4, dev->sm_count), rpc = 256 / lanes;
    st = launch(relu2_glu_backward_kernel, dim3((M + rpc - 1) / rpc), dim3(256), 0, s, false, dh, lddh, q_g, gamma_g,
                q_u, gamma_u, M, N, dg, du, lanes);
  }
  if (st == BITLINEAR_OK) t_last_kernel = "relu2_glu_backward";
  return st;
}

size_t bitlinear_backward_weight_workspace_bytes(int32_t M, int32_t N, int32_t K, int64_t lddy, int64_t ldq) {
  if (check_nk(N, K) != BITLINEAR_OK || M < 1 || M > BITLINEAR_MAX_M || lddy < N || ldq < K) return 0;
  const GgPlan p = bw_plan(N, K, M, plan_sm_count());
  return gg_layout(p, M, N, lddy, bw_b_bytes(p, M, K, ldq)).total;
}

bitlinear_status bitlinear_backward_weight(const uint16_t* dy, int64_t lddy, const int8_t* q, int64_t ldq,
                                           const float* gamma, int32_t M, int32_t N, int32_t K, float* dW,
                                           void* workspace, size_t workspace_bytes, uint32_t flags, void* stream) {
  if (!dy || !q || !gamma || !dW) return BITLINEAR_ERR_NULL;
  bitlinear_status st = check_nk(N, K);
  if (st != BITLINEAR_OK) return st;
  if (M < 1 || M > BITLINEAR_MAX_M || lddy < N || ldq < K) return BITLINEAR_ERR_SHAPE;
  if (flags & ~static_cast<uint32_t>(BITLINEAR_FLAG_ACCUMULATE)) return BITLINEAR_ERR_FLAGS;
  if ((lddy % 8 ? !aligned2(dy) : !aligned16(dy)) || (ldq % 16 == 0 && !aligned16(q)) || !aligned4(gamma) ||
      !aligned4(dW))
    return BITLINEAR_ERR_ALIGN;
  DeviceState* dev = nullptr;
  st = current_device(&dev);
  if (st != BITLINEAR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const GgPlan p = bw_plan(N, K, M, dev->sm_count);
  const GgLayout l = gg_layout(p, M, N, lddy, bw_b_bytes(p, M, K, ldq));
  if (l.total > 0 && (!workspace || !aligned32(workspace) || workspace_bytes < l.total)) return BITLINEAR_ERR_WORKSPACE;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const bool dense = bw_dense(p, M, K);
  int8_t* const padded = !dense && ldq % 16 ? reinterpret_cast<int8_t*>(ws + l.b) : nullptr;
  st = gg_pad(&dy, lddy, q, ldq, padded, M, N, K, ws, l, s);
  if (st == BITLINEAR_OK && dense)
    st = dequant_launch(q, ldq, gamma, M, K, reinterpret_cast<uint16_t*>(ws + l.b), k16(K), s, true, dev->sm_count);
  if (st != BITLINEAR_OK) return st;
  if (padded) {
    q = padded;
    ldq = k16(K);
  }
  CUtensorMap mA, mB;
  if (!make_map_u8(&mA, dy, 2 * static_cast<uint64_t>(N), M, 2 * static_cast<uint64_t>(l.lddy), 128, kGgRed, 128) ||
      !(dense ? make_map_u8(&mB, ws + l.b, 2 * static_cast<uint64_t>(K), M, 2 * static_cast<uint64_t>(k16(K)), 128,
                            kGgRed, 128)
              : make_map_u8(&mB, q, K, M, static_cast<uint64_t>(ldq), 128, kGgRed, 0)))
    return BITLINEAR_ERR_CUDA;
  GradArgs a;
  gg_args(&a, p, N, K, M, workspace, dev);
  a.gamma = gamma;
  a.dw = dW;
  a.accumulate = (flags & BITLINEAR_FLAG_ACCUMULATE) != 0;
  a.vec = K % 8 == 0 && aligned32(dW);
  // by TMA: a row a lane writes 32 lines an instruction (16 x 2560 x 6912: 19.5 us against 15.4)
  a.tma = K % 4 == 0 && aligned16(dW);
  CUtensorMap mC = mA;
  if (a.tma && !make_map(&mC, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, dW, K, N, 4 * static_cast<uint64_t>(K), 32, 32, 128))
    return BITLINEAR_ERR_CUDA;
  st = gg_launch<true>(mA, mB, mC, a, p, dense, s);
  if (st == BITLINEAR_OK) t_last_kernel = "backward_weight";
  return st;
}

size_t bitlinear_backward_input_workspace_bytes(int32_t M, int32_t N, int32_t K, int64_t lddy, int32_t nm_n,
                                                int32_t nm_m) {
  if (check_nk(N, K) != BITLINEAR_OK || M < 1 || M > BITLINEAR_MAX_M || lddy < N || !pattern_ok(nm_n, nm_m)) return 0;
  if (few_tokens(M, K, plan_sm_count())) return bi_few_bytes(N, K, nm_m);
  const GgPlan p = gg_plan(M, K, N, 0.43, plan_sm_count());
  return gg_layout(p, M, N, lddy, bi_b_bytes(p, N, K, nm_m)).total;
}

bitlinear_status bitlinear_backward_input(const bitlinear_weights* w, const uint16_t* dy, int64_t lddy, int32_t M,
                                          const uint16_t* add, uint16_t* dx, void* workspace, size_t workspace_bytes,
                                          void* stream) {
  if (!w || !dy || !dx) return BITLINEAR_ERR_NULL;
  bitlinear_status st = check_matrix(w, dx, nullptr);
  if (st != BITLINEAR_OK) return st;
  const int N = w->N, K = w->K;
  if (M < 1 || M > BITLINEAR_MAX_M || lddy < N) return BITLINEAR_ERR_SHAPE;
  if ((lddy % 8 ? !aligned2(dy) : !aligned16(dy)) || !aligned2(add)) return BITLINEAR_ERR_ALIGN;
  DeviceState* dev = nullptr;
  st = current_device(&dev);
  if (st != BITLINEAR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const int64_t ld = dense_ld(K);
  if (few_tokens(M, K, dev->sm_count)) {
    const size_t need = bi_few_bytes(N, K, w->nm_m);
    if (need > 0 && (!workspace || !aligned32(workspace) || workspace_bytes < need)) return BITLINEAR_ERR_WORKSPACE;
    FewArgs f;
    std::memset(&f, 0, sizeof f);
    f.codes = w->codes;
    f.ldc = ld;
    if (w->nm_m) {
      st = bi_expand(w, ws, false, false, s);
      if (st != BITLINEAR_OK) return st;
      f.codes = ws;
    }
    f.N = N;
    f.K = K;
    f.dy = dy;
    f.lddy = lddy;
    f.M = M;
    f.alpha = w->alpha;
    f.add = add;
    f.dx = dx;
    st = few_launch(f, s, dev->sm_count);
    if (st == BITLINEAR_OK) t_last_kernel = "backward_input_few";
    return st;
  }
  const GgPlan p = gg_plan(M, K, N, 0.43, dev->sm_count);
  const GgLayout l = gg_layout(p, M, N, lddy, bi_b_bytes(p, N, K, w->nm_m));
  if (l.total > 0 && (!workspace || !aligned32(workspace) || workspace_bytes < l.total)) return BITLINEAR_ERR_WORKSPACE;
  st = gg_pad(&dy, lddy, nullptr, 0, nullptr, M, N, K, ws, l, s);
  if (st != BITLINEAR_OK) return st;
  const uint8_t* codes = w->codes;
  const bool dense = bi_dense(p, N, K);
  if (dense || w->nm_m) {
    st = bi_expand(w, ws + l.b, dense, true, s);
    if (st != BITLINEAR_OK) return st;
    codes = ws + l.b;
  }
  CUtensorMap mA, mB;
  if (!make_map_u8(&mA, dy, 2 * static_cast<uint64_t>(N), M, 2 * static_cast<uint64_t>(l.lddy), 128, 128, 128) ||
      !(dense ? make_map_u8(&mB, codes, 2 * static_cast<uint64_t>(K), N, 2 * static_cast<uint64_t>(k16(K)), 128, kGgRed,
                            128)
              : make_map_u8(&mB, codes, static_cast<uint64_t>(ld), N, static_cast<uint64_t>(ld), 32, kGgRed, 0)))
    return BITLINEAR_ERR_CUDA;
  GradArgs a;
  gg_args(&a, p, M, K, N, workspace, dev);
  a.alpha = w->alpha;
  a.add = add;
  a.dx = dx;
  a.vec = K % 16 == 0 && aligned32(dx) && aligned32(add);
  st = gg_launch<false>(mA, mB, mA, a, p, dense, s);
  if (st == BITLINEAR_OK) t_last_kernel = "backward_input";
  return st;
}

}  // extern "C"
