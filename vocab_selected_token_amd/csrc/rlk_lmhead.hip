// rlk_lmhead.hip -- fused LM-head variant for gfx950: selected-token logp of
// z = h . W^T without writing the logits to memory.
//
// The pages name an optional fused kernel without describing it (Issue #323
// "[WS2][Logprob] H100 validation and reproduction guide for Issue #241
// PR1-PR5", "Validation Boundary": the optional PR6 fused kernel).  This file
// keeps the contract of the materialised path (PR #289 "[WS2][PR4][Logp] feat:
// add distributed TP/CP logprob drift report", PR1 commit messages: per-tile
// fp32 (max, sumexp) over real columns, the (-inf, 0) identity, a merge in
// fixed global tile order) and takes the statistics straight from the fp32
// GEMM accumulators.
//
// Two kernels run before the ordinary stage-2 merge (for few tokens the second
// does that merge as well: lmhead_rows):
//   lmhead_segments  bf16 MFMA GEMM of a 256-vocab x 256-token block (or of 128
//                    or 192 tokens, by how many blocks that makes) over the
//                    whole hidden dimension, then, per token, the (max, sumexp)
//                    of each "segment" -- the part of the block's vocabulary
//                    that lies in one tile (a block holds at most one tile
//                    bound, since tiles are at least 256 columns wide) -- and
//                    the fp32 target logit of every token whose target falls in
//                    the block.
//   lmhead_tiles     per (token, tile): merge the tile's segments in ascending
//                    column order into the tile partial, in the same [N][T]
//                    layout that stage 1 of the materialised path writes.
//
// Up to 64 tokens lmhead_stream takes the first kernel's place.
//
// The product is the tile product of rlk_tile.h with W rows as operand A and
// hidden rows as operand B (C[vocab][token]); rlk_lmhead_segments.h turns a
// block's accumulators into its segments.
//
// Determinism: every reduction has a fixed order -- the block's, then the
// segments of a tile in ascending column order, then the tiles in stage 2.  No
// atomics.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rlk_internal.h"
#include "rlk_lmhead_segments.h"
#include "rlk_stream.h"
#include "rlk_tile.h"

namespace rlk {
namespace {

constexpr int kBV = kBA;  // vocabulary rows per block (= kLmheadBlockVocab)
constexpr int kBT = kBB;  // tokens per block, at most

static_assert(kBV == kLmheadBlockVocab, "block width shared with the boundary");
static_assert(kBK == kLmheadSlabK, "slab width shared with the boundary");

constexpr int32_t kStreamTokens = 64;  // the most that lmhead_stream takes

// ---------------------------------------------------------------------------
// lmhead_segments
//   h          bf16 [num_tokens, K] (16-byte chunks, K/8 per row)
//   w          bf16 [>= real_vocab, K]; only rows [row_lo, row_hi) are read
//   seg_m/s    [num_tokens][2 * n_vb]: slot 2*vb holds the block's columns
//              before its inner tile bound (all of them if there is none), slot
//              2*vb+1 those from the bound on ((-inf, 0) if there is none)
//   tlogit     [num_tokens] fp32 target logit, written for effective-active
//              tokens whose target is a column of this block in [row_lo, row_hi)
// One launch covers one virtual shard: the vocabulary blocks vb_begin ..
// vb_begin + n_vbs - 1 of the global 256-column block grid that overlap the
// shard's real columns [row_lo, row_hi).  Rows outside that range are neither
// read nor counted, and a segment slot is written only by the shard whose
// columns [col_lo, col_hi) hold the slot's first column.  A segment lies
// inside one tile, so it holds the same rows, summed in the same order, under
// every grouping of the tiles: the slots, and so the partials, do not depend
// on the shard count.
// ---------------------------------------------------------------------------
template <int kTok>
__global__ __launch_bounds__(kThreads) void lmhead_segments(
    const u32x4* __restrict__ h, const u32x4* __restrict__ w, int32_t hidden_dim, int32_t n_tb,
    int32_t vb_begin, int32_t n_vbs, SegmentArgs a, int64_t blk_begin) {
  constexpr int kTokens = 64 * kTok;
  __shared__ __attribute__((aligned(16))) char smem[2 * kStageBytes<kTok>];
  static_assert(sizeof(smem) >= kTokens * 4 * sizeof(float), "epilogue exchange fits");

  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);

  // Block order for L2 reuse.  Consecutive work indices land on one XCD (the
  // XCD-local renumbering), and 32 consecutive indices -- one XCD's worth of
  // resident blocks -- cover kGroupV vocabulary blocks x 8 token blocks: work
  // index l sits in strip l / (kGroupV * n_tb) of kGroupV vocabulary blocks,
  // token-block major inside the strip.  So each W slice is read by 8 resident
  // blocks and each hidden slice by kGroupV, instead of every vocabulary block
  // re-streaming all hidden states.
  constexpr int32_t kGroupV = 4;
  const int64_t blk = blk_begin + xcd_local_block(blockIdx.x, gridDim.x);
  const int64_t strip = blk / ((int64_t)kGroupV * n_tb);
  const int32_t r_in = (int32_t)(blk - strip * kGroupV * n_tb);
  const int32_t strip_w = min(kGroupV, n_vbs - (int32_t)strip * kGroupV);  // last strip may be narrow
  const int32_t vb = vb_begin + (int32_t)strip * kGroupV + r_in % strip_w;
  const int32_t tb = r_in / strip_w;
  const int32_t v0 = vb * kBV;
  const int32_t t0 = tb * kTokens;
  const int32_t ldc = hidden_dim / 8;  // 16-byte chunks per row
  const int64_t row_bytes = (int64_t)ldc * 16;

  // Rows of W outside [row_lo, row_hi) -- padding, other shards -- and rows past
  // the last token are never read.
  const int32_t w_first = max(v0, a.row_lo);
  const TileOperand wo(w + (int64_t)w_first * ldc, row_bytes, min(v0 + kBV, a.row_hi) - w_first,
                       v0 - w_first, wave, lane);
  const TileOperandOf<kTok> ho(h + (int64_t)t0 * ldc, row_bytes,
                               min(t0 + kTokens, a.num_tokens) - t0, 0, wave, lane);
  f32x4 acc[kVS][kTok];
  tile_product(smem, wo, ho, 0, hidden_dim / kBK, wave, lane, acc);
  write_segments<kTok>(a, acc, reinterpret_cast<float*>(smem), vb, t0, wave >> 2, wave & 3, lane);
}

// ---------------------------------------------------------------------------
// lmhead_stream: lmhead_segments for up to 64 tokens (16 kTok), whose time the weight's
// bytes bound: stream_product in blocks of 256 rows, then z through LDS into the tile
// kernel's layout, and so with its bits.  The whole call takes 70 us for 32 x 1024 x
// 151936 (102 with tiles; the weight at 5.0 TB/s in this kernel), 275 us (327) for 32 x
// 4096, 77 us (108) for 64 x 1024; 64 tokens need 144 registers, and in 128 they spilled
// and took 103.
// ---------------------------------------------------------------------------
template <int kTok>
__global__ __launch_bounds__(kThreads, kTok == 4 ? 2 : 4) void lmhead_stream(const char* __restrict__ h,
                                                             const char* __restrict__ w,
                                                             int32_t hidden_dim, int32_t vb_begin,
                                                             SegmentArgs a, int64_t blk_begin) {
  __shared__ union {
    StreamLds<kTok> stream;
    f32x4 z[kBV / 4][16 * kTok];
  } lds;
  __shared__ float xch[4 * 16 * 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int32_t vb = vb_begin + (int32_t)(blk_begin + blockIdx.x);
  f32x4 acc[2][kTok];
  Bf16Stream math;
  stream_product<2, kThreads>(lds.stream, w, h, (uint32_t)hidden_dim * 2, a.row_lo, a.row_hi,
                              a.num_tokens, vb * kBV, math, acc);
#pragma unroll
  for (int rt = 0; rt < 2; ++rt)
#pragma unroll
    for (int ts = 0; ts < kTok; ++ts)
      lds.z[(wave * 2 + rt) * 4 + (lane >> 4)][ts * 16 + (lane & 15)] = acc[rt][ts];
  __syncthreads();
  const int wv = wave >> 2, wt = wave & 3;  // (waves without tokens only meet the barrier)
  f32x4 z[kVS][1];
#pragma unroll
  for (int vs = 0; vs < kVS; ++vs)
    z[vs][0] = lds.z[(wv * kVS + vs) * 4 + (lane >> 4)][min(wt, kTok - 1) * 16 + (lane & 15)];
  write_segments<1>(a, z, xch, vb, 0, wv, wt, lane);
}

// The partial (M, S) of tile t of a token from its segments, in ascending columns.  A
// tile that starts at or past real_vocab has no real column: the identity (-inf, 0),
// with no read.
__device__ __forceinline__ void tile_of_segments(const float* __restrict__ seg_m,
                                                 const float* __restrict__ seg_s, int32_t tok,
                                                 int32_t t, int32_t n_vb, int32_t real_vocab,
                                                 int32_t padded_vocab, int32_t num_tiles,
                                                 float& M_out, float& S_out) {
  const int32_t c0 = (int32_t)(((int64_t)t * padded_vocab) / num_tiles);
  const int32_t c1 = (int32_t)(((int64_t)(t + 1) * padded_vocab) / num_tiles);
  float M = kNegInf, S = 0.0f;
  // fold one segment into (M, S): identity segments are skipped
  auto fold = [&](float m, float s) __attribute__((always_inline)) {
    if (m == kNegInf) return;
    if (M == kNegInf) {
      M = m;
      S = s;
      return;
    }
    const float nm = maxnan(M, m);
    S = fmaf(s, exp2_hw((m - nm) * kLog2e), S * exp2_hw((M - nm) * kLog2e));
    M = nm;
  };
  if (c0 < real_vocab) {
    const int32_t vb_first = c0 / kBV;
    const int32_t vb_last = min((min(c1, real_vocab) - 1) / kBV, n_vb - 1);
    const int32_t nseg = vb_last - vb_first + 1;
    const int64_t base = (int64_t)tok * 2 * n_vb + 2 * (int64_t)vb_first;
    const int first_slot = (c0 > vb_first * kBV) ? 1 : 0;  // the tile starts inside its first block
    // the first kPre segments' loads all go out before the first fold; the
    // folds then run in ascending column order as before
    constexpr int kPre = 12;
    float pm[kPre], ps[kPre];
#pragma unroll
    for (int i = 0; i < kPre; ++i) {
      if (i < nseg) {
        const int64_t at = base + 2 * i + (i == 0 ? first_slot : 0);
        pm[i] = seg_m[at];
        ps[i] = seg_s[at];
      }
    }
#pragma unroll
    for (int i = 0; i < kPre; ++i)
      if (i < nseg) fold(pm[i], ps[i]);
    for (int32_t i = kPre; i < nseg; ++i) fold(seg_m[base + 2 * i], seg_s[base + 2 * i]);
  }
  M_out = M;
  S_out = (M == kNegInf) ? 0.0f : S;
}

// ---------------------------------------------------------------------------
// lmhead_tiles: one thread per (token, tile) of the tiles [tile_begin,
// tile_begin + n_tiles).
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(256) void lmhead_tiles(
    const float* __restrict__ seg_m, const float* __restrict__ seg_s, int32_t num_tokens,
    int32_t n_vb, int32_t real_vocab, int32_t padded_vocab, int32_t num_tiles,
    int32_t tile_begin, int32_t n_tiles, float* __restrict__ pmax, float* __restrict__ psum,
    int64_t idx_begin) {
  const int64_t idx = idx_begin + (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (idx >= (int64_t)num_tokens * n_tiles) return;
  const int32_t tok = (int32_t)(idx / n_tiles);
  const int32_t t = tile_begin + (int32_t)(idx - (int64_t)tok * n_tiles);
  const int64_t out = (int64_t)tok * num_tiles + t;
  float M, S;
  tile_of_segments(seg_m, seg_s, tok, t, n_vb, real_vocab, padded_vocab, num_tiles, M, S);
  pmax[out] = M;
  psum[out] = S;
}

// ---------------------------------------------------------------------------
// lmhead_rows: lmhead_tiles and the stage-2 merge of few tokens in one launch, one
// wave per token and one tile (of 64 at most) per lane.  The merge is stage 2's, and
// so are its bits: an exact maximum, fp32 exponentials, then an fp64 fma chain in
// ascending tile order, in which an identity partial (0 times 0) changes nothing.
// What it saves is a launch: 17.5 against 18.7 us for 1 token x 128 x 2000, 125.8 against
// 128.1 us for 777 x 1088 x 50021; with 8-bit operands 31.8 against 34.6 us and, 333 x
// 2176 x 50021, 66.8 against 69.5 us.
// ---------------------------------------------------------------------------
constexpr int kRowWaves = 4;  // tokens per block

__global__ __launch_bounds__(kRowWaves * 64) void lmhead_rows(LmheadArgs a, int32_t n_vb,
                                                              float* __restrict__ logp,
                                                              float* __restrict__ lse,
                                                              uint32_t* __restrict__ status,
                                                              int64_t blk_begin) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (blk_begin + blockIdx.x) * kRowWaves + (threadIdx.x >> 6);
  if (r >= a.num_tokens) return;  // uniform over the wave
  float mt = kNegInf, st = 0.0f;
  if (lane < a.num_tiles) {
    tile_of_segments(a.seg_m, a.seg_s, (int32_t)r, lane, n_vb, a.real_vocab, a.padded_vocab,
                     a.num_tiles, mt, st);
    a.pmax[r * a.num_tiles + lane] = mt;
    a.psum[r * a.num_tiles + lane] = st;
  }
  float M = mt;
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) M = maxnan(M, __shfl_xor(M, o));
  float L = kNegInf;
  if (M != kNegInf) {
    const float e = mt != kNegInf ? expf(mt - M) : 0.0f;
    double sum = 0.0;
#pragma unroll
    for (int t = 0; t < 64; ++t)
      sum = fma((double)__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(st), t)),
                (double)__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(e), t)), sum);
    L = (float)((double)M + log(sum));
  }
  if (lane != 0) return;
  lse[r] = L;
  const bool masked = a.mask != nullptr && a.mask[r] == 0;
  const int32_t tgt = masked ? a.ignore_index : a.targets[r];
  if (tgt == a.ignore_index) {
    logp[r] = 0.0f;
  } else if (tgt < 0 || tgt >= a.real_vocab) {
    logp[r] = __builtin_nanf("");
    status[0] = 1u;
  } else {
    logp[r] = a.target_logit[r] - L;
    if (!__builtin_isfinite(L)) status[1] = 1u;
  }
}

}  // namespace

int64_t lmhead_grid_blocks(int32_t num_tokens, int32_t real_vocab) {
  const int64_t n_vb = ((int64_t)real_vocab + kBV - 1) / kBV;
  const int64_t n_tb = ((int64_t)num_tokens + kBT - 1) / kBT;
  return n_vb * n_tb;
}

namespace {

// Time of a round of tiles of 128, 192 and 256 tokens (hidden_dim 4096: 65, 81 and 100
// us; 1024: 19, 24 and 31), see tile_tokens.  It takes narrower tiles for 777 tokens x
// 1088 x 50021 (110 us for the call; 125 with 256 tokens), 333 x 2176 x 50021 (90; 108),
// 128 x 1024 x 151936 (90; 111) and 200 x 2048 x 12003 (38; 54).
constexpr double kTileUnits[] = {2.5, 3.15, 4.0};

// One shard's segments, in launches of at most `limit` threads; a block's work
// index (and so its tile) does not depend on the split.
hipError_t launch_segments(const LmheadArgs& a, const SegmentArgs& sa, int32_t vb_begin,
                           int32_t n_vbs, hipStream_t stream) {
  const int32_t n = a.num_tokens;
  const bool few = n <= kStreamTokens;
  const int k_tok = few ? 0 : tile_tokens(n, n_vbs, kTileUnits);
  const int32_t n_tb = few ? 1 : (n + 64 * k_tok - 1) / (64 * k_tok);
  const auto stream_kernel = n <= 16   ? lmhead_stream<1>
                             : n <= 32 ? lmhead_stream<2>
                                       : lmhead_stream<4>;
  const auto tile_kernel = k_tok == 2   ? lmhead_segments<2>
                           : k_tok == 3 ? lmhead_segments<3>
                                        : lmhead_segments<4>;
  const int64_t max_blocks = launch_thread_limit() / kThreads;
  const int64_t blocks = (int64_t)n_vbs * n_tb;
  for (int64_t b0 = 0; b0 < blocks; b0 += max_blocks) {
    const dim3 grid((unsigned)(blocks - b0 < max_blocks ? blocks - b0 : max_blocks));
    if (few)
      hipLaunchKernelGGL(stream_kernel, grid, dim3(kThreads), 0, stream,
                         static_cast<const char*>(a.hidden), static_cast<const char*>(a.weight),
                         a.hidden_dim, vb_begin, sa, b0);
    else
      hipLaunchKernelGGL(tile_kernel, grid, dim3(kThreads), 0, stream,
                         reinterpret_cast<const u32x4*>(a.hidden),
                         reinterpret_cast<const u32x4*>(a.weight), a.hidden_dim, n_tb, vb_begin,
                         n_vbs, sa, b0);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// Up to here one launch (lmhead_rows) does for both merges (1024 x 512 x 151936: 191.5
// against 195 us); above it is a few thousandths of the product.
constexpr int32_t kRowsTokens = 1024;

hipError_t launch_lmhead(const LmheadArgs& a, const LmheadFp8Args* fp8, const Stage2Args& a2,
                         hipStream_t stream) {
  if (a.num_tokens == 0) return hipSuccess;
  const int32_t n_vb = (a.real_vocab + kBV - 1) / kBV;
  const bool rows = a.num_shards == 1 && a.num_tiles <= 64 && a.num_tokens <= kRowsTokens;
  const int64_t max_items = launch_thread_limit() / 256 * 256;
  auto bound = [&](int64_t t) { return (int32_t)((t * a.padded_vocab) / a.num_tiles); };
  // Virtual shard s owns tiles [floor(s*T/S), floor((s+1)*T/S)): its GEMM
  // blocks, then its tiles' partials.  A block cut by a shard bound is
  // computed by both shards, each over its own rows.
  for (int32_t s = 0; s < a.num_shards; ++s) {
    const int32_t ta = (int32_t)(((int64_t)s * a.num_tiles) / a.num_shards);
    const int32_t tb = (int32_t)(((int64_t)(s + 1) * a.num_tiles) / a.num_shards);
    const int32_t col_lo = bound(ta), col_hi = bound(tb);
    const int32_t row_hi = col_hi < a.real_vocab ? col_hi : a.real_vocab;
    if (col_lo < row_hi) {  // a shard of padding only has no GEMM block
      const int32_t vb_begin = col_lo / kBV;
      const int32_t n_vbs = (row_hi - 1) / kBV + 1 - vb_begin;
      const SegmentArgs sa{a.num_tokens, a.padded_vocab, a.num_tiles, n_vb,
                           col_lo,       row_hi,         col_lo,      col_hi,
                           a.targets,    a.mask,         a.ignore_index,
                           a.seg_m,      a.seg_s,        a.target_logit};
      const hipError_t e = fp8 ? launch_segments_fp8(*fp8, sa, vb_begin, n_vbs, stream)
                               : launch_segments(a, sa, vb_begin, n_vbs, stream);
      if (e != hipSuccess) return e;
    }
    if (rows) break;
    const int64_t items = (int64_t)a.num_tokens * (tb - ta);
    for (int64_t i0 = 0; i0 < items; i0 += max_items) {
      const int64_t ni = items - i0 < max_items ? items - i0 : max_items;
      hipLaunchKernelGGL(lmhead_tiles, dim3((unsigned)((ni + 255) / 256)), dim3(256), 0, stream,
                         a.seg_m, a.seg_s, a.num_tokens, n_vb, a.real_vocab, a.padded_vocab,
                         a.num_tiles, ta, tb - ta, a.pmax, a.psum, i0);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  if (!rows) return launch_stage2(a2, stream);
  const int64_t most = launch_thread_limit() / (kRowWaves * 64);
  const int64_t blocks = (a.num_tokens + kRowWaves - 1) / kRowWaves;
  for (int64_t b = 0; b < blocks; b += most) {
    const int64_t nb = blocks - b < most ? blocks - b : most;
    hipLaunchKernelGGL(lmhead_rows, dim3((unsigned)nb), dim3(kRowWaves * 64), 0, stream, a, n_vb,
                       a2.logp, a2.lse, a2.status, b);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace rlk
