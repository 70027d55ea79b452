// rlk_process.hip -- what a sampler does to logits, for gfx950: penalties for repeated
// tokens, a bias, a temperature and a grammar's mask; and the selected token's
// log-probability under the result, with its gradient to the raw logits.
//
// For a row with raw logits x, column j, s = j occurs in the row's history, c = how often
// among its generated part:
//   x1 = s ? (x > 0 ? x / rho : x rho) : x       x2 = x1 - af c - ap [c > 0]
//   y  = (x2 + bias_j) / T                       y  = -inf where the grammar bars j
//   LSE = log sum_j exp(y_j),  logp = y_t - LSE
//   dx_j = (a g ([j = t] - p_j) + gl p_j) dy/dx,  dy/dx = (s ? (x > 0 ? 1/rho : rho) : 1) / T,
// 0 where j is barred.  A barred column's x takes part in nothing: it is replaced, not
// multiplied, so that NaN or infinity there do no harm.
//
// Three kernels share the code of one piece of a row (2048 columns a wave, 8 a lane four
// times): process_rows writes y, processed_stats each piece's (max, sum of exp(y - max)) and
// the target's y, processed_grad the gradient, from x and the LSE.  y itself goes to memory
// only where the caller wants it.  processed_merge joins the pieces of a row.
//
// Counts: a block clears one 32-bit counter per column of its span in LDS, goes over the
// row's whole history (from the L2: the blocks of a row run on one XCD) and counts the
// tokens that are its own.  LDS atomics on integers: any order gives the same counts.
// Bit 31 marks the tokens of the prompt.
//
// Sums are fp32 within a piece and fp64 over the pieces, in a fixed order; a row's results
// do not depend on what other rows share the call.  No atomics on results.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rlk_internal.h"
#include "rlk_rows.h"
#include "rlk_tile.h"

namespace rlk {
namespace {

constexpr int kPieceChunks = 4;                      // of 8 columns, a lane
constexpr int kPiece = kPieceChunks * 64 * 8;        // columns a wave takes
constexpr uint32_t kOfPrompt = 0x80000000u;
static_assert(kPiece == kProcessPiece, "the boundary sizes the partials by it");

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef int32_t i32x4g __attribute__((ext_vector_type(4)));

// The rules of one row.
struct RowRules {
  float rho, inv_rho, presence, frequency, inv_t;
  int64_t begin, split, end;  // its history, if it counts for anything (else begin == end)
  const float* bias;          // or null
  const uint8_t* allow;       // a bit per column, or null
};

// Row `index[r]` of a table of `rows` rows; without an index row r, or the only one.
__device__ __forceinline__ int64_t table_row(const int32_t* index, int64_t rows, int32_t r) {
  const int64_t at = index ? index[r] : rows == 1 ? 0 : r;
  return at >= 0 && at < rows ? at : -1;
}

__device__ __forceinline__ RowRules row_rules(const RuleArgs& a, int32_t r) {
  RowRules o;
  o.rho = a.repetition ? a.repetition[r] : 1.0f;
  o.presence = a.presence ? a.presence[r] : 0.0f;
  o.frequency = a.frequency ? a.frequency[r] : 0.0f;
  o.inv_rho = 1.0f / o.rho;
  o.inv_t = a.temperature ? 1.0f / a.temperature[r] : 1.0f;
  o.begin = o.split = o.end = 0;
  if (a.history && (o.rho != 1.0f || o.presence != 0.0f || o.frequency != 0.0f)) {
    // whatever the caller's numbers, only the history's own tokens are read
    o.begin = max(a.history_begin[r], (int64_t)0);
    o.end = max(min(a.history_end[r], a.history_len), o.begin);
    o.split = a.history_split ? a.history_split[r] : o.begin;
  }
  const int64_t b = a.bias ? table_row(a.bias_index, a.bias_rows, r) : -1;
  o.bias = b >= 0 ? a.bias + b * a.ld_bias : nullptr;
  const int64_t m = a.allow ? table_row(a.allow_index, a.allow_rows, r) : -1;
  o.allow = m >= 0 ? reinterpret_cast<const uint8_t*>(a.allow + m * a.ld_allow) : nullptr;
  return o;
}

// Counts the history's tokens of the columns [c0, c0 + kSpan); by the whole block.
template <int kSpan, int kThr>
__device__ __forceinline__ void count_tokens(uint32_t* counts, const int32_t* history,
                                             const RowRules& o, int32_t c0) {
  const int tid = threadIdx.x;
#pragma unroll
  for (int i = 0; i < kSpan / 4 / kThr; ++i)
    reinterpret_cast<u32x4*>(counts)[i * kThr + tid] = u32x4{0, 0, 0, 0};
  __syncthreads();
  auto count = [&](int32_t token, int64_t at) __attribute__((always_inline)) {
    const uint32_t col = (uint32_t)token - (uint32_t)c0;
    if (token < 0 || col >= (uint32_t)kSpan) return;
    if (at >= o.split)
      atomicAdd(counts + col, 1u);
    else
      atomicOr(counts + col, kOfPrompt);
  };
  // whole vectors from the first 16-byte boundary on, the ends one by one
  const int64_t skip = (4 - ((reinterpret_cast<uintptr_t>(history + o.begin) >> 2) & 3)) & 3;
  const int64_t first = min(o.begin + skip, o.end), vectors = (o.end - first) / 4;
  const i32x4g* v = reinterpret_cast<const i32x4g*>(history + first);
  for (int64_t q = tid; q < vectors; q += kThr) {
    const i32x4g t = v[q];
#pragma unroll
    for (int e = 0; e < 4; ++e) count(t[e], first + q * 4 + e);
  }
  const int64_t tail = first + vectors * 4;
  if (tid < first - o.begin) count(history[o.begin + tid], o.begin + tid);
  if (tid < o.end - tail) count(history[tail + tid], tail + tid);
  __syncthreads();
}

// One lane's columns of a piece: loads go out together, then each chunk of 8 is worked on.
// visit(i, col, x, y, slope): chunk i's columns from `col` (< real_vocab) on; the columns
// behind the last real one hold -inf and slope 0.
template <bool kSlope, typename Visit>
__device__ __forceinline__ void for_piece(const uint16_t* row, const RowRules& o, bool counted,
                                          const uint32_t* counts, int32_t c0, int32_t real_vocab,
                                          int lane, Visit&& visit) {
  u32x4 raw[kPieceChunks];
  uint32_t bits[kPieceChunks];
#pragma unroll
  for (int i = 0; i < kPieceChunks; ++i) {
    const int32_t col = c0 + (i * 64 + lane) * 8;
    raw[i] = u32x4{0, 0, 0, 0};
    bits[i] = 0;
    if (col < real_vocab) {
      raw[i] = *reinterpret_cast<const u32x4*>(row + col);
      const int32_t left = real_vocab - col;
      bits[i] = left >= 8 ? 0xFFu : (1u << left) - 1;
      if (o.allow) bits[i] &= o.allow[col >> 3];
    }
  }
#pragma unroll
  for (int i = 0; i < kPieceChunks; ++i) {
    const int at = (i * 64 + lane) * 8;
    const int32_t col = c0 + at;
    float y[8], slope[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = __uint_as_float(e & 1 ? raw[i][e / 2] & 0xFFFF0000u : raw[i][e / 2] << 16);
      if (kSlope) slope[e] = o.inv_t;
    }
    if (counted) {
      const u32x4 n0 = *reinterpret_cast<const u32x4*>(counts + at);
      const u32x4 n1 = *reinterpret_cast<const u32x4*>(counts + at + 4);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t n = e < 4 ? n0[e & 3] : n1[e & 3];
        if (n == 0) continue;
        const float by = y[e] > 0.0f ? o.inv_rho : o.rho;
        const uint32_t c = n & ~kOfPrompt;
        y[e] = y[e] * by - (o.frequency * (float)c + (c ? o.presence : 0.0f));
        if (kSlope) slope[e] *= by;
      }
    }
    if (o.bias && col < real_vocab) {
      if (col + 8 <= real_vocab) {
        const f32x4u b0 = *reinterpret_cast<const f32x4u*>(o.bias + col);
        const f32x4u b1 = *reinterpret_cast<const f32x4u*>(o.bias + col + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] += e < 4 ? b0[e & 3] : b1[e & 3];
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e < real_vocab) y[e] += o.bias[col + e];
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const bool on = (bits[i] >> e) & 1;
      y[e] = on ? y[e] * o.inv_t : kNegInf;
      if (kSlope && !on) slope[e] = 0.0f;
    }
    visit(i, col, y, slope);
  }
}

// 8 values of a row, of which `n` are to be written.
__device__ __forceinline__ void put8(uint16_t* out, const float* y, int32_t n) {
  union {
    uint16_t e[8];
    u32x4 x;
  } o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o.e[e] = bf16_bits(y[e]);
  if (n >= 8) {
    *reinterpret_cast<u32x4*>(out) = o.x;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) out[e] = o.e[e];
}
__device__ __forceinline__ void put8(float* out, const float* y, int32_t n) {
  if (n >= 8) {
    reinterpret_cast<f32x4*>(out)[0] = f32x4{y[0], y[1], y[2], y[3]};
    reinterpret_cast<f32x4*>(out)[1] = f32x4{y[4], y[5], y[6], y[7]};
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) out[e] = y[e];
}

// A block's row, and the first column of its span; false past the end.
template <int kSpan>
__device__ __forceinline__ void block_of(int64_t blk_begin, int32_t columns, int32_t& r,
                                         int32_t& c0) {
  const int64_t blk = blk_begin + xcd_local_block(blockIdx.x, gridDim.x);
  const int32_t spans = (columns - 1) / kSpan + 1;
  r = (int32_t)(blk / spans);
  c0 = (int32_t)(blk - (int64_t)r * spans) * kSpan;
}

template <int kWaves, typename OutT>
__global__ __launch_bounds__(64 * kWaves) void process_rows(const uint16_t* logits, int64_t ld,
                                                            int32_t real_vocab,
                                                            int32_t padded_vocab, RuleArgs rules,
                                                            OutT* out, int64_t ld_out,
                                                            int64_t blk_begin) {
  constexpr int kSpan = kWaves * kPiece;
  __shared__ __attribute__((aligned(16))) uint32_t counts[kSpan];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int32_t r, c0;
  block_of<kSpan>(blk_begin, padded_vocab, r, c0);
  const RowRules o = row_rules(rules, r);
  const bool counted = o.end > o.begin;
  if (counted) count_tokens<kSpan, 64 * kWaves>(counts, rules.history, o, c0);
  for_piece<false>(logits + r * ld, o, counted, counts + wave * kPiece, c0 + wave * kPiece,
                   real_vocab, lane, [&](int, int32_t col, const float* y, const float*) {
                     if (col < padded_vocab) put8(out + r * ld_out + col, y, padded_vocab - col);
                   });
}

__device__ __forceinline__ float wave_max(float m) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = maxnan(m, __shfl_xor(m, o));
  return m;
}

template <int kWaves>
__global__ __launch_bounds__(64 * kWaves) void processed_stats(ProcessedArgs a, RuleArgs rules,
                                                               int64_t blk_begin) {
  constexpr int kSpan = kWaves * kPiece;
  __shared__ __attribute__((aligned(16))) uint32_t counts[kSpan];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int32_t r, c0;
  block_of<kSpan>(blk_begin, a.real_vocab, r, c0);
  const RowRules o = row_rules(rules, r);
  const bool counted = o.end > o.begin;
  if (counted) count_tokens<kSpan, 64 * kWaves>(counts, rules.history, o, c0);
  c0 += wave * kPiece;
  if (c0 >= a.real_vocab) return;
  const bool masked = a.mask != nullptr && a.mask[r] == 0;
  const int32_t target = masked ? -1 : a.targets[r];  // (in no column if it is out of range)
  float v[kPieceChunks * 8], top = kNegInf;
  for_piece<false>(static_cast<const uint16_t*>(a.logits) + r * a.ld, o, counted,
                   counts + wave * kPiece, c0, a.real_vocab, lane,
                   [&](int i, int32_t col, const float* y, const float*) {
#pragma unroll
                     for (int e = 0; e < 8; ++e) {
                       v[i * 8 + e] = y[e];
                       top = maxnan(top, y[e]);
                       if (col + e == target && target < a.real_vocab) a.target_logit[r] = y[e];
                     }
                   });
  top = wave_max(top);
  // a piece without a finite column: exp(-inf - 0) = 0, the identity (-inf, 0)
  const float base = top == kNegInf ? 0.0f : top;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kPieceChunks * 8; ++i) sum += exp2_hw((v[i] - base) * kLog2e);
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s);
  if (lane != 0) return;
  const int64_t at = (int64_t)r * a.pieces + c0 / kPiece;
  a.pmax[at] = top;
  a.psum[at] = sum;
}

// One wave a row: an exact maximum, then an fp64 sum of the pieces.
constexpr int kMergeRows = 4;

__global__ __launch_bounds__(64 * kMergeRows) void processed_merge(ProcessedArgs a,
                                                                   int64_t blk_begin) {
  const int lane = threadIdx.x & 63;
  const int64_t r = (blk_begin + blockIdx.x) * kMergeRows + (threadIdx.x >> 6);
  if (r >= a.num_rows) return;
  const float *pmax = a.pmax + r * a.pieces, *psum = a.psum + r * a.pieces;
  float top = kNegInf;
  for (int32_t i = lane; i < a.pieces; i += 64) top = maxnan(top, pmax[i]);
  top = wave_max(top);
  float lse = kNegInf;
  if (top != kNegInf) {
    double sum = 0.0;
    for (int32_t i = lane; i < a.pieces; i += 64)
      sum = fma((double)psum[i], (double)expf(pmax[i] - top), sum);
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s);
    lse = (float)((double)top + log(sum));
  }
  if (lane != 0) return;
  a.lse[r] = lse;
  const bool masked = a.mask != nullptr && a.mask[r] == 0;
  const int32_t target = masked ? a.ignore_index : a.targets[r];
  if (target == a.ignore_index) {
    a.logp[r] = 0.0f;
  } else if (target < 0 || target >= a.real_vocab) {
    a.logp[r] = __builtin_nanf("");
    a.status[0] = 1u;
  } else {
    a.logp[r] = a.target_logit[r] - lse;
    if (!__builtin_isfinite(lse)) a.status[1] = 1u;
  }
}

template <int kWaves, typename OutT>
__global__ __launch_bounds__(64 * kWaves) void processed_grad(ProcessedArgs a, RuleArgs rules,
                                                              OutT* dlogits, int64_t ld_d,
                                                              int64_t blk_begin) {
  constexpr int kSpan = kWaves * kPiece;
  __shared__ __attribute__((aligned(16))) uint32_t counts[kSpan];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int32_t r, c0;
  block_of<kSpan>(blk_begin, a.padded_vocab, r, c0);
  OutT* out = dlogits + r * ld_d;
  const bool masked = a.mask != nullptr && a.mask[r] == 0;
  const int32_t target = masked ? a.ignore_index : a.targets[r];
  const bool act = target != a.ignore_index;
  const float g = act && a.grad ? a.grad[r] : 0.0f, gl = a.grad_lse ? a.grad_lse[r] : 0.0f;
  const bool bad = act && (target < 0 || target >= a.real_vocab);
  c0 += wave * kPiece;
  if (bad || (g == 0.0f && gl == 0.0f)) {  // (the whole block)
    if (bad && c0 == 0 && lane == 0) a.status[0] = 1u;
#pragma unroll
    for (int i = 0; i < kPieceChunks; ++i) {
      const int32_t col = c0 + (i * 64 + lane) * 8;
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = bad && col + e < a.real_vocab ? __builtin_nanf("") : 0.0f;
      if (col < a.padded_vocab) put8(out + col, d, a.padded_vocab - col);
    }
    return;
  }
  const RowRules o = row_rules(rules, r);
  const bool counted = o.end > o.begin;
  if (counted)
    count_tokens<kSpan, 64 * kWaves>(counts, rules.history, o, c0 - wave * kPiece);
  const float coef = gl - g, lse = a.lse[r];
  for_piece<true>(static_cast<const uint16_t*>(a.logits) + r * a.ld, o, counted,
                  counts + wave * kPiece, c0, a.real_vocab, lane,
                  [&](int, int32_t col, const float* y, const float* slope) {
                    float d[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                      const float p = exp2_hw((y[e] - lse) * kLog2e);
                      const float dy = act && col + e == target ? fmaf(coef, p, g) : coef * p;
                      // (not a product with 0: the LSE of a row that is barred altogether
                      // is -inf)
                      d[e] = slope[e] == 0.0f ? 0.0f : dy * slope[e];
                    }
                    if (col < a.padded_vocab) put8(out + col, d, a.padded_vocab - col);
                  });
}

constexpr int kRowWaves = 4;

int64_t blocks_of(int32_t rows, int32_t columns) {
  constexpr int kSpan = kRowWaves * kPiece;
  return (int64_t)rows * ((columns - 1) / kSpan + 1);
}

}  // namespace

hipError_t launch_process(const void* logits, int64_t ld, int32_t num_rows, int32_t real_vocab,
                          int32_t padded_vocab, const RuleArgs& rules, void* out, int64_t ld_out,
                          bool out_bf16, hipStream_t stream) {
  const uint16_t* x = static_cast<const uint16_t*>(logits);
  const dim3 threads(64 * kRowWaves);
  return in_launches(blocks_of(num_rows, padded_vocab), 64 * kRowWaves, [&](int64_t b, int64_t nb) {
    if (out_bf16)
      hipLaunchKernelGGL((process_rows<kRowWaves, uint16_t>), dim3((unsigned)nb), threads, 0, stream, x, ld,
                         real_vocab, padded_vocab, rules, static_cast<uint16_t*>(out), ld_out, b);
    else
      hipLaunchKernelGGL((process_rows<kRowWaves, float>), dim3((unsigned)nb), threads, 0, stream, x, ld,
                         real_vocab, padded_vocab, rules, static_cast<float*>(out), ld_out, b);
  });
}

hipError_t launch_processed_fwd(const ProcessedArgs& a, const RuleArgs& rules,
                                hipStream_t stream) {
  hipError_t e = in_launches(blocks_of(a.num_rows, a.real_vocab), 64 * kRowWaves,
                             [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL(processed_stats<kRowWaves>, dim3((unsigned)nb), dim3(64 * kRowWaves), 0, stream, a,
                       rules, b);
  });
  if (e != hipSuccess) return e;
  return in_launches(((int64_t)a.num_rows + kMergeRows - 1) / kMergeRows, 64 * kMergeRows,
                     [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL(processed_merge, dim3((unsigned)nb), dim3(64 * kMergeRows), 0, stream, a, b);
  });
}

hipError_t launch_processed_bwd(const ProcessedArgs& a, const RuleArgs& rules, void* dlogits,
                                int64_t ld_d, bool out_bf16, hipStream_t stream) {
  const dim3 threads(64 * kRowWaves);
  return in_launches(blocks_of(a.num_rows, a.padded_vocab), 64 * kRowWaves,
                     [&](int64_t b, int64_t nb) {
    if (out_bf16)
      hipLaunchKernelGGL((processed_grad<kRowWaves, uint16_t>), dim3((unsigned)nb), threads, 0, stream, a,
                         rules, static_cast<uint16_t*>(dlogits), ld_d, b);
    else
      hipLaunchKernelGGL((processed_grad<kRowWaves, float>), dim3((unsigned)nb), threads, 0, stream, a, rules,
                         static_cast<float*>(dlogits), ld_d, b);
  });
}

}  // namespace rlk
