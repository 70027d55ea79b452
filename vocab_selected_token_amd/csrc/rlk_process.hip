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
// Counts: a block has one 32-bit counter per column of its span (8192) in LDS, goes over the
// row's whole history (its first 4096 tokens stay in registers for all of the block's spans) and
// counts the tokens that are its own.  LDS atomics on integers: any order gives the same counts.
// Bit 31 marks the tokens of the prompt.  Counters are read back, and cleared, as their columns
// are worked on; where none of a wave's 512 columns is counted the penalties are skipped.
//
// What bounds it: arithmetic and the chain of a span, not yet memory alone.  The statistics of 4096
// rows x 151936 with 2048 tokens of history each take 422-436 us (2.9 TB/s; the vector units are
// busy 68% of it, with 17 instructions a column, half of them for penalties: nearly every 512
// columns hold some token), the gradient 544-557 us (4.5 TB/s); with short histories, 1024 rows,
// 85-95 and 109-112 us (3.3-3.7 and 5.6 TB/s); 512 rows processed 73-75 us (4.3 TB/s).  The logits
// are read through buffers, whose bounds stand in for a test of every load, and a span's are on
// their way while the one before is worked on (with 64-bit addresses, tests and shuffles through
// LDS the statistics took 625 us).
//
// Sums are fp32 within a piece and fp64 over the pieces, in a fixed order; a row's results
// do not depend on what other rows share the call.  No atomics on results.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "rlk_internal.h"
#include "rlk_rows.h"
#include "rlk_tile.h"

namespace rlk {
namespace {

constexpr int kPieceChunks = 4;                      // of 8 columns, a lane
constexpr int kPiece = kPieceChunks * 64 * 8;        // columns a wave takes
constexpr int kSpanThreads = 256;
constexpr int kSpan = kSpanThreads / 64 * kPiece;    // columns a block takes at a time
constexpr uint32_t kOfPrompt = 0x80000000u;
static_assert(kPiece == kProcessPiece, "the boundary sizes the partials by it");

typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));
typedef int32_t i32x4g __attribute__((ext_vector_type(4)));

// How the rows are cut: `parts` blocks a row, each of `per` spans (of a block's pieces).
struct Spans {
  int32_t columns, per, parts;
  int32_t row;     // the launch's first block: a row
  uint32_t first;  // and its part
};

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

// LDS is written and read through this barrier; loads in flight stay there.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// Counts a row's tokens in the columns of one span after another, by the whole block.  Each
// thread keeps up to 16 of the row's tokens in registers; a longer history's others come from
// memory for every span.
struct Counter {
  static constexpr int kHeld = 4;  // vectors of 4 tokens
  uint32_t* counts;  // kSpan of them in LDS
  const i32x4g* v;
  int32_t vectors, ends;  // whole vectors from the first 16-byte boundary on; tokens beside them
  int32_t split;          // where the prompt ends, from the first vector on
  i32x4g held[kHeld];
  int32_t end_token;      // one of the tokens beside the vectors, or -1
  bool end_made;

  __device__ __forceinline__ Counter(uint32_t* counts_, const int32_t* history,
                                     const RowRules& o)
      : counts(counts_) {
    const int tid = threadIdx.x;
    const int64_t skip = (4 - ((reinterpret_cast<uintptr_t>(history + o.begin) >> 2) & 3)) & 3;
    const int64_t first = min(o.begin + skip, o.end);
    v = reinterpret_cast<const i32x4g*>(history + first);
    vectors = (int32_t)((o.end - first) / 4);
    split = (int32_t)(min(max(o.split, o.begin), o.end) - first);
    // at most 3 tokens in front of the vectors and 3 behind
    const int64_t tail = first + (int64_t)vectors * 4;
    const int32_t lead = (int32_t)(first - o.begin);
    ends = lead + (int32_t)(o.end - tail);
    end_token = -1;
    end_made = false;
    if (tid < ends) {
      const int64_t at = tid < lead ? o.begin + tid : tail + (tid - lead);
      end_token = history[at];
      end_made = at >= o.split;
    }
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      held[j] = i32x4g{-1, -1, -1, -1};
      if (tid + j * kSpanThreads < vectors) held[j] = v[tid + j * kSpanThreads];
    }
#pragma unroll
    for (int i = 0; i < kSpan / 4 / kSpanThreads; ++i)
      reinterpret_cast<u32x4*>(counts)[i * kSpanThreads + tid] = u32x4{0, 0, 0, 0};
    lds_barrier();
  }

  __device__ __forceinline__ void one(int32_t token, bool made, int32_t c0) const {
    // (a token below 0 is a column far behind)
    const uint32_t col = (uint32_t)token - (uint32_t)c0;
    if (col >= (uint32_t)kSpan) return;
    if (made)
      atomicAdd(counts + col, 1u);
    else
      atomicOr(counts + col, kOfPrompt);
  }

  // Counts the tokens of the columns [c0, c0 + kSpan): the counters are all zero before.
  __device__ __forceinline__ void count(int32_t c0) const {
    const int tid = threadIdx.x;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      if (j * kSpanThreads >= vectors) break;  // (uniform)
#pragma unroll
      for (int e = 0; e < 4; ++e) one(held[j][e], (tid + j * kSpanThreads) * 4 + e >= split, c0);
    }
#pragma unroll 2
    for (int32_t q = tid + kHeld * kSpanThreads; q < vectors; q += kSpanThreads) {
      const i32x4g t = v[q];
#pragma unroll
      for (int e = 0; e < 4; ++e) one(t[e], q * 4 + e >= split, c0);
    }
    one(end_token, end_made, c0);
    lds_barrier();
  }
};

// A row's logits and its grammar's bits, as buffers: what lies behind the last real column reads
// as 0.  A load's whole position stands in its vector offset: a buffer's bounds are compared with
// that one, and a position in the scalar offset, which can lie behind the row by itself, is not
// sure to be held to them.
struct RowBuffers {
  __amdgpu_buffer_rsrc_t logits, allow;
};

// One lane's columns of a piece: chunk i are 8 columns from (i * 64 + lane) * 8 on.
struct Piece {
  u32x4 raw[kPieceChunks];
  uint32_t bits[kPieceChunks];  // which of a chunk's columns are allowed (with a grammar)
};

__device__ __forceinline__ void load_bits(Piece& p, int i, const RowBuffers& b, int32_t c0,
                                          int lane) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass cannot instantiate the target's builtins
  p.bits[i] = __builtin_amdgcn_raw_buffer_load_b8(
      b.allow, (uint32_t)c0 / 8 + (uint32_t)lane + i * 64, 0, 0);
#endif
}
__device__ __forceinline__ void load_chunk(Piece& p, int i, const RowBuffers& b, bool allow,
                                           int32_t c0, int lane) {
#if defined(__HIP_DEVICE_COMPILE__)
  p.raw[i] = __builtin_bit_cast(
      u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                 b.logits, (uint32_t)c0 * 2 + (uint32_t)lane * 16 + i * 1024, 0, 0));
  if (allow) load_bits(p, i, b, c0, lane);
#endif
}

// x where the bit is set, `other`'s bits where not.
__device__ __forceinline__ float where_bit(uint32_t bits, int e, float x, uint32_t other) {
  const uint32_t m = (uint32_t)((int32_t)(bits << (31 - e)) >> 31);
  return __uint_as_float((__float_as_uint(x) & m) | (other & ~m));
}

// Works on the piece from column c0 on, chunk by chunk, and loads the one from `next` on (if
// >= 0) in its place: visit(i, col, y, by, bits, some) has chunk i's columns from `col` on, with
// by = dy/dx (kSlope), and whether some column of the wave's chunk is barred or padding (y is
// -inf there).  What a chunk or a row has no use for is skipped for the whole wave.  The counters
// (null: none) are zero again afterwards.
template <bool kSlope, typename Visit>
__device__ __forceinline__ void for_piece(Piece& p, const RowBuffers& rb, const RowRules& o,
                                          uint32_t* counts, int32_t c0, int32_t next,
                                          int32_t real_vocab, int lane, Visit&& visit) {
#pragma unroll
  for (int i = 0; i < kPieceChunks; ++i) {
    const int at = (i * 64 + lane) * 8;
    const int32_t col = c0 + at;
    float y[8], by[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = __uint_as_float(e & 1 ? p.raw[i][e / 2] & 0xFFFF0000u : p.raw[i][e / 2] << 16);
      if (kSlope) by[e] = o.inv_t;
    }
    const bool edge = c0 + (i + 1) * 512 > real_vocab;
    uint32_t bits = o.allow ? p.bits[i] : 0xFFu;
    if (edge) {
      const int32_t left = real_vocab - col;
      bits &= left >= 8 ? 0xFFu : left > 0 ? (1u << left) - 1 : 0u;
    }
    if (next >= 0) load_chunk(p, i, rb, o.allow != nullptr, next, lane);
    if (counts) {
      u32x4* n = reinterpret_cast<u32x4*>(counts + at);
      const u32x4 n0 = n[0], n1 = n[1];
      if (__any((n0[0] | n0[1] | n0[2] | n0[3] | n1[0] | n1[1] | n1[2] | n1[3]) != 0)) {
        n[0] = n[1] = u32x4{0, 0, 0, 0};
        float f[8];
        // (not counted: times 1, less 0)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 1.0f;
        if (o.rho != 1.0f) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if ((e < 4 ? n0[e & 3] : n1[e & 3]) != 0) f[e] = y[e] > 0.0f ? o.inv_rho : o.rho;
          if (kSlope) {
#pragma unroll
            for (int e = 0; e < 8; ++e) by[e] *= f[e];
          }
        }
        if (o.frequency != 0.0f || o.presence != 0.0f) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t c = (e < 4 ? n0[e & 3] : n1[e & 3]) & ~kOfPrompt;
            y[e] = fmaf(y[e], f[e], c ? -fmaf(o.frequency, (float)c, o.presence) : 0.0f);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] *= f[e];
        }
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
    for (int e = 0; e < 8; ++e) y[e] *= o.inv_t;
    const bool some = o.allow || edge;
    if (some) {
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = where_bit(bits, e, y[e], 0xFF800000u);
    }
    visit(i, col, y, by, bits, some);
  }
}

// A block's part of the problem: `per` spans of one row, from column c0 up to c1.
struct Part {
  int32_t row, c0, c1;
};
__device__ __forceinline__ Part part_of(const Spans& s) {
  // consecutive indices on one XCD, as in xcd_local_block
  const uint32_t b = blockIdx.x, n = gridDim.x, rem = n % 8, x = b % 8;
  const uint32_t at = s.first + x * (n / 8) + min(x, rem) + b / 8, row = at / (uint32_t)s.parts;
  Part p;
  p.row = s.row + (int32_t)row;
  p.c0 = (int32_t)(at - row * s.parts) * s.per * kSpan;
  p.c1 = (int32_t)min((int64_t)p.c0 + (int64_t)s.per * kSpan, (int64_t)s.columns);
  return p;
}

// The buffers of a row; the first piece's logits are on their way before its rules are known.
__device__ __forceinline__ RowBuffers row_buffers(const uint16_t* row, int32_t real_vocab) {
  RowBuffers b;
  b.logits = __builtin_amdgcn_make_buffer_rsrc(
      const_cast<uint16_t*>(row), 0, (int)(((uint32_t)real_vocab + 7) / 8 * 16), kBufferWord3);
  b.allow = b.logits;
  return b;
}
__device__ __forceinline__ void first_logits(Piece& p, const RowBuffers& b, int32_t c0, int lane) {
#pragma unroll
  for (int i = 0; i < kPieceChunks; ++i) load_chunk(p, i, b, false, c0, lane);
}

// A part's spans one after another, each wave a piece of each: each(its first column, the next
// one's or -1, its counters) works on `p` and loads the next piece in its place.
template <typename Each>
__device__ __forceinline__ void for_spans(const Part& part, int32_t real_vocab,
                                          const RuleArgs& rules, const RowRules& o, RowBuffers& b,
                                          Piece& p, uint32_t* counts, int lane, int wave,
                                          Each&& each) {
  const bool counted = o.end > o.begin;  // (uniform)
  if (o.allow) {
    b.allow = __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(o.allow), 0,
                                                (int)(((uint32_t)real_vocab + 7) / 8),
                                                kBufferWord3);
#pragma unroll
    for (int i = 0; i < kPieceChunks; ++i)
      load_bits(p, i, b, part.c0 + wave * kPiece, lane);
  }
  auto spans = [&](auto&& count, uint32_t* own) __attribute__((always_inline)) {
    for (int32_t c0 = part.c0; c0 < part.c1; c0 += kSpan) {
      count(c0);
      const int32_t cw = c0 + wave * kPiece;
      const bool more = c0 + kSpan < part.c1;
      each(cw, more ? cw + kSpan : -1, own);
      if (!more) break;
      if (own) lds_barrier();  // every counter is zero again
    }
  };
  if (counted) {
    const Counter counter(counts, rules.history, o);
    spans([&](int32_t c0) { counter.count(c0); }, counts + wave * kPiece);
  } else {
    spans([](int32_t) {}, nullptr);
  }
}

// exp(y - base) for many y of one base: exp2(y L - hi), L = log2 e, in one fma, which is exact
// up to its one rounding; what hi took from base L goes into the factor, once.  Below 2^24 that
// is at most 1, half a step of hi < 2^25; a base farther out, whose hi may be off by more than an
// exponential holds, takes the difference first.
struct ExpFrom {
  float base, hi, factor;
  bool near;
  __device__ __forceinline__ explicit ExpFrom(float b) : base(b) {
    near = fabsf(b) < 0x1p24f;
    hi = b * kLog2e;
    factor = near ? exp2_hw(-fmaf(b, kLog2e, -hi)) : 1.0f;
  }
  // without the factor
  template <int kN>
  __device__ __forceinline__ void operator()(const float* y, float* e) const {
    if (near) {
#pragma unroll
      for (int i = 0; i < kN; ++i) e[i] = exp2_hw(fmaf(y[i], kLog2e, -hi));
    } else {
#pragma unroll
      for (int i = 0; i < kN; ++i) e[i] = exp2_hw((y[i] - base) * kLog2e);
    }
  }
};

// 8 values of a row, of which `n` are to be written; kStream: past the caches (512 rows
// processed 85 -> 75 us; the gradient of 1024 rows 110 -> 121, so not there).
template <bool kStream, typename T>
__device__ __forceinline__ void put_vector(T* out, const T& x) {
  if constexpr (kStream)
    __builtin_nontemporal_store(x, out);
  else
    *out = x;
}
template <bool kStream>
__device__ __forceinline__ void put8(uint16_t* out, const float* y, int32_t n) {
  union {
    uint16_t e[8];
    u32x4 x;
  } o;
#pragma unroll
  for (int e = 0; e < 8; ++e) o.e[e] = bf16_bits(y[e]);
  if (n >= 8) {
    put_vector<kStream>(reinterpret_cast<u32x4*>(out), o.x);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) out[e] = o.e[e];
}
template <bool kStream>
__device__ __forceinline__ void put8(float* out, const float* y, int32_t n) {
  if (n >= 8) {
    put_vector<kStream>(reinterpret_cast<f32x4*>(out), f32x4{y[0], y[1], y[2], y[3]});
    put_vector<kStream>(reinterpret_cast<f32x4*>(out) + 1, f32x4{y[4], y[5], y[6], y[7]});
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (e < n) out[e] = y[e];
}

template <typename OutT>
__global__ __launch_bounds__(kSpanThreads, 4) void process_rows(const uint16_t* logits, int64_t ld,
                                                            int32_t real_vocab, Spans spans,
                                                            RuleArgs rules, OutT* out,
                                                            int64_t ld_out) {
  __shared__ __attribute__((aligned(16))) uint32_t counts[kSpan];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Part part = part_of(spans);
  out += part.row * ld_out;
  RowBuffers b = row_buffers(logits + part.row * ld, real_vocab);
  Piece p;
  first_logits(p, b, part.c0 + wave * kPiece, lane);
  const RowRules o = row_rules(rules, part.row);
  for_spans(part, real_vocab, rules, o, b, p, counts, lane, wave,
            [&](int32_t cw, int32_t next, uint32_t* own) __attribute__((always_inline)) {
    for_piece<false>(p, b, o, own, cw, next, real_vocab, lane,
                     [&](int, int32_t col, const float* y, const float*, uint32_t, bool)
                         __attribute__((always_inline)) {
      if (col < spans.columns) put8<true>(out + col, y, spans.columns - col);
    });
  });
}

// Over a wave, in a fixed order: within rows of 16 lanes by rotations, then the four rows.
template <typename F>
__device__ __forceinline__ float wave_reduce(float x, F&& f) {
#if defined(__HIP_DEVICE_COMPILE__)
  auto rotated = [](float v, auto by) {
    return __builtin_bit_cast(
        float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),
                                           0x120 + decltype(by)::value, 0xF, 0xF, false));
  };
  x = f(x, rotated(x, std::integral_constant<int, 8>()));
  x = f(x, rotated(x, std::integral_constant<int, 4>()));
  x = f(x, rotated(x, std::integral_constant<int, 2>()));
  x = f(x, rotated(x, std::integral_constant<int, 1>()));
  auto row = [&](int lane) {
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), lane));
  };
  return f(f(row(0), row(16)), f(row(32), row(48)));
#else
  return x;
#endif
}
__device__ __forceinline__ float wave_max(float m) {
  return wave_reduce(m, [](float x, float y) { return fmaxf(x, y); });
}

// (max, sum of exp(y - max)) of each piece.  The maximum passes over NaN; the sum does not.  A
// piece without a finite column: exp(-inf - 0) = 0, the identity (-inf, 0).
__global__ __launch_bounds__(kSpanThreads, 4) void processed_stats(ProcessedArgs a, Spans spans,
                                                               RuleArgs rules) {
  __shared__ __attribute__((aligned(16))) uint32_t counts[kSpan];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Part part = part_of(spans);
  const int32_t r = part.row;
  RowBuffers b = row_buffers(static_cast<const uint16_t*>(a.logits) + r * a.ld, a.real_vocab);
  Piece p;
  first_logits(p, b, part.c0 + wave * kPiece, lane);
  const bool masked = a.mask != nullptr && a.mask[r] == 0;
  const int32_t target = masked ? -1 : a.targets[r];  // (in no column if it is out of range)
  const RowRules o = row_rules(rules, r);
  for_spans(part, a.real_vocab, rules, o, b, p, counts, lane, wave,
            [&](int32_t cw, int32_t next, uint32_t* own) __attribute__((always_inline)) {
    if (cw >= a.real_vocab) return;
    const bool here = target >= cw && target < cw + kPiece && target < a.real_vocab;
    float v[kPieceChunks * 8], top = kNegInf;
    for_piece<false>(p, b, o, own, cw, next, a.real_vocab, lane,
                     [&](int i, int32_t col, const float* y, const float*, uint32_t, bool)
                         __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i * 8 + e] = y[e];
        top = fmaxf(top, y[e]);
      }
      if (here) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e == target) a.target_logit[r] = y[e];
      }
    });
    top = wave_max(top);
    const ExpFrom exp_of(top == kNegInf ? 0.0f : top);
    exp_of.template operator()<kPieceChunks * 8>(v, v);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < kPieceChunks * 8; ++i) sum += v[i];
    sum = wave_reduce(sum, [](float x, float y) { return x + y; });
    if (lane != 0) return;
    const int64_t at = (int64_t)r * a.pieces + cw / kPiece;
    a.pmax[at] = top;
    a.psum[at] = sum * exp_of.factor;
  });
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
  for (int32_t i = lane; i < a.pieces; i += 64) top = fmaxf(top, pmax[i]);
  top = wave_max(top);
  // (where no piece has a maximum there may still be NaN in the sums; else log 0 = -inf)
  const float base = top == kNegInf ? 0.0f : top;
  double sum = 0.0;
  for (int32_t i = lane; i < a.pieces; i += 64)
    sum = fma((double)psum[i], (double)expf(pmax[i] - base), sum);
#pragma unroll
  for (int s = 32; s >= 1; s >>= 1) sum += __shfl_xor(sum, s);
  const float lse = (float)((double)base + log(sum));
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

template <typename OutT>
__global__ __launch_bounds__(kSpanThreads, 4) void processed_grad(ProcessedArgs a, Spans spans,
                                                              RuleArgs rules, OutT* out,
                                                              int64_t ld_d) {
  __shared__ __attribute__((aligned(16))) uint32_t counts[kSpan];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Part part = part_of(spans);
  const int32_t r = part.row;
  out += r * ld_d;
  const bool masked = a.mask != nullptr && a.mask[r] == 0;
  const int32_t target = masked ? a.ignore_index : a.targets[r];
  const bool act = target != a.ignore_index;
  const float g = act && a.grad ? a.grad[r] : 0.0f, gl = a.grad_lse ? a.grad_lse[r] : 0.0f;
  const bool bad = act && (target < 0 || target >= a.real_vocab);
  if (bad || (g == 0.0f && gl == 0.0f)) {  // (the whole block)
    if (bad && part.c0 == 0 && threadIdx.x == 0) a.status[0] = 1u;
    for (int32_t col = part.c0 + (int32_t)threadIdx.x * 8; col < part.c1; col += kSpanThreads * 8) {
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = bad && col + e < a.real_vocab ? __builtin_nanf("") : 0.0f;
      put8<false>(out + col, d, spans.columns - col);
    }
    return;
  }
  RowBuffers b = row_buffers(static_cast<const uint16_t*>(a.logits) + r * a.ld, a.real_vocab);
  Piece p;
  first_logits(p, b, part.c0 + wave * kPiece, lane);
  const RowRules o = row_rules(rules, r);
  const ExpFrom exp_of(a.lse[r]);
  const float coef = (gl - g) * exp_of.factor;
  for_spans(part, a.real_vocab, rules, o, b, p, counts, lane, wave,
            [&](int32_t cw, int32_t next, uint32_t* own) __attribute__((always_inline)) {
    const bool here = act && target >= cw && target < cw + kPiece;
    for_piece<true>(p, b, o, own, cw, next, a.real_vocab, lane,
                    [&](int, int32_t col, const float* y, const float* by, uint32_t bits,
                        bool some) __attribute__((always_inline)) {
      float d[8];
      exp_of.template operator()<8>(y, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] *= coef;
      if (here) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (col + e == target) d[e] += g;
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] *= by[e];
      if (some) {  // (not a product with 0: p of a barred row is NaN)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] = where_bit(bits, e, d[e], 0u);
      }
      if (col < spans.columns) put8<false>(out + col, d, spans.columns - col);
    });
  });
}

// Spans a block: with few blocks one each, else four, which share the row's rules and tokens
// (1024 rows x 151936, 128-token sequences: statistics 114 -> 95 us, gradient 136 -> 110; 4096
// rows of one sequence: 538 -> 432 and 639 -> 559; 512 rows processed with histories of up to
// 8192: 86 us with one, 92 with four, which leave part of the chip idle at the end).
constexpr int64_t kManyBlocks = 16384;

template <typename F>
hipError_t launch_spans(int32_t rows, int32_t columns, F&& launch) {
  const int32_t n = (columns - 1) / kSpan + 1;
  Spans s;
  s.columns = columns;
  s.per = (int64_t)rows * n < kManyBlocks ? 1 : 4;
  s.parts = (n + s.per - 1) / s.per;
  return in_launches((int64_t)rows * s.parts, kSpanThreads, [&](int64_t b, int64_t nb) {
    s.row = (int32_t)(b / s.parts);
    s.first = (uint32_t)(b % s.parts);
    launch(s, dim3((unsigned)nb), dim3(kSpanThreads));
  });
}

}  // namespace

hipError_t launch_process(const void* logits, int64_t ld, int32_t num_rows, int32_t real_vocab,
                          int32_t padded_vocab, const RuleArgs& rules, void* out, int64_t ld_out,
                          bool out_bf16, hipStream_t stream) {
  const uint16_t* x = static_cast<const uint16_t*>(logits);
  return launch_spans(num_rows, padded_vocab, [&](const Spans& s, dim3 grid, dim3 threads) {
    if (out_bf16)
      hipLaunchKernelGGL((process_rows<uint16_t>), grid, threads, 0, stream, x, ld,
                         real_vocab, s, rules, static_cast<uint16_t*>(out), ld_out);
    else
      hipLaunchKernelGGL((process_rows<float>), grid, threads, 0, stream, x, ld,
                         real_vocab, s, rules, static_cast<float*>(out), ld_out);
  });
}

hipError_t launch_processed_fwd(const ProcessedArgs& a, const RuleArgs& rules,
                                hipStream_t stream) {
  const hipError_t e = launch_spans(
      a.num_rows, a.real_vocab,
      [&](const Spans& s, dim3 grid, dim3 threads) {
        hipLaunchKernelGGL(processed_stats, grid, threads, 0, stream, a,
                           s, rules);
      });
  if (e != hipSuccess) return e;
  return in_launches(((int64_t)a.num_rows + kMergeRows - 1) / kMergeRows, 64 * kMergeRows,
                     [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL(processed_merge, dim3((unsigned)nb), dim3(64 * kMergeRows), 0, stream, a,
                       b);
  });
}

hipError_t launch_processed_bwd(const ProcessedArgs& a, const RuleArgs& rules, void* dlogits,
                                int64_t ld_d, bool out_bf16, hipStream_t stream) {
  return launch_spans(a.num_rows, a.padded_vocab, [&](const Spans& s, dim3 grid, dim3 threads) {
    if (out_bf16)
      hipLaunchKernelGGL((processed_grad<uint16_t>), grid, threads, 0, stream, a, s,
                         rules, static_cast<uint16_t*>(dlogits), ld_d);
    else
      hipLaunchKernelGGL((processed_grad<float>), grid, threads, 0, stream, a, s, rules,
                         static_cast<float*>(dlogits), ld_d);
  });
}

}  // namespace rlk
