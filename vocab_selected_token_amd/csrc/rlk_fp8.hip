// rlk_fp8.hip -- the LM-head in 8-bit floating point (OCP e4m3) for gfx950: the
// cast with one scale per block of 128, and the product of hidden states and
// weight in that form, as bf16 logits or as selected-token statistics without
// logits.
//
// A value is q * s: q in e4m3, s the fp32 scale of its block -- 1 x 128 for hidden
// states (a token, 128 columns of the hidden dimension), 128 x 128 for the weight.
// Both blocks are 128 wide along the dimension that the product sums over, so
//   z[t][v] = sum_b s_h[t][b] s_w[v / 128][b] sum_{k in block b} q_h[t][k] q_w[v][k]
// and four v_mfma_f32_16x16x32_bf16 per 16 x 16 outputs cover a block: its fp32
// result, times the two scales, is added to the fp32 accumulator in ascending b.
// The sums do not depend on the tile, so a token's outputs have the same bits
// whatever the batch, whichever of the two kernels computes them:
//   fp8_tile    256 vocabulary rows x 128 to 256 tokens a block, both operands through
//               LDS (the layout and loads of rlk_tile.h: a slab row is 128 bytes,
//               here 128 columns).
//   fp8_stream  for up to 64 tokens, where the weight's bytes bound the time
//               (rlk_stream.h).
// Precision: the values stay in 8 bits in memory, in LDS and on their way, and become
// bf16, which holds every e4m3 value, in the registers in front of the matrix cores.
// Their products are then exact and all sums fp32: z is 1.4e-7 from 64 bits (root mean
// square, logits of 1.3, hidden_dim 4096).  The 8-bit MFMA (v_mfma_f32_16x16x128_f8f6f4)
// would save the conversions and half of the matrix cores' time, but adds products in groups
// of 8 columns and cuts each towards zero 13 bits below the group's largest exponent: z
// was 1.9e-5 off with it, at any hidden_dim, which is 1e-5 and more of the logp of a token
// that the model is sure of.  4096 tokens x 4096 x 151936 took 2.3 ms that way and take
// 4.0 ms now; 1 token 127 us and 123.
//
// Operand layout of a block: lane l supplies row/column l%16, and of the 128 bytes of
// its row the 16-byte chunks l/16 (the first 8 columns for step 0, the others for step 1)
// and l/16 + 4 (steps 2 and 3).  The matrix cores see the 128 columns in another order
// than they lie in, but in the same for both operands; the result's layout is that of the
// bf16 16 x 16 tiles (4 vocabulary rows of one token per lane).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rlk_internal.h"
#include "rlk_lmhead_segments.h"
#include "rlk_rows.h"
#include "rlk_stream.h"
#include "rlk_tile.h"

namespace rlk {
namespace {

typedef int32_t i32x2 __attribute__((ext_vector_type(2)));

constexpr float kE4m3Max = 448.0f;
constexpr float kSmallestScale = 0x1p-126f;  // the smallest normal number

static_assert(kRowBytes == kFp8Block, "a slab of the tile is one block of columns");

// ---------------------------------------------------------------------------
// The cast: s = max(largest magnitude / 448, 2^-126), q = e4m3(x / s), both
// quotients correctly rounded (many entries lie midway between two e4m3 values,
// so the last bit of the quotient decides them).  A block that holds NaN or
// infinity gets that as its scale, and its product is NaN.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float block_scale(uint32_t top_bits) {
  const float top = __uint_as_float(top_bits << 16);
  return maxnan(top / kE4m3Max, kSmallestScale);
}

// Largest magnitude of 8 bf16 values as bf16 bits: as integers, magnitudes order
// like the values, infinity above them and NaN above that.
__device__ __forceinline__ uint32_t top_bits(const u32x4& x) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max((x[i] >> 16) & 0x7fff, x[i] & 0x7fff));
  return m;
}

// x / s, correctly rounded.  With y = 1 / s correctly rounded, q = x y is off by
// an ulp or two, and one residual step (Markstein), q - (q s - x) y in two fmas,
// gives the rounded quotient: for every pair of a bf16 x and a scale taken from a
// bf16 maximum, which is a finite set of mantissas (all 128 x 128 were compared
// with exact fractions).  The residual's last bit is a number as long as s is
// well above the smallest one; tiny, infinite and NaN scales divide (a choice
// that holds for the whole block).  Against a division per element: 341 and 436 us
// for 151936 x 4096 in 1 x 128 blocks, 317 and 329 us in 128 x 128 blocks.
struct Quotient {
  float s, y;
  bool step;
  __device__ __forceinline__ explicit Quotient(float scale)
      : s(scale), y(1.0f / scale), step(scale >= 0x1p-60f && scale <= 0x1p+120f) {}
  __device__ __forceinline__ float operator()(float x) const {
    const float q = x * y;
    return fmaf(-fmaf(q, s, -x), y, q);  // (the signs as they are, -0 stays -0)
  }
};

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return __builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false),
                                         true);
}

__device__ __forceinline__ uint64_t cast8(const u32x4& x, const Quotient& q) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(x[i] << 16);
    v[2 * i + 1] = __uint_as_float(x[i] & 0xffff0000u);
  }
  if (q.step) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = q(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] / q.s;
  }
  return e4m3x4(v[0], v[1], v[2], v[3]) | (uint64_t)e4m3x4(v[4], v[5], v[6], v[7]) << 32;
}

// 1 x 128 blocks: 16 lanes of 8 columns each, kRowBlocks of them in turn, loaded
// together.  4096 x 4096 takes 12 us; the bytes bound it (5.4 TB/s at 16384 rows).
constexpr int kRowBlocks = 4;

__global__ __launch_bounds__(256) void quantize_rows(const u32x4* __restrict__ x, int64_t ld,
                                                     int64_t rows, int32_t col_blocks,
                                                     uint64_t* __restrict__ q,
                                                     float* __restrict__ scale, int64_t row_stride,
                                                     int64_t col_stride, int64_t blk_begin) {
  const int lane = threadIdx.x & 15;
  // the thread block's 16 groups take kRowBlocks x 16 consecutive blocks of the matrix
  const int64_t b0 = (blk_begin + blockIdx.x) * (16 * kRowBlocks) + (threadIdx.x >> 4);
  const int64_t n = rows * col_blocks;
  u32x4 v[kRowBlocks];
#pragma unroll
  for (int i = 0; i < kRowBlocks; ++i) {
    const int64_t b = min(b0 + 16 * i, n - 1), r = b / col_blocks;
    v[i] = x[r * ld + (b - r * col_blocks) * 16 + lane];
  }
#pragma unroll
  for (int i = 0; i < kRowBlocks; ++i) {
    const int64_t b = b0 + 16 * i;
    uint32_t m = top_bits(v[i]);
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    const float s = block_scale(m);
    if (b >= n) continue;
    q[b * 16 + lane] = cast8(v[i], Quotient(s));
    const int64_t r = b / col_blocks;
    if (lane == 0) scale[r * row_stride + (b - r * col_blocks) * col_stride] = s;
  }
}

// 128 x 128 blocks: one per thread block, 8 rows apart per thread, kept in
// registers between the maximum and the cast.  151936 x 4096 takes 317 us, 5.9 TB/s
// of the bytes it has to move (348 us without the nontemporal loads and stores:
// nothing here is read again soon).
__global__ __launch_bounds__(256) void quantize_blocks(
    const u32x4* __restrict__ x, int64_t ld, int64_t rows, int32_t col_blocks,
    uint64_t* __restrict__ q, float* __restrict__ scale, int64_t row_stride, int64_t col_stride,
    int64_t blk_begin) {
  __shared__ uint32_t part[4];
  const int64_t b = blk_begin + blockIdx.x;
  const int64_t rb = b / col_blocks;
  const int32_t c = (int32_t)(b - rb * col_blocks);
  const int64_t r0 = rb * kFp8Block + (threadIdx.x >> 4);
  const int lane = threadIdx.x & 15;
  u32x4 v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = u32x4{0, 0, 0, 0};
    if (r0 + i * 16 < rows) v[i] = __builtin_nontemporal_load(x + (r0 + i * 16) * ld + c * 16 + lane);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, top_bits(v[i]));
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, o));
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = m;
  __syncthreads();
  m = max(max(part[0], part[1]), max(part[2], part[3]));
  const float s = block_scale(m);
  const Quotient quot(s);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (r0 + i * 16 < rows)
      __builtin_nontemporal_store(cast8(v[i], quot),
                                  q + (r0 + i * 16) * (col_blocks * 16) + c * 16 + lane);
  if (threadIdx.x == 0) scale[rb * row_stride + c * col_stride] = s;
}

// ---------------------------------------------------------------------------
// The product.
// ---------------------------------------------------------------------------
// 8 e4m3 values as bf16, which holds each of them exactly (NaN stays NaN).
[[maybe_unused]] __device__ __forceinline__ bf16x8 widen(int32_t lo, int32_t hi) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass has no such builtins
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  union {
    bf16x2 pair[4];
    bf16x8 whole;
  } w;
  w.pair[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  w.pair[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  w.pair[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  w.pair[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return w.whole;
#else
  return bf16x8{};
#endif
}

[[maybe_unused]] __device__ __forceinline__ f32x4 mfma_step(const bf16x8& a, const bf16x8& b,
                                                            const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

[[maybe_unused]] __device__ __forceinline__ void add_scaled(f32x4& acc, const f32x4& z, float f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = fmaf(z[i], f, acc[i]);
}

// What both kernels read.
struct Fp8Operands {
  const char* __restrict__ hq;     // [num_tokens][hidden_dim]
  const float* __restrict__ hs;    // (token, block) at token * hs_row + block * hs_col
  const char* __restrict__ wq;     // [>= real_vocab][hidden_dim]
  const float* __restrict__ ws;    // (128-row block, block)
  int64_t hs_row, hs_col, ws_row, ws_col;
  int32_t hidden_dim;
};

// Where logits go (kLogits kernels).
struct LogitsOut {
  uint16_t* __restrict__ out;  // bf16 [num_tokens][ld]
  int64_t ld;
  int32_t num_tokens, real_vocab, padded_vocab;
};

// Work index -> (vocabulary block, token block): see lmhead_segments.
__device__ __forceinline__ void block_of(int64_t blk, int32_t n_vbs, int32_t n_tb, int32_t& vb,
                                         int32_t& tb) {
  constexpr int32_t kGroupV = 4;
  const int64_t strip = blk / ((int64_t)kGroupV * n_tb);
  const int32_t r_in = (int32_t)(blk - strip * kGroupV * n_tb);
  const int32_t strip_w = min(kGroupV, n_vbs - (int32_t)strip * kGroupV);
  vb = (int32_t)strip * kGroupV + r_in % strip_w;
  tb = r_in / strip_w;
}

// 4 logits of a token, columns from v on, as bf16; -inf from the real vocabulary's end.
__device__ __forceinline__ uint64_t logits_of(const LogitsOut& o, int32_t v, const f32x4& z) {
  union {
    uint16_t e[4];
    uint64_t x;
  } u;
#pragma unroll
  for (int i = 0; i < 4; ++i) u.e[i] = v + i < o.real_vocab ? bf16_bits(z[i]) : (uint16_t)0xff80;
  return u.x;
}

// Stores the kCount logits `x` of token t, columns from v on (a multiple of kCount),
// as far as the padded vocabulary goes.  kNt: past the caches (1024 tokens x 151936:
// 555 against 575 us, and no loss to a forward that reads the logits next; nothing
// gained where few tokens are streamed).
template <int kCount, bool kNt, typename T>
__device__ __forceinline__ void store_logits(const LogitsOut& o, int32_t t, int32_t v,
                                             const T& x) {
  static_assert(sizeof(T) == kCount * 2, "bf16");
  if (t >= o.num_tokens || v >= o.padded_vocab) return;
  uint16_t* out = o.out + (int64_t)t * o.ld + v;
  if (v + kCount <= o.padded_vocab) {
    if constexpr (kNt)
      __builtin_nontemporal_store(x, reinterpret_cast<T*>(out));
    else
      *reinterpret_cast<T*>(out) = x;
  } else {
    union {
      T whole;
      uint16_t e[kCount];
    } u;
    u.whole = x;
    for (int i = 0; i < kCount; ++i)
      if (v + i < o.padded_vocab) out[i] = u.e[i];
  }
}

// What a tile of 64 kTok tokens keeps in LDS, twice over: a slab of 256 weight rows,
// of its tokens, and the tokens' scales (64 floats a wave).
template <int kTok>
struct Fp8Tile {
  static constexpr int kTokens = 64 * kTok;
  static constexpr int kStage = kSlabBytes + kTokens * kRowBytes;
  static constexpr int kScaleBytes = kThreads * 4;
  static constexpr int kLds = 2 * (kStage + kScaleBytes);
};

// acc: z of the vocabulary rows [v0, +256) and tokens [t0, +64 kTok), in 2 x 4 waves
// of 128 x 16 kTok.  Some row and token of the tile exist.
// A wave takes a slab in eight 16-row tiles of A, a tile in four steps of 32 columns, a
// step in kTok MFMAs.  Beside these it widens the next step of A (4 conversions) and adds
// the previous tile's block sums, scaled, to the accumulators; B is widened once a slab, step
// by step as the last tile has done with it.
// What bounds it: 128 MFMAs a slab and wave (kTok = 4) take 2048 cycles of a SIMD, their issue
// with 192 conversions and 128 fmas 1792, with two waves on it: 4096 x 4096 x 151936 in 4.0
// ms, 1.27 PFLOP/s, where a library's bf16 product reaches 1.43.  Registers decide the
// shape: 128 accumulators, 64 of B and 16 sums leave no room to hold A's raw chunks a tile
// ahead (255 of 256 are in use, none spilled); addresses are one offset and immediates,
// scales come from LDS and the scalar cache, and the body has no branch, for the same reason.
template <int kTok>
__device__ __forceinline__ void fp8_product(char* smem, const Fp8Operands& p,
                                            const SegmentArgs& a, int32_t v0, int32_t t0,
                                            int wave, int lane, f32x4 (&acc)[kVS][kTok]) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass cannot instantiate the target's builtins
  typedef Fp8Tile<kTok> T;
  const int wv = wave >> 2, wt = wave & 3;
#pragma unroll
  for (int vs = 0; vs < kVS; ++vs)
#pragma unroll
    for (int ts = 0; ts < kTok; ++ts) acc[vs][ts] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t row_bytes = p.hidden_dim;
  const int32_t w_first = max(v0, a.row_lo);
  const TileOperand wo(p.wq + (int64_t)w_first * row_bytes, row_bytes,
                       min(v0 + kBA, a.row_hi) - w_first, v0 - w_first, wave, lane);
  const TileOperandOf<kTok> ho(p.hq + (int64_t)t0 * row_bytes, row_bytes,
                       min(t0 + T::kTokens, a.num_tokens) - t0, 0, wave, lane);
  const int nslab = p.hidden_dim / kFp8Block;
  // token scales: each wave loads those of its 16 kTok tokens, one per lane (and
  // some that it does not use)
  const int32_t last = min(t0 + T::kTokens, a.num_tokens) - t0 - 1;
  const __amdgpu_buffer_rsrc_t srs =
      buffer_of(p.hs + (int64_t)t0 * p.hs_row, (last * p.hs_row + (nslab - 1) * p.hs_col + 1) * 4);
  const uint32_t s_off = (uint32_t)(min(wt * (16 * kTok) + lane, last) * p.hs_row * 4);
  const uint32_t s_step = (uint32_t)p.hs_col * 4;
  // this wave's weight scale: its 128 rows are one block (rows past the real
  // vocabulary's last block are not used: clamped)
  const int32_t wb = min(v0 / kFp8Block + wv, (a.row_hi - 1) / kFp8Block);
  const float* __restrict__ wsp = p.ws + (int64_t)wb * p.ws_row;

  auto issue = [&](int slab, int stage) __attribute__((always_inline)) {
    char* base = smem + stage * T::kStage;
    wo.issue(base, wave, slab);
    ho.issue(base + kSlabBytes, wave, slab);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        srs, (lds_ptr)(smem + 2 * T::kStage + stage * T::kScaleBytes + wave * 256), 4, s_off,
        (uint32_t)slab * s_step, 0, 0);
  };
  // Fragment reads.  Rows 16 apart have the same swizzle, so a fragment is at a
  // fixed distance from the wave's first: the lane's offset of its two chunks
  // (the second's position differs in one bit) plus an immediate.
  const int fr = lane & 15, fc = lane >> 4;
  const int lo0 = swizzled(fr, fc) * 16, lo1 = lo0 ^ 64;
  // chunk `c` (columns for the steps 2c and 2c + 1) of A's 16-row tile `at`
  auto read_a = [&](const char* stage, int at, int c) __attribute__((always_inline)) {
    return *reinterpret_cast<const i32x4*>(stage + wv * 128 * kRowBytes + (c ? lo1 : lo0) +
                                           at * 16 * kRowBytes);
  };
  // step ks of B's tile `ts`
  auto read_b = [&](const char* stage, int ts, int ks) __attribute__((always_inline)) {
    return *reinterpret_cast<const i32x2*>(stage + kSlabBytes + wt * (16 * kTok) * kRowBytes +
                                           (ks < 2 ? lo0 : lo1) + ts * 16 * kRowBytes +
                                           (ks & 1) * 8);
  };
  auto scale_of = [&](int s, int ts) __attribute__((always_inline)) {
    const char* at = smem + 2 * T::kStage + (s & 1) * T::kScaleBytes;
    return reinterpret_cast<const float*>(at)[wave * 64 + ts * 16 + fr];
  };

  i32x4 ra[2];         // A's chunks as they are read, the next steps' still to be widened
  i32x2 rb[kTok];      // a step of B's
  bf16x8 fa, b[kTok][4];
  f32x4 z[kTok];       // the tile's block sums
  float f[kTok], g[kTok];
  issue(0, 0);
  if (nslab > 1) issue(1, 1);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  ra[0] = read_a(smem, 0, 0);
  ra[1] = read_a(smem, 0, 1);
  fa = widen(ra[0][0], ra[0][1]);
#pragma unroll
  for (int ts = 0; ts < kTok; ++ts) {
#pragma unroll
    for (int ks = 0; ks < 4; ++ks) {
      rb[ts] = read_b(smem, ts, ks);
      if (ks < 3) b[ts][ks] = widen(rb[ts][0], rb[ts][1]);
    }
    z[ts] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    f[ts] = 0.0f;
  }
  float sw = scalar_load(wsp);
  for (int s = 0; s < nslab; ++s) {
    const char* cur = smem + (s & 1) * T::kStage;
    const char* nxt = smem + ((s + 1) & 1) * T::kStage;
#pragma unroll
    for (int at = 0; at < kVS; ++at) {
      const char* from = at < kVS - 1 ? cur : nxt;  // A's next tile
      const int to = (at + 1) % kVS;
      if (at == kVS - 1) {
        // every wave has read slab s into registers, and slab s+1 has landed
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0);
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        // the last two steps reload the last slab and read fragments that nothing
        // uses: unconditional, and in bounds
        issue(min(s + 2, nslab - 1), s & 1);
      }
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        // the next step's fragment of A
        const bf16x8 an = ks == 0   ? widen(ra[0][2], ra[0][3])
                          : ks == 1 ? widen(ra[1][0], ra[1][1])
                          : ks == 2 ? widen(ra[1][2], ra[1][3])
                                    : widen(ra[0][0], ra[0][1]);
        if (ks == 1) ra[0] = read_a(from, to, 0);
        if (ks == 3) ra[1] = read_a(from, to, 1);
        // B's steps are replaced one by one once the last tile has them
        if (at == 0 && ks == 0)
#pragma unroll
          for (int ts = 0; ts < kTok; ++ts) {
            b[ts][3] = widen(rb[ts][0], rb[ts][1]);
            g[ts] = scale_of(s, ts);
          }
        if (at == kVS - 1) {
          if (ks > 0)
#pragma unroll
            for (int ts = 0; ts < kTok; ++ts) b[ts][ks - 1] = widen(rb[ts][0], rb[ts][1]);
#pragma unroll
          for (int ts = 0; ts < kTok; ++ts) rb[ts] = read_b(nxt, ts, ks);
        }
#pragma unroll
        for (int ts = 0; ts < kTok; ++ts) {
          if (ks == 0) add_scaled(acc[(at + kVS - 1) % kVS][ts], z[ts], f[ts]);
          z[ts] = mfma_step(fa, b[ts][ks], ks ? z[ts] : f32x4{0.0f, 0.0f, 0.0f, 0.0f});
        }
        fa = an;
        if (at == 0 && ks == 2) {
#pragma unroll
          for (int ts = 0; ts < kTok; ++ts) f[ts] = g[ts] * sw;
          sw = scalar_load(wsp + min(s + 1, nslab - 1) * p.ws_col);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
#pragma unroll
  for (int ts = 0; ts < kTok; ++ts) add_scaled(acc[kVS - 1][ts], z[ts], f[ts]);
  // the reloads of the last two steps land before the stages are used again
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
#endif
}

// A tile's fixed part -- first loads, exponentials or stores, drain -- takes 8 us
// (statistics) or 10 (logits) beside 3 us a slab.
template <bool kLogits, int kTok>
__global__ __launch_bounds__(kThreads) void fp8_tile(Fp8Operands p, SegmentArgs a, LogitsOut lo,
                                                     int32_t n_tb, int32_t vb_begin,
                                                     int32_t n_vbs, int64_t blk_begin) {
  typedef Fp8Tile<kTok> T;
  __shared__ __attribute__((aligned(16))) char smem[T::kLds];
  static_assert(T::kLds >= T::kTokens * 4 * (int)sizeof(float), "epilogue exchange fits");
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wv = wave >> 2, wt = wave & 3;
  int32_t vb, tb;
  block_of(blk_begin + xcd_local_block(blockIdx.x, gridDim.x), n_vbs, n_tb, vb, tb);
  vb += vb_begin;
  const int32_t v0 = vb * kBA, t0 = tb * T::kTokens;
  f32x4 acc[kVS][kTok] = {};
  // else a block of padding: only logits has them, and stores no sum
  if (!kLogits || v0 < a.row_hi) fp8_product<kTok>(smem, p, a, v0, t0, wave, lane, acc);
  if constexpr (kLogits) {
    static_assert(T::kLds >= kWaves * 4096 * kTok, "the rows fit");
    store_rows<kTok>(
        smem, wave, lane,
        [&](int vs, int ts) __attribute__((always_inline)) {
          return logits_of(lo, v0 + wv * 128 + vs * 16 + 4 * (lane >> 4), acc[vs][ts]);
        },
        [&](int r, int c, const u32x4& x) __attribute__((always_inline)) {
          store_logits<8, true>(lo, t0 + wt * (16 * kTok) + r, v0 + wv * 128 + c * 8, x);
        });
  } else {
    write_segments<kTok>(a, acc, reinterpret_cast<float*>(smem), vb, t0, wv, wt, lane);
  }
}

// The stream kernel's fp32 z, kept between it and segments_of_z.
struct ZOut {
  float* __restrict__ z;  // [num_tokens][ld]
  int64_t ld;
  int32_t num_tokens;
};

__device__ __forceinline__ void store_z(const ZOut& o, int32_t t, int32_t v, const f32x4& z) {
  if (t < o.num_tokens) *reinterpret_cast<f32x4*>(o.z + (int64_t)t * o.ld + v) = z;
}

// What the 8-bit head adds to stream_product: the tokens' scales, staged like the
// hidden states (one per thread at most), and the weight's.
template <int kTok>
struct Fp8Stream {
  static constexpr int kTokens = 16 * kTok;
  static_assert(kBuf * kTokens <= kStreamThreads, "a scale per thread at most");

  float (*lds)[kBuf * kTokens];
  const float* __restrict__ hs;
  const float* __restrict__ ws;  // the block's: its 64 rows lie in one of 128
  int64_t hs_row, hs_col, ws_col;
  int32_t num_tokens, nslab;
  float scale, sw;

  __device__ __forceinline__ void load_stage(int s) {
    const int tid = threadIdx.x, r = tid % kTokens, i = min(tid / kTokens, kBuf - 1);
    scale = hs[min(r, num_tokens - 1) * hs_row + min(s + i, nslab - 1) * hs_col];
  }
  __device__ __forceinline__ void store_stage(int at) {
    if (threadIdx.x < kBuf * kTokens) lds[at][threadIdx.x] = scale;
  }
  __device__ __forceinline__ void begin(int slab) { sw = scalar_load(ws + slab * ws_col); }
  __device__ __forceinline__ void multiply(f32x4& acc, const i32x4& a0, const i32x4& a1,
                                           const i32x4& b0, const i32x4& b1, int at,
                                           int place) const {
    f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
    z = mfma_step(widen(a0[0], a0[1]), widen(b0[0], b0[1]), z);
    z = mfma_step(widen(a0[2], a0[3]), widen(b0[2], b0[3]), z);
    z = mfma_step(widen(a1[0], a1[1]), widen(b1[0], b1[1]), z);
    z = mfma_step(widen(a1[2], a1[3]), widen(b1[2], b1[3]), z);
    add_scaled(acc, z, lds[at][place] * sw);
  }
};

// Few tokens (16 kTok at most).  No block waits for another: the statistics, whose
// order spans 128 rows, are taken from z by segments_of_z.  The weight's bytes bound it:
// 1 token x 4096 x 151936 in 111-115 us, 5.4-5.6 TB/s; reading alone, row pieces in this
// order, reaches 6.1.  From 32 tokens on every wave's conversions of the hidden states weigh
// as well (64 tokens: 172 us).
template <bool kLogits, int kTok>
__global__ __launch_bounds__(kStreamThreads) void fp8_stream(Fp8Operands p, SegmentArgs a,
                                                             LogitsOut lo, ZOut zo,
                                                             int32_t v_begin, int64_t blk_begin) {
  __shared__ StreamLds<kTok> lds;
  __shared__ float scales[2][kBuf * 16 * kTok];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int32_t v0 = v_begin + (int32_t)(blk_begin + blockIdx.x) * kStreamRows;
  const int32_t vw = v0 + wave * 16;
  f32x4 acc[1][kTok] = {};  // outside the rows: zeros, which segments_of_z passes over
  if (v0 < a.row_hi && v0 + kStreamRows > a.row_lo) {
    Fp8Stream<kTok> math;
    math.lds = scales;
    math.hs = p.hs;
    math.ws = p.ws + (int64_t)(max(v0, a.row_lo) / kFp8Block) * p.ws_row;
    math.hs_row = p.hs_row;
    math.hs_col = p.hs_col;
    math.ws_col = p.ws_col;
    math.num_tokens = a.num_tokens;
    math.nslab = p.hidden_dim / kFp8Block;
    stream_product(lds, p.wq, p.hq, (uint32_t)p.hidden_dim, a.row_lo, a.row_hi, a.num_tokens, v0,
                   math, acc);
  }
  if (!kLogits && vw >= a.row_hi) return;  // z ends with the vocabulary's last 256 columns
#pragma unroll
  for (int ts = 0; ts < kTok; ++ts) {
    const int32_t t = ts * 16 + (lane & 15), v = vw + 4 * (lane >> 4);
    if constexpr (kLogits)
      store_logits<4, false>(lo, t, v, logits_of(lo, v, acc[0][ts]));
    else
      store_z(zo, t, v, acc[0][ts]);
  }
}

// The segments of a 256-column block from z, in the tile kernel's layout and so
// with its bits: two waves of 128 vocabulary rows x 16 tokens.  A launch's latency: 6 us
// for 1 token x 151936 columns.
__global__ __launch_bounds__(128) void segments_of_z(ZOut zo, SegmentArgs a, int32_t vb_begin,
                                                     int32_t n_tg, int64_t blk_begin) {
  __shared__ float xch[16 * 4];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t blk = blk_begin + blockIdx.x;
  const int32_t vb = vb_begin + (int32_t)(blk / n_tg);
  const int32_t t0 = (int32_t)(blk % n_tg) * 16;
  const int32_t t = min(t0 + (lane & 15), a.num_tokens - 1);
  const float* __restrict__ z =
      zo.z + (int64_t)t * zo.ld + vb * kBA + wv * 128 + 4 * (lane >> 4);
  f32x4 acc[kVS][1];
#pragma unroll
  for (int vs = 0; vs < kVS; ++vs) acc[vs][0] = *reinterpret_cast<const f32x4*>(z + vs * 16);
  write_segments<1>(a, acc, xch, vb, t0, wv, 0, lane);
}

template <bool kLogits, int kTok>
hipError_t launch_stream(const Fp8Operands& p, const SegmentArgs& sa, const LogitsOut& lo,
                         const ZOut& zo, int32_t v_begin, int32_t columns, hipStream_t stream) {
  return in_launches(columns / kStreamRows, kStreamThreads, [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL((fp8_stream<kLogits, kTok>), dim3((unsigned)nb), dim3(kStreamThreads), 0,
                       stream, p, sa, lo, zo, v_begin, b);
  });
}

template <bool kLogits, int kTok>
hipError_t launch_tile(const Fp8Operands& p, const SegmentArgs& sa, const LogitsOut& lo,
                       int32_t vb_begin, int32_t n_vbs, hipStream_t stream) {
  const int32_t n_tb = (sa.num_tokens + 64 * kTok - 1) / (64 * kTok);
  return in_launches((int64_t)n_vbs * n_tb, kThreads, [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL((fp8_tile<kLogits, kTok>), dim3((unsigned)nb), dim3(kThreads), 0, stream,
                       p, sa, lo, n_tb, vb_begin, n_vbs, b);
  });
}

// Time of a round of tiles of 128, 192 and 256 tokens, see tile_tokens: 68, 87 and 107 us
// at hidden_dim 4096, 37, 47 and 58 at 2048, 23, 29 and 35 at 1024, 15, 19 and 23 at 512 (logits
// of 65536 columns): near the same ratios throughout.  333 tokens x 2176 x 50021 take 118 us
// in tiles of 256, 97 in tiles of 192 and 111 in tiles of 128; 65 tokens x 4096 x 151936 317, 260
// and 211; 4096 tokens 4.02, 4.38 and 4.77 ms.
constexpr double kTileUnits[] = {2.55, 3.2, 4.0};

// The product over the columns [256 vb_begin, +256 n_vbs).  Up to 64 tokens the
// weight's bytes bound the time and the stream kernel's registers hold all
// tokens (64 tokens x 151936 columns at hidden_dim 4096: 187 us against 211 us for a
// tile); above, the tile shares each weight slab among its tokens.
template <bool kLogits>
hipError_t launch_product(const Fp8Operands& p, const SegmentArgs& sa, const LogitsOut& lo,
                          const ZOut& zo, int32_t vb_begin, int32_t n_vbs, hipStream_t stream) {
  const int32_t n = sa.num_tokens;
  if (n > kFp8FewTokens) {
    switch (tile_tokens(n, n_vbs, kTileUnits)) {
      case 2: return launch_tile<kLogits, 2>(p, sa, lo, vb_begin, n_vbs, stream);
      case 3: return launch_tile<kLogits, 3>(p, sa, lo, vb_begin, n_vbs, stream);
      default: return launch_tile<kLogits, 4>(p, sa, lo, vb_begin, n_vbs, stream);
    }
  }
  const int32_t v = vb_begin * kBA, columns = n_vbs * kBA;
  hipError_t e;
  if (n <= 16)
    e = launch_stream<kLogits, 1>(p, sa, lo, zo, v, columns, stream);
  else if (n <= 32)
    e = launch_stream<kLogits, 2>(p, sa, lo, zo, v, columns, stream);
  else
    e = launch_stream<kLogits, 4>(p, sa, lo, zo, v, columns, stream);
  if (e != hipSuccess || kLogits) return e;
  const int32_t n_tg = (n + 15) / 16;
  return in_launches((int64_t)n_vbs * n_tg, 128, [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL(segments_of_z, dim3((unsigned)nb), dim3(128), 0, stream, zo, sa, vb_begin,
                       n_tg, b);
  });
}

Fp8Operands operands(const LmheadFp8Args& a) {
  return {static_cast<const char*>(a.hidden_q), a.hidden_scale,
          static_cast<const char*>(a.weight_q), a.weight_scale,
          a.hidden_row_stride, a.hidden_col_stride, a.weight_row_stride, a.weight_col_stride,
          a.hidden_dim};
}

}  // namespace

hipError_t launch_fp8_quantize(const Fp8QuantizeArgs& a, hipStream_t stream) {
  const int32_t col_blocks = (int32_t)(a.cols / kFp8Block);
  const bool wide = a.block_rows > 1;
  const int64_t items = wide ? (a.rows + kFp8Block - 1) / kFp8Block * col_blocks
                             : (a.rows * col_blocks + 16 * kRowBlocks - 1) / (16 * kRowBlocks);
  const u32x4* x = reinterpret_cast<const u32x4*>(a.x);
  uint64_t* q = reinterpret_cast<uint64_t*>(a.q);
  return in_launches(items, 256, [&](int64_t b, int64_t nb) {
    if (wide)
      hipLaunchKernelGGL(quantize_blocks, dim3((unsigned)nb), dim3(256), 0, stream, x, a.ld / 8,
                         a.rows, col_blocks, q, a.scale, a.scale_row_stride, a.scale_col_stride, b);
    else
      hipLaunchKernelGGL(quantize_rows, dim3((unsigned)nb), dim3(256), 0, stream, x, a.ld / 8,
                         a.rows, col_blocks, q, a.scale, a.scale_row_stride, a.scale_col_stride, b);
  });
}

hipError_t launch_segments_fp8(const LmheadFp8Args& f, const SegmentArgs& sa, int32_t vb_begin,
                               int32_t n_vbs, hipStream_t stream) {
  const ZOut zo{f.z, (int64_t)sa.n_vb * kBA, sa.num_tokens};
  return launch_product<false>(operands(f), sa, LogitsOut{}, zo, vb_begin, n_vbs, stream);
}

hipError_t launch_logits_fp8(const LmheadFp8Args& f, int32_t num_tokens, int32_t real_vocab,
                             int32_t padded_vocab, void* logits, int64_t ld,
                             hipStream_t stream) {
  SegmentArgs sa{};
  sa.num_tokens = num_tokens;
  sa.row_hi = real_vocab;
  const LogitsOut lo{reinterpret_cast<uint16_t*>(logits), ld, num_tokens, real_vocab,
                     padded_vocab};
  return launch_product<true>(operands(f), sa, lo, ZOut{}, 0, (padded_vocab + kBA - 1) / kBA,
                              stream);
}

}  // namespace rlk
