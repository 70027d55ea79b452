// rlk_linear.hip -- dense products with bias, activation and residual in the epilogue, and
// their gradients, for gfx950:
//   z = x . W^T + b,   y = residual + act(z)
//   dz = dy act'(z),   dx = dz . W,   dW = dz^T . x,   db = sum over tokens of dz
// (the residual's gradient is dy).  y is rounded to bf16 once; z, the activation and the
// residual's sum are fp32.
//
// The tile product of rlk_tile.h does the work: W's rows as operand A and x's as B give
// C[out][token], so that a lane holds 4 consecutive outputs of one token.  Up to 64 tokens
// linear_few streams the weight instead.
//
// What the backward pass needs of z (z / cap for the soft cap) is kept in fp16, for its 11 bits,
// clamped to +-65504, where every activation here has reached its last slope.  The rounding, 2^-11
// relative, moves act'(z) by at most 2^-12 (the soft cap's by 2^-11.6): less than rounding dz to
// bf16, 2^-8 of it, wherever |act'(z)| > 0.05.  Where the slope all but vanishes it is more: GELU's
// moves by 0.7% of itself at z = -4 and 1.2% at -5 (by tanh 0.9 and 1.6), SiLU's by 0.4% at -10,
// the soft cap's by 0.4% at |z / cap| = 4 and 0.8% at 8.  A bias in fp32 has a gradient in fp32,
// which that rounding would show in (1e-4 relative): z is kept in fp32 then, and by the C call
// wherever it is asked to.
//
// dz is rounded to bf16 for its two products, whose matrix instructions take operands of 16 bits
// (those of fp32 operands have a small part of their rate); with the results' own rounding dx and
// dW are off by 0.0023 of their size, where products of an fp32 dz would be off by 0.0017.
//
// Sums are fp32 in a fixed order: repeated calls give the same bits.  No atomics.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rlk_internal.h"
#include "rlk_rows.h"
#include "rlk_stream.h"
#include "rlk_tile.h"

namespace rlk {
namespace {

static_assert(kBK == kLmheadSlabK, "slab width shared with the boundary");

// 16 bytes at any element's address
typedef uint32_t u32x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint16_t u16x4u __attribute__((ext_vector_type(4), aligned(2)));
typedef float f32x4u __attribute__((ext_vector_type(4), aligned(4)));

__device__ __forceinline__ float bf16_float(uint16_t b) {
  return __uint_as_float((uint32_t)b << 16);
}
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

// ---------------------------------------------------------------------------
// The activations.  exp2 and the reciprocal are the hardware's (1 step of fp32), which
// rounding to bf16 hides.
// ---------------------------------------------------------------------------
constexpr float kGeluC = 0.7978845608028654f;       // sqrt(2 / pi)
constexpr float kGeluA = 0.044715f;
constexpr float kInvSqrt2Pi = 0.3989422804014327f;

__device__ __forceinline__ float sigmoid(float z) {
  return rcp_hw(1.0f + exp2_hw(-z * kLog2e));
}
// exp(-z^2 / 2).
__device__ __forceinline__ float bell(float z) { return exp2_hw(z * z * (-0.5f * kLog2e)); }
// The normal distribution's Phi(z), bell = exp(-z^2 / 2): Phi(-a) = bell P(t), t = 1 / (1 + 0.3 a),
// with P fitted to erfcx(a / sqrt 2) / 2 over 0 <= a <= 14 for the least relative error
// (1.7e-7; behind, bell is 0).  Half the instructions of the library's erfcf, whose share of 1024
// tokens x 2048 x 151936 was a fifth (GELU 819 us, SiLU 648).
__device__ __forceinline__ float normal_cdf(float z, float bell) {
  const float t = rcp_hw(fmaf(0.3f, fabsf(z), 1.0f));
  float p = 0.035674773156642914f;
  p = fmaf(p, t, -0.1572030782699585f);
  p = fmaf(p, t, 0.20635350048542023f);
  p = fmaf(p, t, -0.05368363857269287f);
  p = fmaf(p, t, 0.12856163084506989f);
  p = fmaf(p, t, 0.09991349279880524f);
  p = fmaf(p, t, 0.12075395882129669f);
  p = fmaf(p, t, 0.11962930113077164f);
  const float q = p * t * bell;
  return z < 0.0f ? q : 1.0f - q;
}
// cap tanh(u), u = z / cap: cap - 2 cap / (1 + exp(2u)); below 2^-4, where that would cancel, the
// series z (1 - u^2 / 3 + 2 u^4 / 15), whose next term is 2^-28 of it.
__device__ __forceinline__ float soft_cap(float z, float cap, float inv_cap) {
  const float u = z * inv_cap, q = u * u;
  const float far = fmaf(-2.0f * cap, rcp_hw(1.0f + exp2_hw(u * (2.0f * kLog2e))), cap);
  const float near = z * fmaf(fmaf(q, 2.0f / 15.0f, -1.0f / 3.0f), q, 1.0f);
  return fabsf(u) < 0.0625f ? near : far;
}

template <int kAct>
__device__ __forceinline__ float act_of(float z, float cap, float inv_cap) {
  if constexpr (kAct == kActRelu) return z < 0.0f ? 0.0f : z;  // (NaN stays)
  if constexpr (kAct == kActSilu) return z * sigmoid(z);
  if constexpr (kAct == kActGelu) return z * normal_cdf(z, bell(z));
  if constexpr (kAct == kActGeluTanh)  // (1 + tanh(u)) / 2 = sigmoid(2u)
    return z * sigmoid(2.0f * kGeluC * (z + kGeluA * z * z * z));
  if constexpr (kAct == kActSoftcap) return soft_cap(z, cap, inv_cap);
  return z;
}

// act'(z) from what was kept: z, or z / cap.
template <int kAct>
__device__ __forceinline__ float slope_of(float z) {
  if constexpr (kAct == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
  if constexpr (kAct == kActSilu) {
    const float s = sigmoid(z);
    return s * (1.0f + z * (1.0f - s));
  }
  if constexpr (kAct == kActGelu) {
    const float b = bell(z);
    return normal_cdf(z, b) + z * kInvSqrt2Pi * b;
  }
  if constexpr (kAct == kActGeluTanh) {
    const float s = sigmoid(2.0f * kGeluC * (z + kGeluA * z * z * z));
    return s + z * s * (1.0f - s) * 2.0f * kGeluC * (1.0f + 3.0f * kGeluA * z * z);
  }
  if constexpr (kAct == kActSoftcap) {  // 1 - tanh^2, without the difference
    const float e = exp2_hw(fabsf(z) * (-2.0f * kLog2e)), r = rcp_hw(1.0f + e);
    return 4.0f * e * r * r;
  }
  return 1.0f;
}

// use(slope): the slope of the call's activation, one for all of its outputs.
template <typename Use>
__device__ __forceinline__ void with_slope(int activation, Use&& use) {
  switch (activation) {
    case kActRelu: return use(slope_of<kActRelu>);
    case kActGelu: return use(slope_of<kActGelu>);
    case kActGeluTanh: return use(slope_of<kActGeluTanh>);
    case kActSilu: return use(slope_of<kActSilu>);
    case kActSoftcap: return use(slope_of<kActSoftcap>);
  }
  use(slope_of<kActNone>);
}

// What is kept of z, before its rounding (NaN stays).
__device__ __forceinline__ float clamped(float z) {
  return z > 65504.0f ? 65504.0f : z < -65504.0f ? -65504.0f : z;
}
// In fp16 a positive z keeps at least `least`: under ReLU the smallest positive value, since its
// slope is z's sign, which rounding to 0 would take from z up to 2^-25.
__device__ __forceinline__ float least_kept(const LinearArgs& a) {
  return a.activation == kActRelu ? 0x1p-24f : 0.0f;
}
__device__ __forceinline__ uint16_t fp16_bits(float z, float least) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass cannot instantiate the target's builtins
  const float kept = z > 0.0f ? __builtin_amdgcn_fmed3f(z, least, 65504.0f) : clamped(z);
  return __builtin_bit_cast(uint16_t, (_Float16)kept);
#else
  return 0;
#endif
}
__device__ __forceinline__ f32x4 clamped(const f32x4& z) {
  return f32x4{clamped(z[0]), clamped(z[1]), clamped(z[2]), clamped(z[3])};
}

// finish(act): the call's activation, one for all of its outputs.
template <typename Finish>
__device__ __forceinline__ void with_activation(const LinearArgs& a, Finish&& finish) {
  const float cap = a.cap, inv_cap = 1.0f / a.cap;
  switch (a.activation) {
    case kActRelu: return finish([](float z) { return act_of<kActRelu>(z, 0.0f, 0.0f); });
    case kActGelu: return finish([](float z) { return act_of<kActGelu>(z, 0.0f, 0.0f); });
    case kActGeluTanh: return finish([](float z) { return act_of<kActGeluTanh>(z, 0.0f, 0.0f); });
    case kActSilu: return finish([](float z) { return act_of<kActSilu>(z, 0.0f, 0.0f); });
    case kActSoftcap:
      return finish([=](float z) { return act_of<kActSoftcap>(z, cap, inv_cap); });
  }
  finish([](float z) { return z; });
}

__device__ __forceinline__ f32x4 floats_of(const u16x4u& b) {
  return f32x4{bf16_float(b[0]), bf16_float(b[1]), bf16_float(b[2]), bf16_float(b[3])};
}
// 4 consecutive elements from n on (0 from `end` on).
__device__ __forceinline__ f32x4 four_of(const uint16_t* from, int32_t n, int32_t end) {
  if (n + 4 <= end) return floats_of(*reinterpret_cast<const u16x4u*>(from + n));
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < end) x[e] = bf16_float(from[n + e]);
  return x;
}
__device__ __forceinline__ f32x4 four_of(const float* from, int32_t n, int32_t end) {
  if (n + 4 <= end) return *reinterpret_cast<const f32x4u*>(from + n);
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < end) x[e] = from[n + e];
  return x;
}
// The bias of 4 consecutive outputs.
__device__ __forceinline__ f32x4 bias_of(const LinearArgs& a, int32_t n) {
  if (!a.bias) return f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  return a.bias_bf16 ? four_of(static_cast<const uint16_t*>(a.bias), n, a.out_dim)
                     : four_of(static_cast<const float*>(a.bias), n, a.out_dim);
}

constexpr uint16_t kNegInfBf16 = 0xFF80;

// 8 outputs of a token from output n on: those behind out_dim are -inf up to padded_out.
__device__ __forceinline__ void put_out(const LinearArgs& a, int32_t m, int32_t n,
                                        const u32x4& x) {
  if (m >= a.tokens || n >= a.padded_out) return;
  uint16_t* out = static_cast<uint16_t*>(a.out) + m * a.ld_out + n;
  union {
    u32x4 x;
    uint16_t e[8];
  } o;
  o.x = x;
  if (n + 8 > a.out_dim) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (n + e >= a.out_dim) o.e[e] = kNegInfBf16;
  }
  if (n + 8 <= a.padded_out) {
    *reinterpret_cast<u32x4*>(out) = o.x;
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (n + e < a.padded_out) out[e] = o.e[e];
}

// ---------------------------------------------------------------------------
// linear_tiles: 32 kVSn outputs x 16 kTok kWB tokens a block, by the tile product; then bias,
// activation, residual and z's copy on a lane's 4 outputs, and whole rows out through LDS.
// Bound by what stands beside the matrix cores, which are busy 41-44% of the time in the large
// cases (8% at 777 x 1088 x 2501): a slab of the 256 x 256 tile takes 1.45 us, which is 1.48
// PFLOP/s, and a tile 12-20 us more for its first loads, its epilogue and its stores, which
// nothing hides at one block a CU; small tiles wait for their slabs.  In a row of calls 1024 x
// 2048 x 151936 takes 606-625 us without an activation (1.02-1.05 PFLOP/s) and 651-661 with the soft cap, 4096 x
// 4096 x 4096 109-111 us (1.24-1.26) and 117-123 with a bias, a residual, SiLU and z kept; single
// calls under a trace 679-717 with the soft cap and 133-140 with everything.
// ---------------------------------------------------------------------------
template <int kVSn, int kTok, int kWB>
struct Shape {
  static constexpr int kA = 32 * kVSn, kB = 16 * kTok * kWB;
  static constexpr int kWavesN = 2 * kWB, kThr = 64 * kWavesN;
  static constexpr int kLds = 2 * (kA + kB) * kRowBytes;
  static constexpr int kOwn = 512 * kVSn * kTok;  // bytes of a wave's rows
  static constexpr bool kSplits = kB == 256;      // see launch_tiles
  static_assert(kLds >= kWavesN * kOwn, "the rows fit");
  typedef TileOperandOf<kA / (kWavesN * kRowsPerLoad)> OperandA;
  typedef TileOperandOf<kB / (kWavesN * kRowsPerLoad)> OperandB;
  typedef TileOperandTOf<kA, kWavesN> OperandAT;
  typedef TileOperandTOf<kB, kWavesN> OperandBT;
};

template <int kVSn, int kTok, int kWB>
__device__ __forceinline__ void linear_tile(const LinearArgs& a, char* smem, int32_t n0,
                                            int32_t m0) {
  typedef Shape<kVSn, kTok, kWB> S;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t row_bytes = (int64_t)a.in_dim * 2;
  f32x4 acc[kVSn][kTok] = {};
  if (n0 < a.out_dim) {  // (else a tile of padding)
    const typename S::OperandA wo(static_cast<const char*>(a.weight) + n0 * row_bytes, row_bytes,
                                  min(S::kA, a.out_dim - n0), 0, wave, lane);
    const typename S::OperandB xo(static_cast<const char*>(a.x) + m0 * row_bytes, row_bytes,
                                  min(S::kB, a.tokens - m0), 0, wave, lane);
    tile_product<kWB>(smem, wo, xo, 0, a.in_dim / kBK, wave, lane, acc);
  }
  const int32_t nw = n0 + wave / kWB * (16 * kVSn), mw = m0 + wave % kWB * (16 * kTok);
  char* own = smem + wave * S::kOwn;
  const bool inside = nw + 16 * kVSn <= a.out_dim;  // (all of the wave's outputs)
  auto add_bias = [&](auto&& at) __attribute__((always_inline)) {
    constexpr int kBatch = kVSn < 4 ? kVSn : 4;
#pragma unroll
    for (int vs = 0; vs < kVSn; vs += kBatch) {
      f32x4 b[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) b[i] = at(nw + (vs + i) * 16 + 4 * (lane >> 4));
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int ts = 0; ts < kTok; ++ts) acc[vs + i][ts] += b[i];
    }
  };
  if (a.bias) {
    if (!inside)
      add_bias([&](int32_t n) { return bias_of(a, n); });
    else if (a.bias_bf16)
      add_bias([&](int32_t n) {
        return floats_of(
            *reinterpret_cast<const u16x4u*>(static_cast<const uint16_t*>(a.bias) + n));
      });
    else
      add_bias([&](int32_t n) {
        return (f32x4)*reinterpret_cast<const f32x4u*>(static_cast<const float*>(a.bias) + n);
      });
  }
  // The residual comes in by whole rows, all on their way before z's copy goes out (tokens from
  // the last on again: they are not written).  A wave at the outputs' end takes them later.
  const uint16_t* res = static_cast<const uint16_t*>(a.residual);
  const bool ahead = res && inside;
  u32x4 held[kVSn * kTok / 2];
  if (ahead) {
    int j = 0;
    whole_rows<kTok, kVSn>(own, lane, [&](int r, int c, u32x4*) __attribute__((always_inline)) {
      held[j++] = *reinterpret_cast<const u32x4u*>(res + min(mw + r, a.tokens - 1) *
                                                   a.ld_residual + nw + c * 8);
    });
  }
  const float by = a.activation == kActSoftcap ? 1.0f / a.cap : 1.0f;
  if (a.saved && a.saved_f32) {
#pragma unroll
    for (int ts = 0; ts < kTok; ++ts) {
      const int32_t m = mw + ts * 16 + (lane & 15);
      if (m >= a.tokens) continue;
      float* to = static_cast<float*>(a.saved) + m * a.ld_saved;
#pragma unroll
      for (int vs = 0; vs < kVSn; ++vs) {
        const int32_t n = nw + vs * 16 + 4 * (lane >> 4);
        if (n < a.ld_saved) *reinterpret_cast<f32x4*>(to + n) = clamped(acc[vs][ts] * by);
      }
    }
  } else if (a.saved) {
    const float least = least_kept(a);
    store_rows<kTok, kVSn>(
        smem, wave, lane,
        [&](int vs, int ts) __attribute__((always_inline)) {
          union {
            uint16_t e[4];
            uint64_t x;
          } o;
#pragma unroll
          for (int e = 0; e < 4; ++e) o.e[e] = fp16_bits(acc[vs][ts][e] * by, least);
          return o.x;
        },
        [&](int r, int c, const u32x4& x) __attribute__((always_inline)) {
          const int32_t m = mw + r, n = nw + c * 8;
          if (m < a.tokens && n < a.ld_saved)
            *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(a.saved) + m * a.ld_saved + n) = x;
        });
  }
  if (ahead) {
    int j = 0;
    whole_rows<kTok, kVSn>(own, lane, [&](int, int, u32x4* at) __attribute__((always_inline)) {
      *at = held[j++];
    });
  } else if (res) {
    whole_rows<kTok, kVSn>(own, lane, [&](int r, int c, u32x4* at)
                                          __attribute__((always_inline)) {
      const int32_t m = mw + r, n = nw + c * 8;
      union {
        u32x4 x;
        uint16_t e[8];
      } o;
      o.x = u32x4{0, 0, 0, 0};
      if (m < a.tokens) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < a.out_dim) o.e[e] = res[m * a.ld_residual + n + e];
      }
      *at = o.x;
    });
  }
  const bool add = res != nullptr;
  with_activation(a, [&](auto&& act) __attribute__((always_inline)) {
    store_rows<kTok, kVSn>(
        smem, wave, lane,
        [&](int vs, int ts) __attribute__((always_inline)) {
          union {
            uint16_t e[4];
            uint64_t x;
          } o, r;
          float y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) y[e] = act(acc[vs][ts][e]);
          if (add) {
            r.x = *reinterpret_cast<const uint64_t*>(row_slot<kVSn>(own, lane, vs, ts));
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] += bf16_float(r.e[e]);
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) o.e[e] = bf16_bits(y[e]);
          return o.x;
        },
        [&](int r, int c, const u32x4& x) __attribute__((always_inline)) {
          put_out(a, mw + r, nw + c * 8, x);
        });
  });
}

// Blocks [0, n_whole) take a tile each, the others half a tile's tokens.
template <int kVSn, int kTok, int kWB>
__global__ __launch_bounds__((Shape<kVSn, kTok, kWB>::kThr), 2) void linear_tiles(
    LinearArgs a, int32_t n_a, int32_t n_b, int64_t n_whole, int64_t blk_begin) {
  typedef Shape<kVSn, kTok, kWB> S;
  __shared__ __attribute__((aligned(16))) char smem[S::kLds];
  // (the halves are the last to be dispatched)
  const uint32_t whole =
      (uint32_t)max((int64_t)0, min(n_whole - blk_begin, (int64_t)gridDim.x));
  int32_t ta, tb;
  if (blockIdx.x < whole) {
    tile_of(blk_begin + xcd_local_block(blockIdx.x, whole), n_a, n_b, ta, tb);
    linear_tile<kVSn, kTok, kWB>(a, smem, ta * S::kA, tb * S::kB);
  } else if constexpr (S::kSplits) {
    const int64_t at = blk_begin + whole - n_whole +
                       xcd_local_block(blockIdx.x - whole, gridDim.x - whole);
    tile_of(n_whole + at / 2, n_a, n_b, ta, tb);
    const int32_t m0 = tb * S::kB + (int32_t)(at % 2) * (S::kB / 2);
    if (m0 < a.tokens) linear_tile<kVSn, kTok / 2, kWB>(a, smem, ta * S::kA, m0);
  }
}

// What the epilogue adds to 4 outputs of token m from output n (a multiple of 4) on.
struct Added {
  f32x4 bias, residual;
};
__device__ __forceinline__ Added added_to(const LinearArgs& a, int32_t m, int32_t n) {
  Added o;
  o.bias = bias_of(a, n);
  o.residual = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (a.residual)
    o.residual = four_of(static_cast<const uint16_t*>(a.residual) + m * a.ld_residual, n,
                         a.out_dim);
  return o;
}

// Those outputs: the rest of the epilogue.
__device__ __forceinline__ void finish4(const LinearArgs& a, int32_t m, int32_t n, f32x4 z,
                                        const Added& add) {
  uint16_t* out = static_cast<uint16_t*>(a.out) + m * a.ld_out + n;
  union {
    uint16_t e[4];
    uint64_t x;
  } o;
  o.x = 0xFF80FF80FF80FF80ull;
  if (n < a.out_dim) {
    if (a.bias) z += add.bias;
    if (a.saved) {
      const float by = a.activation == kActSoftcap ? 1.0f / a.cap : 1.0f;
      if (a.saved_f32) {
        *reinterpret_cast<f32x4*>(static_cast<float*>(a.saved) + m * a.ld_saved + n) =
            clamped(z * by);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) o.e[e] = fp16_bits(z[e] * by, least_kept(a));
        *reinterpret_cast<uint64_t*>(static_cast<uint16_t*>(a.saved) + m * a.ld_saved + n) = o.x;
      }
    }
    with_activation(a, [&](auto&& act) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) z[e] = act(z[e]);
    });
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (a.residual) z[e] += add.residual[e];
      o.e[e] = n + e < a.out_dim ? bf16_bits(z[e]) : kNegInfBf16;
    }
  }
  if (n + 4 <= a.padded_out) {
    *reinterpret_cast<uint64_t*>(out) = o.x;
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < a.padded_out) out[e] = o.e[e];
}

// ---------------------------------------------------------------------------
// linear_few: up to 64 tokens (16 kTok), whose time the weight's bytes bound.  A block takes
// 16 outputs; its four waves take every fourth slab of 64 of the sum each, operands
// straight from memory to registers, kDepth slabs ahead, and meet only at the end, where the
// four sums are added in order.  What the epilogue adds is fetched first.  One token x 4096 x
// 4096 with bias and residual: 8.0-8.2 us (4.1 TB/s, of which the launch's start and end take a
// third; fetched last, 8.8).
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 4;
constexpr int kDepth = 4;

template <int kTok>
__global__ __launch_bounds__(64 * kFewWaves) void linear_few(LinearArgs a, int64_t blk_begin) {
  constexpr int kTokens = 16 * kTok;
  __shared__ f32x4 part[kFewWaves][kTokens][4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int32_t n0 = (int32_t)(blk_begin + blockIdx.x) * 16;
  const int fr = lane & 15, fc = lane >> 4;
  // 4 outputs of a token in the end: what is added to them is on its way first
  const int m = threadIdx.x / 4, at = threadIdx.x % 4;
  static_assert(kTokens * 4 <= 64 * kFewWaves, "a thread takes 4 outputs of a token");
  const bool mine = m < min(kTokens, a.tokens) && n0 + at * 4 < a.padded_out;
  Added add = {};
  if (mine) add = added_to(a, m, n0 + at * 4);
  if (n0 < a.out_dim) {
    const uint16_t *w, *x[kTok];
    w = static_cast<const uint16_t*>(a.weight) +
        (int64_t)min(n0 + fr, a.out_dim - 1) * a.in_dim + fc * 8;
#pragma unroll
    for (int ts = 0; ts < kTok; ++ts)
      x[ts] = static_cast<const uint16_t*>(a.x) +
              (int64_t)min(ts * 16 + fr, a.tokens - 1) * a.in_dim + fc * 8;
    f32x4 acc[kTok] = {};
    bf16x8 wf[kDepth][2], xf[kDepth][kTok][2];
    const int nslab = a.in_dim / kBK;
    const int turn = (int)((blk_begin + blockIdx.x) % nslab);
    auto load = [&](int s, int at) __attribute__((always_inline)) {
      // past the end the last slab is loaded again, unused
      const int t = min(s, nslab - 1) + turn;
      const int64_t k = (int64_t)(t < nslab ? t : t - nslab) * kBK;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        wf[at][h] = *reinterpret_cast<const bf16x8*>(w + k + h * 32);
#pragma unroll
        for (int ts = 0; ts < kTok; ++ts)
          xf[at][ts][h] = *reinterpret_cast<const bf16x8*>(x[ts] + k + h * 32);
      }
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d) load(wave + d * kFewWaves, d);
    for (int s = wave; s < nslab; s += kDepth * kFewWaves) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        if (s + d * kFewWaves < nslab) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int ts = 0; ts < kTok; ++ts)
              acc[ts] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wf[d][h], xf[d][ts][h], acc[ts],
                                                                0, 0, 0);
        }
        load(s + (d + kDepth) * kFewWaves, d);
      }
    }
#pragma unroll
    for (int ts = 0; ts < kTok; ++ts) part[wave][ts * 16 + fr][fc] = acc[ts];
  }
  __syncthreads();
  if (!mine) return;
  f32x4 z = {0.0f, 0.0f, 0.0f, 0.0f};
  if (n0 < a.out_dim) {
    z = part[0][m][at];
#pragma unroll
    for (int i = 1; i < kFewWaves; ++i) z += part[i][m][at];
  }
  finish4(a, m, n0 + at * 4, z, add);
}

// ---------------------------------------------------------------------------
// linear_stream: up to 64 tokens and a weight of many rows: the stream product, 64 kRT outputs a
// block, the whole sum.  Each block begins its sum at another slab and goes around: the weight's
// rows are a power of two apart, and blocks in step would all ask the same few memory
// channels (16 tokens x 4096 x 151936: 255 us in step, 218 so, 5.7 TB/s; 64 tokens 283 and 248).
// ---------------------------------------------------------------------------
template <int kTok, int kRT>
__global__ __launch_bounds__(kStreamThreads) void linear_stream(LinearArgs a, int64_t blk_begin) {
  __shared__ StreamLds<kTok> lds;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int64_t blk = blk_begin + blockIdx.x;
  const int32_t n0 = (int32_t)blk * (kStreamRows * kRT);
  f32x4 acc[kRT][kTok] = {};
  Bf16Stream math;
  if (n0 < a.out_dim)
    stream_product<kRT, kStreamThreads, true>(
        lds, static_cast<const char*>(a.weight), static_cast<const char*>(a.x),
        (uint32_t)a.in_dim * 2, 0, a.out_dim, a.tokens, n0, math, acc,
        (int)(blk % (a.in_dim / kBK)));
#pragma unroll
  for (int rt = 0; rt < kRT; ++rt)
#pragma unroll
    for (int ts = 0; ts < kTok; ++ts) {
      const int32_t m = ts * 16 + (lane & 15), n = n0 + (wave * kRT + rt) * 16 + 4 * (lane >> 4);
      if (m < a.tokens && n < a.padded_out) finish4(a, m, n, acc[rt][ts], added_to(a, m, n));
    }
}

// ---------------------------------------------------------------------------
// linear_dz: dz = dy act'(z) in bf16, its rows and columns filled up with zeros to multiples
// of 64, and what 64 tokens add to db.  A block takes 64 tokens x 128 outputs, a thread 4 tokens
// x 8 outputs, whose loads go out together.  The blocks behind copy x's and W's last rows, those
// behind the last whole 64, followed by zeros: the slabs of dW's and dx's sums that they do not
// fill.  Bound by its bytes: 4096 x 4096 23-24 us (4.2-4.4 TB/s); 777 x 2501 with z in fp32 11 us,
// of which the smallest launch's 5.4 are one half and 3 would do for the bytes (rows that are
// not 16-byte aligned are read by whole vectors at their elements' addresses).
// ---------------------------------------------------------------------------
constexpr int kDzRows = 64, kDzCols = 128;

struct TailArgs {
  const u32x4* x;  // the first of the last rows
  const u32x4* w;
  int32_t x_rows, w_rows;  // how many (0: no such slab)
  int32_t ldc;             // 16-byte chunks per row
  int32_t blocks;          // that copy each of them
};

__global__ __launch_bounds__(256) void linear_dz(LinearBwdArgs a, TailArgs t, int64_t n_dz,
                                                 int64_t blk_begin) {
  __shared__ float sums[16][kDzCols + 4];
  const LinearBwdLayout& l = a.layout;
  int64_t blk = blk_begin + blockIdx.x;
  if (blk >= n_dz) {
    blk -= n_dz;
    const bool of_w = t.x_rows == 0 || blk >= t.blocks;
    const int64_t i = (blk % t.blocks) * 256 + threadIdx.x;
    u32x4* to = reinterpret_cast<u32x4*>(a.workspace + (of_w ? l.w_tail : l.x_tail));
    if (i < (int64_t)kBK * t.ldc)
      to[i] = i < (int64_t)(of_w ? t.w_rows : t.x_rows) * t.ldc ? (of_w ? t.w : t.x)[i]
                                                               : u32x4{0, 0, 0, 0};
    return;
  }
  const int group = threadIdx.x >> 4, at = (threadIdx.x & 15) * 8;
  const int32_t n_cols = (l.cols + kDzCols - 1) / kDzCols;
  const int32_t rb = (int32_t)(blk / n_cols), c0 = (int32_t)(blk % n_cols) * kDzCols;
  const int32_t n = c0 + at;
  const LinearArgs& f = a.f;
  const uint16_t* dy = static_cast<const uint16_t*>(a.dy);
  union Eight {
    u32x4 x;
    uint16_t e[8];
    _Float16 h[8];
  };
  float sum[8] = {};
  if (n < l.cols) {
    Eight g[4], h[4];
    f32x4 z[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t m = rb * kDzRows + i * 16 + group;
      g[i].x = h[i].x = u32x4{0, 0, 0, 0};
      z[i][0] = z[i][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (m >= f.tokens || n >= f.out_dim) continue;
      const uint16_t* from = dy + m * a.ld_dy + n;
      if (n + 8 <= f.out_dim) {
        g[i].x = *reinterpret_cast<const u32x4u*>(from);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < f.out_dim) g[i].e[e] = from[e];
      }
      if (!f.saved) continue;
      if (f.saved_f32) {
        const f32x4* kept = reinterpret_cast<const f32x4*>(static_cast<const float*>(f.saved) +
                                                           m * f.ld_saved + n);
        z[i][0] = kept[0];
        z[i][1] = kept[1];
      } else {
        h[i].x = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(f.saved) +
                                                 m * f.ld_saved + n);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t m = rb * kDzRows + i * 16 + group;
      with_slope(f.activation, [&](auto&& slope) __attribute__((always_inline)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float kept = f.saved_f32 ? z[i][e / 4][e % 4] : (float)h[i].h[e];
          // (columns behind out_dim hold anything in z)
          const float d = n + e < f.out_dim ? bf16_float(g[i].e[e]) * slope(kept) : 0.0f;
          sum[e] += d;
          g[i].e[e] = bf16_bits(d);
        }
      });
      *reinterpret_cast<u32x4*>(a.workspace + l.dz + ((int64_t)m * l.cols + n) * 2) = g[i].x;
    }
  }
  if (!a.dbias) return;
#pragma unroll
  for (int e = 0; e < 8; ++e) sums[group][at + e] = sum[e];
  __syncthreads();
  if (threadIdx.x >= kDzCols || c0 + (int32_t)threadIdx.x >= l.cols) return;
  float all = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) all += sums[i][threadIdx.x];
  reinterpret_cast<float*>(a.workspace + l.bias_part)[(int64_t)rb * l.cols + c0 + threadIdx.x] =
      all;
}

// ---------------------------------------------------------------------------
// linear_grads: dx, dW and db in one launch, so that the last blocks of one fill the chip
// beside the next (4096 x 4096 x 4096: 205-215 us in a row of calls, 1.28-1.34 PFLOP/s, and 219-226
// in single ones; the library's two products 247).  Blocks [0, n_dx) are dx's (A = W by its rows,
// the sum's index; B = dz: C[in][token]), the next n_dw dW's (A = x and B = dz by their rows:
// C[in][out]), the rest db's.
// ---------------------------------------------------------------------------
template <int kVSn, int kTok, int kWB>
__global__ __launch_bounds__((Shape<kVSn, kTok, kWB>::kThr), 2) void linear_grads(
    LinearBwdArgs a, int64_t n_dx, int64_t n_dw, int64_t blk_begin) {
  typedef Shape<kVSn, kTok, kWB> S;
  __shared__ __attribute__((aligned(16))) char smem[S::kLds];
  const LinearBwdLayout& l = a.layout;
  const LinearArgs& f = a.f;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  int64_t blk = blk_begin + blockIdx.x;
  if (blk >= n_dx + n_dw) {
    const int64_t n = (blk - n_dx - n_dw) * S::kThr + threadIdx.x;
    if (n >= f.out_dim) return;
    const float* part = reinterpret_cast<const float*>(a.workspace + l.bias_part) + n;
    float sum = 0.0f;
#pragma unroll 8
    for (int32_t i = 0; i < l.row_blocks; ++i) sum += part[(int64_t)i * l.cols];
    if (f.bias_bf16)
      static_cast<uint16_t*>(a.dbias)[n] = bf16_bits(sum);
    else
      static_cast<float*>(a.dbias)[n] = sum;
    return;
  }
  const bool is_dx = blk < n_dx;
  const int32_t n_k = (f.in_dim + S::kA - 1) / S::kA;
  int32_t ta, tb;
  if (is_dx)
    tile_of(xcd_local_block(blk, n_dx), n_k, (f.tokens + S::kB - 1) / S::kB, ta, tb);
  else
    tile_of(xcd_local_block(blk - n_dx, n_dw), n_k, (f.out_dim + S::kB - 1) / S::kB, ta, tb);
  const int32_t k0 = ta * S::kA, b0 = tb * S::kB;
  const int64_t k_bytes = (int64_t)f.in_dim * 2, dz_bytes = (int64_t)l.cols * 2;
  const char* dz = a.workspace + l.dz;
  const int32_t rows = is_dx ? f.out_dim : f.tokens;  // of the operand by its rows
  const typename S::OperandAT ao(
      static_cast<const char*>(is_dx ? f.weight : f.x) + k0 * 2, k_bytes,
      min(S::kA, f.in_dim - k0), a.workspace + (is_dx ? l.w_tail : l.x_tail) + k0 * 2,
      rows % kBK ? rows / kBK : -1, wave, lane);
  f32x4 acc[kVSn][kTok];
  if (is_dx) {
    const typename S::OperandB bo(dz + b0 * dz_bytes, dz_bytes, min(S::kB, l.rows - b0), 0, wave,
                                  lane);
    tile_product<kWB>(smem, ao, bo, 0, l.cols / kBK, wave, lane, acc);
  } else {
    const typename S::OperandBT bo(dz + b0 * 2, dz_bytes, min(S::kB, l.cols - b0), nullptr, -1,
                                   wave, lane);
    tile_product<kWB>(smem, ao, bo, 0, l.rows / kBK, wave, lane, acc);
  }
  const int32_t kw = k0 + wave / kWB * (16 * kVSn), bw = b0 + wave % kWB * (16 * kTok);
  const int32_t last = is_dx ? f.tokens : f.out_dim;
  uint16_t* out = static_cast<uint16_t*>(is_dx ? a.dx : a.dweight);
  store_rows<kTok, kVSn>(
      smem, wave, lane,
      [&](int vs, int ts) __attribute__((always_inline)) {
        union {
          uint16_t e[4];
          uint64_t x;
        } o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.e[e] = bf16_bits(acc[vs][ts][e]);
        return o.x;
      },
      [&](int r, int c, const u32x4& x) __attribute__((always_inline)) {
        const int32_t row = bw + r, k = kw + c * 8;
        if (row < last && k < f.in_dim)
          *reinterpret_cast<u32x4*>(out + (int64_t)row * f.in_dim + k) = x;
      });
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

int64_t tiles_of(int64_t a, int64_t b, int64_t edge_a, int64_t edge_b) {
  return ((a + edge_a - 1) / edge_a) * ((b + edge_b - 1) / edge_b);
}

// The tiles, and what a slab of the sum takes (us, 4096 in) with 1, 2, ... of them on each of the
// chip's 256 CUs, up to as many as fit: many small tiles fill the chip where few large ones would
// not, and multiply more slowly where there is work for both.
struct TileCost {
  int a, b, fit;
  double time[5];
};
constexpr TileCost kTileCosts[] = {{256, 256, 1, {1.45}},
                                   {128, 128, 2, {0.65, 1.0}},
                                   {128, 64, 3, {0.55, 0.65, 0.81}},
                                   {64, 64, 5, {0.46, 0.50, 0.60, 0.75, 0.95}}};

// Which of them: blocks(edge of A, edge of B) tiles in all.  Of the four, 4096 x 4096 x 4096
// take 124, 136, 160 and 200 us, 1024 x 4096 x 4096 94, 46, 42 and 48, 512 x 4096 x 4096 93, 43,
// 38 and 32, 777 x 1088 x 2501 35, 16, 12.2 and 12.0, 333 x 2048 x 50021 110, 86, 100 and 115.
template <typename Blocks>
int best_tile(Blocks&& blocks) {
  int best = 0;
  double least = 0.0;
  for (int i = 0; i < 4; ++i) {
    const TileCost& c = kTileCosts[i];
    const int64_t n = blocks(c.a, c.b), full = n / (256 * c.fit), rest = n % (256 * c.fit);
    const double cost = (double)full * c.time[c.fit - 1] + (rest ? c.time[(rest - 1) / 256] : 0.0);
    if (i == 0 || cost < least) {
      least = cost;
      best = i;
    }
  }
  return best;
}

// Of the largest tiles one fits a CU.  What they leave for a last round, if it is at most half
// of one, goes in halves of a tile, to twice as many CUs (1024 x 2048 x 151936, 9.3 rounds:
// 617 -> 606 us; 1024 x 2048 x 33280, 2.03: 159 -> 140; 1024 x 1024 x 21504, 1.3: 60.5 -> 50.8).
template <int kVSn, int kTok, int kWB>
hipError_t launch_tiles(const LinearArgs& a, hipStream_t stream) {
  typedef Shape<kVSn, kTok, kWB> S;
  const int32_t n_a = (a.padded_out + S::kA - 1) / S::kA, n_b = (a.tokens + S::kB - 1) / S::kB;
  const int64_t n = (int64_t)n_a * n_b, rest = n % 256;
  const int64_t halves = S::kSplits && n > 256 && rest <= 128 ? rest : 0;
  return in_launches(n + halves, S::kThr, [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL((linear_tiles<kVSn, kTok, kWB>), dim3((unsigned)nb), dim3(S::kThr), 0,
                       stream, a, n_a, n_b, n - halves, b);
  });
}

// Up to 64 tokens.  A weight of few rows needs every block's waves on one sum; one of many is
// read fastest by blocks of 128 rows, where that leaves enough of them.  Of linear_few, blocks of
// 64 and of 128 rows, 16 tokens x 4096 x 8192 outputs take 19.6, 20.0 and 35.5 us, x 16384 37.6,
// 25.6 and 37.0, x 24576 55, 43.5 and 38.9; 64 tokens x 4096 x 4096 23.6, 26.6 and 43, x 8192
// 44.6, 28.0 and 44.
template <int kTok>
hipError_t launch_few(const LinearArgs& a, hipStream_t stream) {
  const int64_t n = a.padded_out;
  auto stream_blocks = [&](auto kernel, int rows) {
    return in_launches((n + rows - 1) / rows, kStreamThreads, [&](int64_t b, int64_t nb) {
      hipLaunchKernelGGL(kernel, dim3((unsigned)nb), dim3(kStreamThreads), 0, stream, a, b);
    });
  };
  if (n > 16384) return stream_blocks(linear_stream<kTok, 2>, 2 * kStreamRows);
  if (n > (kTok == 1 ? 8192 : 4096)) return stream_blocks(linear_stream<kTok, 1>, kStreamRows);
  return in_launches((n + 15) / 16, 64 * kFewWaves, [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL(linear_few<kTok>, dim3((unsigned)nb), dim3(64 * kFewWaves), 0, stream, a,
                       b);
  });
}

template <int kVSn, int kTok, int kWB>
hipError_t launch_grads(const LinearBwdArgs& a, hipStream_t stream) {
  typedef Shape<kVSn, kTok, kWB> S;
  const LinearArgs& f = a.f;
  const int64_t n_dx = a.dx ? tiles_of(f.in_dim, f.tokens, S::kA, S::kB) : 0;
  const int64_t n_dw = a.dweight ? tiles_of(f.in_dim, f.out_dim, S::kA, S::kB) : 0;
  const int64_t n_db = a.dbias ? ((int64_t)f.out_dim + S::kThr - 1) / S::kThr : 0;
  return in_launches(n_dx + n_dw + n_db, S::kThr, [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL((linear_grads<kVSn, kTok, kWB>), dim3((unsigned)nb), dim3(S::kThr), 0,
                       stream, a, n_dx, n_dw, b);
  });
}

}  // namespace

constexpr int32_t kLinearFewTokens = 64;

hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t stream) {
  if (a.tokens <= kLinearFewTokens) {
    if (a.tokens <= 16) return launch_few<1>(a, stream);
    if (a.tokens <= 32) return launch_few<2>(a, stream);
    return launch_few<4>(a, stream);
  }
  switch (best_tile([&](int ea, int eb) { return tiles_of(a.padded_out, a.tokens, ea, eb); })) {
    case 0: return launch_tiles<8, 4, 4>(a, stream);
    case 1: return launch_tiles<4, 4, 2>(a, stream);
    case 2: return launch_tiles<4, 2, 2>(a, stream);
    default: return launch_tiles<2, 2, 2>(a, stream);
  }
}

LinearBwdLayout linear_bwd_layout(int64_t tokens, int64_t in_dim, int64_t out_dim) {
  LinearBwdLayout l{};
  const int64_t rows = (tokens + kBK - 1) / kBK * kBK, cols = (out_dim + kBK - 1) / kBK * kBK;
  l.rows = (int32_t)rows;
  l.cols = (int32_t)cols;
  l.row_blocks = (int32_t)(rows / kDzRows);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  l.dz = take((size_t)rows * cols * 2);
  l.x_tail = take((size_t)kBK * in_dim * 2);
  l.w_tail = take((size_t)kBK * in_dim * 2);
  l.bias_part = take((size_t)l.row_blocks * cols * 4);
  l.total = at;
  return l;
}

hipError_t launch_linear_bwd(const LinearBwdArgs& a, hipStream_t stream) {
  const LinearArgs& f = a.f;
  const LinearBwdLayout& l = a.layout;
  if (f.tokens == 0) {  // no token: no gradient, and db's sums have no term
    if (a.dweight) {
      const hipError_t e =
          launch_fill_zero(a.dweight, (int64_t)f.out_dim * f.in_dim * 2, stream);
      if (e != hipSuccess) return e;
    }
    LinearBwdArgs of_db = a;
    of_db.dweight = nullptr;
    return launch_grads<4, 4, 2>(of_db, stream);
  }
  TailArgs t;
  t.ldc = f.in_dim / 8;
  t.x_rows = a.dweight ? f.tokens % kBK : 0;
  t.w_rows = a.dx ? f.out_dim % kBK : 0;
  t.x = static_cast<const u32x4*>(f.x) + (int64_t)(f.tokens / kBK * kBK) * t.ldc;
  t.w = static_cast<const u32x4*>(f.weight) + (int64_t)(f.out_dim / kBK * kBK) * t.ldc;
  t.blocks = (int32_t)(((int64_t)kBK * t.ldc + 255) / 256);
  const int64_t n_dz = (int64_t)l.row_blocks * ((l.cols + kDzCols - 1) / kDzCols);
  const int64_t tails = (t.x_rows ? t.blocks : 0) + (t.w_rows ? t.blocks : 0);
  hipError_t e = in_launches(n_dz + tails, 256, [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL(linear_dz, dim3((unsigned)nb), dim3(256), 0, stream, a, t, n_dz, b);
  });
  if (e != hipSuccess) return e;
  switch (best_tile([&](int ea, int eb) {
    return (a.dx ? tiles_of(f.in_dim, f.tokens, ea, eb) : 0) +
           (a.dweight ? tiles_of(f.in_dim, f.out_dim, ea, eb) : 0);
  })) {
    case 0: return launch_grads<8, 4, 4>(a, stream);
    case 1: return launch_grads<4, 4, 2>(a, stream);
    case 2: return launch_grads<4, 2, 2>(a, stream);
    default: return launch_grads<2, 2, 2>(a, stream);
  }
}

}  // namespace rlk
