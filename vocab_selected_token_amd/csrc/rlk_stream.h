// rlk_stream.h -- few tokens times a weight that is streamed from memory, shared by
// the LM-head kernels: the weight's bytes bound the time.
//
// A block is four waves of 16 vocabulary rows x all tokens (16 kTok at most), or, where
// its results belong together, eight of 32.  The
// weight is read once, from memory into registers, kBuf - 1 slabs (of 128 bytes a
// row) ahead of the one that is multiplied; the hidden states come through LDS,
// kBuf slabs at a time, loaded while the previous ones are multiplied (read by every
// wave from memory they cost as much as the weight: the loads of 16 rows x 64 bytes,
// not the bytes, bound a CU's rate; with the smaller blocks 1 token x 4096 x 151936 in
// 8 bits went from 171 to 125 us for the whole call).  The blocks are small -- 64 rows, thousands of
// them -- so that every CU ends at about the same time.  Lane l supplies row l%16 at
// the 16-byte chunks l/16 and l/16 + 4 of a slab, of the weight as operand A and of
// the hidden states as B; accumulator i of lane l is C[4*(l/16) + i][l%16].
#pragma once

#include "rlk_tile.h"

namespace rlk {
namespace {

constexpr int kStreamRows = 64;     // vocabulary rows per block
constexpr int kStreamThreads = 256;
constexpr int kBuf = 4;  // slabs of the weight in registers; slabs per LDS stage

typedef int32_t i32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, kBufferWord3);
}

// Read through the scalar cache (a uniform address; written before the launch).
__device__ __forceinline__ float scalar_load(const float* p) {
  return *(const __attribute__((address_space(4))) float*)(uintptr_t)p;
}

template <int kTok>
struct StreamLds {
  static constexpr int kTokens = 16 * kTok;
  static constexpr int kBytes = kTokens * kRowBytes;  // a slab's hidden states
  __attribute__((aligned(16))) char hidden[2][kBuf * kBytes];
};

// acc: C of this wave's 16 kRT rows of the block's [v0, +kThr / 4 kRT) and the tokens.
// w: the weight's rows [row_lo, row_hi) (some of them in the block; others are not read:
// the row is clamped), row_bytes each, a multiple of 128; h: num_tokens rows.  `math`
// multiplies a slab and may stage data of its own beside the hidden states.
// Every wave of the block calls it; on return all have done with `lds`.
template <int kRT = 1, int kThr = kStreamThreads, int kTok, typename Math>
__device__ __forceinline__ void stream_product(StreamLds<kTok>& lds, const char* w, const char* h,
                                               uint32_t row_bytes, int32_t row_lo, int32_t row_hi,
                                               int32_t num_tokens, int32_t v0, Math& math,
                                               f32x4 (&acc)[kRT][kTok]) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass cannot instantiate the target's builtins
  typedef StreamLds<kTok> T;
  constexpr int kCopies = kBuf * T::kBytes / 16 / kThr;  // per thread and stage
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int nslab = (int)(row_bytes / kRowBytes);
#pragma unroll
  for (int rt = 0; rt < kRT; ++rt)
#pragma unroll
    for (int ts = 0; ts < kTok; ++ts) acc[rt][ts] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // a wave outside the rows reads one of them all the same, unused
  const int32_t w_first = max(v0, row_lo);
  const int32_t w_rows = min(v0 + kThr / 4 * kRT, row_hi) - w_first;
  const __amdgpu_buffer_rsrc_t wrs =
      buffer_of(w + (int64_t)w_first * row_bytes, (int64_t)w_rows * row_bytes);
  const __amdgpu_buffer_rsrc_t hrs = buffer_of(h, (int64_t)num_tokens * row_bytes);
  const int fr = lane & 15, fc = lane >> 4;
  uint32_t woff[kRT];
#pragma unroll
  for (int rt = 0; rt < kRT; ++rt)
    woff[rt] = (uint32_t)min(max(v0 + (wave * kRT + rt) * 16 + fr - w_first, 0), w_rows - 1) *
                   row_bytes +
               fc * 16;

  u32x4 copy[kCopies];
  auto load_stage = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const int e = j * kThr + tid, c = e & 7, r = (e >> 3) % T::kTokens,
                i = (e >> 3) / T::kTokens;
      copy[j] = __builtin_bit_cast(
          u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                     hrs,
                     (uint32_t)min(r, num_tokens - 1) * row_bytes +
                         (uint32_t)min(s + i, nslab - 1) * kRowBytes + c * 16,
                     0, 0));
    }
    math.load_stage(s);
  };
  auto store_stage = [&](int at) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kCopies; ++j) {
      const int e = j * kThr + tid, c = e & 7, r = (e >> 3) % T::kTokens,
                i = (e >> 3) / T::kTokens;
      *reinterpret_cast<u32x4*>(lds.hidden[at] + i * T::kBytes + swizzled(r, c) * 16) = copy[j];
    }
    math.store_stage(at);
  };
  // LDS is written and read through this barrier; loads in flight stay there
  auto barrier = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
  };

  i32x4 a[kBuf][kRT][2];
  auto load = [&](int slab, int at) __attribute__((always_inline)) {
    const uint32_t off = (uint32_t)slab * kRowBytes;
#pragma unroll
    for (int rt = 0; rt < kRT; ++rt)
#pragma unroll
      for (int c = 0; c < 2; ++c)
        a[at][rt][c] = __builtin_bit_cast(
            i32x4, __builtin_amdgcn_raw_buffer_load_b128(wrs, woff[rt] + c * 64, off, 0));
  };
  load_stage(0);
  // past the end the last slab is loaded again, unused
#pragma unroll
  for (int i = 0; i < kBuf - 1; ++i) load(min(i, nslab - 1), i);
  store_stage(0);
  barrier();
  for (int s = 0, at = 0; s < nslab; s += kBuf, at ^= 1) {
    load_stage(min(s + kBuf, nslab - 1));
#pragma unroll
    for (int i = 0; i < kBuf; ++i) {
      load(min(s + i + kBuf - 1, nslab - 1), (i + kBuf - 1) % kBuf);
      __builtin_amdgcn_sched_barrier(0);
      if (s + i < nslab) {
        const char* hs = lds.hidden[at] + i * T::kBytes;
        math.begin(s + i);
#pragma unroll
        for (int ts = 0; ts < kTok; ++ts) {
          const i32x4 b0 = *reinterpret_cast<const i32x4*>(hs + swizzled(ts * 16 + fr, fc) * 16);
          const i32x4 b1 =
              *reinterpret_cast<const i32x4*>(hs + swizzled(ts * 16 + fr, 4 + fc) * 16);
#pragma unroll
          for (int rt = 0; rt < kRT; ++rt)
            math.multiply(acc[rt][ts], a[i][rt][0], a[i][rt][1], b0, b1, at,
                          i * T::kTokens + ts * 16 + fr);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    store_stage(at ^ 1);
    barrier();
  }
#endif
}

// bf16: two k-steps of 32 a slab, in the order of the tile product.
struct Bf16Stream {
  __device__ __forceinline__ void load_stage(int) {}
  __device__ __forceinline__ void store_stage(int) {}
  __device__ __forceinline__ void begin(int) {}
  __device__ __forceinline__ void multiply(f32x4& acc, const i32x4& a0, const i32x4& a1,
                                           const i32x4& b0, const i32x4& b1, int, int) const {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a0),
                                                  __builtin_bit_cast(bf16x8, b0), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a1),
                                                  __builtin_bit_cast(bf16x8, b1), acc, 0, 0, 0);
  }
};

}  // namespace
}  // namespace rlk
