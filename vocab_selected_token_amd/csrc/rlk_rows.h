// rlk_rows.h -- a tile of accumulators out to memory in whole rows, shared by the
// LM-head kernels that write their products.
#pragma once

#include "rlk_tile.h"

namespace rlk {
namespace {

__device__ __forceinline__ uint16_t bf16_bits(float x) {
  const __bf16 b = (__bf16)x;  // to nearest even
  return __builtin_bit_cast(uint16_t, b);
}

// Where 4 columns (of A, 4 * (lane / 16) on in its 16-row tile vs) of a wave's row
// ts * 16 + lane % 16 (of B) lie in LDS, 2 bytes each: rows of 32 kVSn bytes, chunk c of row
// r at c ^ (r % (2 kVSn)), so that 16 rows spread over all banks.
template <int kVSn>
__device__ __forceinline__ char* row_slot(char* own, int lane, int vs, int ts) {
  const int r = ts * 16 + (lane & 15), c = vs * 2 + (lane >> 5);
  return own + r * (32 * kVSn) + (c ^ (r & (2 * kVSn - 1))) * 16 + ((lane >> 4) & 1) * 8;
}

// A wave's 16 kTok rows in 16-byte pieces of whole rows: visit(row, chunk, its place in LDS).
template <int kTok, int kVSn, typename Visit>
__device__ __forceinline__ void whole_rows(char* own, int lane, Visit&& visit) {
  constexpr int kChunks = 2 * kVSn, kRowsAt = 64 / kChunks;
#pragma unroll
  for (int j = 0; j < 16 * kTok / kRowsAt; ++j) {
    const int r = j * kRowsAt + lane / kChunks, at = lane % kChunks;
    visit(r, at ^ (r & (kChunks - 1)),
          reinterpret_cast<u32x4*>(own + r * (32 * kVSn) + at * 16));
  }
}

// A wave's 16 kTok rows (of operand B) x 16 kVSn columns (of A) in bf16, through LDS: 8
// bytes a lane as the accumulators lie, out in 16-byte pieces of whole rows.
// pack(vs, ts) gives 4 columns; put(row, chunk, x) stores 8 of them.  smem: 512 kTok kVSn
// bytes a wave, free; each wave uses its own part.
template <int kTok, int kVSn = kVS, typename Pack, typename Put>
__device__ __forceinline__ void store_rows(char* smem, int wave, int lane, Pack&& pack,
                                           Put&& put) {
  char* own = smem + wave * (16 * kTok * 32 * kVSn);
#pragma unroll
  for (int ts = 0; ts < kTok; ++ts)
#pragma unroll
    for (int vs = 0; vs < kVSn; ++vs)
      *reinterpret_cast<uint64_t*>(row_slot<kVSn>(own, lane, vs, ts)) = pack(vs, ts);
  whole_rows<kTok, kVSn>(own, lane, [&](int r, int c, const u32x4* x)
                                        __attribute__((always_inline)) { put(r, c, *x); });
}

}  // namespace
}  // namespace rlk
