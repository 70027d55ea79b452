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

// A wave's 16 kTok rows (of operand B) x 128 columns (of A) in bf16, through LDS: 8
// bytes a lane as the accumulators lie, out in 16-byte pieces of whole 256-byte rows.
// pack(vs, ts) gives 4 columns; put(row, chunk, x) stores 8 of them.  smem: 4096 kTok
// bytes a wave, free; each wave uses its own part.
template <int kTok, typename Pack, typename Put>
__device__ __forceinline__ void store_rows(char* smem, int wave, int lane, Pack&& pack,
                                           Put&& put) {
  char* own = smem + wave * (16 * kTok * 256);
#pragma unroll
  for (int ts = 0; ts < kTok; ++ts)
#pragma unroll
    for (int vs = 0; vs < kVS; ++vs) {
      // chunk c of row r lies at c ^ (r % 16): 16 rows spread over all banks
      const int r = ts * 16 + (lane & 15), c = vs * 2 + (lane >> 5);
      *reinterpret_cast<uint64_t*>(own + r * 256 + (c ^ (lane & 15)) * 16 +
                                   ((lane >> 4) & 1) * 8) = pack(vs, ts);
    }
#pragma unroll
  for (int j = 0; j < 4 * kTok; ++j) {
    const int r = j * 4 + (lane >> 4), c = (lane & 15) ^ (r & 15);
    put(r, c, *reinterpret_cast<const u32x4*>(own + r * 256 + (lane & 15) * 16));
  }
}

}  // namespace
}  // namespace rlk
