// rlk_lmhead_segments.h -- from a block's fp32 logits to its segment statistics,
// shared by the LM-head kernels that keep no logits.
//
// A block holds z[256 vocabulary rows][kTokens tokens] in its accumulators, two
// halves of 128 vocabulary rows in different waves; each lane holds 4
// consecutive vocabulary rows of one token per 16 x 16 tile, so a wave's rows of
// one token sit in the four lanes l%16 + 16g.  Every reduction has a fixed order
// that does not depend on the number of tokens in the block -- each lane over
// its rows in register order, then the four lanes of a token by xor-shuffles
// over 16 and 32 lanes (commutative additions, so all four lanes hold the same
// bits), then the two vocabulary halves (the lower half first).  No atomics.
#pragma once

#include "rlk_internal.h"
#include "rlk_tile.h"

namespace rlk {
namespace {

// Column bound of the first tile boundary strictly inside [v0, v0 + kLmheadBlockVocab), or
// v0 + kLmheadBlockVocab if there is none.  Tile t spans [floor(t*V/T), floor((t+1)*V/T)).
__device__ __forceinline__ int32_t inner_tile_bound(int32_t v0, int32_t padded_vocab,
                                                    int32_t num_tiles) {
  // the tile holding column v0 is the largest t with floor(t*V/T) <= v0
  const int64_t t = ((int64_t)(v0 + 1) * num_tiles - 1) / padded_vocab;
  const int32_t b = (int32_t)(((t + 1) * padded_vocab) / num_tiles);
  return (b > v0 && b < v0 + kLmheadBlockVocab) ? b : v0 + kLmheadBlockVocab;
}

// acc: this wave's z of vocabulary rows [v0 + 128 wv, +128) and tokens
// [t0 + 16 kTok wt, +16 kTok); xch: 4 floats per token of the block (LDS).
// Every wave of the block calls it.  `vb` is v0 / 256.
template <int kTok>
__device__ __forceinline__ void write_segments(const SegmentArgs& a, f32x4 (&acc)[kVS][kTok],
                                               float* xch, int32_t vb, int32_t t0, int wv, int wt,
                                               int lane) {
  const int32_t v0 = vb * kLmheadBlockVocab;
  const int32_t num_tokens = a.num_tokens, row_lo = a.row_lo, row_hi = a.row_hi;
  const int32_t ignore_index = a.ignore_index;
  const int32_t* __restrict__ targets = a.targets;
  const uint8_t* __restrict__ mask = a.mask;
  const int32_t bnd = inner_tile_bound(v0, a.padded_vocab, a.num_tiles);
  const int32_t vw0 = v0 + wv * 128;            // first vocabulary row of this wave
  const int32_t row_lane = 4 * (lane >> 4);     // lane-group offset inside a 16-row tile
  // every row of the block is in [row_lo, row_hi) and no tile bound cuts it:
  // one segment, no masks
  const bool simple = (v0 >= row_lo) && (v0 + kLmheadBlockVocab <= row_hi) && (bnd == v0 + kLmheadBlockVocab);

#pragma unroll
  for (int ts = 0; ts < kTok; ++ts) {
    const int32_t tok = t0 + (wt * kTok + ts) * 16 + (lane & 15);
    int32_t trow = -1;  // the target's column if this wave holds it
    if (tok < num_tokens && (mask == nullptr || mask[tok] != 0)) {
      const int32_t tg = targets[tok];
      if (tg != ignore_index && tg >= vw0 && tg < vw0 + 128 && tg >= row_lo && tg < row_hi)
        trow = tg;
    }
    if (__any(trow >= 0)) {  // rare: some token of this wave has its target here
      float tz = 0.0f;
      bool have_t = false;
#pragma unroll
      for (int vs = 0; vs < kVS; ++vs)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t row = vw0 + vs * 16 + row_lane + i;
          if (row == trow) {
            tz = acc[vs][ts][i];
            have_t = true;
          }
        }
      if (have_t) a.tlogit[tok] = tz;
    }
    float m0 = kNegInf, m1 = kNegInf, s0 = 0.0f, s1 = 0.0f;
    if (simple) {
#pragma unroll
      for (int vs = 0; vs < kVS; ++vs)
#pragma unroll
        for (int i = 0; i < 4; ++i) m0 = maxnan(m0, acc[vs][ts][i]);
      // the lanes l%16 + 16g hold the other rows of the same token
      m0 = maxnan(m0, __shfl_xor(m0, 16));
      m0 = maxnan(m0, __shfl_xor(m0, 32));
      const float b0 = (m0 == kNegInf) ? 0.0f : m0;
#pragma unroll
      for (int vs = 0; vs < kVS; ++vs)
#pragma unroll
        for (int i = 0; i < 4; ++i) s0 += exp2_hw((acc[vs][ts][i] - b0) * kLog2e);
    } else {
      // Segment 0 is the rows [row_lo, min(row_hi, bnd)), segment 1 the rows
      // [max(row_lo, bnd), row_hi).  A 16-row tile wholly inside one segment
      // takes its rows without per-row tests; only a tile that a bound cuts
      // tests each row.  Rows outside both segments add nothing, exactly as
      // the per-row form's exp(-inf) = +0 addends do, so the sums keep their
      // bits; the maxima do not depend on the order.
      const int32_t end0 = min(row_hi, bnd), beg1 = max(row_lo, bnd);
      // pass 1: per-segment maxima over this lane's rows
#pragma unroll
      for (int vs = 0; vs < kVS; ++vs) {
        const int32_t r0 = vw0 + vs * 16;
        if (r0 >= row_lo && r0 + 16 <= end0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) m0 = maxnan(m0, acc[vs][ts][i]);
        } else if (r0 >= beg1 && r0 + 16 <= row_hi) {
#pragma unroll
          for (int i = 0; i < 4; ++i) m1 = maxnan(m1, acc[vs][ts][i]);
        } else if (r0 + 16 > row_lo && r0 < row_hi) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int32_t row = r0 + row_lane + i;
            const float z = acc[vs][ts][i];
            const bool in = row >= row_lo && row < row_hi;
            if (in && row < bnd) m0 = maxnan(m0, z);
            if (in && row >= bnd) m1 = maxnan(m1, z);
          }
        }
      }
      m0 = maxnan(m0, __shfl_xor(m0, 16));
      m0 = maxnan(m0, __shfl_xor(m0, 32));
      m1 = maxnan(m1, __shfl_xor(m1, 16));
      m1 = maxnan(m1, __shfl_xor(m1, 32));
      // pass 2: sums of exp(z - max) relative to the token's maxima, in the
      // same row order as the one-segment form
      const float b0 = (m0 == kNegInf) ? 0.0f : m0;
      const float b1 = (m1 == kNegInf) ? 0.0f : m1;
#pragma unroll
      for (int vs = 0; vs < kVS; ++vs) {
        const int32_t r0 = vw0 + vs * 16;
        if (r0 >= row_lo && r0 + 16 <= end0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) s0 += exp2_hw((acc[vs][ts][i] - b0) * kLog2e);
        } else if (r0 >= beg1 && r0 + 16 <= row_hi) {
#pragma unroll
          for (int i = 0; i < 4; ++i) s1 += exp2_hw((acc[vs][ts][i] - b1) * kLog2e);
        } else if (r0 + 16 > row_lo && r0 < row_hi) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int32_t row = r0 + row_lane + i;
            const float z = (row >= row_lo && row < row_hi) ? acc[vs][ts][i] : kNegInf;
            const bool hi = row >= bnd;
            const float e = exp2_hw((z - (hi ? b1 : b0)) * kLog2e);
            s0 += hi ? 0.0f : e;
            s1 += hi ? e : 0.0f;
          }
        }
      }
    }
    // the four lanes of the token: pairs over 16 lanes, then over 32; each
    // addition has the same two addends in both lanes, so all four agree
    s0 += __shfl_xor(s0, 16);
    s1 += __shfl_xor(s1, 16);
    s0 += __shfl_xor(s0, 32);
    s1 += __shfl_xor(s1, 32);
    if (wv == 1 && lane < 16) {
      float* x = xch + (((wt * kTok + ts) * 16 + lane) * 4);
      x[0] = m0;
      x[1] = s0;
      x[2] = m1;
      x[3] = s1;
    }
    // keep this token's values in registers of the lower-half wave
    if (wv == 0) {
      acc[0][ts][0] = m0;
      acc[0][ts][1] = s0;
      acc[0][ts][2] = m1;
      acc[0][ts][3] = s1;
    }
  }
  __syncthreads();
  // slot 0 starts at v0; slot 1 at the inner bound, or (an identity slot that
  // nothing reads) at v0 when there is none
  const int32_t c_slot1 = (bnd < v0 + kLmheadBlockVocab) ? bnd : v0;
  const bool own0 = v0 >= a.col_lo && v0 < a.col_hi;
  const bool own1 = c_slot1 >= a.col_lo && c_slot1 < a.col_hi;
  if (wv == 0 && lane < 16) {
    const int64_t seg_ld = 2 * (int64_t)a.n_vb;
#pragma unroll
    for (int ts = 0; ts < kTok; ++ts) {
      const int32_t tok = t0 + (wt * kTok + ts) * 16 + lane;
      if (tok >= num_tokens) continue;
      const float* x = xch + (((wt * kTok + ts) * 16 + lane) * 4);
      float out_m[2], out_s[2];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        // lower vocabulary half first, then the upper half
        const float ma = acc[0][ts][2 * g], sa_ = acc[0][ts][2 * g + 1];
        const float mb = x[2 * g], sb_ = x[2 * g + 1];
        const float M = maxnan(ma, mb);
        float S = 0.0f;
        if (M != kNegInf) {
          if (ma != kNegInf) S = sa_ * exp2_hw((ma - M) * kLog2e);
          if (mb != kNegInf) S = fmaf(sb_, exp2_hw((mb - M) * kLog2e), S);
        }
        out_m[g] = M;
        out_s[g] = S;
      }
      float* om = a.seg_m + (int64_t)tok * seg_ld + 2 * vb;
      float* os = a.seg_s + (int64_t)tok * seg_ld + 2 * vb;
      if (own0) {
        om[0] = out_m[0];
        os[0] = out_s[0];
      }
      if (own1) {
        om[1] = out_m[1];
        os[1] = out_s[1];
      }
    }
  }
}

}  // namespace
}  // namespace rlk
