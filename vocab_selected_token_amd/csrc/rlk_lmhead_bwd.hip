// rlk_lmhead_bwd.hip -- gradients of the fused LM-head for gfx950: from logp and
// LSE of z = h . W^T back to h and W, without keeping the logits.
//
// With p = exp(z - LSE), g and gl the upstream gradients of logp and LSE and a
// the effective-active flag of a row,
//   dz = a g (onehot(target) - p) + gl p,   dh = dz . W,   dW = dz^T . h.
// z is computed again, a piece of the vocabulary at a time, and each piece's dz
// is used for both products while it is at hand.
//
// Only rows that some term reaches ("live": effective-active with g != 0, or gl
// != 0) take part.  They are gathered to the front first, in ascending order, so
// that prompt and padding tokens cost nothing in the three products and a NaN in
// a hidden state that is masked out meets no product (0 * NaN would be NaN).
//
// dz is rounded to bf16 for the matrix cores: half a step, at most 2^-8 relative, once
// per element, as much as rounding the results to bf16 does (in norm, dhidden ends up
// 0.0017 from 64 bits and dweight 0.0023; results rounded alone 0.0017).  Two things
// keep that rounding from adding up.  All rows are divided by the largest |g|, |gl|
// before it (and the results multiplied by it), so that the equal gradients of a
// mean become +-1 and a target's entry near 1 - p rounds without a bias that
// every row shares; and for dh what the rounding took from the target's entry,
// which dominates its row, is added back in fp32 (dh_finish).
//
// Sums over K, over the vocabulary and over tokens are held in fp32, in a fixed
// order: repeated calls give the same bits.  No atomics.
//
// What it costs: three products of the live rows, one of them the forward's again; the
// alternative, logits kept from the forward, is what the caller comes here to avoid.
// 4096 tokens (3405 live) x 4096 x 151936 take 10.1 ms, 1.26 PFLOP/s in the products; a
// library's bf16 product of that size runs at 1.43.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "rlk_internal.h"
#include "rlk_rows.h"
#include "rlk_stream.h"
#include "rlk_tile.h"

namespace rlk {
namespace {

static_assert(kBK == kLmheadSlabK, "slab width shared with the boundary");

constexpr int kT = 64;  // tile edge of the gather and transpose kernels
constexpr int kScanThreads = 1024;
constexpr int32_t kScanFew = 1024;

__device__ __forceinline__ float bf16_float(uint16_t b) {
  return __uint_as_float((uint32_t)b << 16);
}

// What the kernels know of one live row, normalised by the call's scale.
struct LiveRows {
  int32_t* idx;    // its row in the batch
  int32_t* tgt;    // its target column, or -1 (not active)
  float* lse;
  float* cg;       // a g / scale: added at the target
  float* cc;       // (gl - a g) / scale: times p
  float* resid;    // the target entry of dz less its bf16 rounding
  int32_t* inv;    // [num_tokens] batch row -> live row, or -1
  uint32_t* head;  // [0] number of live rows, [1] the scale's bits
};

__device__ __forceinline__ LiveRows live_rows(char* ws, const LmheadBwdLayout& l) {
  return {reinterpret_cast<int32_t*>(ws + l.idx),   reinterpret_cast<int32_t*>(ws + l.tgt),
          reinterpret_cast<float*>(ws + l.lse),     reinterpret_cast<float*>(ws + l.cg),
          reinterpret_cast<float*>(ws + l.cc),      reinterpret_cast<float*>(ws + l.resid),
          reinterpret_cast<int32_t*>(ws + l.inv),   reinterpret_cast<uint32_t*>(ws + l.head)};
}

// What is known of the batch's rows.
struct RowArgs {
  const int32_t* __restrict__ targets;
  const uint8_t* __restrict__ mask;
  const float* __restrict__ lse;
  const float* __restrict__ grad;
  const float* __restrict__ grad_lse;
  uint32_t* __restrict__ status;
  int32_t num_tokens, padded_tokens, real_vocab, ignore_index;
};

template <int kThr>
struct ScanLds {
  float top[kThr / 64];
  int32_t sum[kThr / 64];
};

// By a whole block: the scale (largest finite |a g|, |gl|; 1 if all are 0), then the
// live rows in ascending order.  Returns their number; at(i, r) hears that live row i
// is row r of the batch.  With `write`, they and the scale go to the workspace; slots
// from the last live row up to a multiple of 256 hold rows that give dz = 0.  An
// effective-active row with a target outside [0, V_real) is live with NaN factors,
// and so is one whose LSE is not finite (exp(z - inf) would be a plausible 0): its dz is
// NaN.
template <int kThr, typename At>
__device__ __forceinline__ int32_t scan_rows(const RowArgs& a, const LiveRows& live,
                                             ScanLds<kThr>& lds, bool write, At&& at_row) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  auto row = [&](int32_t r, float& g, float& gl, int32_t& tgt, bool& act, bool& bad) {
    act = (a.mask == nullptr || a.mask[r] != 0);
    tgt = act ? a.targets[r] : -1;
    act = act && tgt != a.ignore_index;
    bad = act && (tgt < 0 || tgt >= a.real_vocab);
    g = (act && a.grad) ? a.grad[r] : 0.0f;
    gl = a.grad_lse ? a.grad_lse[r] : 0.0f;
  };

  float scale = 1.0f;
  if (write) {
    float top = 0.0f;
    for (int32_t r = tid; r < a.num_tokens; r += kThr) {
      float g, gl;
      int32_t tgt;
      bool act, bad;
      row(r, g, gl, tgt, act, bad);
      const float m = fmaxf(isfinite(g) ? fabsf(g) : 0.0f, isfinite(gl) ? fabsf(gl) : 0.0f);
      top = fmaxf(top, m);
    }
#pragma unroll
    for (int o = 32; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
    if (lane == 0) lds.top[wave] = top;
    __syncthreads();
    for (int w = 0; w < kThr / 64; ++w) top = fmaxf(top, lds.top[w]);
    if (top > 0.0f) scale = top;
  }

  int32_t base = 0;
  for (int32_t r0 = 0; r0 < a.num_tokens; r0 += kThr) {
    const int32_t r = r0 + tid;
    float g = 0.0f, gl = 0.0f;
    int32_t tgt = -1;
    bool act = false, bad = false;
    if (r < a.num_tokens) row(r, g, gl, tgt, act, bad);
    const bool on = bad || g != 0.0f || gl != 0.0f;
    const uint64_t votes = __ballot(on);
    const int32_t before = __popcll(votes & ((1ull << lane) - 1));
    __syncthreads();  // the previous round's sums have been read
    if (lane == 0) lds.sum[wave] = __popcll(votes);
    __syncthreads();
    int32_t at = base + before;
    for (int w = 0; w < kThr / 64; ++w) {
      if (w < wave) at += lds.sum[w];
      base += lds.sum[w];
    }
    if (on) at_row(at, r);
    if (!write) continue;
    if (on) {
      const float nan = __builtin_nanf("");
      live.idx[at] = r;
      live.tgt[at] = (act && !bad) ? tgt : -1;
      const float l = a.lse[r];
      const bool none = bad || !isfinite(l);
      live.lse[at] = l;
      live.cg[at] = none ? nan : g / scale;
      live.cc[at] = none ? nan : gl / scale - g / scale;
      live.resid[at] = 0.0f;
      if (bad) a.status[0] = 1u;
    }
    if (r < a.num_tokens) live.inv[r] = on ? at : -1;
  }
  if (!write) return base;
  const int32_t end = min((base + 255) / 256 * 256, a.padded_tokens);
  for (int32_t i = base + tid; i < end; i += kThr) {
    live.idx[i] = -1;
    live.tgt[i] = -1;
    live.lse[i] = 0.0f;
    live.cg[i] = 0.0f;
    live.cc[i] = 0.0f;
    live.resid[i] = 0.0f;
  }
  if (tid == 0) {
    live.head[0] = (uint32_t)base;
    live.head[1] = __float_as_uint(scale);
  }
  return base;
}

// ---------------------------------------------------------------------------
// live_rows_scan: one block, for more than kScanFew tokens (4096: 12 us).
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kScanThreads) void live_rows_scan(RowArgs a, char* ws,
                                                               LmheadBwdLayout lay) {
  __shared__ ScanLds<kScanThreads> lds;
  scan_rows(a, live_rows(ws, lay), lds, true, [](int32_t, int32_t) {});
}

// How dh's blocks share its sums.  The grid is made for tiles of all tokens; where
// some have no live row, their blocks take a part of the others' sums: `splits` parts
// to each of `tiles` tiles of live rows, padded to `rows` (777 tokens, 660 of them live,
// x 1088 x 50021: grad_piece 108 -> 89 us; the blocks that are left over end at once, and
// the others are numbered without them, so that every XCD gets its share: 4096 x 4096 x
// 151936, 3405 live, backward 10.40 -> 10.14 ms).
struct DhParts {
  int32_t tiles, splits, rows;
  __device__ __forceinline__ DhParts(int32_t count, const LmheadBwdLayout& l)
      : tiles((count + kBA - 1) / kBA),
        splits(tiles ? min(l.splits * (l.padded_tokens / kBA) / tiles, l.most_splits) : 0),
        rows(tiles * kBA) {}
};

// A 64 x 64 bf16 tile read by rows (row r of the source at src[r], or zeros) and
// written by columns: dst[c][r] = src[r][c].  256 threads; rows of 72 elements
// in LDS keep both directions at most 2-way conflicting.
struct Tile64 {
  uint16_t v[kT][kT + 8];
};

// ---------------------------------------------------------------------------
// gather_rows: hc[i] = h[idx[i]] (zeros in the slots behind the last live row)
// and, when asked for, its transpose ht[k][i].  The blocks behind those of the rows
// copy the weight's last rows, those behind the last whole 64, followed by zeros: the
// slab of dh's sum that they do not fill.
// kScan: up to kScanFew tokens every block scans the rows itself, and the first
// writes what the scan found (a launch less: the backward of 1 x 64 x 1000 takes 25.0 us
// for 30.5, of 64 x 512 x 12003 45.0 for 49.2).
// ---------------------------------------------------------------------------
struct GatherArgs {
  const u32x4* __restrict__ h;
  u32x4* __restrict__ hc;
  uint16_t* __restrict__ ht;
  const u32x4* __restrict__ w_tail;  // the weight's last rows
  u32x4* __restrict__ tail;
  int64_t n_rows;     // blocks of rows
  int32_t tail_rows;  // 0: no such slab
  int32_t ldc;        // 16-byte chunks per row
};

template <bool kScan>
__global__ __launch_bounds__(256) void gather_rows(GatherArgs a, RowArgs rows, char* ws,
                                                   LmheadBwdLayout lay, int64_t blk_begin) {
  __shared__ Tile64 t;
  __shared__ int32_t from[kT];
  const int64_t blk = blk_begin + blockIdx.x;
  if (blk >= a.n_rows) {
    const int64_t i = (blk - a.n_rows) * 256 + threadIdx.x;
    if (i < (int64_t)kBK * a.ldc)
      a.tail[i] = i < (int64_t)a.tail_rows * a.ldc ? a.w_tail[i] : u32x4{0, 0, 0, 0};
    return;
  }
  const LiveRows live = live_rows(ws, lay);
  const int32_t k_tiles = a.ldc / (kT / 8);
  const int32_t i0 = (int32_t)(blk / k_tiles) * kT;
  const int32_t kc0 = (int32_t)(blk % k_tiles) * (kT / 8);
  int32_t count;
  if constexpr (kScan) {
    __shared__ ScanLds<256> lds;
    if (threadIdx.x < kT) from[threadIdx.x] = -1;
    __syncthreads();
    count = scan_rows(rows, live, lds, blk == 0, [&](int32_t at, int32_t r) {
      if (at >= i0 && at < i0 + kT) from[at - i0] = r;
    });
  } else {
    count = (int32_t)live.head[0];
    if (threadIdx.x < kT) from[threadIdx.x] = live.idx[i0 + threadIdx.x];
  }
  if (i0 >= (count + 255) / 256 * 256) return;
  __syncthreads();
  for (int q = threadIdx.x; q < kT * kT / 8; q += 256) {
    const int r = q >> 3, c = q & 7;
    u32x4 x = {0, 0, 0, 0};
    if (from[r] >= 0) x = a.h[(int64_t)from[r] * a.ldc + kc0 + c];
    a.hc[(int64_t)(i0 + r) * a.ldc + kc0 + c] = x;
    if (a.ht) *reinterpret_cast<u32x4*>(&t.v[r][c * 8]) = x;
  }
  if (!a.ht) return;
  __syncthreads();
  for (int q = threadIdx.x; q < kT * kT / 8; q += 256) {
    const int c = q >> 3, r = (q & 7) * 8;
    union {
      uint16_t e[8];
      u32x4 x;
    } o;
#pragma unroll
    for (int i = 0; i < 8; ++i) o.e[i] = t.v[r + i][c];
    *reinterpret_cast<u32x4*>(a.ht + (int64_t)(kc0 * 8 + c) * rows.padded_tokens + i0 + r) = o.x;
  }
}

// Work index -> (tile of A, tile of B): strips of 4 A tiles, B-major inside, so
// that the blocks resident on one XCD share operand rows (see lmhead_segments).
__device__ __forceinline__ void tile_of(int64_t blk, int32_t n_a, int32_t n_b, int32_t& ta,
                                        int32_t& tb) {
  constexpr int32_t kGroup = 4;
  const int64_t strip = blk / ((int64_t)kGroup * n_b);
  const int32_t r_in = (int32_t)(blk - strip * kGroup * n_b);
  const int32_t strip_w = min(kGroup, n_a - (int32_t)strip * kGroup);
  ta = (int32_t)strip * kGroup + r_in % strip_w;
  tb = r_in / strip_w;
}

// dz of one column from its logit (nl = -LSE log2 e), before its rounding to bf16;
// what the rounding takes is kept where the column is the target's.
__device__ __forceinline__ float plain_dz(float z, float nl, float cc) {
  return exp2_hw(fmaf(z, kLog2e, nl)) * cc;
}
__device__ __forceinline__ float dz_of(float z, float nl, float cg, float cc, bool real,
                                       bool target, float* resid) {
  const float p = plain_dz(z, nl, 1.0f);
  const float d = !real ? 0.0f : target ? fmaf(p, cc, cg) : p * cc;
  if (target) *resid = d - bf16_float(bf16_bits(d));
  return d;
}

// Whole rows out of a 256 x 256 tile, past the caches (what is written outlives them:
// the backward of 1024 tokens x 2048 x 151936 takes 1784 us this way, 1837 us with
// ordinary stores; dw_few below gains most, 32 tokens 228 us for 267).
static_assert(kTileLds >= kWaves * 4096 * kTS, "the rows fit");
__device__ __forceinline__ void put_row(uint16_t* out, const u32x4& x) {
  __builtin_nontemporal_store(x, reinterpret_cast<u32x4*>(out));
}

// ---------------------------------------------------------------------------
// dz_piece: dz of the columns [c0, c0 + piece) for the live rows, in bf16
// (dz[i][c], ld = piece).  The exponentials and the stores of a tile follow its
// product and nothing hides them, so a wave without target and padding tests no
// column (this kernel for 1024 x 64 x 65536: 69 -> 45 us; 777 x 1088 x 50021: 111 -> 101;
// 1024 x 2048 x 151936: 629 -> 577).
// ---------------------------------------------------------------------------
template <int kTok>
__global__ __launch_bounds__(kThreads) void dz_piece(
    const u32x4* __restrict__ hc, const u32x4* __restrict__ w, int32_t hidden_dim,
    int32_t real_vocab, int32_t c0, int32_t piece, uint16_t* __restrict__ dz, char* ws,
    LmheadBwdLayout lay, int64_t blk_begin) {
  constexpr int kTokens = 64 * kTok;
  __shared__ __attribute__((aligned(16))) char smem[2 * kStageBytes<kTok>];
  static_assert(sizeof(smem) >= kWaves * 4096 * kTok, "the rows fit");
  const LiveRows live = live_rows(ws, lay);
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wv = wave >> 2, wt = wave & 3;
  // only tiles with a live row
  const int32_t n_va = piece / kBA, n_tb = ((int32_t)live.head[0] + kTokens - 1) / kTokens;
  const int64_t blk = blk_begin + blockIdx.x, used = (int64_t)n_va * n_tb;
  if (blk >= used) return;
  int32_t va, tb;
  tile_of(xcd_local_block(blk, used), n_va, n_tb, va, tb);
  const int32_t t0 = tb * kTokens, v0 = va * kBA;  // v0: column inside the piece
  f32x4 acc[kVS][kTok] = {};  // a tile of padding: z = 0, of which no dz is made
  if (c0 + v0 < real_vocab) {
    const int64_t row_bytes = (int64_t)hidden_dim * 2;
    const TileOperand wo(reinterpret_cast<const char*>(w) + (int64_t)(c0 + v0) * row_bytes,
                         row_bytes, min(kBA, real_vocab - c0 - v0), 0, wave, lane);
    const TileOperandOf<kTok> ho(reinterpret_cast<const char*>(hc) + (int64_t)t0 * row_bytes,
                                 row_bytes, kTokens, 0, wave, lane);
    tile_product(smem, wo, ho, 0, hidden_dim / kBK, wave, lane, acc);
  }
  const int32_t cw = v0 + wv * 128;  // this wave's first column
#pragma unroll
  for (int ts = 0; ts < kTok; ++ts) {
    const int32_t i = t0 + (wt * kTok + ts) * 16 + (lane & 15);
    const float nl = -live.lse[i] * kLog2e, cg = live.cg[i], cc = live.cc[i];
    const int32_t tgt = live.tgt[i] - c0;
    // columns from here on are padding; all of them for a slot behind the last live row
    // (its z may be NaN: a hidden state of zero times an infinite weight)
    const int32_t last = i < (int32_t)live.head[0] ? real_vocab - c0 : 0;
    // neither target nor padding in the wave's columns of these tokens: nothing to test
    if (!__any((tgt >= cw && tgt < cw + 128) || last < cw + 128)) {
#pragma unroll
      for (int vs = 0; vs < kVS; ++vs)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[vs][ts][e] = plain_dz(acc[vs][ts][e], nl, cc);
    } else {
#pragma unroll
      for (int vs = 0; vs < kVS; ++vs)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int32_t c = cw + vs * 16 + 4 * (lane >> 4) + e;
          acc[vs][ts][e] =
              dz_of(acc[vs][ts][e], nl, cg, cc, c < last, c == tgt, live.resid + i);
        }
    }
  }
  store_rows<kTok>(
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
        put_row(dz + (int64_t)(t0 + wt * (16 * kTok) + r) * piece + v0 + wv * 128 + c * 8, x);
      });
}

// ---------------------------------------------------------------------------
// grad_piece: both products of one piece in one launch, so that the last blocks
// of one fill the chip beside the other's.  The blocks [0, n_dh) are dh's (the
// longer sums first), the rest dW's.
//   dh:  part[s][k][i] (+)= sum over split s (DhParts) of the piece's columns of
//        dz[i][c] W[c0 + c][k], in fp32; the first piece writes, the others add.
//        A = dz, B = W by its rows, so a lane holds 4 consecutive tokens of one k.
//   dW:  dW[c0 + c][k] = scale * sum_i dz[i][c] ht[k][i], in bf16; +0 from the
//        real vocabulary's end on.  A = ht, B = dz by its rows: 4 consecutive k of
//        one column.
// The MFMAs bound it: 2.15 ms a piece of a third of 151936 columns at 3405 live rows and
// hidden_dim 4096, 1.31 PFLOP/s.  (With copies of W and dz turned beforehand instead
// of the transposing reads the backward took 12.8 ms for 11.5.)  With few tokens dW's
// sums are short and its stores weigh more: 1024 x 2048 x 151936 1.07 ms, 1.19 PFLOP/s.
// ---------------------------------------------------------------------------
struct GradArgs {
  const uint16_t* __restrict__ dz;    // [padded_tokens][piece]
  const uint16_t* __restrict__ ht;    // [hidden_dim][padded_tokens]
  const uint16_t* __restrict__ w;     // [>= real_vocab][hidden_dim]
  const uint16_t* __restrict__ tail;  // [64][hidden_dim], see gather_rows
  float* __restrict__ part;           // [DhParts::splits][hidden_dim][DhParts::rows]
  uint16_t* __restrict__ dw;          // [padded_vocab][hidden_dim]
  int32_t hidden_dim, real_vocab, padded_vocab;
  int32_t c0, piece;
  int32_t padded_tokens;
  bool add;
  int64_t n_dh, n_dw;
};

__global__ __launch_bounds__(kThreads) void grad_piece(GradArgs a, char* ws, LmheadBwdLayout lay,
                                                       int64_t blk_begin) {
  __shared__ __attribute__((aligned(16))) char smem[kTileLds];
  const LiveRows live = live_rows(ws, lay);
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wv = wave >> 2, wt = wave & 3;
  const int32_t n_k = (a.hidden_dim + kBA - 1) / kBA;
  const int32_t count = (int32_t)live.head[0];
  const int64_t blk = blk_begin + blockIdx.x;
  const bool is_dh = blk < a.n_dh;
  const DhParts parts(count, lay);

  int32_t ta, tb, s0 = 0, nslab;
  if (is_dh) {
    const int64_t per = (int64_t)n_k * parts.tiles, used = per * parts.splits;
    if (blk >= used) return;
    const int64_t b = xcd_local_block(blk, used);
    const int32_t split = (int32_t)(b / per);
    tile_of(b - split * per, parts.tiles, n_k, ta, tb);
    const int32_t slabs = (min(a.piece, a.real_vocab - a.c0) + kBK - 1) / kBK;
    s0 = (int32_t)((int64_t)split * slabs / parts.splits);
    nslab = (int32_t)((int64_t)(split + 1) * slabs / parts.splits) - s0;
    a.part += (int64_t)split * a.hidden_dim * parts.rows;
  } else {
    tile_of(xcd_local_block(blk - a.n_dh, a.n_dw), n_k, a.piece / kBB, ta, tb);
    if (a.c0 + tb * kBB >= a.padded_vocab) return;
    nslab = a.c0 + tb * kBB < a.real_vocab ? (count + kBK - 1) / kBK : 0;
  }
  const int32_t a0 = ta * kBA, b0 = tb * kBB;

  f32x4 acc[kVS][kTS];
  if (nslab > 0) {
    const int64_t k_bytes = (int64_t)a.hidden_dim * 2, t_bytes = (int64_t)a.padded_tokens * 2,
                  c_bytes = (int64_t)a.piece * 2;
    const TileOperand ao(is_dh ? a.dz + (int64_t)a0 * a.piece : a.ht + (int64_t)a0 * a.padded_tokens,
                         is_dh ? c_bytes : t_bytes, is_dh ? kBA : min(kBA, a.hidden_dim - a0), 0,
                         wave, lane);
    const TileOperandT bo(is_dh ? a.w + (int64_t)a.c0 * a.hidden_dim + b0 : a.dz + b0,
                          is_dh ? k_bytes : c_bytes, is_dh ? min(kBB, a.hidden_dim - b0) : kBB,
                          a.tail + b0, is_dh ? (a.real_vocab - a.c0) / kBK : -1, wave, lane);
    tile_product(smem, ao, bo, s0, nslab, wave, lane, acc);
  } else {
#pragma unroll
    for (int vs = 0; vs < kVS; ++vs)
#pragma unroll
      for (int ts = 0; ts < kTS; ++ts) acc[vs][ts] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  }

  if (is_dh) {
#pragma unroll
    for (int ts = 0; ts < kTS; ++ts) {
      const int32_t k = b0 + (wt * kTS + ts) * 16 + (lane & 15);
      if (k >= a.hidden_dim) continue;
      float* out = a.part + (int64_t)k * parts.rows + a0 + wv * 128 + 4 * (lane >> 4);
#pragma unroll
      for (int vs = 0; vs < kVS; ++vs) {
        f32x4* o = reinterpret_cast<f32x4*>(out + vs * 16);
        *o = a.add ? *o + acc[vs][ts] : acc[vs][ts];
      }
    }
    return;
  }
  const float scale = __uint_as_float(live.head[1]);
  store_rows<kTS>(
      smem, wave, lane,
      [&](int vs, int ts) __attribute__((always_inline)) {
        union {
          uint16_t e[4];
          uint64_t x;
        } o;
        const bool on = a.c0 + b0 + (wt * kTS + ts) * 16 + (lane & 15) < a.real_vocab;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.e[e] = on ? bf16_bits(acc[vs][ts][e] * scale) : (uint16_t)0;
        return o.x;
      },
      [&](int r, int c, const u32x4& x) __attribute__((always_inline)) {
        const int32_t row = a.c0 + b0 + wt * 64 + r, k = a0 + wv * 128 + c * 8;
        if (row < a.padded_vocab && k < a.hidden_dim)
          put_row(a.dw + (int64_t)row * a.hidden_dim + k, x);
      });
}

// ---------------------------------------------------------------------------
// Few tokens (16 kTok at most): the weight's and dW's bytes bound the time, and the
// tiles of the kernels above would leave most of their rows empty.
//   dz_stream  z by stream_product, then dz by tokens (dz[i][c], as dz_piece) and by
//              columns (dzt[c][i], 64 tokens apart) for dw_few.
//   dw_few     a block takes 64 columns: dz's fragments stay in registers, and each
//              of its four waves goes over every fourth 64 of hidden_dim, operands
//              straight from memory (the L2 holds ht), one or two MFMA steps for a
//              whole sum, out through LDS in rows of 128 bytes.
// 32 x 1024 x 151936: dz_stream 65 us (the weight at 4.8 TB/s), dw_few 64 us (dW at
// 4.9 TB/s; 76 with each step's ht loaded as it is used), dh_few 65 us; the tiles took
// 340 us for the whole backward, these 215.
// ---------------------------------------------------------------------------
constexpr int kFewLd = 64;  // tokens a row of dzt has room for

template <int kTok>
__global__ __launch_bounds__(kStreamThreads) void dz_stream(
    const char* __restrict__ hc, const char* __restrict__ w, int32_t hidden_dim,
    int32_t real_vocab, int32_t c0, int32_t piece, uint16_t* __restrict__ dz,
    uint16_t* __restrict__ dzt, char* ws, LmheadBwdLayout lay, int64_t blk_begin) {
  __shared__ StreamLds<kTok> lds;
  const LiveRows live = live_rows(ws, lay);
  if (live.head[0] == 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int32_t v0 = c0 + (int32_t)(blk_begin + blockIdx.x) * kStreamRows;
  f32x4 acc[1][kTok];
  Bf16Stream math;
  // the gathered rows behind the last live one are zeros
  stream_product(lds, w, hc, (uint32_t)hidden_dim * 2, 0, real_vocab, 16 * kTok, v0, math, acc);
  const int32_t v = v0 + wave * 16 + 4 * (lane >> 4);
#pragma unroll
  for (int ts = 0; ts < kTok; ++ts) {
    const int32_t i = ts * 16 + (lane & 15);
    const float nl = -live.lse[i] * kLog2e, cg = live.cg[i], cc = live.cc[i];
    const int32_t tgt = live.tgt[i];
    const int32_t last = i < (int32_t)live.head[0] ? real_vocab : 0;  // as in dz_piece
    union {
      uint16_t e[4];
      uint64_t x;
    } o;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      o.e[e] = bf16_bits(
          dz_of(acc[0][ts][e], nl, cg, cc, v + e < last, v + e == tgt, live.resid + i));
      if (dzt) dzt[(int64_t)(v + e - c0) * kFewLd + i] = o.e[e];
    }
    *reinterpret_cast<uint64_t*>(dz + (int64_t)i * piece + (v - c0)) = o.x;
  }
}

template <int kTok>
__global__ __launch_bounds__(256) void dw_few(const uint16_t* __restrict__ ht,
                                              const uint16_t* __restrict__ dzt,
                                              int32_t hidden_dim, int32_t real_vocab,
                                              int32_t padded_vocab, int32_t c0,
                                              int32_t padded_tokens, uint16_t* __restrict__ dw,
                                              char* ws, LmheadBwdLayout lay, int64_t blk_begin) {
  constexpr int kSteps = kTok > 2 ? 2 : 1;  // of 32 tokens
  __shared__ __attribute__((aligned(16))) char stage[4][64 * 128];
  const LiveRows live = live_rows(ws, lay);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int32_t b0 = (int32_t)(blk_begin + blockIdx.x) * 64;  // column inside the piece
  const float scale = __uint_as_float(live.head[1]);
  const bool any = live.head[0] != 0 && c0 + b0 < real_vocab;
  const int fr = lane & 15, fg = lane >> 4;
  const i32x4 none = {0, 0, 0, 0};
  i32x4 b[4][kSteps];
#pragma unroll
  for (int ts = 0; ts < 4; ++ts)
#pragma unroll
    for (int s = 0; s < kSteps; ++s)  // 16 tokens fill half a step
      b[ts][s] = any && s * 32 + fg * 8 < 16 * kTok
                     ? *reinterpret_cast<const i32x4*>(
                           dzt + (int64_t)(b0 + ts * 16 + fr) * kFewLd + s * 32 + fg * 8)
                     : none;
  char* own = stage[wave];
  i32x4 a[4][kSteps];
  auto load_a = [&](int32_t k0) __attribute__((always_inline)) {
#pragma unroll
    for (int vs = 0; vs < 4; ++vs)
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        a[vs][s] = any ? *reinterpret_cast<const i32x4*>(
                             ht + (int64_t)(k0 + vs * 16 + fr) * padded_tokens + s * 32 + fg * 8)
                       : none;
  };
  if (wave * 64 < hidden_dim) load_a(wave * 64);
  for (int32_t k0 = wave * 64; k0 < hidden_dim; k0 += 256) {
    f32x4 acc[4][4];
#pragma unroll
    for (int vs = 0; vs < 4; ++vs) {
#pragma unroll
      for (int ts = 0; ts < 4; ++ts) {
        acc[vs][ts] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
          acc[vs][ts] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(bf16x8, a[vs][s]), __builtin_bit_cast(bf16x8, b[ts][s]),
              acc[vs][ts], 0, 0, 0);
      }
    }
    // the next step's, on their way while this one's results leave (in place of the last
    // step's the last 64 again, unused)
    load_a(min(k0 + 256, hidden_dim - 64));
#pragma unroll
    for (int ts = 0; ts < 4; ++ts) {
      const int r = ts * 16 + fr;
      const bool on = c0 + b0 + r < real_vocab;
#pragma unroll
      for (int vs = 0; vs < 4; ++vs) {
        union {
          uint16_t e[4];
          uint64_t x;
        } o;
#pragma unroll
        for (int e = 0; e < 4; ++e) o.e[e] = on ? bf16_bits(acc[vs][ts][e] * scale) : (uint16_t)0;
        *reinterpret_cast<uint64_t*>(own + swizzled(r, vs * 2 + (lane >> 5)) * 16 +
                                     (fg & 1) * 8) = o.x;
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int r = j * 8 + (lane >> 3), c = (lane & 7) ^ ((r >> 1) & 7);
      const u32x4 x = *reinterpret_cast<const u32x4*>(own + r * 128 + (lane & 7) * 16);
      if (c0 + b0 + r < padded_vocab)
        __builtin_nontemporal_store(
            x, reinterpret_cast<u32x4*>(dw + (int64_t)(c0 + b0 + r) * hidden_dim + k0 + c * 8));
    }
  }
}

// dh_few: part[s][k][i] (+)= the sum of dh_piece for the same split, for few tokens:
// a block takes 256 columns of hidden_dim, its eight waves 32 each with all tokens.
// W goes through LDS in slabs of 64 of its rows, two stages (64 KB: two blocks a CU,
// one slab of each in flight); dz's fragments come from memory, a slab ahead.
template <int kTok>
__global__ __launch_bounds__(kThreads) void dh_few(GradArgs a, char* ws, LmheadBwdLayout lay,
                                                   int64_t blk_begin) {
#if defined(__HIP_DEVICE_COMPILE__)  // the host pass cannot instantiate the target's builtins
  __shared__ __attribute__((aligned(16))) char smem[2 * kSlabBytes];
  const LiveRows live = live_rows(ws, lay);
  if (live.head[0] == 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int32_t n_k = (a.hidden_dim + kBB - 1) / kBB;
  const int64_t blk = blk_begin + blockIdx.x;
  const int32_t split = (int32_t)(blk / n_k), k0 = (int32_t)(blk % n_k) * kBB;
  const int32_t slabs = (min(a.piece, a.real_vocab - a.c0) + kBK - 1) / kBK;
  const int32_t s0 = (int32_t)((int64_t)split * slabs / lay.splits);
  const int32_t s1 = (int32_t)((int64_t)(split + 1) * slabs / lay.splits);
  const TileOperandT wo(a.w + (int64_t)a.c0 * a.hidden_dim + k0, (int64_t)a.hidden_dim * 2,
                        min(kBB, a.hidden_dim - k0), a.tail + k0, (a.real_vocab - a.c0) / kBK,
                        wave, lane);
  f32x4 acc[kTok][2];
#pragma unroll
  for (int t = 0; t < kTok; ++t) acc[t][0] = acc[t][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  if (s1 > s0) {
    const uint16_t* dz = a.dz + (int64_t)(lane & 15) * a.piece + (lane >> 4) * 8;
    bf16x8 d[kTok][2], nd[kTok][2];
    auto load_dz = [&](int s, bf16x8 (&to)[kTok][2]) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < kTok; ++t)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
          to[t][ks] = *reinterpret_cast<const bf16x8*>(dz + (int64_t)t * 16 * a.piece + s * kBK +
                                                       ks * 32);
    };
    wo.issue(smem, wave, s0);
    wo.issue(smem + kSlabBytes, wave, min(s0 + 1, s1 - 1));
    load_dz(s0, d);
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    for (int s = s0; s < s1; ++s) {
      char* cur = smem + ((s - s0) & 1) * kSlabBytes;
      bf16x8 b[2][2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          b[j][ks] = TileOperandT::fragment(cur, wave * 32 + j * 16, ks, lane);
      __builtin_amdgcn_sched_barrier(0);
      // every wave has read slab s into registers, and slab s+1 has landed
      __builtin_amdgcn_s_waitcnt(0);
      __syncthreads();
      __builtin_amdgcn_sched_barrier(0);
      // the last two steps load the last slab again, unused
      wo.issue(cur, wave, min(s + 2, s1 - 1));
      load_dz(min(s + 1, s1 - 1), nd);
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int t = 0; t < kTok; ++t)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            acc[t][j] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(d[t][ks], b[j][ks], acc[t][j], 0, 0, 0);
#pragma unroll
      for (int t = 0; t < kTok; ++t)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) d[t][ks] = nd[t][ks];
    }
    __builtin_amdgcn_s_waitcnt(0);  // no load into LDS outlives the block
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int32_t k = k0 + wave * 32 + j * 16 + (lane & 15);
    if (k >= a.hidden_dim) continue;
    float* out = a.part + ((int64_t)split * a.hidden_dim + k) * a.padded_tokens + 4 * (lane >> 4);
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      f32x4* o = reinterpret_cast<f32x4*>(out + t * 16);
      *o = a.add ? *o + acc[t][j] : acc[t][j];
    }
  }
#endif
}

// ---------------------------------------------------------------------------
// dh_finish: dh[r] = scale * (sum of the splits' partials in a fixed order + resid
// W[target]) in bf16; +0 on rows that are not live.  A block takes 64 live rows x kCols
// columns, through LDS from the partials' layout to rows, and writes the zeros of the 64
// batch rows of the same numbers.  Few rows make few blocks of many splits: kCols is
// small then, and kGroups of threads sum a range of the splits each.  The partials'
// bytes bound it where there are many rows: 27 us for 3405 x 4096 (59 MB of them);
// 32 x 1024 in 128 splits take 8 us (12 with one group).
// ---------------------------------------------------------------------------
template <int kCols, int kGroups>
__global__ __launch_bounds__(256 * kGroups) void dh_finish(const float* __restrict__ part,
                                                           int32_t num_tokens, int32_t ldc,
                                                           const u32x4* __restrict__ w,
                                                           u32x4* __restrict__ dh, char* ws,
                                                           LmheadBwdLayout lay,
                                                           int64_t blk_begin) {
  __shared__ float t[kGroups][kCols][kT + 1];  // [group of splits][k][i]
  const LiveRows live = live_rows(ws, lay);
  const int64_t blk = blk_begin + blockIdx.x;
  const int32_t k_tiles = ldc * 8 / kCols;
  const int32_t i0 = (int32_t)(blk / k_tiles) * kT;
  const int32_t kc0 = (int32_t)(blk % k_tiles) * (kCols / 8);
  const int32_t count = (int32_t)live.head[0];
  const DhParts parts(count, lay);
  const int64_t split_size = (int64_t)parts.rows * ldc * 8;
  const int tid = threadIdx.x & 255, group = threadIdx.x >> 8;
  const int32_t s0 = group * parts.splits / kGroups, s1 = (group + 1) * parts.splits / kGroups;
  if (i0 < count) {
    for (int q = tid; q < kT * kCols / 4; q += 256) {
      const int k = q >> 4, i = (q & 15) * 4;
      if (i0 + i >= count) continue;
      const float* p = part + (int64_t)(kc0 * 8 + k) * parts.rows + i0 + i;
      f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
      for (int32_t s = s0; s < s1; ++s)
        sum += *reinterpret_cast<const f32x4*>(p + s * split_size);
#pragma unroll
      for (int e = 0; e < 4; ++e) t[group][k][i + e] = sum[e];
    }
  }
  __syncthreads();
  const float scale = __uint_as_float(live.head[1]);
  for (int q = threadIdx.x; q < kT * kCols / 8; q += 256 * kGroups) {
    const int r = q / (kCols / 8), c = q % (kCols / 8);
    const int32_t at = i0 + r;
    if (at < num_tokens && live.inv[at] < 0) dh[(int64_t)at * ldc + kc0 + c] = u32x4{0, 0, 0, 0};
    if (at >= count) continue;
    const float rs = live.resid[at];
    union {
      uint16_t e[8];
      u32x4 x;
    } o, wr;
    wr.x = u32x4{0, 0, 0, 0};
    if (rs != 0.0f) wr.x = w[(int64_t)live.tgt[at] * ldc + kc0 + c];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float x = t[0][c * 8 + e][r];
#pragma unroll
      for (int g = 1; g < kGroups; ++g) x += t[g][c * 8 + e][r];
      if (rs != 0.0f) x = fmaf(rs, bf16_float(wr.e[e]), x);
      o.e[e] = bf16_bits(x * scale);
    }
    dh[(int64_t)live.idx[at] * ldc + kc0 + c] = o.x;
  }
}

__global__ __launch_bounds__(256) void fill_zero(u32x4* __restrict__ out, int64_t n,
                                                 int64_t begin) {
  const int64_t i = begin + (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) out[i] = u32x4{0, 0, 0, 0};
}

// Launches `blocks` blocks in pieces of at most the launch limit.
template <typename F>
hipError_t in_launches(int64_t blocks, int threads, F&& launch) {
  const int64_t most = launch_thread_limit() / threads;
  for (int64_t b = 0; b < blocks; b += most) {
    launch(b, blocks - b < most ? blocks - b : most);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace

// Pieces of equal size whose dz holds at most 2^28 elements (512 MiB of bf16), but
// at least 16384 columns; 4096 tokens take a 151936-column vocabulary in three.
// Small pieces leave part of the chip idle at the end of every launch (backward of
// 3405 live tokens: 11.1 ms in ten pieces, 10.95 in five, 10.75 in three, 10.7 in
// two).  Splits: enough blocks of dh for the chip's 256 CUs, but at least kSplitSlabs
// slabs to each.
constexpr int64_t kSplitSlabs = 4;

LmheadBwdLayout lmhead_bwd_layout(int64_t n, int64_t k, int64_t padded_vocab, bool want_dh,
                                  bool want_dw) {
  LmheadBwdLayout l{};
  const int64_t np = (n + 255) / 256 * 256;
  const int64_t blocks_v = (padded_vocab + 255) / 256;
  int64_t piece = (int64_t{1} << 28) / (np > 0 ? np : 1);
  piece = piece < 16384 ? 16384 : piece;
  const int64_t pieces = (blocks_v * 256 + piece - 1) / piece;
  piece = (blocks_v + pieces - 1) / pieces * 256;
  const int64_t blocks = np / 256 * ((k + 255) / 256);
  const int64_t most_splits = piece / (kBK * kSplitSlabs) > 1 ? piece / (kBK * kSplitSlabs) : 1;
  const int64_t want = n <= kFewLd ? 512 : 256;  // two blocks of dh_few fit a CU
  int64_t splits = blocks > 0 && blocks < want ? want / blocks : 1;
  splits = splits < most_splits ? splits : most_splits;
  l.padded_tokens = (int32_t)np;
  l.piece = (int32_t)piece;
  l.splits = (int32_t)splits;
  l.most_splits = (int32_t)most_splits;
  size_t at = 256;  // the status words
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  };
  l.head = take(8);
  l.idx = take(np * 4);
  l.tgt = take(np * 4);
  l.lse = take(np * 4);
  l.cg = take(np * 4);
  l.cc = take(np * 4);
  l.resid = take(np * 4);
  l.inv = take(n * 4);
  l.hc = take((size_t)np * k * 2);
  l.dz = take((size_t)np * piece * 2);
  if (want_dw) l.ht = take((size_t)np * k * 2);
  if (want_dw && n <= kFewLd) l.dzt = take((size_t)piece * kFewLd * 2);
  if (want_dh) {
    l.tail = take((size_t)kBK * k * 2);
    l.part = take((size_t)splits * np * k * 4);
  }
  l.total = at;
  return l;
}

hipError_t launch_fill_zero(void* out, int64_t bytes, hipStream_t stream) {
  const int64_t n = bytes / 16;
  return in_launches((n + 255) / 256, 256, [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL(fill_zero, dim3((unsigned)nb), dim3(256), 0, stream,
                       reinterpret_cast<u32x4*>(out), n, b * 256);
  });
}

namespace {

// One piece for few tokens.
template <int kTok>
hipError_t launch_few(const LmheadBwdArgs& a, const GradArgs& g, hipStream_t stream) {
  const LmheadBwdLayout& l = a.layout;
  const int32_t c0 = g.c0, piece = g.piece;
  char* ws = a.workspace;
  uint16_t* dzt = a.dweight ? reinterpret_cast<uint16_t*>(ws + l.dzt) : nullptr;
  const int32_t real = a.real_vocab - c0 < piece ? a.real_vocab - c0 : piece;
  if (real > 0) {
    const hipError_t e = in_launches(
        ((int64_t)real + kStreamRows - 1) / kStreamRows, kStreamThreads,
        [&](int64_t b, int64_t nb) {
          hipLaunchKernelGGL(dz_stream<kTok>, dim3((unsigned)nb), dim3(kStreamThreads), 0, stream,
                             ws + l.hc, static_cast<const char*>(a.weight), a.hidden_dim,
                             a.real_vocab, c0, piece, reinterpret_cast<uint16_t*>(ws + l.dz), dzt,
                             ws, l, b);
        });
    if (e != hipSuccess) return e;
  }
  if (a.dhidden && real > 0) {
    const int64_t n_k = (a.hidden_dim + kBB - 1) / kBB;
    const hipError_t e = in_launches(l.splits * n_k, kThreads, [&](int64_t b, int64_t nb) {
      hipLaunchKernelGGL(dh_few<kTok>, dim3((unsigned)nb), dim3(kThreads), 0, stream, g, ws, l, b);
    });
    if (e != hipSuccess) return e;
  }
  if (!a.dweight) return hipSuccess;
  return in_launches(piece / 64, 256, [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL(dw_few<kTok>, dim3((unsigned)nb), dim3(256), 0, stream,
                       reinterpret_cast<const uint16_t*>(ws + l.ht), dzt, a.hidden_dim,
                       a.real_vocab, a.padded_vocab, c0, l.padded_tokens,
                       static_cast<uint16_t*>(a.dweight), ws, l, b);
  });
}

}  // namespace

hipError_t launch_lmhead_bwd(const LmheadBwdArgs& a, hipStream_t stream) {
  const LmheadBwdLayout& l = a.layout;
  char* ws = a.workspace;
  const int32_t np = l.padded_tokens, k = a.hidden_dim, ldc = k / 8;
  u32x4* hc = reinterpret_cast<u32x4*>(ws + l.hc);
  uint16_t* dz = reinterpret_cast<uint16_t*>(ws + l.dz);
  uint16_t* ht = a.dweight ? reinterpret_cast<uint16_t*>(ws + l.ht) : nullptr;
  const u32x4* w = reinterpret_cast<const u32x4*>(a.weight);

  const RowArgs rows{a.targets, a.mask, a.lse, a.grad, a.grad_lse, a.status, a.num_tokens, np,
                     a.real_vocab, a.ignore_index};
  const bool scan = a.num_tokens <= kScanFew;
  hipError_t e;
  if (!scan) {
    hipLaunchKernelGGL(live_rows_scan, dim3(1), dim3(kScanThreads), 0, stream, rows, ws, l);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int32_t whole = a.real_vocab / kBK * kBK;
  GatherArgs ga;
  ga.h = reinterpret_cast<const u32x4*>(a.hidden);
  ga.hc = hc;
  ga.ht = ht;
  ga.w_tail = w + (int64_t)whole * ldc;
  ga.tail = reinterpret_cast<u32x4*>(ws + l.tail);
  ga.n_rows = (int64_t)(np / kT) * (k / kT);
  ga.tail_rows = a.dhidden ? a.real_vocab - whole : 0;
  ga.ldc = ldc;
  const int64_t tail_blocks = ga.tail_rows ? ((int64_t)kBK * ldc + 255) / 256 : 0;
  e = in_launches(ga.n_rows + tail_blocks, 256, [&](int64_t b, int64_t nb) {
    hipLaunchKernelGGL(scan ? gather_rows<true> : gather_rows<false>, dim3((unsigned)nb),
                       dim3(256), 0, stream, ga, rows, ws, l, b);
  });
  if (e != hipSuccess) return e;

  const int32_t n_k = (k + kBA - 1) / kBA, n_t = np / kBB;
  GradArgs g;
  g.dz = dz;
  g.ht = ht;
  g.w = static_cast<const uint16_t*>(a.weight);
  g.tail = reinterpret_cast<const uint16_t*>(ws + l.tail);
  g.part = reinterpret_cast<float*>(ws + l.part);
  g.dw = static_cast<uint16_t*>(a.dweight);
  g.hidden_dim = k;
  g.real_vocab = a.real_vocab;
  g.padded_vocab = a.padded_vocab;
  g.padded_tokens = np;
  const int few = a.num_tokens <= 16 ? 1 : a.num_tokens <= 32 ? 2 : a.num_tokens <= kFewLd ? 4 : 0;
  // pieces of the columns that need work: dW's rows go on to V_pad (as +0)
  const int32_t columns = a.dweight ? a.padded_vocab : a.real_vocab;
  for (int64_t begin = 0; begin < columns; begin += l.piece) {
    const int32_t c0 = (int32_t)begin;
    const int64_t left = (columns - begin + 255) / 256 * 256;
    const int32_t piece = left < l.piece ? (int32_t)left : l.piece;
    g.c0 = c0;
    g.piece = piece;
    g.add = c0 > 0;
    if (few) {
      e = few == 1   ? launch_few<1>(a, g, stream)
          : few == 2 ? launch_few<2>(a, g, stream)
                     : launch_few<4>(a, g, stream);
      if (e != hipSuccess) return e;
      continue;
    }
    if (c0 < a.real_vocab) {
      // tiles of 128 tokens where one holds them all (128 x 1024 x 151936: backward 305 us
      // for 331; 90 x 512 x 12003: 62 for 71)
      const bool narrow = a.num_tokens <= 128;
      const int64_t tiles = (int64_t)(piece / kBA) * (narrow ? 1 : n_t);
      e = in_launches(tiles, kThreads, [&](int64_t b, int64_t nb) {
        hipLaunchKernelGGL((narrow ? dz_piece<2> : dz_piece<4>), dim3((unsigned)nb),
                           dim3(kThreads), 0, stream, hc, w, k, a.real_vocab, c0, piece, dz, ws,
                           l, b);
      });
      if (e != hipSuccess) return e;
    }
    // a piece of padding only adds nothing to dh
    g.n_dh = a.dhidden && c0 < a.real_vocab ? (int64_t)l.splits * n_t * n_k : 0;
    g.n_dw = a.dweight ? (int64_t)(piece / kBB) * n_k : 0;
    e = in_launches(g.n_dh + g.n_dw, kThreads, [&](int64_t b, int64_t nb) {
      hipLaunchKernelGGL(grad_piece, dim3((unsigned)nb), dim3(kThreads), 0, stream, g, ws, l, b);
    });
    if (e != hipSuccess) return e;
  }
  if (a.dhidden) {
    const int32_t cols = few ? 16 : kT, groups = few ? 4 : 1;
    e = in_launches((int64_t)(np / kT) * (k / cols), 256 * groups, [&](int64_t b, int64_t nb) {
      hipLaunchKernelGGL((few ? dh_finish<16, 4> : dh_finish<kT, 1>), dim3((unsigned)nb),
                         dim3(256 * groups), 0, stream,
                         reinterpret_cast<const float*>(ws + l.part), a.num_tokens, ldc, w,
                         reinterpret_cast<u32x4*>(a.dhidden), ws, l, b);
    });
  }
  return e;
}

}  // namespace rlk
