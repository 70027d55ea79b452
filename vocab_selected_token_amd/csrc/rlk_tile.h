// rlk_tile.h -- the bf16 MFMA tile product shared by the LM-head kernels.
//
// A block of 512 threads computes C[a][b] = sum_k A[a][k] B[b][k] for 256 rows
// of A and 256 rows of B, both K-contiguous in memory.  With
// v_mfma_f32_16x16x32_bf16, lane l supplies row/col l%16 and k in
// [8*(l/16), 8*(l/16)+8) of a 32-wide k-step; accumulator i of lane l is
// C[4*(l/16) + i][l%16].  So each lane holds 4 A rows of one B row per 16x16
// tile, and a wave's A rows of one B row sit in the four lanes l%16 + 16g.  The
// 512 threads form 2 x 4 waves of 128 A rows x 64 B rows (8 x 4 MFMA tiles, 128
// fp32 accumulators per lane), two waves per SIMD, so one wave's MFMAs run
// while the other waits on memory.
//
// K advances in slabs of 64 (two k-steps) through two LDS stages filled by
// direct global-to-LDS loads (buffer_load_dwordx4 ... lds: lane i of an
// instruction writes bytes [16i, 16i + 16) after the wave's LDS base; the
// address is a buffer resource per operand based at the block's first row, a
// fixed 32-bit byte offset per lane and the slab's offset in a scalar
// register, so a load needs no address arithmetic).  LDS
// rows are 128 bytes with the 16-byte chunks XOR-swizzled by row -- chunk c of
// row r sits at position c ^ ((r >> 1) & 7) -- so that fragment reads of
// consecutive rows at one chunk spread over the bank groups; each load lane
// fetches the chunk that belongs at its position.  One barrier per slab, placed
// before the slab's last k-step: by then every wave has read the slab's
// fragments into registers, so the DMA for slab s+2 can go into the stage just
// released, and the first fragments of slab s+1 are read while the last k-step's
// MFMAs run.  Inside each k-step the next fragment reads (and the slab loads)
// are spread between the MFMAs.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rlk {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
// 16 bytes as a native vector: arrays of it stay in registers (HIP's uint4 is
// a struct around a union, which keeps arrays of it in scratch memory)
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNegInf = -__builtin_huge_valf();

constexpr int kThreads = 512;
constexpr int kWaves = kThreads / 64;
constexpr int kBA = 256;  // rows of A per block
constexpr int kBB = 256;  // rows of B per block
constexpr int kRowBytes = 128;  // one row of a slab: 64 bf16, 8 chunks of 16 bytes
constexpr int kBK = kRowBytes / 2;
constexpr int kSlabBytes = kBA * kRowBytes;  // one operand, one stage
constexpr int kTileLds = 2 * 2 * kSlabBytes;
constexpr int kRowsPerLoad = 64 / (kRowBytes / 16);  // 8 rows per load instruction
constexpr int kRowsPerWave = kBA / kWaves;           // 32 rows of each operand per wave
constexpr int kLoads = kRowsPerWave / kRowsPerLoad;  // 4 instructions per operand per slab
constexpr int kVS = 8;  // 16-row tiles of A per wave
constexpr int kTS = 4;  // 16-row tiles of B per wave

static_assert(kBA == kBB, "the load mapping assumes square blocks");

typedef __attribute__((address_space(3))) void* lds_ptr;

// Word 3 of a raw (untyped) buffer resource on gfx9: 32-bit data format, no
// swizzle, no thread-id addressing.
constexpr int kBufferWord3 = 0x00020000;

// s_waitcnt immediate with lgkmcnt = 0 and the other counters at their maxima
constexpr int kWaitLds = 0xC07F;

// LDS position (in 16-byte units) of chunk c of row r inside one operand stage.
__device__ __forceinline__ int swizzled(int r, int c) { return r * 8 + (c ^ ((r >> 1) & 7)); }

__device__ __forceinline__ float maxnan(float a, float b) {
  return __builtin_elementwise_maximum(a, b);
}
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// Consecutive work indices on one XCD (blocks are dealt to the 8 XCDs in turn).
__device__ __forceinline__ int64_t xcd_local_block(int64_t b, int64_t nb) {
  constexpr int64_t kXcds = 8;
  const int64_t per = nb / kXcds, rem = nb % kXcds, x = b % kXcds, l = b / kXcds;
  return x * per + (x < rem ? x : rem) + l;
}

// One operand's slab loads.  Wave w moves rows [32w, 32w + 32), 8 rows per
// instruction; lane i of instruction j fetches row 32w + 8j + i/8 at the chunk
// that belongs at LDS position i%8.  The resource starts at `first` and covers
// `rows` (1..256) rows of row_bytes; block row r reads row r + shift of them,
// clamped into [0, rows): rows outside are never read.  256 rows span less than
// 2^31 bytes (the boundary limits hidden_dim).
struct TileOperand {
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t off[kLoads];  // byte offsets from the resource's base

  __device__ __forceinline__ TileOperand(const void* first, int64_t row_bytes, int32_t rows,
                                         int32_t shift, int wave, int lane) {
    rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(first), 0,
                                             (int)((int64_t)rows * row_bytes), kBufferWord3);
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int row = wave * kRowsPerWave + j * kRowsPerLoad + (lane >> 3);
      const int c = (lane & 7) ^ ((row >> 1) & 7);
      off[j] = (uint32_t)((int64_t)min(max(row + shift, 0), rows - 1) * row_bytes + c * 16);
    }
  }

  // the slab at byte `soff` of the rows into the LDS stage at `stage`
  __device__ __forceinline__ void issue(char* stage, int wave, uint32_t soff) const {
    char* base = stage + (wave * kRowsPerWave) * kRowBytes;
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc,
                                               (lds_ptr)(base + j * kRowsPerLoad * kRowBytes), 16,
                                               off[j], soff, 0, 0);
  }
};

// acc = the product over the slabs [slab0, slab0 + nslab) (nslab >= 1) of the
// operands' rows.  smem: kTileLds bytes, free for other use on return (every
// load has landed and every wave has passed the last barrier).
__device__ __forceinline__ void tile_product(char* smem, const TileOperand& A,
                                             const TileOperand& B, int slab0, int nslab, int wave,
                                             int lane, f32x4 (&acc)[kVS][kTS]) {
  const int wv = wave >> 2;  // half of A's rows
  const int wt = wave & 3;   // quarter of B's rows
#pragma unroll
  for (int a = 0; a < kVS; ++a)
#pragma unroll
    for (int b = 0; b < kTS; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[a][b][i] = 0.0f;

  // slab `slab` into LDS stage `stage` (A rows at the stage base, B rows after);
  // all A rows, then all B rows (about 0.6% faster than alternating)
  auto issue = [&](int slab, int stage) __attribute__((always_inline)) {
    char* base = smem + stage * 2 * kSlabBytes;
    const uint32_t soff = (uint32_t)(slab0 + slab) * kRowBytes;  // the slab's bytes in a row
    A.issue(base, wave, soff);
    B.issue(base + kSlabBytes, wave, soff);
  };
  // fragment reads of k-step ks: lane l takes row l%16 of each 16-row tile at
  // chunk 4ks + l/16 (k in [32ks + 8(l/16), +8))
  const int frag_row = lane & 15;
  const int frag_c = lane >> 4;
  auto fetch = [&](const char* As, int ks, bf16x8 (&af)[kVS], bf16x8 (&bf)[kTS])
      __attribute__((always_inline)) {
    const char* Bs = As + kSlabBytes;
#pragma unroll
    for (int vs = 0; vs < kVS; ++vs)
      af[vs] = *reinterpret_cast<const bf16x8*>(
          As + swizzled(wv * 128 + vs * 16 + frag_row, ks * 4 + frag_c) * 16);
#pragma unroll
    for (int ts = 0; ts < kTS; ++ts)
      bf[ts] = *reinterpret_cast<const bf16x8*>(
          Bs + swizzled(wt * 64 + ts * 16 + frag_row, ks * 4 + frag_c) * 16);
  };
  auto mma = [&](const bf16x8 (&af)[kVS], const bf16x8 (&bf)[kTS]) __attribute__((always_inline)) {
#pragma unroll
    for (int vs = 0; vs < kVS; ++vs)
#pragma unroll
      for (int ts = 0; ts < kTS; ++ts)
        acc[vs][ts] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[vs], bf[ts], acc[vs][ts], 0, 0, 0);
  };
  // Instruction order inside a k-step: 4 MFMAs, then one fragment read (and,
  // after the barrier, one slab load) per 2 MFMAs, then the remaining MFMAs.
  // The reads thus overlap the MFMAs that do not need them.
  constexpr int kReads = kVS + kTS, kMfmas = kVS * kTS, kLead = 4, kPer = 2;
  static_assert(kLead + kPer * kReads <= kMfmas, "the reads fit inside the step");
  static_assert(2 * kLoads <= kReads, "one load per read at most");
  auto order_step = [&](bool with_loads) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_group_barrier(0x008, kLead, 0);  // MFMA
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
      if (with_loads && i < 2 * kLoads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM
      __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, kMfmas - kLead - kPer * kReads, 0);
  };

  issue(0, 0);
  if (nslab > 1) issue(1, 1);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  bf16x8 a0[kVS], b0[kTS], a1[kVS], b1[kTS];
  fetch(smem, 0, a0, b0);
  for (int s = 0; s < nslab; ++s) {
    const char* cur = smem + (s & 1) * 2 * kSlabBytes;
    const char* nxt = smem + ((s + 1) & 1) * 2 * kSlabBytes;
    // the fragments of this k-step were read during the previous one; wait for
    // them before more reads go out (the LDS counter holds at most 15)
    __builtin_amdgcn_s_waitcnt(kWaitLds);
    fetch(cur, 1, a1, b1);
    mma(a0, b0);
    order_step(false);
    __builtin_amdgcn_sched_barrier(0);
    // every wave has read slab s into registers, and slab s+1 (issued one
    // slab ago) has landed in the other stage
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    __builtin_amdgcn_sched_barrier(0);
    // slab s+2 into the stage just released.  The last two steps reload slab
    // nslab-1 there and read the other stage's first fragments, which nothing
    // uses: the loads and reads stay unconditional, so they can be interleaved
    // with the MFMAs, and stay in bounds.
    issue(min(s + 2, nslab - 1), s & 1);
    fetch(nxt, 0, a0, b0);
    mma(a1, b1);
    order_step(true);
    __builtin_amdgcn_sched_barrier(0);
  }
  // the reloads of the last two steps land before the epilogue reuses the stages
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
}

}  // namespace
}  // namespace rlk
