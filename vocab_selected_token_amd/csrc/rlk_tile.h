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
//
// B may also lie the other way in memory (TileOperandT): rows of the sum's index,
// its own index contiguous.  A slab is then 64 rows of 512 bytes, and a fragment
// comes from two transposing LDS reads (ds_read_b64_tr_b16): of 16 lanes, lane i
// names 4 consecutive columns (4 (i % 4) on) of row i/4, and gets column i of the
// four rows.  The product runs as fast as with both operands along the sum, and saves
// the copy.  The chunks of row r are XOR-swizzled by 2 (r % 4) + 8 (r / 8 % 2):
// the 8 rows that 32 lanes read at once lie 32 bytes apart over all 64 banks.
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

// One operand's slab loads.  Wave w moves rows [32w, 32w + 32), 8 rows per
// instruction; lane i of instruction j fetches row 32w + 8j + i/8 at the chunk
// that belongs at LDS position i%8.  The resource starts at `first` and covers
// `rows` (1..256) rows of row_bytes; block row r reads row r + shift of them,
// clamped into [0, rows): rows outside are never read.  256 rows span less than
// 2^31 bytes (the boundary limits hidden_dim).  (kLoadsT: 8 kLoadsT rows a wave,
// for tiles of fewer rows.)
template <int kLoadsT>
struct TileOperandOf {
  static constexpr int kLoads = kLoadsT;
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t off[kLoadsT];  // byte offsets from the resource's base

  __device__ __forceinline__ TileOperandOf(const void* first, int64_t row_bytes, int32_t rows,
                                           int32_t shift, int wave, int lane) {
    rsrc = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(first), 0,
                                             (int)((int64_t)rows * row_bytes), kBufferWord3);
#pragma unroll
    for (int j = 0; j < kLoadsT; ++j) {
      const int row = wave * (kRowsPerLoad * kLoadsT) + j * kRowsPerLoad + (lane >> 3);
      const int c = (lane & 7) ^ ((row >> 1) & 7);
      off[j] = (uint32_t)((int64_t)min(max(row + shift, 0), rows - 1) * row_bytes + c * 16);
    }
  }

  static constexpr int kReadsPerFragment = 1;

  // slab `slab` into the LDS stage at `stage`
  __device__ __forceinline__ void issue(char* stage, int wave, int slab) const {
    const uint32_t soff = (uint32_t)slab * kRowBytes;  // the slab's bytes in a row
    char* base = stage + wave * (kRowsPerLoad * kLoadsT) * kRowBytes;
#pragma unroll
    for (int j = 0; j < kLoadsT; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rsrc,
                                               (lds_ptr)(base + j * kRowsPerLoad * kRowBytes), 16,
                                               off[j], soff, 0, 0);
  }

  // The fragment of the 16 rows from `row` on for k-step ks: lane l takes row
  // l%16 at chunk 4ks + l/16 (k in [32ks + 8(l/16), +8)).
  static __device__ __forceinline__ bf16x8 fragment(const char* stage, int row, int ks, int lane) {
    return *reinterpret_cast<const bf16x8*>(
        stage + swizzled(row + (lane & 15), ks * 4 + (lane >> 4)) * 16);
  }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

// The restrict pointer tells the compiler that the read's memory is its own:
// without that (or a type to tell it by) it takes every direct load in flight for
// a write to what is read here, and waits for it.  tile_product's barrier and
// waits keep the two apart.
__device__ __forceinline__ s16x4 transposed_read(lds_s16x4 __restrict__ at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(at);
}

typedef TileOperandOf<kLoads> TileOperand;

// An operand whose rows are the sum's index: row k of the slab holds B[0..255][k]
// (kCols of them).  Of 256, wave w moves rows [8w, 8w + 8) of a slab, 2 per instruction;
// lane i of instruction j fetches row 8w + 2j + i/32 at the chunk that belongs at position
// i%32.  Columns from `cols` (a multiple of 8) on are never read: clamped.  Slab
// tail_slab, if any, is read at `tail` (64 whole rows) instead: the one that the
// last rows do not fill.
template <int kCols, int kWavesT>
struct TileOperandTOf {
  const char* first;
  const char* tail;
  int tail_slab;
  int64_t slab_bytes;

  static constexpr int kRowBytesT = kCols * 2;
  static constexpr int kReadsPerFragment = 2;
  static constexpr int kChunks = kCols / 8;            // of 16 bytes, per row
  static constexpr int kRowsPerLoadT = 64 / kChunks;   // rows per load instruction
  static constexpr int kRowsPerWaveT = kBK / kWavesT;
  static constexpr int kLoads = kRowsPerWaveT / kRowsPerLoadT;
  uint32_t off[kLoads];

  // (64 columns: rows are half as long as the banks, so odd rows lie apart from even ones)
  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (kChunks == 8) return (row & 2) | (((row >> 3) & 1) << 2);
    return ((row & 3) << 1) | (((row >> 3) & 1) << 3);
  }
  static_assert(kChunks >= 8, "a chunk stays in its row");

  __device__ __forceinline__ TileOperandTOf(const void* first_, int64_t row_bytes, int32_t cols,
                                            const void* tail_, int tail_slab_, int wave, int lane)
      : first(static_cast<const char*>(first_)),
        tail(static_cast<const char*>(tail_)),
        tail_slab(tail_slab_),
        slab_bytes(kBK * row_bytes) {
#pragma unroll
    for (int j = 0; j < kLoads; ++j) {
      const int row = wave * kRowsPerWaveT + j * kRowsPerLoadT + lane / kChunks;
      const int c = min((lane % kChunks) ^ swizzle(row), cols / 8 - 1);
      off[j] = (uint32_t)(row * row_bytes + c * 16);
    }
  }

  __device__ __forceinline__ void issue(char* stage, int wave, int slab) const {
    // (a select, not a branch: the loads stay among the MFMAs)
    const int64_t from_tail = -(int64_t)(slab == tail_slab);
    const char* at = first + ((slab * slab_bytes & ~from_tail) | ((tail - first) & from_tail));
    const __amdgpu_buffer_rsrc_t rsrc = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<char*>(at), 0, (int)slab_bytes, kBufferWord3);
    char* base = stage + wave * kRowsPerWaveT * kRowBytesT;
#pragma unroll
    for (int j = 0; j < kLoads; ++j)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          rsrc, (lds_ptr)(base + j * kRowsPerLoadT * kRowBytesT), 16, off[j], 0, 0, 0);
  }

  static __device__ __forceinline__ bf16x8 fragment(const char* stage, int row, int ks, int lane) {
    const int i = lane & 15;
    // the lane's row in the k-step's first four of its eight, and its column
    const int r = ks * 32 + (lane >> 4) * 8 + (i >> 2), col = row + (i & 3) * 4;
    const char* at = stage + r * kRowBytesT + ((col >> 3) ^ swizzle(r)) * 16 + (col & 7) * 2;
    union {
      s16x4 half[2];
      bf16x8 whole;
    } f;
    // rows 4 apart have the same swizzle
    f.half[0] = transposed_read((lds_s16x4)at);
    f.half[1] = transposed_read((lds_s16x4)(at + 4 * kRowBytesT));
    return f.whole;
  }
};

typedef TileOperandTOf<kBB, kWaves> TileOperandT;

// LDS of a tile whose B has 64 kTok rows (each wave takes 16 kTok of them).
template <int kTok>
constexpr int kStageBytes = kSlabBytes + 64 * kTok * kRowBytes;

// acc = the product over the slabs [slab0, slab0 + nslab) (nslab >= 1) of the
// operands' rows, by waves of 16 kVSn rows of A x 16 kTok of B, kWB of them along B and two
// along A.  smem: two stages, free for other use on return (every load has landed and
// every wave has passed the last barrier).
template <int kWB = 4, int kVSn, int kTok, typename OperandA, typename OperandB>
__device__ __forceinline__ void tile_product(char* smem, const OperandA& A, const OperandB& B,
                                             int slab0, int nslab, int wave, int lane,
                                             f32x4 (&acc)[kVSn][kTok]) {
  constexpr int kSlabA = 2 * 16 * kVSn * kRowBytes;
  constexpr int kStage = kSlabA + kWB * 16 * kTok * kRowBytes;
  const int wv = wave / kWB;  // half of A's rows
  const int wt = wave % kWB;  // part of B's rows
#pragma unroll
  for (int a = 0; a < kVSn; ++a)
#pragma unroll
    for (int b = 0; b < kTok; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[a][b][i] = 0.0f;

  // slab `slab` into LDS stage `stage` (A rows at the stage base, B rows after);
  // all A rows, then all B rows (about 0.6% faster than alternating)
  auto issue = [&](int slab, int stage) __attribute__((always_inline)) {
    char* base = smem + stage * kStage;
    A.issue(base, wave, slab0 + slab);
    B.issue(base + kSlabA, wave, slab0 + slab);
  };
  auto fetch = [&](const char* As, int ks, bf16x8 (&af)[kVSn], bf16x8 (&bf)[kTok])
      __attribute__((always_inline)) {
    const char* Bs = As + kSlabA;
#pragma unroll
    for (int vs = 0; vs < kVSn; ++vs)
      af[vs] = OperandA::fragment(As, wv * (16 * kVSn) + vs * 16, ks, lane);
#pragma unroll
    for (int ts = 0; ts < kTok; ++ts)
      bf[ts] = OperandB::fragment(Bs, wt * (16 * kTok) + ts * 16, ks, lane);
  };
  auto mma = [&](const bf16x8 (&af)[kVSn], const bf16x8 (&bf)[kTok])
      __attribute__((always_inline)) {
#pragma unroll
    for (int vs = 0; vs < kVSn; ++vs)
#pragma unroll
      for (int ts = 0; ts < kTok; ++ts)
        acc[vs][ts] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(af[vs], bf[ts], acc[vs][ts], 0, 0, 0);
  };
  // Instruction order inside a k-step: 4 MFMAs, then one LDS read (and, after the
  // barrier, one slab load) per 2 MFMAs -- per MFMA, where fragments take two reads,
  // and in narrower tiles -- then the remaining MFMAs.  The reads thus overlap
  // the MFMAs that do not need them.  (With fewer MFMAs than reads the order is left to the
  // compiler.)
  constexpr int kReads = OperandA::kReadsPerFragment * kVSn + OperandB::kReadsPerFragment * kTok,
                kMfmas = kVSn * kTok;
  constexpr int kPer = 4 + 2 * kReads <= kMfmas ? 2 : 1;
  constexpr int kSpare = kMfmas - kPer * kReads, kLead = kSpare < 4 ? kSpare : 4;
  constexpr int kSlabLoads = OperandA::kLoads + OperandB::kLoads;
  static_assert(kSpare < 0 || kSlabLoads <= kReads, "one load per read at most");
  auto order_step = [&](bool with_loads) __attribute__((always_inline)) {
    if constexpr (kSpare < 0) return;
    __builtin_amdgcn_sched_group_barrier(0x008, kLead, 0);  // MFMA
#pragma unroll
    for (int i = 0; i < kReads; ++i) {
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // LDS read
      if (with_loads && i < kSlabLoads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);  // VMEM
      __builtin_amdgcn_sched_group_barrier(0x008, kPer, 0);
    }
    __builtin_amdgcn_sched_group_barrier(0x008, kSpare - kLead, 0);
  };

  issue(0, 0);
  if (nslab > 1) issue(1, 1);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  bf16x8 a0[kVSn], b0[kTok], a1[kVSn], b1[kTok];
  fetch(smem, 0, a0, b0);
  for (int s = 0; s < nslab; ++s) {
    const char* cur = smem + (s & 1) * kStage;
    const char* nxt = smem + ((s + 1) & 1) * kStage;
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
