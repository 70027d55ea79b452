// rlk_internal.h -- launch arguments shared by the boundary and the kernels.
// Internal to librlk_logp.so; every field has been validated by the boundary
// before a launcher sees it.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rlk {

struct Stage1Args {
  const void* logits;  // bf16 [num_rows, ld]
  int64_t ld;          // elements, multiple of 8
  int32_t num_rows;
  int32_t real_vocab;
  int32_t padded_vocab;
  int32_t num_tiles;
  int32_t tile_width;  // V_pad / T if exact, else 0
  int32_t tile_begin;  // this virtual shard's tiles
  int32_t tile_count;
  float* pmax;  // [num_rows][num_tiles]
  float* psum;
  float* pent;  // entropy statistic [num_rows][num_tiles], or null
};

struct Stage2Args {
  const void* logits;           // bf16 logits for the target gather, or
  const float* target_logit;    // if non-null: the fp32 target logit of each row
  int64_t ld;
  int32_t num_rows;
  int32_t real_vocab;
  int32_t num_tiles;
  const float* pmax;
  const float* psum;
  const float* pent;  // with entropy: the stage-1 entropy statistic
  const int32_t* targets;
  const uint8_t* mask;  // may be null
  int32_t ignore_index;
  float* logp;
  float* lse;
  float* entropy;  // per-row entropy out, or null
  uint32_t* status;
};

struct BwdArgs {
  const void* logits;
  int64_t ld;
  int32_t num_rows;
  int32_t real_vocab;
  int32_t padded_vocab;
  const int32_t* targets;
  const uint8_t* mask;  // may be null
  int32_t ignore_index;
  const float* lse;
  const float* grad;      // may be null with grad_lse or grad_ent given
  const float* grad_lse;  // null = zero
  const float* grad_ent;  // null = zero
  const float* entropy;   // read where grad_ent is nonzero
  void* dlogits;
  int64_t ld_d;
  bool out_bf16;
  uint32_t* status;
};

// Forward and backward in one launch (g known before the forward): one block
// per row keeps the row's tile partials in LDS, so T is bounded.
constexpr int32_t kFbMaxTiles = 1024;

struct FwdBwdArgs {
  const void* logits;
  int64_t ld;
  int32_t num_rows;
  int32_t real_vocab;
  int32_t padded_vocab;
  int32_t num_tiles;
  int32_t tile_width;  // V_pad / T if exact, else 0
  const int32_t* targets;
  const uint8_t* mask;  // may be null
  int32_t ignore_index;
  const float* grad;
  float* logp;
  float* lse;
  void* dlogits;
  int64_t ld_d;
  bool out_bf16;
  uint32_t* status;
  // Unit schedule: [num_rows][num_tiles] 64-bit partial slots (two such arrays
  // with the entropy), or null for the one-block-per-row schedule (the same
  // bits either way).
  uint64_t* slots;
  // The extended form (unit schedule only): entropy out [num_rows] (non-null:
  // the forward of rlk_logp_fwd_ex); grad_lse / grad_ent (either non-null: the
  // gradient of rlk_logp_bwd_ex, with grad, grad_lse and grad_ent each null =
  // zero).
  float* entropy = nullptr;
  const float* grad_lse = nullptr;
  const float* grad_ent = nullptr;
};

// Whether the unit schedule of the one-launch forward+backward takes this
// geometry: T <= 64, tiles of at least 8 columns, and every tile's full
// chunks within the passes a lane group keeps in registers.
bool fwd_bwd_units_fit(int32_t real_vocab, int32_t padded_vocab, int32_t num_tiles);
// Polls of a row's partial slots before a block computes them itself (read
// once per process: RLK_FB_SPIN_LIMIT, default 16384; 0 makes every block
// compute its row's partials itself -- a hook for tests).
int32_t fwd_bwd_spin_limit();

// Fused LM-head variant: vocabulary rows per GEMM block (tiles must be at
// least this wide, so a block holds at most one tile bound).
constexpr int32_t kLmheadBlockVocab = 256;
constexpr int32_t kLmheadSlabK = 64;  // hidden_dim must be a multiple of this
// and at most this: a block's 256 rows of one operand then span under 2^31
// bytes, the range of the buffer resource its loads go through
constexpr int64_t kLmheadMaxHidden = int64_t{1} << 21;

struct LmheadArgs {
  const void* hidden;  // bf16 [num_tokens, hidden_dim]
  const void* weight;  // bf16 [>= real_vocab, hidden_dim]
  int32_t hidden_dim;
  int32_t num_tokens;
  int32_t real_vocab;
  int32_t padded_vocab;
  int32_t num_tiles;
  int32_t num_shards;  // virtual shards: launched one after another
  const int32_t* targets;
  const uint8_t* mask;  // may be null
  int32_t ignore_index;
  float* seg_m;  // [num_tokens][2 * ceil(real_vocab / 256)]
  float* seg_s;
  float* target_logit;  // [num_tokens]
  float* pmax;          // [num_tokens][num_tiles]
  float* psum;
};

// Where a block's statistics go, and what they cover.
struct SegmentArgs {
  int32_t num_tokens;
  int32_t padded_vocab;
  int32_t num_tiles;
  int32_t n_vb;            // vocabulary blocks of the whole problem
  int32_t row_lo, row_hi;  // the shard's real rows: others neither read nor counted
  int32_t col_lo, col_hi;  // the shard's columns: it writes the slots that start there
  const int32_t* __restrict__ targets;
  const uint8_t* __restrict__ mask;
  int32_t ignore_index;
  float* __restrict__ seg_m;  // [num_tokens][2 * n_vb]
  float* __restrict__ seg_s;
  float* __restrict__ tlogit;  // [num_tokens]
};

// A matrix in 8-bit floating point: columns that share a scale.
constexpr int32_t kFp8Block = 128;

struct Fp8QuantizeArgs {
  const void* x;  // bf16 [rows, ld]
  int64_t ld;
  int64_t rows;
  int64_t cols;        // a multiple of 128
  int32_t block_rows;  // 1 or 128
  void* q;             // e4m3 [rows, cols]
  float* scale;        // (row block, column block) at these strides
  int64_t scale_row_stride;
  int64_t scale_col_stride;
};

// Up to this many tokens the 8-bit LM-head streams the weight, and its statistics
// take z (fp32) through the workspace.
constexpr int32_t kFp8FewTokens = 64;

// The operands of an 8-bit LM-head.
struct LmheadFp8Args {
  const void* hidden_q;       // e4m3 [num_tokens, hidden_dim]
  const float* hidden_scale;  // (token, column block)
  const void* weight_q;       // e4m3 [>= real_vocab, hidden_dim]
  const float* weight_scale;  // (128-row block, column block)
  int64_t hidden_row_stride, hidden_col_stride;
  int64_t weight_row_stride, weight_col_stride;
  int32_t hidden_dim;
  float* z;  // statistics of few tokens: [num_tokens][real_vocab rounded up to 256]
};

// Gradients of the fused LM-head.  Byte offsets into its workspace (the status
// words come first): what is known of the live rows, their hidden states by
// tokens and by columns, a piece of dz (also by columns, for few tokens), the
// weight's last rows and the fp32 partials of dh.
struct LmheadBwdLayout {
  int32_t padded_tokens;  // num_tokens rounded up to 256
  int32_t piece;          // vocabulary columns at a time (a multiple of 256)
  int32_t splits;         // dh: parts a piece's columns are summed in, if all rows are live
  int32_t most_splits;    // and at most, if not
  size_t head, idx, tgt, lse, cg, cc, resid, inv;
  size_t hc, ht, dz, dzt, tail, part, total;
};

// ht rows of padded_tokens elements must span under 2^31 bytes by 256.
constexpr int64_t kLmheadBwdMaxTokens = int64_t{1} << 21;

struct LmheadBwdArgs {
  const void* hidden;  // bf16 [num_tokens, hidden_dim]
  const void* weight;  // bf16 [>= real_vocab, hidden_dim]
  int32_t hidden_dim;
  int32_t num_tokens;
  int32_t real_vocab;
  int32_t padded_vocab;
  const int32_t* targets;
  const uint8_t* mask;  // may be null
  int32_t ignore_index;
  const float* lse;
  const float* grad;      // null = zero
  const float* grad_lse;  // null = zero
  void* dhidden;          // bf16 [num_tokens, hidden_dim], or null: not wanted
  void* dweight;          // bf16 [padded_vocab, hidden_dim], or null: not wanted
  char* workspace;
  LmheadBwdLayout layout;
  uint32_t* status;
};

// What a sampler does to logits (rlk_logits_rules).
struct RuleArgs {
  const float* repetition;  // [num_rows] each, or null: 1, 0, 0, 1
  const float* presence;
  const float* frequency;
  const float* temperature;
  const int32_t* history;  // null: none
  int64_t history_len;
  const int64_t* history_begin;  // [num_rows]
  const int64_t* history_split;  // null: no prompt
  const int64_t* history_end;
  const float* bias;  // [bias_rows][ld_bias], or null
  int64_t bias_rows, ld_bias;
  const int32_t* bias_index;  // null: row r, or the only one
  const uint32_t* allow;  // [allow_rows][ld_allow], a bit per column, or null
  int64_t allow_rows, ld_allow;
  const int32_t* allow_index;
};

constexpr int32_t kProcessPiece = 2048;  // columns whose statistics are one partial

struct ProcessedArgs {
  const void* logits;  // bf16 [num_rows, ld]
  int64_t ld;
  int32_t num_rows;
  int32_t real_vocab;
  int32_t padded_vocab;
  int32_t pieces;  // ceil(real_vocab / kProcessPiece)
  const int32_t* targets;
  const uint8_t* mask;  // may be null
  int32_t ignore_index;
  float* pmax;  // [num_rows][pieces]
  float* psum;
  float* target_logit;  // [num_rows]
  float* logp;
  float* lse;
  const float* grad;      // null = zero
  const float* grad_lse;  // null = zero
  uint32_t* status;
};

// A dense product with its epilogue: out = residual + act(x . weight^T + bias).
enum Activation : int32_t { kActNone, kActRelu, kActGelu, kActGeluTanh, kActSilu, kActSoftcap };
constexpr int64_t kLinearMaxOut = int64_t{1} << 21;  // with a backward pass

struct LinearArgs {
  const void* x;       // bf16 [tokens, in_dim]
  const void* weight;  // bf16 [out_dim, in_dim]
  const void* bias;    // [out_dim], or null
  bool bias_bf16;
  const void* residual;  // bf16 [tokens, ld_residual], or null
  int64_t ld_residual;
  int32_t tokens, in_dim, out_dim, padded_out;
  int32_t activation;
  float cap;
  void* out;  // bf16 [tokens, ld_out]
  int64_t ld_out;
  void* saved;  // fp16 or float [tokens, ld_saved], or null
  bool saved_f32;
  int64_t ld_saved;
};

// Byte offsets into the workspace of the backward pass.
struct LinearBwdLayout {
  int32_t rows, cols;  // of dz: tokens and out_dim rounded up to 64
  int32_t row_blocks;  // partials of the bias' gradient
  size_t dz, x_tail, w_tail, bias_part, total;
};

struct LinearBwdArgs {
  LinearArgs f;   // x, weight, sizes, activation, saved
  const void* dy;  // bf16 [tokens, ld_dy]
  int64_t ld_dy;
  void* dx;       // bf16 [tokens, in_dim], or null
  void* dweight;  // bf16 [out_dim, in_dim], or null
  void* dbias;    // [out_dim], or null
  char* workspace;
  LinearBwdLayout layout;
};

// Most threads one launch may have.  A dispatch holds its grid size in 32 bits
// of threads: at 2^32 the launch fails, and above it the size wraps around and
// the kernel silently runs on a fraction of the grid.  Every launcher splits
// its work into launches of at most this many threads (2^31, or less when the
// RLK_MAX_LAUNCH_THREADS environment variable says so at the process's first
// launch -- a hook for tests, which check that any split gives the same bits).
int64_t launch_thread_limit();

// Launches `blocks` blocks of `threads` in pieces of at most that limit: launch(first block,
// how many).
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

// The allocation-free forward's workspace: a device array of the library's own,
// one per GPU, of this many bytes (status words plus 2 * N * T fp32 partials:
// N * T <= 4,194,304, e.g. 65,536 rows of 64 tiles).
constexpr size_t kNoAllocScratchBytes = (size_t{32} << 20) + 256;
// Its device address on the current device (looked up once per device).
hipError_t noalloc_scratch(void** ptr);

// Tokens of an LM-head tile, in 64s (2 to 4), for n tokens and n_vbs vocabulary blocks:
// unit is the time of a round -- the chip's 256 CUs, a block each -- of such tiles.  The
// last round of blocks and the last tile of tokens are paid in full, which narrower
// tiles may save; one has to be clearly ahead, for it reads the weight more often.
inline int tile_tokens(int32_t n, int32_t n_vbs, const double (&unit)[3]) {
  int best = 4;
  double least = 0.0;
  for (int k = 4; k >= 2; --k) {
    const int64_t blocks = (int64_t)n_vbs * (((int64_t)n + 64 * k - 1) / (64 * k));
    const double cost = (double)((blocks + 255) / 256) * unit[k - 2];
    if (k == 4 || cost < 0.95 * least) {
      least = cost;
      best = k;
    }
  }
  return best;
}

int64_t stage1_blocks(int64_t items);
int64_t lmhead_grid_blocks(int32_t num_tokens, int32_t real_vocab);
// The LM-head's segments, tile partials and stage-2 merge; with fp8 its operands (a.hidden and
// a.weight are not used).
hipError_t launch_lmhead(const LmheadArgs& a, const LmheadFp8Args* fp8, const Stage2Args& a2,
                         hipStream_t stream);
// One shard's segments: the blocks [vb_begin, vb_begin + n_vbs) of the grid.
hipError_t launch_segments_fp8(const LmheadFp8Args& f, const SegmentArgs& sa, int32_t vb_begin,
                               int32_t n_vbs, hipStream_t stream);
hipError_t launch_logits_fp8(const LmheadFp8Args& f, int32_t num_tokens, int32_t real_vocab,
                             int32_t padded_vocab, void* logits, int64_t ld, hipStream_t stream);
hipError_t launch_fp8_quantize(const Fp8QuantizeArgs& a, hipStream_t stream);
LmheadBwdLayout lmhead_bwd_layout(int64_t num_tokens, int64_t hidden_dim, int64_t padded_vocab,
                                  bool want_dhidden, bool want_dweight);
hipError_t launch_lmhead_bwd(const LmheadBwdArgs& a, hipStream_t stream);
hipError_t launch_fill_zero(void* out, int64_t bytes, hipStream_t stream);  // bytes % 16 == 0
int64_t bwd_col_blocks(int32_t padded_vocab);
hipError_t launch_stage1(const Stage1Args& a, hipStream_t stream);
hipError_t launch_stage2(const Stage2Args& a, hipStream_t stream);
hipError_t launch_bwd(const BwdArgs& a, hipStream_t stream);
hipError_t launch_fwd_bwd(const FwdBwdArgs& a, hipStream_t stream);
hipError_t launch_process(const void* logits, int64_t ld, int32_t num_rows, int32_t real_vocab,
                          int32_t padded_vocab, const RuleArgs& rules, void* out, int64_t ld_out,
                          bool out_bf16, hipStream_t stream);
hipError_t launch_processed_fwd(const ProcessedArgs& a, const RuleArgs& rules, hipStream_t stream);
hipError_t launch_processed_bwd(const ProcessedArgs& a, const RuleArgs& rules, void* dlogits,
                                int64_t ld_d, bool out_bf16, hipStream_t stream);
hipError_t launch_linear_fwd(const LinearArgs& a, hipStream_t stream);
LinearBwdLayout linear_bwd_layout(int64_t tokens, int64_t in_dim, int64_t out_dim);
hipError_t launch_linear_bwd(const LinearBwdArgs& a, hipStream_t stream);
hipError_t launch_clear_status(uint32_t* status, hipStream_t stream);

}  // namespace rlk
