// Internal interface between the host side of the cache and beam entry points
// (kda_cache_api.cu) and their kernels.  Plain structs of device pointers and
// element strides, validated on the host before any launch.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

// The pages of one KV cache tensor, [num_pages, page_size, Hkv, D] by strides.
struct PageView {
  void* data;
  int64_t page, token, head;  // element strides
};

// Rotary positions of R token rows and the write of their keys and values.
struct RopeArgs {
  const void* q; const void* k; const void* v;
  int64_t q_rs, q_hs, k_rs, k_hs, v_rs, v_hs;
  const uint64_t* steps;       // [rot/2] turns per position, 64-bit fixed point (8-byte aligned)
  const int32_t* cu;           // [N+1], or null: one row per sequence
  const int32_t* lens;         // [N]
  const int32_t* table; int64_t table_rs; int32_t table_cols;
  PageView kp, vp;
  int32_t num_pages, page_size;
  void* q_out; int64_t o_rs, o_hs;
  int32_t R, N, Hq, Hkv, D, rot;
  int32_t interleaved;
  float amplitude;
  int32_t in_dtype, page_dtype;
  int32_t vec;                 // elements per access: 8 (bf16 -> bf16, 16-byte aligned rows) or 4
  int32_t sms;                 // SMs of the device
  // Rows with a position on each of several axes and a slot each; cu, lens and table are not used then.
  const int32_t* positions;    // [R, num_axes], or null
  int64_t p_rs, p_as;
  const int32_t* slots;        // [R]: page * page_size + place
  const int32_t* pair_axes;    // [rot/2]
  int32_t num_axes;
};
constexpr int kRopeAxes = 4;   // most axes

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t s);

// Copies of slots within each of up to kMovePools pools, byte by byte.
constexpr int kMovePools = 64;
constexpr int kMoveBeams = 32;
struct MovePool {
  char* base;
  int64_t stride, bytes;     // slot stride and slot size
  int64_t first;             // first block of this pool (set by the launcher)
};
struct MoveArgs {
  const int32_t* src; const int32_t* dst; const int32_t* parents;  // [N, K]; parents may be null
  int64_t src_rs, dst_rs, par_rs;
  int32_t N, K, num_slots;
  int32_t pools, align;      // align: 16, 4 or 2 bytes, of every base, stride and size
  MovePool pool[kMovePools];
};

// Sets the pools' first blocks and launches; the block count must stay below 2^31 (false: it does not).
bool plan_pool_move(MoveArgs& a, int64_t* blocks);
cudaError_t launch_pool_move(const MoveArgs& a, int64_t blocks, cudaStream_t s);

// Pages of a step's sequences.
constexpr int kPageSequences = 8192;  // most sequences of a call
struct PagesArgs {
  const int32_t* old_lens; const int32_t* new_lens;  // [N]
  const int32_t* shared_lens;                        // [N], or null
  int32_t* table; int64_t table_rs; int32_t table_cols;
  int32_t* ring; int32_t capacity;                   // free pages
  const int32_t* state;                              // {head, count}
  int32_t* lens_out; int32_t* state_out;             // may be old_lens or new_lens, and state
  int32_t* cu; int32_t* slots;                       // [N + 1], [R]
  int32_t N, page_size;
  int64_t R;
  // A place / page_size is (place * page_factor) >> page_shift for places below 2^31 (set by the launcher).
  uint32_t page_factor; int32_t page_shift;
};
cudaError_t launch_page_assign(const PagesArgs& a, cudaStream_t s);

// Parts of results that another kernel joins: unnormalised outputs with their
// row's maximum (units of log 2) and sum.  The piece that begins a unit leaves
// part [warp][row of the batch's N * Hq] with a note of that piece, how many more
// follow and the row's place in the unit (part_note); piece c of those that follow
// leaves part [c][warp][place].
struct Parts {
  float* first_o; float2* first_ml; int2* first_note;
  float* more_o; float2* more_ml;
  int32_t ctas, warps, rows;  // pieces, parts a piece and places a unit
};

// Attention of one new token per sequence over paged keys and values.
struct AttendArgs {
  const void* q; int64_t q_rs, q_hs;      // [N, Hq, D]
  PageView kp, vp;
  int32_t num_pages, page_size;
  const int32_t* table; int64_t table_rs; int32_t table_cols;
  const int32_t* lens;                    // [N]
  void* out;                              // bf16 [N, Hq, D] contiguous
  float* lse;                             // [N, Hq] contiguous, or null
  float* work;                            // attend_floats()
  int32_t N, Hq, Hkv, D, dtype;
  int32_t window;                         // 0: all
  float scale_log2;                       // scale * log2(e)
  int32_t vec16;                          // q rows, key and value vectors start on 16-byte boundaries
  // Under shared prefixes (zero otherwise).  Group g is sequences starts[g] .. starts[g + 1] - 1, whose first
  // prefix_lens[g] positions are attended to by one kernel and left out by the other, which is told so by `own`.
  // Both leave parts.
  const int32_t* starts; const int32_t* prefix_lens; int32_t num_groups;
  int32_t own;
  Parts parts;
};
constexpr int kAttendWarps = 4;  // of a block of the tensor-core kernel
// Of these, those that take a piece of sequences' own positions under a shared prefix each; else the block takes one.
constexpr int own_warps_alone(int D) { return D < 256 ? kAttendWarps : 1; }

// Grid and workspace of the attention kernels: `ctas` workers that each may
// leave two partial results of `heads` query heads.
struct AttendPlan {
  int32_t ctas, heads;
  int64_t floats;
};
// Floats of workspace for either kernel that may serve the dtype.
int64_t attend_floats(int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype, int32_t sms);
cudaError_t launch_paged_attention(const AttendArgs& a, int32_t sms, cudaStream_t s);

// Attention of sequences that share prefixes, group by group (starts, prefix_lens and num_groups set).
int64_t prefix_floats(int64_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype, int32_t sms);
cudaError_t launch_prefix_attention(const AttendArgs& a, int32_t sms, cudaStream_t s);

// Beam selection over beams x vocabulary.
constexpr int kBeamMax = 32;      // beams of a request
constexpr int kBeamOutMax = 64;   // candidates returned
struct BeamArgs {
  const void* logits; int64_t ns, bs;   // [N, B, V] element strides
  const float* scores;                  // [N, B]
  const int32_t* finished;              // [N, B], or null
  float* out_scores; int32_t* out_parents; int32_t* out_tokens;  // [N, M]
  float* work;
  int32_t N, B, V, M, eos, dtype;
};
// A block scans `batches` times 256 * `loads` vectors of 16 bytes of one beam; `splits` blocks a beam.
struct BeamPlan {
  int32_t loads, batches, splits;
  bool aligned;  // every row starts on a 16-byte boundary
  int64_t floats;
};
// `splits` and `floats` are the same for either alignment.
BeamPlan beam_plan(int64_t N, int32_t B, int32_t V, int32_t M, int32_t dtype, bool aligned, int32_t sms);
cudaError_t launch_beam_select(const BeamArgs& a, const BeamPlan& p, cudaStream_t s);

}  // namespace kda
