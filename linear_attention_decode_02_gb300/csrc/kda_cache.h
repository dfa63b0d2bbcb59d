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
};

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
};

// Grid and workspace of the attention kernels: `ctas` workers that each may
// leave two partial results of `heads` query heads.
struct AttendPlan {
  int32_t ctas, heads;
  int64_t floats;
};
// Floats of workspace for either kernel that may serve the dtype.
int64_t attend_floats(int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype, int32_t sms);
cudaError_t launch_paged_attention(const AttendArgs& a, int32_t sms, cudaStream_t s);

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
