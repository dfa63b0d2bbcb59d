// How the attention kernels share their work, and how partial results join.
//
// A unit is one sequence, one key head and one group of at most HG of its
// query heads; its work is a row of tiles of kTile positions, at least one.
// All units' tiles form one line, cut into `ctas` equal pieces whatever the
// sequences' lengths, so ragged batches and a few very long sequences load
// the SMs alike, and the host needs no lengths.  A unit inside one piece is
// finished there; one that crosses a cut leaves an unnormalised partial
// (maximum, sum, output) per piece, which a second kernel joins.  A piece
// cuts at most two units, so the workspace is fixed by the grid.
#pragma once

#include "kda_cache.h"
#include "kda_device.cuh"

namespace kda {

constexpr int kTile = 64;  // positions of a tile

// The tensor-core kernel (kda_attend_mma.cu), for bfloat16 whose vectors start on 16-byte boundaries.
AttendPlan attend_mma_plan(int32_t G, int32_t D, int32_t sms);
cudaError_t launch_attend_mma(const AttendArgs& a, const AttendPlan& p, cudaStream_t s);

// First tile of piece c.
__device__ __forceinline__ int64_t piece_start(int64_t c, int64_t T, int C) { return c * T / C; }
// Piece that owns tile t.
__device__ __forceinline__ int64_t piece_of(int64_t t, int64_t T, int C) { return ((t + 1) * C + T - 1) / T - 1; }

// What a piece tells the join about the unit at its first tile.
struct PieceNote {
  int64_t unit_start, unit_end, tiles;  // the unit's tiles; all tiles
  int32_t n, group;                     // n < 0: nothing to join here
};
constexpr int kNoteFloats = sizeof(PieceNote) / 4;
static_assert(kNoteFloats == 8, "workspace layout");

// Workspace: notes [ctas], then maximum and sum [2 * ctas][heads][2], then outputs [2 * ctas][heads][D].
struct Workspace {
  PieceNote* note;
  float* ml;
  float* o;
  int heads, D;
  __device__ __forceinline__ Workspace(float* w, int ctas, int heads_, int D_)
      : note(reinterpret_cast<PieceNote*>(w)), ml(w + (int64_t)ctas * kNoteFloats),
        o(ml + (int64_t)4 * ctas * heads_), heads(heads_), D(D_) {}
  __device__ __forceinline__ float* ml_of(int64_t slot, int h) const { return ml + (slot * heads + h) * 2; }
  __device__ __forceinline__ float* o_of(int64_t slot, int h) const { return o + (slot * heads + h) * D; }
};

// Positions a sequence attends to: [first, end), and its tiles [tile0, tile0 + tiles).
struct Span {
  int first, end, tile0, tiles;
};
__device__ __forceinline__ Span span_of(const AttendArgs& a, int n) {
  const int64_t cap = (int64_t)a.table_cols * a.page_size;
  const int len = __ldg(a.lens + n);
  Span s;
  s.end = (int)min((int64_t)max(len, 0), cap);
  s.first = a.window > 0 && len > a.window ? len - a.window : 0;
  if (s.first >= s.end) s.first = s.end = 0;
  s.tile0 = s.first / kTile;
  s.tiles = s.end == 0 ? 1 : (s.end - 1) / kTile - s.tile0 + 1;
  return s;
}

// Finds, with the whole block, the number of tiles per (key head, group) of
// all sequences and the sequence where tile `c * T / C` lies.
struct Place {
  int64_t T;       // all tiles
  int64_t start, stop;
  int n;           // sequence of tile `start`
  int64_t before;  // tiles before sequence n
};
template <int THREADS>
__device__ __forceinline__ Place find_place(const AttendArgs& a, int units, int c, int C) {
  __shared__ int64_t s_warp[THREADS / 32];
  __shared__ int s_n;
  __shared__ int64_t s_before;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.N + THREADS - 1) / THREADS;
  const int n0 = min(a.N, tid * per), n1 = min(a.N, n0 + per);
  int64_t mine = 0;
  for (int n = n0; n < n1; ++n) mine += span_of(a, n).tiles;
  int64_t scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += up;
  }
  if (lane == 31) s_warp[warp] = scan;
  __syncthreads();
  int64_t prior = 0, total = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) prior += s_warp[w];
    total += s_warp[w];
  }
  Place p;
  p.T = total * units;
  p.start = piece_start(c, p.T, C);
  p.stop = piece_start(c + 1, p.T, C);
  int64_t at = (prior + scan - mine) * units;  // tiles before sequence n0
  if (n0 < n1 && p.start >= at && p.start < at + mine * units) {
    int n = n0;
    for (; n < n1 - 1; ++n) {
      const int64_t t = (int64_t)span_of(a, n).tiles * units;
      if (p.start < at + t) break;
      at += t;
    }
    s_n = n;
    s_before = at;
  }
  __syncthreads();
  p.n = s_n;
  p.before = s_before;
  return p;
}

// out[h][d] of a finished head from its sum of weights and unnormalised output.
__device__ __forceinline__ float finished(float o, float l) { return l == 0.f ? 0.f : o / l; }
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace kda
