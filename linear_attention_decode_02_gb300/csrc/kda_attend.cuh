// How the attention kernels share their work, and how partial results join.
//
// A unit is one sequence, one key head and one group of at most HG of its
// query heads; its work is a row of tiles of kTile positions, at least one.
// All units' tiles form one line, cut into equal pieces, one for each block of
// the grid but at least a tile, whatever the sequences' lengths, so ragged
// batches and a few very long sequences load the SMs alike, and the host needs
// no lengths.  A unit inside one piece is finished there; one that crosses a
// cut leaves an unnormalised partial (maximum, sum, output) per piece, which a
// second kernel joins.  A piece cuts at most two units, so the workspace is
// fixed by the grid.
#pragma once

#include <atomic>

#include "kda_cache.h"
#include "kda_device.cuh"

namespace kda {

// Lets `k` use `bytes` of dynamic shared memory on the current device; `set`
// (one flag a device) remembers where that was done.
template <typename Kernel>
inline cudaError_t allow_shared(Kernel k, int bytes, std::atomic<bool> (&set)[64]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  // idempotent, so two host threads that both get here set the same value
  e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) set[dev].store(true, std::memory_order_release);
  return e;
}

constexpr int kTile = 64;  // positions of a tile

// The tensor-core kernel (kda_attend_mma.cu), for bfloat16 whose vectors start on 16-byte boundaries.
AttendPlan attend_mma_plan(int32_t G, int32_t D, int32_t sms);
cudaError_t launch_attend_mma(const AttendArgs& a, const AttendPlan& p, cudaStream_t s);
// Float32 in matrix instructions (kda_attend_tf32.cu), for many query heads a key head.
AttendPlan attend_tf32_plan(int32_t G, int32_t D, int32_t sms);
cudaError_t launch_attend_tf32(const AttendArgs& a, const AttendPlan& p, cudaStream_t s);

// a / b, neither negative; 32-bit where they fit (a 64-bit division is a long call).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
  return a / b;
}
// Pieces of T tiles, their first tiles, and the piece that owns a tile.
__device__ __forceinline__ int pieces_of(int64_t T, int ctas) { return T < ctas ? (int)T : ctas; }
__device__ __forceinline__ int64_t piece_start(int64_t c, int64_t T, int pieces) { return quotient(c * T, pieces); }
__device__ __forceinline__ int64_t piece_of(int64_t t, int64_t T, int pieces) {
  return quotient((t + 1) * pieces + T - 1, T) - 1;
}

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

// The tiles of all sequences and where piece c lies in them, found by the whole
// block; start == stop where there is no such piece.
struct Place {
  int64_t T;       // all tiles
  int64_t start, stop;
  int n;           // sequence of tile `start`
  int64_t before;  // tiles before sequence n
  // False where there is no piece c.
  __device__ __forceinline__ bool cut(int64_t tiles, int c, int ctas) {
    T = tiles;
    const int pieces = pieces_of(T, ctas);
    start = stop = before = 0;
    n = 0;
    if (c >= pieces) return false;
    start = piece_start(c, T, pieces);
    stop = piece_start(c + 1, T, pieces);
    return true;
  }
};
template <int THREADS>
__device__ __forceinline__ Place find_place(const AttendArgs& a, int units, int c, int ctas) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Place p;
  if (a.N <= 32) {  // a sequence a lane, every warp alone
    const int64_t mine = lane < a.N ? (int64_t)span_of(a, lane).tiles * units : 0;
    int64_t scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += up;
    }
    if (!p.cut(__shfl_sync(0xffffffffu, scan, 31), c, ctas)) return p;
    p.n = __popc(__ballot_sync(0xffffffffu, scan <= p.start));
    p.before = __shfl_sync(0xffffffffu, scan - mine, p.n);
    return p;
  }
  __shared__ int64_t s_warp[THREADS / 32];
  __shared__ int s_n;
  __shared__ int64_t s_before;
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
  if (!p.cut(total * units, c, ctas)) return p;  // the whole block
  int64_t at = (prior + scan - mine) * units;    // tiles before sequence n0
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

// Where a walk over the piece's tiles stands.
struct Walk {
  int64_t tile, unit_start, unit_end;
  int n, group;
  Span sp;
  __device__ __forceinline__ void start(const AttendArgs& a, const Place& p) {
    tile = p.start;
    n = p.n;
    sp = span_of(a, n);
    group = (int)quotient(tile - p.before, sp.tiles);
    unit_start = p.before + (int64_t)group * sp.tiles;
    unit_end = unit_start + sp.tiles;
  }
  __device__ __forceinline__ void next_unit(const AttendArgs& a, int units) {
    unit_start = unit_end;
    if (++group == units) {
      group = 0;
      if (++n < a.N) sp = span_of(a, n);
    }
    unit_end = unit_start + sp.tiles;
  }
};

__device__ __forceinline__ PieceNote note_of(const Walk& w, const Place& p) {
  PieceNote note;
  note.unit_start = w.unit_start; note.unit_end = w.unit_end; note.tiles = p.T;
  note.n = w.unit_start < p.start ? w.n : -1;
  note.group = w.group;
  return note;
}

// 16 bytes to shared memory; zeros where live is false (src is then not read).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// One warp's copies of keys and values into its ring of stages, KEYS positions
// each.  A block of WARPS warps shares a tile; a warp's part of it is SUBS
// stages.  The pages of a stage are looked up two stages before it is issued,
// so that the table's latency is not in the way.  Positions not attended to
// become zeros.  SWIZZLE puts 16-byte chunk c of row r at c ^ (r & 7).
template <typename T, int D, int KEYS, int STAGES, int WARPS, bool SWIZZLE>
struct PageCopies {
  static constexpr int SUBS = kTile / WARPS / KEYS;
  static constexpr int ROW = D * (int)sizeof(T);
  static constexpr int TENSOR = KEYS * ROW;
  static constexpr int STAGE = 2 * TENSOR;
  static constexpr int RING = STAGES * STAGE;  // bytes of a warp
  static constexpr int CHUNKS = ROW / 16;
  // One pass of the warp copies 32 chunks: part of a row, or PASS_ROWS rows.
  static constexpr int PASSES = KEYS * CHUNKS / 32;
  static_assert(SUBS >= 1 && SUBS * KEYS * WARPS == kTile && 2 * KEYS <= 32 && PASSES * 32 == KEYS * CHUNKS, "bad shape");
  struct Notes {
    const char* row[2 * KEYS];  // keys, then values; of a position not attended to: the first page
    uint32_t live[STAGES];
  };

  const AttendArgs& a;
  const Place& place;
  Notes& notes;
  uint32_t ring;
  int units, groups, warp, lane;
  const char* data;                                // of keys for the first KEYS lanes, of values for the next
  int64_t page_stride, token_stride, head_stride;  // elements
  struct Look {
    int page, token, head;  // of this lane's position (page 0: none) and of the stage; head -1: no stage
  };
  Look next, second;
  Walk at;  // of the next look-up
  int sub;

  __device__ __forceinline__ PageCopies(const AttendArgs& a_, const Place& p, Notes& n, const void* ring_, int units_,
                                        int groups_, int warp_, int lane_)
      : a(a_), place(p), notes(n), ring(static_cast<uint32_t>(__cvta_generic_to_shared(ring_))), units(units_),
        groups(groups_), warp(warp_), lane(lane_), sub(0) {
    const PageView& mine = lane < KEYS ? a.kp : a.vp;
    data = static_cast<const char*>(mine.data);
    page_stride = mine.page;
    token_stride = mine.token;
    head_stride = mine.head;
    at.start(a, place);
    next = look_up();
    second = look_up();
  }
  __device__ __forceinline__ Look look_up() {
    Look l{0, 0, -1};
    if (at.tile < place.stop) {
      l.head = groups == 1 ? at.group : at.group / groups;
      const int t = (at.sp.tile0 + (int)(at.tile - at.unit_start)) * kTile + (warp * SUBS + sub) * KEYS + lane % KEYS;
      if (lane < 2 * KEYS && t >= at.sp.first && t < at.sp.end) {
        const int col = t / a.page_size;
        l.token = t - col * a.page_size;
        l.page = __ldg(a.table + (int64_t)at.n * a.table_rs + col);
      }
      if (++sub == SUBS) {
        sub = 0;
        if (++at.tile == at.unit_end) at.next_unit(a, units);
      }
    }
    return l;
  }
  // Pass i: its row among keys and values, its chunk of the row, and where that goes in a stage.
  __device__ __forceinline__ int row_of(int i) const { return (i * 32 + lane) / CHUNKS; }
  __device__ __forceinline__ int chunk_of(int i) const { return (i * 32 + lane) % CHUNKS; }
  __device__ __forceinline__ uint32_t target(int i) const {
    return row_of(i) * ROW + ((SWIZZLE ? chunk_of(i) ^ (row_of(i) & 7) : chunk_of(i)) << 4);
  }
  // Copies the next stage's positions to `stage` and closes a copy group, empty at the end of the piece.
  __device__ __forceinline__ void copy(int stage) {
    if (next.head >= 0) {
      const bool live = next.page > 0 && next.page < a.num_pages;
      const uint32_t mask = __ballot_sync(0xffffffffu, live) & ((1u << KEYS) - 1);
      __syncwarp();
      if (lane < 2 * KEYS) {
        const int64_t offset = next.page * page_stride + next.token * token_stride + next.head * head_stride;
        notes.row[lane] = data + (live ? offset * (int)sizeof(T) : 0);
      }
      if (lane == 0) notes.live[stage] = mask;
      __syncwarp();
      const uint32_t base = ring + stage * STAGE;
      if (mask == (1u << KEYS) - 1) {
#pragma unroll
        for (int i = 0; i < 2 * PASSES; ++i) copy16(base + target(i), notes.row[row_of(i)] + chunk_of(i) * 16);
      } else {
#pragma unroll
        for (int i = 0; i < 2 * PASSES; ++i)
          copy16(base + target(i), notes.row[row_of(i)] + chunk_of(i) * 16, mask >> (row_of(i) % KEYS) & 1);
      }
      next = second;
      second = look_up();
    }
    copy_commit();
  }
};

}  // namespace kda
