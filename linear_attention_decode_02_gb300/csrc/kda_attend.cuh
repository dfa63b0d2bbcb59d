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
// The same under shared prefixes, for 64 and 128 channels: sequences' own positions, up to 8 heads a key head, and the
// groups' common ones, in units of p.heads query rows.  Both leave parts of as many warps.
constexpr int kTf32PartWarps = 8;
cudaError_t launch_attend_tf32_own(const AttendArgs& a, const AttendPlan& p, cudaStream_t s);
cudaError_t launch_attend_tf32_groups(const AttendArgs& a, const AttendPlan& p, cudaStream_t s);

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

// Where a result's later parts are: the piece that began it, how many after that
// hold more of it, and its place in them (below 256).
__device__ __forceinline__ int2 part_note(int piece, int more, int row) { return make_int2(piece, more << 8 | row); }

// Positions a sequence attends to: [first, end), and its tiles [tile0, tile0 + tiles).
struct Span {
  int first, end, tile0, tiles;
};
// `skip`: positions at the beginning that are left out.
template <int TILE = kTile>
__device__ __forceinline__ Span span_of(const AttendArgs& a, int n, int skip = 0) {
  const int64_t cap = (int64_t)a.table_cols * a.page_size;
  const int len = __ldg(a.lens + n);
  Span s;
  s.end = (int)min((int64_t)max(len, 0), cap);
  s.first = a.window > 0 && len > a.window ? len - a.window : 0;
  if (skip > 0) s.first = max(s.first, skip);
  if (s.first >= s.end) s.first = s.end = 0;
  s.tile0 = s.first / TILE;
  s.tiles = s.end == 0 ? 1 : (s.end - 1) / TILE - s.tile0 + 1;
  return s;
}

// A sequence takes part in its group's common positions where it attends to all of them.
__device__ __forceinline__ bool takes_part(const AttendArgs& a, int n, int prefix) {
  const int64_t cap = (int64_t)a.table_cols * a.page_size;
  const int len = __ldg(a.lens + n);
  return prefix > 0 && min((int64_t)max(len, 0), cap) >= prefix && (a.window == 0 || len <= a.window);
}

// Positions that a sequence leaves to its group's kernel, for sequences that go by in order: none, or found by their groups;
// and positions of a tile.
struct Whole {
  static constexpr int TILE = kTile;
  __device__ __forceinline__ int shared(const AttendArgs&, int) { return 0; }
};
template <int T>
struct Own {
  static constexpr int TILE = T;
  int end = 0, prefix = 0;  // the sequences before `end` that are left have `prefix` positions in common
  __device__ __forceinline__ int shared(const AttendArgs& a, int n) {
    if (n >= end) {
      int g = 0, hi = a.num_groups;
      end = INT32_MAX;
      while (g < hi) {  // the first group that ends behind n
        const int mid = (int)(((unsigned)g + (unsigned)hi) >> 1), e = __ldg(a.starts + mid + 1);
        if (e <= n) {
          g = mid + 1;
        } else {
          hi = mid;
          end = e;
        }
      }
      prefix = 0;
      if (g < a.num_groups) {
        const int first = __ldg(a.starts + g), common = __ldg(a.prefix_lens + g);
        if (n < first) end = first;
        else prefix = (int)min((int64_t)max(common, 0), (int64_t)a.table_cols * a.page_size);
      }
    }
    return takes_part(a, n, prefix) ? prefix : 0;
  }
};

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
// With EACH a block has a piece for every warp, c is the warp's own and ctas counts warps.
template <int THREADS, typename Part = Whole, bool EACH = false>
__device__ __forceinline__ Place find_place(const AttendArgs& a, int units, int c, int ctas) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  Place p;
  if (a.N <= 32) {  // a sequence a lane, every warp alone
    const int64_t mine = lane < a.N ? (int64_t)span_of<Part::TILE>(a, lane, Part().shared(a, lane)).tiles * units : 0;
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
  constexpr int PIECES = EACH ? THREADS / 32 : 1;
  __shared__ int s_n[PIECES];
  __shared__ int64_t s_before[PIECES];
  const int per = (a.N + THREADS - 1) / THREADS;
  const int n0 = min(a.N, tid * per), n1 = min(a.N, n0 + per);
  int64_t mine = 0;
  Part part;
  for (int n = n0; n < n1; ++n) mine += span_of<Part::TILE>(a, n, part.shared(a, n)).tiles;
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
  if (!p.cut(total * units, c, ctas) && !EACH) return p;  // the whole block
  const int64_t before = (prior + scan - mine) * units;   // tiles before sequence n0
#pragma unroll
  for (int w = 0; w < PIECES; ++w) {
    Place q = p;
    if (EACH && !q.cut(total * units, c - warp + w, ctas)) break;
    if (n0 < n1 && q.start >= before && q.start < before + mine * units) {
      int64_t at = before;
      Part again;
      int n = n0;
      for (; n < n1 - 1; ++n) {
        const int64_t t = (int64_t)span_of<Part::TILE>(a, n, again.shared(a, n)).tiles * units;
        if (q.start < at + t) break;
        at += t;
      }
      s_n[w] = n;
      s_before[w] = at;
    }
  }
  __syncthreads();
  if (p.start < p.stop) {
    p.n = s_n[EACH ? warp : 0];
    p.before = s_before[EACH ? warp : 0];
  }
  return p;
}

// ---- groups of sequences that share a prefix -------------------------------------

// A group's sequences and what its unit, a key head and ROWS query rows, has of
// tiles of KT positions.  Query row i of a key head is its query head i % G (G to a
// key head) in sequence i / G of the group.
struct Group {
  int first, rows, prefix, tiles, row_tiles;  // first sequence; query rows of a key head; common positions
};
template <int KT, int ROWS>
__device__ __forceinline__ Group group_of(const AttendArgs& a, int g) {
  Group r;
  r.first = min(max(__ldg(a.starts + g), 0), a.N);
  const int end = min(max(__ldg(a.starts + g + 1), r.first), a.N);
  const int64_t cap = (int64_t)a.table_cols * a.page_size;
  r.prefix = (int)min((int64_t)max(__ldg(a.prefix_lens + g), 0), cap);
  r.rows = (end - r.first) * (a.Hq / a.Hkv);
  // a prefix longer than the window is left to its sequences, none of which takes part: 16 x 4 of 8192 + 300 positions of
  // 32 / 8 heads of 128, window 4096, 145 us, 235 where its tiles were worked on for nobody, 165 as a paged call
  r.tiles = a.window > 0 && r.prefix > a.window ? 0 : (r.prefix + KT - 1) / KT;
  r.row_tiles = r.tiles > 0 ? (r.rows + ROWS - 1) / ROWS : 0;
  return r;
}

// Warp w of `warps`: empty parts for the sequences that take no part in their groups' positions.
__device__ __forceinline__ void leave_empty_parts(const AttendArgs& a, int w, int warps, int lane) {
  const int64_t heads = (int64_t)a.N * a.Hq;
  for (int n = w; n < a.N; n += warps) {
    const int g = find_sequence(a.starts, a.num_groups, n, lane);
    if (g < a.num_groups && n >= __ldg(a.starts + g) && takes_part(a, n, group_of<1, 1>(a, g).prefix)) continue;
    for (int h = lane; h < a.Hq; h += 32) {
      const int64_t head = (int64_t)n * a.Hq + h;
      a.parts.first_note[head] = part_note(0, 0, 0);
      for (int i = 0; i < a.parts.warps; ++i) a.parts.first_ml[i * heads + head] = make_float2(-INFINITY, 0.f);
    }
  }
}

// Where a walk over the tiles of groups' units stands; the key head's row tiles lie together.
template <int KT, int ROWS>
struct GroupWalk {
  static constexpr int TILE = KT;
  int64_t tile, unit_start, unit_end;
  int g, n, group, row_tile;  // n: the sequence whose pages are read; group: the key head
  Span sp;
  Group of;
  __device__ __forceinline__ void enter(const AttendArgs& a) {
    of = group_of<KT, ROWS>(a, g);
    n = of.first;
    sp = Span{0, of.prefix, 0, of.tiles};
  }
  __device__ __forceinline__ void start(const AttendArgs& a, const Place& p) {
    tile = p.start;
    g = p.n;
    enter(a);
    const int64_t u = quotient(tile - p.before, of.tiles);
    group = (int)quotient(u, of.row_tiles);
    row_tile = (int)(u - (int64_t)group * of.row_tiles);
    unit_start = p.before + u * of.tiles;
    unit_end = unit_start + of.tiles;
  }
  __device__ __forceinline__ void next_unit(const AttendArgs& a, int = 0) {
    unit_start = unit_end;
    if (++row_tile == of.row_tiles) {
      row_tile = 0;
      if (++group == a.Hkv) {
        group = 0;
        do {
          if (++g >= a.num_groups) return;
          enter(a);
        } while (of.row_tiles == 0);
      }
    }
    unit_end = unit_start + of.tiles;
  }
  __device__ __forceinline__ int rows_left() const { return of.rows - row_tile * ROWS; }
  // Sequence and query head of row r of the unit.
  __device__ __forceinline__ int2 row(const AttendArgs& a, int r) const {
    const int G = a.Hq / a.Hkv, i = row_tile * ROWS + r;
    return make_int2(of.first + i / G, group * G + i % G);
  }
};

// The tiles of all groups' units and where piece c lies in them (p.n: the group), found by the whole block.
template <int THREADS, int KT, int ROWS>
__device__ __forceinline__ Place find_group_place(const AttendArgs& a, int c, int ctas) {
  __shared__ int64_t s_warp[THREADS / 32], s_before;
  __shared__ int s_g;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.num_groups + THREADS - 1) / THREADS;
  const int g0 = min(a.num_groups, tid * per), g1 = min(a.num_groups, g0 + per);
  const auto tiles_of = [&](int g) {
    const Group r = group_of<KT, ROWS>(a, g);
    return (int64_t)r.row_tiles * a.Hkv * r.tiles;
  };
  int64_t mine = 0;
  for (int g = g0; g < g1; ++g) mine += tiles_of(g);
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
  if (!p.cut(total, c, ctas)) return p;  // the whole block
  int64_t before = prior + scan - mine;
  if (p.start < p.stop && p.start >= before && p.start < before + mine) {
    int g = g0;
    for (; g < g1 - 1; ++g) {
      const int64_t t = tiles_of(g);
      if (p.start < before + t) break;
      before += t;
    }
    s_g = g;
    s_before = before;
  }
  __syncthreads();
  p.n = s_g;
  p.before = s_before;
  return p;
}

// out[h][d] of a finished head from its sum of weights and unnormalised output.
__device__ __forceinline__ float finished(float o, float l) { return l == 0.f ? 0.f : o / l; }
__device__ __forceinline__ float log_sum(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

// Where a walk over the piece's tiles stands.
template <typename Part>
struct WalkOf {
  static constexpr int TILE = Part::TILE;
  int64_t tile, unit_start, unit_end;
  int n, group;
  Span sp;
  Part part;
  __device__ __forceinline__ void start(const AttendArgs& a, const Place& p) {
    tile = p.start;
    n = p.n;
    sp = span_of<TILE>(a, n, part.shared(a, n));
    group = (int)quotient(tile - p.before, sp.tiles);
    unit_start = p.before + (int64_t)group * sp.tiles;
    unit_end = unit_start + sp.tiles;
  }
  __device__ __forceinline__ void next_unit(const AttendArgs& a, int units) {
    unit_start = unit_end;
    if (++group == units) {
      group = 0;
      if (++n < a.N) sp = span_of<TILE>(a, n, part.shared(a, n));
    }
    unit_end = unit_start + sp.tiles;
  }
};
using Walk = WalkOf<Whole>;

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
template <typename T, int D, int KEYS, int STAGES, int WARPS, bool SWIZZLE, typename W = Walk>
struct PageCopies {
  static constexpr int SUBS = W::TILE / WARPS / KEYS;
  static constexpr int ROW = D * (int)sizeof(T);
  static constexpr int TENSOR = KEYS * ROW;
  static constexpr int STAGE = 2 * TENSOR;
  static constexpr int RING = STAGES * STAGE;  // bytes of a warp
  static constexpr int CHUNKS = ROW / 16;
  // One pass of the warp copies 32 chunks: part of a row, or PASS_ROWS rows.
  static constexpr int PASSES = KEYS * CHUNKS / 32;
  static_assert(SUBS >= 1 && SUBS * KEYS * WARPS == W::TILE && 2 * KEYS <= 32 && PASSES * 32 == KEYS * CHUNKS, "bad shape");
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
  W at;  // of the next look-up
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
      const int t = (at.sp.tile0 + (int)(at.tile - at.unit_start)) * W::TILE + (warp * SUBS + sub) * KEYS + lane % KEYS;
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
