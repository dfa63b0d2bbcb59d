// Attention of one new token per sequence where groups of sequences begin with
// the same positions: the common part is read once a group, by the tensor cores,
// with all the group's queries of a key head as rows; each sequence's own part is
// left to the paged kernel; a last kernel joins both.
//
// For a row with maximum m, sum l and unnormalised output o over a part of its
// positions (weights 2^(s - m)), parts 1 and 2 join as
//   m = max(m1, m2),  l = l1 2^(m1 - m) + l2 2^(m2 - m),  o alike,
// so it does not matter how the positions were cut or who took them.
//
// A unit is a group, a key head and RT x 128 query rows (row i is query head
// i % G of the key head in sequence i / G of the group, G query heads a key head).
// Units' tiles of KT positions form one line, which is cut into equal pieces, one
// for each SM, as in the paged kernel; positions come through the table row of
// the group's first sequence.  The part of a unit in the piece that begins it goes
// to the row's own place, later parts to a place of their piece.
//
// Roles of a CTA:
//   warps 0 .. 4 W - 1    softmax, a group of four for each of W lanes: thread = row
//   the next warp         allocates tensor memory, issues the matrix products
//   the last four         copy queries, keys and values into shared memory
// A lane is a buffer of scores S (128 rows x KT positions, float32), an output O
// and the warps between them.  With two row tiles each lane is one of them and both
// use every tile of keys and values; with one they take the tiles in turn, each to
// an output and statistics of its own, which are joined at the unit's end.  Either
// way one lane's softmax runs under the other's products.  256 channels leave room
// for one output: its softmax takes both buffers in turn.
// The row's thread puts the weights back over S as the next product's left operand,
// in two bfloat16 pieces, p = hi + lo to 2^-16, for 16 positions at a time 8 columns
// of hi and 8 of lo.  It reads S twice, for the row's maximum and for the weights,
// which are taken relative to a reference that follows the maximum only when that
// has passed it by 2^kSlack: O, which lies in tensor memory, is seldom rescaled.
//
// A barrier's parity tells two phases apart, so each is waited for, or known to be
// over, before the next: S of a buffer is issued behind the product of the weights
// that were in it, so a lane's O is at rest while its warps work on new scores.
//
// Every mbarrier wait is bounded in time: a role whose wait runs out records a bit
// in the error word, raises the CTA's abort flag and leaves its loop; all meet at
// the end before tensor memory is freed.
#include <algorithm>

#include "kda_attend_rows.cuh"
#include "kda_tcgen05.cuh"

namespace kda {

// bit 4: a wait of the shared-prefix attention kernel timed out.
__device__ unsigned int g_kda_prefix_error = 0;

namespace {

constexpr int kRows = 128;       // rows of a tile
constexpr int kLoaders = 128;    // threads
constexpr float kSlack = 4.f;    // in units of log 2
constexpr int kLiveDepth = 16;   // tiles whose masks are kept

template <int D, int RT>
struct PrefixShape {
  static constexpr int KT = D == 256 ? 64 : 128;   // positions of a tile
  static constexpr int BLOCKS = D / 64;            // 128-byte wide column blocks of an operand
  static constexpr int Q_TILE = BLOCKS * kRows * 128;
  static constexpr int QSLOTS = RT == 1 && D < 256 ? 2 : 1;
  static constexpr int HALF = BLOCKS * KT * 128;   // keys or values of a tile
  static constexpr int SLOTS = D == 64 ? 12 : 5;
  static constexpr int BYTES = QSLOTS * RT * Q_TILE + SLOTS * HALF + 1024;
  static constexpr int LANES = D == 256 ? 1 : 2;
  static constexpr bool SPLIT = RT < LANES;        // lanes take tiles in turn
  static constexpr int THREADS = (4 * LANES + 1) * 32 + kLoaders;
  static constexpr uint32_t S_COL = 0, O_COL = 2 * KT;   // two buffers of S, then O of each lane
  static constexpr uint32_t COLS = 512;
  static_assert(O_COL + LANES * D <= COLS && RT <= LANES, "tensor memory");
  static_assert(SLOTS / 2 + 4 <= kLiveDepth, "ring");
};

struct PrefixWork {
  float4* note;   // [N * Hq]
  float* o;       // [N * Hq][D]
  float2* ml;     // [ctas][RT * 128]: continued units
  float* more;    // [ctas][RT * 128][D]
  int32_t* skip;  // [N]
};

// Groups' sequences and tiles.
struct Group {
  int first, rows, prefix, tiles, row_tiles;  // sequences first .. ; query rows of a key head; positions
  __device__ __forceinline__ int64_t units(int Hkv) const { return (int64_t)row_tiles * Hkv; }
};
template <int KT, int ROWS>
__device__ __forceinline__ Group group_of(const PrefixArgs& a, int g) {
  const AttendArgs& at = a.attend;
  Group r;
  r.first = min(max(__ldg(a.starts + g), 0), at.N);
  const int end = min(max(__ldg(a.starts + g + 1), r.first), at.N);
  const int64_t cap = (int64_t)at.table_cols * at.page_size;
  r.prefix = (int)min((int64_t)max(__ldg(a.prefix_lens + g), 0), cap);
  r.rows = (end - r.first) * (at.Hq / at.Hkv);
  r.tiles = (r.prefix + KT - 1) / KT;
  r.row_tiles = r.tiles > 0 ? (r.rows + ROWS - 1) / ROWS : 0;
  return r;
}

// A sequence takes part in its group's common positions where it attends to all of them.
__device__ __forceinline__ bool takes_part(const AttendArgs& a, int n, int prefix) {
  const int64_t cap = (int64_t)a.table_cols * a.page_size;
  const int len = __ldg(a.lens + n);
  return prefix > 0 && min((int64_t)max(len, 0), cap) >= prefix && (a.window == 0 || len <= a.window);
}

// Where a walk over the piece's tiles stands.
template <int KT, int ROWS>
struct PrefixWalk {
  int64_t tile, unit_start, unit_end;
  int g, head, row_tile;
  Group group;
  __device__ __forceinline__ void start(const PrefixArgs& a, int64_t tile_, int g_, int64_t before) {
    tile = tile_;
    g = g_;
    group = group_of<KT, ROWS>(a, g);
    const int64_t u = quotient(tile - before, group.tiles);
    head = (int)quotient(u, group.row_tiles);
    row_tile = (int)(u - (int64_t)head * group.row_tiles);
    unit_start = before + u * group.tiles;
    unit_end = unit_start + group.tiles;
  }
  // False behind the last unit.
  __device__ __forceinline__ void next_unit(const PrefixArgs& a) {
    unit_start = unit_end;
    if (++row_tile == group.row_tiles) {
      row_tile = 0;
      if (++head == a.attend.Hkv) {
        head = 0;
        do {
          if (++g >= a.G) return;
          group = group_of<KT, ROWS>(a, g);
        } while (group.row_tiles == 0);
      }
    }
    unit_end = unit_start + group.tiles;
  }
  __device__ __forceinline__ int rows_left() const { return group.rows - row_tile * ROWS; }
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Scores of 32 positions, those not attended to set to minus infinity.
__device__ __forceinline__ void masked(uint32_t (&x)[32], uint32_t live) {
  if (live == 0xffffffffu) return;
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = live >> i & 1 ? x[i] : 0xff800000u;
}

template <int D, int RT>
__global__ void __launch_bounds__(PrefixShape<D, RT>::THREADS, 1)
    kda_prefix_kernel(const __grid_constant__ PrefixArgs a, const PrefixWork ws) {
  using P = PrefixShape<D, RT>;
  constexpr int KT = P::KT, ROWS = RT * kRows, SLOTS = P::SLOTS, LANES = P::LANES, WARPS = P::THREADS / 32;
  using Walker = PrefixWalk<KT, ROWS>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                       ~static_cast<uintptr_t>(1023));
  unsigned char* const s_q = sm;
  unsigned char* const s_ring = sm + P::QSLOTS * RT * P::Q_TILE;
  __shared__ uint64_t full[SLOTS], empty[SLOTS], s_full[2], p_full[2], o_done[2], q_empty[P::QSLOTS], live_full[kLiveDepth],
      x_full, x_empty, drained;
  __shared__ float2 s_ml[P::SPLIT ? kRows : 1];
  __shared__ uint32_t s_live[kLiveDepth][KT / 32];
  __shared__ uint32_t s_taddr;
  __shared__ volatile int s_abort;
  __shared__ int64_t s_warp[WARPS], s_before;
  __shared__ int s_g;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const AttendArgs& at = a.attend;
  const int C = gridDim.x, c = blockIdx.x, G = at.Hq / at.Hkv;

  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&full[i], kLoaders);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kRows / 32);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < P::QSLOTS; ++i) mbar_init(&q_empty[i], 1);
    for (int i = 0; i < kLiveDepth; ++i) mbar_init(&live_full[i], kLoaders / 32);
    mbar_init(&x_full, kRows);
    mbar_init(&x_empty, kRows);
    mbar_init(&drained, 1);
    s_abort = 0;
    mbar_fence_init();
  }
  if (warp == 4 * LANES) tc::alloc(&s_taddr, P::COLS);
  pdl_wait();
  pdl_launch_dependents();

  // The piece: groups' tiles summed by the whole block.
  const int per = (a.G + P::THREADS - 1) / P::THREADS;
  const int g0 = min(a.G, tid * per), g1 = min(a.G, g0 + per);
  const auto tiles_of = [&](int g) {
    const Group r = group_of<KT, ROWS>(a, g);
    return r.units(at.Hkv) * r.tiles;
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
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t taddr = s_taddr;
  int64_t prior = 0, T = 0;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) prior += s_warp[w];
    T += s_warp[w];
  }
  const int pieces = pieces_of(T, C);
  const int64_t start = c < pieces ? piece_start(c, T, pieces) : 0, stop = c < pieces ? piece_start(c + 1, T, pieces) : 0;
  {
    int64_t before = prior + scan - mine;
    if (start < stop && start >= before && start < before + mine) {
      int g = g0;
      for (; g < g1 - 1; ++g) {
        const int64_t t = tiles_of(g);
        if (start < before + t) break;
        before += t;
      }
      s_g = g;
      s_before = before;
    }
  }
  __syncthreads();

  // Nearly every wait ends with its first try, which looks at nothing else.
  auto wait_or_abort = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_sleep_try(bar, parity))) return true;
    const bool stopped = s_abort;  // by another role
    const bool ok = !stopped && mbar_sleep_wait(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    if (lane == 0 && !stopped) {
      atomicOr(&g_kda_prefix_error, 16u);
      s_abort = 1;
    }
    return false;
  };
  const bool any = start < stop;
  Walker walk;
  if (any) walk.start(a, start, s_g, s_before);

  if (warp < 4 * LANES) {
    // ---------------- which sequences take part, and softmax ----------------
    for (int n = c * 4 * LANES + warp; n < at.N; n += C * 4 * LANES) {
      const int g = find_sequence(a.starts, a.G, n, lane);
      bool part = false;
      int prefix = 0;
      if (g < a.G && n >= __ldg(a.starts + g)) {
        prefix = group_of<KT, ROWS>(a, g).prefix;
        part = takes_part(at, n, prefix);
      }
      if (lane == 0) ws.skip[n] = part ? prefix : 0;
      if (!part)
        for (int h = lane; h < at.Hq; h += 32) ws.note[(int64_t)n * at.Hq + h] = first_note(-INFINITY, 0.f, 0, 0, 0);
    }
    const int me = LANES == 1 ? 0 : warp >> 2;   // lane of the CTA
    const int row_tile = RT == 1 ? 0 : me;
    const int row = (warp & 3) * 32 + lane;      // of the row tile, and tensor-memory lane
    const uint32_t tl = taddr + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_addr = tl + P::O_COL + me * D;
    int tile = 0, job = 0, unit = 0;  // tiles of the piece, this lane's tiles and units so far
    bool run = any;
    while (run && walk.tile < stop) {
      const int valid = walk.rows_left() - row_tile * kRows;  // rows of this tile that exist
      const bool idle = valid <= (warp & 3) * 32;             // none of this warp's
      float m = -INFINITY, l = 0.f;
      const int64_t end = min(walk.unit_end, stop);
      const int count = (int)(end - walk.tile);
      const bool begins = walk.unit_start >= start;
      for (int j = P::SPLIT ? me : 0; j < count; j += P::SPLIT ? 2 : 1, ++job) {
        const int b = LANES == 1 ? job & 1 : me, at_mask = (tile + j) % kLiveDepth;
        const uint32_t phase = LANES == 1 ? (job >> 1) & 1 : job & 1;
        const bool first = j < (P::SPLIT ? 2 : 1);  // O holds nothing yet
        if (!wait_or_abort(&s_full[b], phase) || !wait_or_abort(&live_full[at_mask], ((tile + j) / kLiveDepth) & 1)) {
          run = false;
          break;
        }
        tc::fence_after_sync();
        if (!idle) {
          const uint32_t s_addr = tl + P::S_COL + b * KT;
          // The maximum first, for all positions: 128 columns of S pass through 64 registers.
          uint32_t s[2][32];
          float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          tc::ld32_async(s_addr, s[0]);
#pragma unroll
          for (int k = 0; k < KT / 32; ++k) {
            tc::ld_wait(s[k & 1]);
            tc::ld32_async(s_addr + (k + 1 < KT / 32 ? 32 * (k + 1) : 0), s[(k + 1) & 1]);  // the first again at the end
            masked(s[k & 1], s_live[at_mask][k]);
#pragma unroll
            for (int i = 0; i < 32; i += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                top[e] = max3(top[e], __uint_as_float(s[k & 1][i + 2 * e]), __uint_as_float(s[k & 1][i + 2 * e + 1]));
          }
          const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * at.scale_log2;
          const bool rises = most > m + kSlack || (m == -INFINITY && most > m);
          if (__any_sync(0xffffffffu, rises)) {
            const float fall = rises ? (m == -INFINITY ? 0.f : ex2(m - most)) : 1.f;
            if (rises) m = most;
            l *= fall;
            if (!first) {
              // with one lane the last tile's product may still run
              if (LANES == 1 && !wait_or_abort(&o_done[(job - 1) & 1], ((job - 1) >> 1) & 1)) { run = false; break; }
              tc::fence_after_sync();
#pragma unroll 1
              for (int i = 0; i < D; i += 16) {
                float o[16];
                tc::ld16(o_addr + i, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = fall == 0.f ? 0.f : o[e] * fall;
                tc::st16(o_addr + i, o);
              }
            }
          }
          const float ref = m == -INFINITY ? 0.f : m;
          const float2 scale2 = dup2(at.scale_log2), ref2 = dup2(-ref), minus2 = dup2(-1.f);
          float2 sum[4] = {dup2(0.f), dup2(0.f), dup2(0.f), dup2(0.f)};
#pragma unroll
          for (int k = 0; k < KT / 32; ++k) {
            uint32_t(&x)[32] = s[(k + KT / 32) & 1];
            tc::ld_wait(x);
            if (k + 1 < KT / 32) tc::ld32_async(s_addr + 32 * (k + 1), s[(k + 1 + KT / 32) & 1]);
            masked(x, s_live[at_mask][k]);
#pragma unroll
            for (int h = 0; h < 32; h += 16) {
              uint32_t w[16];  // 8 columns of hi, 8 of lo
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float2 y =
                    fma2(make_float2(__uint_as_float(x[h + 2 * i]), __uint_as_float(x[h + 2 * i + 1])), scale2, ref2);
                const float2 p = make_float2(ex2(y.x), ex2(y.y));
                sum[i & 3] = add2(sum[i & 3], p);
                // hi is the upper half of the float32, cut off; lo what is left, rounded
                const uint32_t u = __float_as_uint(p.x), v = __float_as_uint(p.y);
                w[i] = __byte_perm(u, v, 0x7632);
                const float2 rest =
                    fma2(make_float2(__uint_as_float(u & 0xffff0000u), __uint_as_float(v & 0xffff0000u)), minus2, p);
                w[8 + i] = pack_bf2(rest.x, rest.y);
              }
              tc::st16_async(s_addr + 32 * k + h, w);
            }
          }
          tc::st_wait();
          const float2 all = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
          l += all.x + all.y;
        }
        // The other lane's warps have read this one's last output.
        if (P::SPLIT && me == 1 && j < 2 && unit > 0 && !wait_or_abort(&x_empty, (unit - 1) & 1)) { run = false; break; }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[b]);
      }
      if (!run) break;
      // The unit's end in this piece: its rows' statistics and outputs.
      const int last = job - 1;
      if ((!P::SPLIT || me < count) &&
          !wait_or_abort(&o_done[LANES == 1 ? last & 1 : me], LANES == 1 ? (last >> 1) & 1 : last & 1)) {
        run = false;
        break;
      }
      tc::fence_after_sync();
      if (P::SPLIT && me == 1) {
        if (count < 2 && unit > 0 && !wait_or_abort(&x_empty, (unit - 1) & 1)) { run = false; break; }
        s_ml[row] = make_float2(m, l);
        tc::fence_before_sync();
        mbar_arrive(&x_full);
      } else {
        float other_scale = 0.f, scale = 1.f;
        if constexpr (P::SPLIT) {
          if (!wait_or_abort(&x_full, unit & 1)) { run = false; break; }
          tc::fence_after_sync();
          const float2 other = s_ml[row];
          const float top = fmaxf(m, other.x), ref = top == -INFINITY ? 0.f : top;
          scale = exp2f(m - ref);
          other_scale = exp2f(other.x - ref);
          l = fmaf(l, scale, other.y == 0.f ? 0.f : other.y * other_scale);
          m = top;
        }
        if (!idle) {
          const int i = walk.row_tile * ROWS + row_tile * kRows + row;  // query row
          const int n = walk.group.first + i / G;
          const bool mine = row < valid && takes_part(at, n, walk.group.prefix);
          float* dst = nullptr;
          if (mine) {
            const int64_t head = (int64_t)n * at.Hq + walk.head * G + i % G;
            if (begins) {
              ws.note[head] =
                  first_note(m, l, c, (int)piece_of(walk.unit_end - 1, T, pieces) - c, row_tile * kRows + row);
              dst = ws.o + head * D;
            } else {
              const int64_t at_piece = (int64_t)c * ROWS + row_tile * kRows + row;
              ws.ml[at_piece] = make_float2(m, l);
              dst = ws.more + at_piece * D;
            }
          }
#pragma unroll 1
          for (int k = 0; k < D / 32; ++k) {
            float o[32];
            tc::ld32(o_addr + 32 * k, o);
            if constexpr (P::SPLIT) {
              if (count > 1) {
                float x[32];
                tc::ld32(o_addr + D + 32 * k, x);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = fmaf(o[e], scale, x[e] * other_scale);
              }
            }
            if (mine) {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                reinterpret_cast<float4*>(dst + 32 * k)[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
          }
        }
        tc::fence_before_sync();
        if (P::SPLIT) mbar_arrive(&x_empty);
      }
      tile += count;
      ++unit;
      walk.tile = end;
      walk.next_unit(a);
    }
  } else if (warp == 4 * LANES) {
    // ---------------- matrix products ----------------
    constexpr uint32_t ID_S = tc::idesc_bf16(kRows, KT, false, false), ID_O = tc::idesc_bf16(kRows, D, false, true);
    const uint32_t q_addr = smem_addr(s_q), ring = smem_addr(s_ring);
    int half = 0;           // of the next K; its V is the one after it
    int unit = 0;
    uint32_t weighed = 0;  // parity of the outputs issued from each buffer
    bool run = any;
    // A half that has landed; the tensor cores read it through another proxy than the copies wrote it.
    const auto slot_wait = [&](int h) {
      const bool ok = wait_or_abort(&full[h % SLOTS], (h / SLOTS) & 1);
      fence_proxy_async_smem();
      return ok;
    };
    const uint32_t issue = tc::elect();
    const auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    // S of row tile r into buffer b from the keys in half h.
    const auto scores = [&](int q_slot, int r, int b, int h) {
      tc::fence_after_sync();
      const uint64_t q = tc::desc_sw128(q_addr + uniform(q_slot * RT + r) * P::Q_TILE, 16, 1024);
      const uint64_t k = tc::desc_sw128(ring + uniform(h % SLOTS) * P::HALF, 16, 1024);
      const int buffer = uniform(b);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)  // descriptors count in 16 bytes
        tc::mma_bf16_by(issue, taddr + P::S_COL + buffer * KT, q + ((ks >> 2) * (kRows * 128) + (ks & 3) * 32) / 16,
                        k + ((ks >> 2) * (KT * 128) + (ks & 3) * 32) / 16, ID_S, ks > 0);
      tc::commit_by(issue, &s_full[buffer]);
    };
    // Waits for the weights in buffer b; the output of lane o += them times the values in half h.
    const auto outputs = [&](int o, int b, int h, bool first) -> bool {
      const int buffer = uniform(b);
      if (!wait_or_abort(&p_full[buffer], weighed >> buffer & 1)) return false;
      weighed ^= 1u << buffer;
      tc::fence_after_sync();
      const uint64_t v = tc::desc_sw128(ring + uniform(h % SLOTS) * P::HALF, KT * 128, 1024);
      const uint32_t p = taddr + P::S_COL + buffer * KT, d = taddr + P::O_COL + uniform(o) * D;
      const bool onto = uniform(!first);
#pragma unroll
      for (int ks = 0; ks < KT / 16; ++ks)
#pragma unroll
        for (int piece = 0; piece < 2; ++piece)
          tc::mma_bf16_ta_by(issue, d, p + ks * 16 + piece * 8, v + ks * 2048 / 16, ID_O, onto || ks > 0 || piece > 0);
      tc::commit_by(issue, &o_done[buffer]);
      return true;
    };
    const auto release = [&](uint64_t* bar) { tc::commit_by(issue, bar); };
    int job = 0;
    while (run && walk.tile < stop) {
      const int count = (int)(min(walk.unit_end, stop) - walk.tile);
      const int q_slot = unit % P::QSLOTS;
      // the products of tile j with its keys, of tile j - 1 with its values
      for (int j = 0; j <= count && run; ++j) {
        const int hk = half + 2 * j, hv = hk - 1;
        if (j < count && !slot_wait(hk)) { run = false; break; }
        if constexpr (RT == 1) {
          const int b = P::SPLIT ? j & 1 : (job + j) & 1;
          if (j < count) {
            scores(q_slot, 0, b, hk);
            release(&empty[uniform(hk % SLOTS)]);
          }
          if (j > 0) {
            if (!slot_wait(hv) || !outputs(P::SPLIT ? b ^ 1 : 0, b ^ 1, hv, j <= (P::SPLIT ? 2 : 1))) { run = false; break; }
            release(&empty[uniform(hv % SLOTS)]);
          }
        } else {
          if (j > 0 && !slot_wait(hv)) { run = false; break; }
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            if (j > 0 && run && !outputs(r, r, hv, j == 1)) run = false;
            if (r == RT - 1 && j > 0 && run) release(&empty[uniform(hv % SLOTS)]);
            if (j < count && run) scores(q_slot, r, r, hk);
          }
          if (!run) break;
          if (j < count) release(&empty[uniform(hk % SLOTS)]);
        }
        if (j == count - 1) release(&q_empty[uniform(q_slot)]);
      }
      half += 2 * count;
      job += count;
      ++unit;
      walk.tile += count;
      if (walk.tile < stop) walk.next_unit(a);
    }
    release(&drained);  // every product issued has completed before the columns are freed
    mbar_sleep_wait(&drained, 0);
  } else {
    // ---------------- copies ----------------
    constexpr int CHUNKS = D / 8;                    // 16-byte pieces of a row
    constexpr int WARP_ROWS = KT / 4;                // keys of a warp
    constexpr int STEP_ROWS = 32 / CHUNKS;           // keys of one instruction
    static_assert(CHUNKS <= 32 && WARP_ROWS <= 32, "a row or more an instruction, a key or less a lane");
    const int lw = warp - (4 * LANES + 1);
    const int chunk = lane % CHUNKS, sub = lane / CHUNKS;
    const uint32_t ring = smem_addr(s_ring), q_addr = smem_addr(s_q);
    const auto place = [](int row, int ch, int rows) {  // of a 16-byte piece in an operand of `rows` rows
      return (uint32_t)((ch >> 3) * rows * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
    };
    // This lane's key of a tile: found a tile ahead of its copy.
    Walker ahead = walk;
    struct Look {
      int page, token, head;  // page 0: none
    };
    const auto look_up = [&]() {
      Look l{0, 0, 0};
      if (ahead.tile < stop) {
        const int t = (int)(ahead.tile - ahead.unit_start) * KT + lw * WARP_ROWS + lane;
        if (lane < WARP_ROWS && t < ahead.group.prefix) {
          const int col = t / at.page_size;
          l.token = t - col * at.page_size;
          l.page = __ldg(at.table + (int64_t)ahead.group.first * at.table_rs + col);
        }
        l.head = ahead.head;
        if (++ahead.tile == ahead.unit_end) ahead.next_unit(a);
      }
      return l;
    };
    int half = 0, tile = 0, unit = 0;
    bool run = any;
    const auto copy_half = [&](const void* data, int64_t offset, uint32_t mask) {
      const uint32_t base = ring + (half % SLOTS) * P::HALF;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(data);
#pragma unroll 4
      for (int i = 0; i < WARP_ROWS / STEP_ROWS; ++i) {
        const int k = i * STEP_ROWS + sub;
        const int64_t from = __shfl_sync(0xffffffffu, offset, k);
        copy16(base + place(lw * WARP_ROWS + k, chunk, KT), src + from + chunk * 8, mask >> k & 1);
      }
      copy_arrive(&full[half % SLOTS]);
      ++half;
    };
    Look look = any ? look_up() : Look{0, 0, 0};
    while (run && walk.tile < stop) {
      const int64_t end = min(walk.unit_end, stop);
      const int q_slot = unit % P::QSLOTS;
      if (unit >= P::QSLOTS) {
        if (!wait_or_abort(&q_empty[q_slot], (unit / P::QSLOTS - 1) & 1)) { run = false; break; }
      }
      {
        const int left = min(walk.rows_left(), ROWS), rows = (left + 31) & ~31;
        for (int i = tid - (4 * LANES + 1) * 32; i < rows * CHUNKS; i += kLoaders) {
          const int row = i / CHUNKS, ch = i % CHUNKS;
          const int q = walk.row_tile * ROWS + row;
          const bool real = row < left;
          const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(at.q);
          if (real)
            src += (int64_t)(walk.group.first + q / G) * at.q_rs + (int64_t)(walk.head * G + q % G) * at.q_hs + ch * 8;
          copy16(q_addr + (q_slot * RT + row / kRows) * P::Q_TILE + place(row % kRows, ch, kRows), src, real);
        }
      }
      for (; walk.tile < end; ++walk.tile, ++tile) {
        const Look next = look_up();
        const bool live = look.page > 0 && look.page < at.num_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, live);
        const auto offset = [&](const PageView& p) {
          return live ? look.page * p.page + look.token * p.token + look.head * p.head : 0;
        };
        if (half >= SLOTS && !wait_or_abort(&empty[half % SLOTS], (half / SLOTS - 1) & 1)) { run = false; break; }
        if (WARP_ROWS == 32) {
          if (lane == 0) s_live[tile % kLiveDepth][lw] = mask;
        } else if (lane == 0) {  // two warps a word
          reinterpret_cast<uint16_t*>(s_live[tile % kLiveDepth])[lw] = (uint16_t)mask;
        }
        if (lane == 0) mbar_arrive(&live_full[tile % kLiveDepth]);
        copy_half(at.kp.data, offset(at.kp), mask);
        if (half >= SLOTS && !wait_or_abort(&empty[half % SLOTS], (half / SLOTS - 1) & 1)) { run = false; break; }
        copy_half(at.vp.data, offset(at.vp), mask);
        look = next;
      }
      if (!run) break;
      ++unit;
      walk.next_unit(a);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // none lands when the CTA is gone
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == 4 * LANES) {
    tc::fence_after_sync();
    tc::dealloc(taddr, P::COLS);
  }
}

// Joins the parts of one query head of a sequence: of the common positions and of
// its own, each a first part and those of later pieces.  WARPS warps share the
// parts; a block of four warps joins one head or four.
template <int D, int WARPS>
__global__ void __launch_bounds__(128) kda_prefix_join_kernel(const __grid_constant__ AttendArgs a, const PrefixWork pre,
                                                              int ctas, int own_rows, int pre_ctas,
                                                              int pre_rows) {
  constexpr int VEC = D / 32, AHEAD = 4;
  __shared__ float s_m[4], s_l[4], s_o[WARPS > 1 ? 4 : 1][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t head = WARPS == 1 ? (int64_t)blockIdx.x * 4 + warp : blockIdx.x;
  if (head >= (int64_t)a.N * a.Hq) return;
  const Workspace own(a.work, ctas, own_rows, D);
  const float4 notes[2] = {pre.note[head], a.first_note[head]};
  // A kernel that gave up a wait has left notes that say anything: no part outside the workspace is read for them.
  int piece[2], row[2], more[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int packed = __float_as_int(notes[w].w), last = (w == 0 ? pre_ctas : ctas) - 1;
    piece[w] = __float_as_int(notes[w].z);
    row[w] = packed & 255;
    more[w] = packed >> 8;
    if (piece[w] < 0 || more[w] < 0 || piece[w] > last || more[w] > last - piece[w] ||
        row[w] >= (w == 0 ? pre_rows : own_rows))
      more[w] = 0;
  }
  const int parts0 = 1 + more[0], parts = parts0 + 1 + more[1];
  float m = -INFINITY, l = 0.f, o[VEC] = {};
#pragma unroll 1
  for (int i = WARPS == 1 ? 0 : warp; i < parts; i += WARPS * AHEAD) {
    float pm[AHEAD], pl[AHEAD], po[AHEAD][VEC];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int p = i + k * WARPS;
      pm[k] = -INFINITY;
      pl[k] = 0.f;
      const float* from = nullptr;
      if (p < parts) {
        const bool w = p >= parts0;
        const int j = w ? p - parts0 : p;
        if (j == 0) {
          pm[k] = w ? notes[1].x : notes[0].x;
          pl[k] = w ? notes[1].y : notes[0].y;
          from = (w ? a.first_o : pre.o) + head * D;
        } else {
          const int64_t place = w ? 2 * (int64_t)(piece[1] + j) * own_rows + row[1] : (int64_t)(piece[0] + j) * pre_rows + row[0];
          const float2 ml = w ? *reinterpret_cast<const float2*>(own.ml + 2 * place) : pre.ml[place];
          pm[k] = ml.x;
          pl[k] = ml.y;
          from = (w ? own.o : pre.more) + place * D;
        }
      }
#pragma unroll
      for (int v = 0; v < VEC; ++v) po[k][v] = 0.f;
      if (pl[k] != 0.f) {  // a part of no positions may have left no output
#pragma unroll
        for (int v = 0; v < VEC; v += 2) {
          const float2 x = *reinterpret_cast<const float2*>(from + lane * VEC + v);
          po[k][v] = x.x;
          po[k][v + 1] = x.y;
        }
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) top = fmaxf(top, pm[k]);
    const float ref = top == -INFINITY ? 0.f : top, f = exp2f(m - ref);
    l *= f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) o[v] *= f;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const float w = exp2f(pm[k] - ref);
      l = fmaf(pl[k], w, l);
#pragma unroll
      for (int v = 0; v < VEC; ++v) o[v] = fmaf(po[k][v], w, o[v]);
    }
    m = top;
  }
  const auto finish = [&](float M, float L, const float (&x)[VEC]) {
    const float scale = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int v = 0; v < VEC; v += 2)
      *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + head * D + lane * VEC + v) =
          pack_bf2(x[v] * scale, x[v + 1] * scale);
    if (a.lse != nullptr && lane == 0) a.lse[head] = log_sum(M == -INFINITY ? 0.f : M, L);
  };
  if constexpr (WARPS == 1) {
    finish(m, l, o);
  } else {
    if (lane == 0) {
      s_m[warp] = m;
      s_l[warp] = l;
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) s_o[warp][lane * VEC + v] = o[v];
    __syncthreads();
    if (warp > 0) return;
    float M = -INFINITY, L = 0.f, x[VEC] = {};
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, s_m[w]);
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = exp2f(s_m[w] - ref);
      L = fmaf(f, s_l[w], L);
#pragma unroll
      for (int v = 0; v < VEC; ++v) x[v] = fmaf(f, s_o[w][lane * VEC + v], x[v]);
    }
    finish(M, L, x);
  }
}

// Places of the workspace, in floats: the paged kernel's own, then both kernels'
// first parts, the prefix kernel's later ones and the sequences' skips.
struct PrefixPlan {
  AttendPlan own;
  int64_t own_note, own_o, note, o, ml, more, skip, floats;
};
PrefixPlan prefix_plan(int64_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t sms) {
  PrefixPlan p;
  p.own = attend_mma_plan(Hq / Hkv, D, sms);
  const int64_t heads = N * Hq, rows = (int64_t)sms * 2 * kRows;
  int64_t at = (p.own.floats + 3) & ~int64_t{3};
  const auto take = [&](int64_t floats) {
    const int64_t r = at;
    at += (floats + 3) & ~int64_t{3};
    return r;
  };
  p.own_note = take(4 * heads);
  p.own_o = take(heads * D);
  p.note = take(4 * heads);
  p.o = take(heads * D);
  p.ml = take(2 * rows);
  p.more = take(rows * D);
  p.skip = take(N);
  p.floats = at;
  return p;
}

template <int D, int RT>
cudaError_t launch_prefix(const PrefixArgs& a, const PrefixWork& ws, int sms, cudaStream_t s) {
  using P = PrefixShape<D, RT>;
  static std::atomic<bool> set[64];
  const cudaError_t e = allow_shared(kda_prefix_kernel<D, RT>, P::BYTES, set);
  if (e != cudaSuccess) return e;
  return launch_pdl(kda_prefix_kernel<D, RT>, dim3(sms), dim3(P::THREADS), P::BYTES, s, 1, a, ws);
}

template <int D>
cudaError_t launch_prefix_join(const AttendArgs& a, const PrefixWork& ws, const AttendPlan& own, int rows, int sms,
                               cudaStream_t s) {
  const int64_t heads = (int64_t)a.N * a.Hq;
  if (heads >= 16LL * sms)
    return launch_pdl(kda_prefix_join_kernel<D, 1>, dim3((unsigned)((heads + 3) / 4)), dim3(128), 0, s, 1, a, ws, own.ctas,
                      own.heads, sms, rows);
  return launch_pdl(kda_prefix_join_kernel<D, 4>, dim3((unsigned)heads), dim3(128), 0, s, 1, a, ws, own.ctas,
                      own.heads, sms, rows);
}

}  // namespace

int64_t prefix_floats(int64_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype, int32_t sms) {
  const int64_t paged = attend_floats(Hq, Hkv, D, dtype, sms);
  return dtype == KDA_DT_F32 ? paged : std::max(paged, prefix_plan(N, Hq, Hkv, D, sms).floats);
}

cudaError_t launch_prefix_attention(const PrefixArgs& given, int32_t sms, cudaStream_t s) {
  PrefixArgs a = given;
  AttendArgs& t = a.attend;
  if (t.dtype == KDA_DT_F32 || !t.vec16 || a.G >= t.N) return launch_paged_attention(t, sms, s);
  const PrefixPlan p = prefix_plan(t.N, t.Hq, t.Hkv, t.D, sms);
  PrefixWork ws;
  ws.note = reinterpret_cast<float4*>(t.work + p.note);
  ws.o = t.work + p.o;
  ws.ml = reinterpret_cast<float2*>(t.work + p.ml);
  ws.more = t.work + p.more;
  ws.skip = reinterpret_cast<int32_t*>(t.work + p.skip);
  const bool two = t.D < 256 && (int64_t)t.N * (t.Hq / t.Hkv) > (int64_t)kRows * a.G;
  cudaError_t e = cudaErrorInvalidValue;
  switch (t.D) {
    case 64: e = two ? launch_prefix<64, 2>(a, ws, sms, s) : launch_prefix<64, 1>(a, ws, sms, s); break;
    case 128: e = two ? launch_prefix<128, 2>(a, ws, sms, s) : launch_prefix<128, 1>(a, ws, sms, s); break;
    case 256: e = launch_prefix<256, 1>(a, ws, sms, s); break;
  }
  if (e != cudaSuccess) return e;
  t.skip = ws.skip;
  t.first_note = reinterpret_cast<float4*>(t.work + p.own_note);
  t.first_o = t.work + p.own_o;
  e = launch_attend_mma(t, p.own, s);
  if (e != cudaSuccess) return e;
  const int rows = two ? 2 * kRows : kRows;
  if (t.D == 64) return launch_prefix_join<64>(t, ws, p.own, rows, sms, s);
  if (t.D == 128) return launch_prefix_join<128>(t, ws, p.own, rows, sms, s);
  return launch_prefix_join<256>(t, ws, p.own, rows, sms, s);
}

cudaError_t read_prefix_error(unsigned int* flags, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_kda_prefix_error, sizeof(unsigned int));
  if (e != cudaSuccess || !clear) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_kda_prefix_error, &zero, sizeof(unsigned int));
}

}  // namespace kda
