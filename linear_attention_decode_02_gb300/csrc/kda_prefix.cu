// Attention of one new token per sequence where groups of sequences begin with
// the same positions: the common part is read once for up to 256 rows, the queries of a
// key head in all the group's sequences, by the tensor cores; each sequence's own part is
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
//   the next W warps      issue a lane's matrix products each (one warp for both was
//                         at work on issuing them for longer than they took)
//   four more             copy keys and values into shared memory
//   two more              copy queries
// Work goes in steps of 64 positions.  A lane has two buffers of scores S (128 rows x
// 64, float32), an output O and the warps between them: the scores of a step are
// issued before the output of the last one, so they are there when its softmax ends.
// With two row tiles each lane is one of them and both use every tile of keys and
// values; with one they take the tiles in turn, each to an output and statistics of
// its own, which are joined at the unit's end.  256 channels leave room for one
// output, and one lane.
// The row's thread puts the weights back over S as the next product's left operand,
// in two bfloat16 pieces, p = hi + lo to 2^-17, for 16 positions at a time 8 columns
// of hi and 8 of lo: one piece alone would cost each output 2^-9 of its weights'
// largest.  hi is rounded to nearest, as in the paged kernel; cut off, which leaves lo
// a bit more to hold, weights are good to 2^-16 and 256 users take 228 us instead of 232.
// Sums in tensor memory are cut to float32, not rounded: outputs over 7000 positions of
// a piece lean towards zero by 1.2e-5 of themselves, those of the paged kernel by 0.7e-5.
// Weights are relative to a reference that follows the row's maximum only
// where that has passed it by 2^kSlack, so O, which lies in tensor memory, is seldom
// rescaled.
//
// Products of one accumulator and shape complete in the order in which they are issued;
// for others PTX promises none.  So scores that go where weights were wait for the
// product that read those.
//
// A barrier's parity tells two phases apart, so each is waited for, or known to be
// over, before the next: the scores of a buffer wait for every product of the weights
// that were in it, so no second phase of that product passes unseen.  Lanes that
// take tiles in turn do not wait for each other's halves of the ring: a tile's mask is
// given when what was in both its slots has been used, and a lane waits for the mask
// before it waits for either half (given with the keys' slot, the values' barrier could
// still be in the phase before the last one, which looks like the one waited for).
//
// What bounds it, at 32 / 8 heads of 128 (the launch alone under a profiler, in us):
//   16 prompts of 8192 positions, four beams each (one row tile): 77, 392 MB at 64 % of DRAM's rate;
//     the steps of a lane wait for one another, and a ring of five halves holds little
//   256 users of one system prompt of 32768 (two row tiles): 158, tensor pipe 55 %; a step of 64 positions
//     takes both lanes 2300 cycles, 1536 of them the tensor pipe's for its products, 1250 its softmax
// Tried: one warp that issues both lanes' products (246 -> 300 us a call), tiles of 64
// positions (76 -> 104, 155 -> 171: twice the copies' bookkeeping, and values held
// through two more tiles), scores first at a tile's end with one row tile (76 -> 88),
// parts laid out in planes of 8 channels, so that a warp's stores join (152 -> 153, and
// the join 16 -> 18).  Of a piece's 283000 cycles 26000 pass before its first weights
// (lengths and groups 6000, table, keys and queries 16000), 12000 with its last output.
// Compiled for 128 registers a thread, 80 bytes of one spill (with 256 channels, 150 registers, none).
//
// The kernel of own positions reads nothing that this one writes and writes elsewhere.
// So it begins as this one's blocks leave, all of which have waited for what came
// before the call, and waits for this one at its own end: 101 -> 94 us for the 16
// prompts, 243 -> 229 for the 256 users.
//
// Every mbarrier wait is bounded in time: a role whose wait runs out records a bit
// in the error word, raises the CTA's abort flag and leaves its loop; all meet at
// the end before tensor memory is freed.
#include <algorithm>

#include "kda_attend_rows.cuh"
#include "kda_stream_common.cuh"
#include "kda_tcgen05.cuh"

namespace kda {

// bit 4: a wait of the shared-prefix attention kernel timed out.
__device__ unsigned int g_kda_prefix_error = 0;

namespace {

constexpr int kRows = 128;       // rows of a tile
constexpr int kLoaders = 128;    // threads
constexpr int kQueryThreads = 64;
constexpr float kSlack = 4.f;    // in units of log 2
constexpr int kLiveDepth = 16;   // tiles whose masks are kept
constexpr int kStep = 64;        // positions that a softmax takes at once

template <int D, int RT>
struct PrefixShape {
  static constexpr int KT = D == 256 ? 64 : 128;   // positions of a tile
  static constexpr int STEPS = KT / kStep;         // of a tile
  static constexpr int BLOCKS = D / 64;            // 128-byte wide column blocks of an operand
  static constexpr int Q_TILE = BLOCKS * kRows * 128;
  static constexpr int QSLOTS = RT == 1 && D < 256 ? 2 : 1;
  static constexpr int HALF = BLOCKS * KT * 128;   // keys or values of a tile
  static constexpr int SLOTS = D == 64 ? 12 : 5;
  static constexpr int BYTES = QSLOTS * RT * Q_TILE + SLOTS * HALF + 1024;
  static constexpr int LANES = D == 256 ? 1 : 2;
  static constexpr bool SPLIT = RT < LANES;        // lanes take tiles in turn
  static constexpr int THREADS = LANES == 1 ? 11 * 32 : 16 * 32;
  // first warps of the roles
  static constexpr int LOADER0 = LANES == 1 ? 5 : 8, PRODUCT0 = LANES == 1 ? 4 : 12, QUERY0 = LANES == 1 ? 9 : 14;
  static constexpr uint32_t S_COL = 0, O_COL = LANES * 2 * kStep;   // two buffers of S for each lane, then its O
  static constexpr uint32_t COLS = 512;
  static_assert(O_COL + LANES * D <= COLS && RT <= LANES, "tensor memory");
  static_assert(SLOTS / 2 + 4 <= kLiveDepth, "ring");
};

// Registers of the four warps of a group: up to N, down to -N, 0: as they are.
template <int N>
__device__ __forceinline__ void more_registers() {
  if constexpr (N > 0) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
  if constexpr (N < 0) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(-N));
}
// A box of rows x 64 channels to shared memory, its 16-byte pieces swizzled over 128-byte rows.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int token, int head, int page,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(token), "r"(head), "r"(page), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(map)) : "memory");
}
// mbar_sleep_wait behind a try that gave up, with another before the clock is read: 256 users 232.4 us without, 231.2 with it.
__device__ __forceinline__ bool wait_longer(uint64_t* bar, uint32_t parity) {
  return mbar_sleep_try(bar, parity) || mbar_sleep_wait(bar, parity);
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int D, int RT>
__global__ void __launch_bounds__(PrefixShape<D, RT>::THREADS, 1)
    kda_prefix_kernel(const __grid_constant__ AttendArgs a, int box,
                      const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  using P = PrefixShape<D, RT>;
  constexpr int KT = P::KT, ROWS = RT * kRows, SLOTS = P::SLOTS, LANES = P::LANES;
  using Walker = GroupWalk<KT, ROWS>;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* sm = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                       ~static_cast<uintptr_t>(1023));
  unsigned char* const s_q = sm;
  unsigned char* const s_ring = sm + P::QSLOTS * RT * P::Q_TILE;
  __shared__ uint64_t full[SLOTS], empty[SLOTS], s_full[2 * LANES], p_full[2 * LANES], o_done[2 * LANES],
      q_full[P::QSLOTS], q_empty[P::QSLOTS], live_full[kLiveDepth], x_full, x_empty, drained[LANES];
  __shared__ float2 s_ml[P::SPLIT ? kRows : 1];
  __shared__ __align__(8) uint32_t s_live[kLiveDepth][KT / 32];
  __shared__ uint32_t s_taddr;
  __shared__ volatile int s_abort;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int C = gridDim.x, c = blockIdx.x;

  if (tid == 0) {
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&full[i], kLoaders);
      mbar_init(&empty[i], RT);  // the lanes that use a half
    }
    for (int i = 0; i < 2 * LANES; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], kRows / 32);
      mbar_init(&o_done[i], 1);
    }
    for (int i = 0; i < P::QSLOTS; ++i) {
      mbar_init(&q_full[i], kQueryThreads);
      mbar_init(&q_empty[i], LANES);
    }
    for (int i = 0; i < kLiveDepth; ++i) mbar_init(&live_full[i], kLoaders / 32);
    mbar_init(&x_full, kRows);
    mbar_init(&x_empty, kRows);
    for (int i = 0; i < LANES; ++i) mbar_init(&drained[i], 1);
    s_abort = 0;
    mbar_fence_init();
  }
  if (tid == P::LOADER0 * 32 && box > 0) {
    prefetch_map(&k_map);
    prefetch_map(&v_map);
  }
  if (warp == P::PRODUCT0) tc::alloc(&s_taddr, P::COLS);
  pdl_wait();
  pdl_launch_dependents();

  tc::fence_before_sync();
  const Place piece = find_group_place<P::THREADS, KT, ROWS>(a, c, C);  // every thread passes a barrier in it
  tc::fence_after_sync();
  const uint32_t taddr = s_taddr;
  const int64_t start = piece.start, stop = piece.stop;

  // Nearly every wait ends with its first try, which looks at nothing else.
  auto wait_or_abort = [&](uint64_t* bar, uint32_t parity) -> bool {
    if (__all_sync(0xffffffffu, mbar_sleep_try(bar, parity))) return true;
    const bool stopped = s_abort;  // by another role
    const bool ok = !stopped && wait_longer(bar, parity);
    if (__all_sync(0xffffffffu, ok)) return true;
    if (lane == 0 && !stopped) {
      atomicOr(&g_kda_prefix_error, 16u);
      s_abort = 1;
    }
    return false;
  };
  constexpr int CHUNKS = D / 8;  // 16-byte pieces of a row
  const auto place = [](int row, int ch, int rows) {  // of a 16-byte piece in an operand of `rows` rows
    return (uint32_t)((ch >> 3) * rows * 128 + row * 128 + (((ch & 7) ^ (row & 7)) << 4));
  };
  const bool any = start < stop;
  Walker walk;
  if (any) walk.start(a, piece);

  if (warp < 4 * LANES) {
    more_registers<LANES == 1 ? 0 : 144>();
    // ---------------- softmax ----------------
    leave_empty_parts(a, c * 4 * LANES + warp, C * 4 * LANES, lane);
    const int me = LANES == 1 ? 0 : warp >> 2;   // lane of the CTA
    const int row_tile = RT == 1 ? 0 : me;
    const int row = (warp & 3) * 32 + lane;      // of the row tile, and tensor-memory lane
    const uint32_t tl = taddr + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t o_addr = tl + P::O_COL + me * D;
    int tile = 0, job = 0, unit = 0;  // tiles of the piece, this lane's steps and units so far
    bool run = any;
    while (run && walk.tile < stop) {
      const int valid = walk.rows_left() - row_tile * kRows;  // rows of this tile that exist
      const bool idle = valid <= (warp & 3) * 32;             // none of this warp's
      float m = -INFINITY, l = 0.f;
      const int64_t end = min(walk.unit_end, stop);
      const int count = (int)(end - walk.tile);
      const bool begins = walk.unit_start >= start;
      const int steps = (P::SPLIT ? (count + 1 - me) / 2 : count) * P::STEPS;  // this lane's
      for (int i = 0; i < steps; ++i, ++job) {
        const int j = tile + i / P::STEPS * (P::SPLIT ? 2 : 1) + (P::SPLIT ? me : 0), at_mask = j % kLiveDepth;
        const int b = 2 * me + (job & 1);
        if (!wait_or_abort(&s_full[b], (job >> 1) & 1) ||
            (i % P::STEPS == 0 && !wait_or_abort(&live_full[at_mask], (j / kLiveDepth) & 1))) {
          run = false;
          break;
        }
        tc::fence_after_sync();
        if (!idle) {
          const uint32_t s_addr = tl + P::S_COL + b * kStep;
          uint32_t x[kStep];
          tc::ld64_async(s_addr, x);
          const uint2 word = *reinterpret_cast<const uint2*>(&s_live[at_mask][i % P::STEPS * 2]);
          tc::ld_wait(x);
          if ((word.x & word.y) != 0xffffffffu) {
#pragma unroll
            for (int e = 0; e < kStep; ++e) x[e] = (e < 32 ? word.x : word.y) >> (e & 31) & 1 ? x[e] : 0xff800000u;  // -infinity
          }
          float tops[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            tops[e] = __uint_as_float(x[e]);
#pragma unroll
            for (int k = 4; k < 60; k += 8) tops[e] = max3(tops[e], __uint_as_float(x[k + e]), __uint_as_float(x[k + e + 4]));
            tops[e] = fmaxf(tops[e], __uint_as_float(x[60 + e]));
          }
          const float top = max3(fmaxf(tops[0], tops[1]), tops[2], tops[3]) * a.scale_log2;
          const bool rises = top > m + kSlack || (m == -INFINITY && top > m);
          if (__any_sync(0xffffffffu, rises)) {
            const float fall = rises ? (m == -INFINITY ? 0.f : ex2(m - top)) : 1.f;
            if (rises) m = top;
            l *= fall;
            if (i > 0) {  // the last step's product may still run
              if (!wait_or_abort(&o_done[2 * me + ((job - 1) & 1)], ((job - 1) >> 1) & 1)) { run = false; break; }
              tc::fence_after_sync();
#pragma unroll 1
              for (int k = 0; k < D; k += 16) {
                float o[16];
                tc::ld16(o_addr + k, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = fall == 0.f ? 0.f : o[e] * fall;
                tc::st16(o_addr + k, o);
              }
            }
          }
          const float2 scale2 = dup2(a.scale_log2), minus2 = dup2(-1.f), ref2 = dup2(m == -INFINITY ? 0.f : -m);
          float2 sum[4] = {dup2(0.f), dup2(0.f), dup2(0.f), dup2(0.f)};
#pragma unroll
          for (int h = 0; h < kStep; h += 16) {
            uint32_t w[16];  // 8 columns of hi, 8 of lo
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 y =
                  fma2(make_float2(__uint_as_float(x[h + 2 * e]), __uint_as_float(x[h + 2 * e + 1])), scale2, ref2);
              const float2 p = make_float2(ex2(y.x), ex2(y.y));
              sum[e & 3] = add2(sum[e & 3], p);
              w[e] = pack_bf2(p.x, p.y);
              const float2 rest = fma2(make_float2(bf_lo(w[e]), bf_hi(w[e])), minus2, p);
              w[8 + e] = pack_bf2(rest.x, rest.y);
            }
            tc::st16_async(s_addr + h, w);
          }
          tc::st_wait();
          const float2 all = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
          l += all.x + all.y;
        }
        // The other lane's warps have read this one's last output.
        if (P::SPLIT && me == 1 && i == 0 && unit > 0 && !wait_or_abort(&x_empty, (unit - 1) & 1)) { run = false; break; }
        tc::fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[b]);
      }
      if (!run) break;
      // The unit's end in this piece: its rows' statistics and outputs.
      if (steps > 0 && !wait_or_abort(&o_done[2 * me + ((job - 1) & 1)], ((job - 1) >> 1) & 1)) { run = false; break; }
      tc::fence_after_sync();
      if (P::SPLIT && me == 1) {
        if (steps == 0 && unit > 0 && !wait_or_abort(&x_empty, (unit - 1) & 1)) { run = false; break; }
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
          const int r = row_tile * kRows + row;  // of the unit
          const int2 of = walk.row(a, r);
          const bool mine = row < valid && takes_part(a, of.x, walk.of.prefix);
          float* dst = nullptr;
          if (mine) {
            const int64_t head = (int64_t)of.x * a.Hq + of.y, later = (int64_t)c * ROWS + r;
            if (begins) {
              const int pieces = pieces_of(piece.T, C);
              a.parts.first_note[head] = part_note(c, (int)piece_of(walk.unit_end - 1, piece.T, pieces) - c, r);
            }
            (begins ? a.parts.first_ml[head] : a.parts.more_ml[later]) = make_float2(m, l);
            dst = begins ? a.parts.first_o + head * D : a.parts.more_o + later * D;
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
  } else if (warp >= P::PRODUCT0 && warp < P::PRODUCT0 + LANES) {
    more_registers<LANES == 1 ? 0 : -112>();
    // ---------------- matrix products, a warp for each lane ----------------
    constexpr uint32_t ID_S = tc::idesc_bf16(kRows, kStep, false, false), ID_O = tc::idesc_bf16(kRows, D, false, true);
    const uint32_t q_addr = smem_addr(s_q), ring = smem_addr(s_ring);
    const uint32_t issue = tc::elect();
    const auto uniform = [](int x) { return __shfl_sync(0xffffffffu, x, 0); };
    const int me = uniform(warp - P::PRODUCT0), row_tile = RT == 1 ? 0 : me;
    int half = 0, tile = 0, unit = 0, job = 0;  // of the next K, whose V is the one after it; tiles, units and steps so far
    bool run = any;
    const auto release = [&](uint64_t* bar) { tc::commit_by(issue, bar); };
    // A half that has landed.  What threads copied the tensor cores read through another proxy.
    const auto slot_wait = [&](int h, bool threads) {
      if (!wait_or_abort(&full[h % SLOTS], (h / SLOTS) & 1)) return false;
      if (threads) fence_proxy_async_smem();
      return true;
    };
    while (run && walk.tile < stop) {
      const int count = (int)(min(walk.unit_end, stop) - walk.tile);
      const int q_slot = unit % P::QSLOTS;
      const int steps = (P::SPLIT ? (count + 1 - me) / 2 : count) * P::STEPS;
      bool threads = true, behind = true;  // whether threads copied any of this step's tile, and of the last one's
      const auto tile_of = [&](int i) { return i / P::STEPS * (P::SPLIT ? 2 : 1) + (P::SPLIT ? me : 0); };
      const auto scores = [&](int i) {
        const int j = tile_of(i), hk = half + 2 * j, sub = i % P::STEPS;
        behind = threads;
        if (i == 0 && !wait_or_abort(&q_full[q_slot], (unit / P::QSLOTS) & 1)) return false;
        if (sub == 0) {
          const int at_mask = (tile + j) % kLiveDepth;
          if (!wait_or_abort(&live_full[at_mask], ((tile + j) / kLiveDepth) & 1)) return false;
          threads = box == 0;
#pragma unroll
          for (int k = 0; k < KT / 32; ++k) threads = threads || s_live[at_mask][k] != 0xffffffffu;
          if (!slot_wait(hk, threads || i == 0)) return false;  // the queries are always copied by threads
        }
        const int g = job + i, b = uniform(2 * me + (g & 1));
        if (g >= 2 && !wait_or_abort(&o_done[b], ((g >> 1) - 1) & 1)) return false;  // has read the weights that were in S
        tc::fence_after_sync();
        const uint64_t q = tc::desc_sw128(q_addr + uniform(q_slot * RT + row_tile) * P::Q_TILE, 16, 1024);
        const uint64_t k = tc::desc_sw128(ring + uniform(hk % SLOTS) * P::HALF + uniform(sub) * (kStep * 128), 16, 1024);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)  // descriptors count in 16 bytes
          tc::mma_bf16_by(issue, taddr + P::S_COL + b * kStep, q + ((ks >> 2) * (kRows * 128) + (ks & 3) * 32) / 16,
                          k + ((ks >> 2) * (KT * 128) + (ks & 3) * 32) / 16, ID_S, ks > 0);
        release(&s_full[b]);
        if (sub == P::STEPS - 1) release(&empty[uniform(hk % SLOTS)]);
        return true;
      };
      const auto output = [&](int i, bool by_threads) {
        const int hv = half + 2 * tile_of(i) + 1, sub = i % P::STEPS, b = uniform(2 * me + ((job + i) & 1));
        if (sub == 0 && !slot_wait(hv, by_threads)) return false;
        if (!wait_or_abort(&p_full[b], ((job + i) >> 1) & 1)) return false;
        tc::fence_after_sync();
        const uint64_t v = tc::desc_sw128(ring + uniform(hv % SLOTS) * P::HALF + uniform(sub) * (kStep * 128), KT * 128, 1024);
        const uint32_t p = taddr + P::S_COL + b * kStep, d = taddr + P::O_COL + me * D;
        const bool onto = uniform(i > 0);
#pragma unroll
        for (int ks = 0; ks < kStep / 16; ++ks)
#pragma unroll
          for (int piece = 0; piece < 2; ++piece)
            tc::mma_bf16_ta_by(issue, d, p + ks * 16 + piece * 8, v + ks * 2048 / 16, ID_O, onto || ks > 0 || piece > 0);
        release(&o_done[b]);
        if (sub == P::STEPS - 1) release(&empty[uniform(hv % SLOTS)]);
        return true;
      };
      // Scores of step i, then the output of step i - 1, whose softmax ran meanwhile.  Lanes that take tiles in turn run
      // under each other, and would only hold the values while the next keys are on their way: output first between tiles.
      for (int i = 0; run && i <= steps; ++i) {
        const bool first = P::SPLIT && i % P::STEPS == 0;
        if (first && i > 0) run = output(i - 1, threads);
        if (run && i < steps) run = scores(i);
        if (!first && run && i > 0) run = output(i - 1, i < steps ? behind : threads);
      }
      // A lane without a tile of the unit waits for its queries all the same: it would run ahead, and its arrivals for this
      // unit and the next in the slot would pass for both lanes' of one.
      if (steps == 0 && run) run = wait_or_abort(&q_full[q_slot], (unit / P::QSLOTS) & 1);
      if (!run) break;
      release(&q_empty[uniform(q_slot)]);
      half += 2 * count;
      tile += count;
      job += steps;
      ++unit;
      walk.tile += count;
      if (walk.tile < stop) walk.next_unit(a);
    }
    release(&drained[me]);  // every product issued has completed before the columns are freed
    wait_longer(&drained[me], 0);
  } else if (warp >= P::LOADER0 && warp < P::LOADER0 + kLoaders / 32) {
    more_registers<LANES == 1 ? 0 : -112>();
    // ---------------- copies ----------------
    constexpr int WARP_ROWS = KT / 4;                // keys of a warp
    constexpr int STEP_ROWS = 32 / CHUNKS;           // keys of one instruction
    static_assert(CHUNKS <= 32 && WARP_ROWS <= 32, "a row or more an instruction, a key or less a lane");
    const int lw = warp - P::LOADER0;
    const int chunk = lane % CHUNKS, sub = lane / CHUNKS;
    const uint32_t ring = smem_addr(s_ring);
    // This lane's key of a tile: found a tile ahead of its copy.
    Walker ahead = walk;
    struct Look {
      int page, token, head;  // page 0: none
    };
    const auto look_up = [&]() {
      Look l{0, 0, 0};
      if (ahead.tile < stop) {
        const int t = (int)(ahead.tile - ahead.unit_start) * KT + lw * WARP_ROWS + lane;
        if (lane < WARP_ROWS && t < ahead.of.prefix) {
          const int col = t / a.page_size;
          l.token = t - col * a.page_size;
          l.page = __ldg(a.table + (int64_t)ahead.of.first * a.table_rs + col);
        }
        l.head = ahead.group;
        if (++ahead.tile == ahead.unit_end) ahead.next_unit(a);
      }
      return l;
    };
    int half = 0, tile = 0;
    bool run = any;
    // This warp's keys or values of a tile: by TMA where all are there and pages hold whole boxes, by threads, which put
    // zeros in the place of what is not attended to, otherwise.
    const auto copy_half = [&](const PageView& view, const CUtensorMap* map, const Look& look, uint32_t mask) {
      const uint32_t base = ring + (half % SLOTS) * P::HALF;
      uint64_t* const bar = &full[half % SLOTS];
      if (box > 0 && mask == (WARP_ROWS == 32 ? 0xffffffffu : (1u << WARP_ROWS) - 1)) {
        if (lane == 0) mbar_expect_tx(bar, WARP_ROWS * D * 2);
        __syncwarp();
        if (lane < WARP_ROWS && lane % box == 0) {
#pragma unroll
          for (int b = 0; b < P::BLOCKS; ++b)
            tma_load_4d(base + (b * KT + lw * WARP_ROWS + lane) * 128, map, 64 * b, look.token, look.head, look.page, bar);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_many(bar, 32);
        ++half;
        return;
      }
      const int64_t offset =
          mask >> lane & 1 ? look.page * view.page + look.token * view.token + look.head * view.head : 0;
      const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(view.data);
#pragma unroll 4
      for (int i = 0; i < WARP_ROWS / STEP_ROWS; ++i) {
        const int k = i * STEP_ROWS + sub;
        const int64_t from = __shfl_sync(0xffffffffu, offset, k);
        copy16(base + place(lw * WARP_ROWS + k, chunk, KT), src + from + chunk * 8, mask >> k & 1);
      }
      copy_arrive(bar);
      ++half;
    };
    Look look = any ? look_up() : Look{0, 0, 0};
    while (run && walk.tile < stop) {
      const int64_t end = min(walk.unit_end, stop);
      for (; walk.tile < end; ++walk.tile, ++tile) {
        const Look next = look_up();
        const bool live = look.page > 0 && look.page < a.num_pages;
        const uint32_t mask = __ballot_sync(0xffffffffu, live);
        if (half >= SLOTS && !wait_or_abort(&empty[half % SLOTS], (half / SLOTS - 1) & 1)) { run = false; break; }
        if (WARP_ROWS == 32) {
          if (lane == 0) s_live[tile % kLiveDepth][lw] = mask;
        } else if (lane == 0) {  // two warps a word
          reinterpret_cast<uint16_t*>(s_live[tile % kLiveDepth])[lw] = (uint16_t)mask;
        }
        copy_half(a.kp, &k_map, look, mask);
        if (half >= SLOTS && !wait_or_abort(&empty[half % SLOTS], (half / SLOTS - 1) & 1)) { run = false; break; }
        if (lane == 0) mbar_arrive(&live_full[tile % kLiveDepth]);  // both halves' slots are free
        copy_half(a.vp, &v_map, look, mask);
        look = next;
      }
      if (!run) break;
      walk.next_unit(a);
    }
    // No copy lands when the CTA is gone; all have been waited for but where a role gave up.
    asm volatile("cp.async.wait_all;" ::: "memory");
    for (int h = max(0, half - SLOTS); h < half; ++h) wait_longer(&full[h % SLOTS], (h / SLOTS) & 1);
  } else {
    more_registers<LANES == 1 ? 0 : -112>();
    // ---------------- queries of the units ----------------
    // A thread's rows are STEP apart; addresses only step (with divisions and products for
    // each row, on the loaders, a unit's queries took 10000 cycles).
    constexpr int STEP = kQueryThreads / CHUNKS;
    const int t = tid - P::QUERY0 * 32, chunk = t % CHUNKS, first_row = t / CHUNKS;
    const int G = a.Hq / a.Hkv, over = STEP % G;
    const int64_t step = STEP / G * a.q_rs + over * a.q_hs, wrap = a.q_rs - G * a.q_hs;
    const __nv_bfloat16* const q = static_cast<const __nv_bfloat16*>(a.q) + chunk * 8;
    for (int unit = 0; walk.tile < stop && any; ++unit) {
      const int q_slot = unit % P::QSLOTS;
      if (unit >= P::QSLOTS && !wait_or_abort(&q_empty[q_slot], (unit / P::QSLOTS - 1) & 1)) break;
      const int left = min(walk.rows_left(), ROWS), rows = (left + 31) & ~31, i = walk.row_tile * ROWS + first_row;
      int head = i % G;
      const __nv_bfloat16* src = q + (walk.of.first + i / G) * a.q_rs + (walk.group * G + head) * a.q_hs;
      const uint32_t dst = smem_addr(s_q) + q_slot * RT * P::Q_TILE + place(first_row, chunk, kRows);
#pragma unroll 4
      for (int row = first_row; row < rows; row += STEP) {
        const int on = row - first_row, tile = RT == 1 ? 0 : row / kRows;
        copy16((dst + on * 128 + tile * (P::Q_TILE - kRows * 128)) ^ ((on & 7) << 4), row < left ? src : q, row < left);
        src += step;
        head += over;
        if (head >= G) {
          head -= G;
          src += wrap;
        }
      }
      copy_arrive(&q_full[q_slot]);
      walk.tile = min(walk.unit_end, stop);
      if (walk.tile < stop) walk.next_unit(a);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }

  tc::fence_before_sync();
  __syncthreads();
  if (warp == P::PRODUCT0) {
    tc::fence_after_sync();
    tc::dealloc(taddr, P::COLS);
  }
}

// Joins the parts of one query head of a sequence, `pre` of the common positions
// and `own` of its own.  WARPS warps share the parts; a block of four warps joins one
// head or four.
template <int D, int WARPS>
__global__ void __launch_bounds__(128) kda_prefix_join_kernel(const __grid_constant__ AttendArgs a, const Parts pre,
                                                              const Parts own) {
  // Parts read at once: 34 parts of 64 channels (7 groups of 20, 12 heads) 37 -> 32 us a call for eight, 128 channels 97 -> 98
  constexpr int VEC = D / 32, AHEAD = D == 64 ? 8 : 4;
  __shared__ float s_m[4], s_l[4], s_o[WARPS > 1 ? 4 : 1][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t heads = (int64_t)a.N * a.Hq, head = WARPS == 1 ? (int64_t)blockIdx.x * 4 + warp : blockIdx.x;
  if (head >= heads) return;
  const int2 notes[2] = {pre.first_note[head], own.first_note[head]};
  // A kernel that gave up a wait has left notes that say anything: no part outside the workspace is read for them.
  int piece[2], row[2], more[2];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int ctas = w == 0 ? pre.ctas : own.ctas;
    piece[w] = notes[w].x;
    row[w] = notes[w].y & 255;
    more[w] = notes[w].y >> 8;
    if (piece[w] < 0 || more[w] < 0 || piece[w] >= ctas || more[w] >= ctas - piece[w] ||
        row[w] >= (w == 0 ? pre.rows : own.rows))
      more[w] = 0;
  }
  const int parts0 = pre.warps * (1 + more[0]), parts = parts0 + own.warps * (1 + more[1]);
  float m = -INFINITY, l = 0.f, o[VEC] = {};
#pragma unroll 1
  for (int i = WARPS == 1 ? 0 : warp; i < parts; i += WARPS * AHEAD) {
    float pm[AHEAD], pl[AHEAD], po[AHEAD][VEC];
    const float* from[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int q = i + k * WARPS;
      pm[k] = -INFINITY;
      pl[k] = 0.f;
      from[k] = nullptr;
      if (q < parts) {
        const bool w = q >= parts0;
        const int at = w ? q - parts0 : q, warps = w ? own.warps : pre.warps;
        const bool first = at < warps;  // of the piece that begins the unit
        const int64_t place = first ? at * heads + head
                                    : ((int64_t)(w ? piece[1] : piece[0]) * warps + at) * (w ? own.rows : pre.rows) +
                                          (w ? row[1] : row[0]);
        const float2 ml = (w ? (first ? own.first_ml : own.more_ml) : (first ? pre.first_ml : pre.more_ml))[place];
        pm[k] = ml.x;
        pl[k] = ml.y;
        from[k] = (w ? (first ? own.first_o : own.more_o) : (first ? pre.first_o : pre.more_o)) + place * D;
      }
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) po[k][v] = 0.f;
      if (pl[k] != 0.f) {  // a part of no positions may have left no output
#pragma unroll
        for (int v = 0; v < VEC; v += 2) {
          const float2 x = *reinterpret_cast<const float2*>(from[k] + lane * VEC + v);
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

// The paged kernel's grid for sequences' own positions, the kernel over the groups' common ones, both kernels' parts
// in the workspace, and its size.
struct PrefixPlan {
  AttendPlan own, pre;
  Parts own_parts, pre_parts;
  int64_t floats;
};
PrefixPlan prefix_plan(float* work, int64_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype, int32_t sms, int64_t groups) {
  PrefixPlan p;
  int64_t at = 0;
  const auto take = [&](int64_t floats) {
    float* r = reinterpret_cast<float*>(reinterpret_cast<uintptr_t>(work) + 4 * at);  // work may be null, for the size
    at += (floats + 3) & ~int64_t{3};
    return r;
  };
  const int64_t heads = N * Hq;
  const auto parts = [&](int ctas, int warps, int rows, int most_rows) {
    Parts r;
    const int64_t later = (int64_t)ctas * warps * most_rows;
    r.first_note = reinterpret_cast<int2*>(take(2 * heads));
    r.first_ml = reinterpret_cast<float2*>(take(2 * warps * heads));
    r.first_o = take(warps * heads * D);
    r.more_ml = reinterpret_cast<float2*>(take(2 * later));
    r.more_o = take(later * D);
    r.ctas = ctas;
    r.warps = warps;
    r.rows = rows;
    return r;
  };
  const int32_t G = Hq / Hkv;
  // Query rows that a group has a key head, on average, decide how many a unit takes.
  const double rows = groups > 0 ? (double)N * G / groups : 0;
  if (dtype == KDA_DT_F32) {
    p.own = attend_tf32_plan(G, D, sms);
    p.pre = attend_tf32_plan(rows <= 8 ? 8 : 16, D, sms);
    p.own_parts = parts(p.own.ctas, kTf32PartWarps, p.own.heads, p.own.heads);
    p.pre_parts = parts(p.pre.ctas, kTf32PartWarps, p.pre.heads, 16);
  } else {
    p.own = attend_mma_plan(G, D, sms);
    p.pre.ctas = sms;
    p.pre.heads = D < 256 && rows > kRows ? 2 * kRows : kRows;
    const int alone = own_warps_alone(D);
    p.own_parts = parts(p.own.ctas * alone, kAttendWarps / alone, p.own.heads, p.own.heads);
    p.pre_parts = parts(p.pre.ctas, 1, p.pre.heads, 2 * kRows);
  }
  p.floats = at;
  return p;
}

// The pages as [num_pages][Hkv][page_size][D], boxes of `rows` positions and 64 channels.
bool encode_pages(CUtensorMap* map, const PageView& p, const AttendArgs& a, int rows) {
  EncodeTiledFn encode = encode_tiled();
  if (encode == nullptr) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)a.D, (cuuint64_t)a.page_size, (cuuint64_t)a.Hkv, (cuuint64_t)a.num_pages};
  // an axis of one element may have any stride, which the map need not accept
  const auto bytes = [&](int64_t stride, int64_t extent) { return (cuuint64_t)(extent > 1 ? stride : a.D) * 2; };
  const cuuint64_t strides[3] = {bytes(p.token, a.page_size), bytes(p.head, a.Hkv), bytes(p.page, a.num_pages)};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, 1, 1}, steps[4] = {1, 1, 1, 1};
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, p.data, dims, strides, box, steps,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, int RT>
cudaError_t launch_prefix(const AttendArgs& a, int sms, cudaStream_t s) {
  using P = PrefixShape<D, RT>;
  static std::atomic<bool> set[64];
  const cudaError_t e = allow_shared(kda_prefix_kernel<D, RT>, P::BYTES, set);
  if (e != cudaSuccess) return e;
  // A warp's positions of a tile are whole boxes, of whole eights as the swizzle repeats, and a page whole boxes too.
  CUtensorMap k_map = {}, v_map = {};
  int box = P::KT / 4;
  if (a.page_size < box) box = a.page_size >= 8 && box % a.page_size == 0 ? a.page_size : 0;
  if (box > 0 && a.page_size % box != 0) box = 0;
  if (box > 0 && !(encode_pages(&k_map, a.kp, a, box) && encode_pages(&v_map, a.vp, a, box))) box = 0;
  return launch_pdl(kda_prefix_kernel<D, RT>, dim3(sms), dim3(P::THREADS), P::BYTES, s, 1, a, box, k_map, v_map);
}

template <int D>
cudaError_t launch_prefix_join(const AttendArgs& a, const PrefixPlan& p, int sms, cudaStream_t s) {
  const int64_t heads = (int64_t)a.N * a.Hq;
  if (heads >= 16LL * sms)  // 1404 heads of 34 parts, by one warp each, 37 -> 61 us
    return launch_pdl(kda_prefix_join_kernel<D, 1>, dim3((unsigned)((heads + 3) / 4)), dim3(128), 0, s, 1, a, p.pre_parts,
                      p.own_parts);
  return launch_pdl(kda_prefix_join_kernel<D, 4>, dim3((unsigned)heads), dim3(128), 0, s, 1, a, p.pre_parts, p.own_parts);
}

// Bytes of keys and values from which sharing is worth its two launches more, by
// what it could save at the table's width, or the window's (the host knows no lengths; a
// sequence that shares is no longer than the window): below, every sequence is on its
// own.  Measured shared and alone, us (groups x sequences x common positions, 64 own
// ones; the bytes that sharing saves):
//   32 / 8 heads of 128   1 x 2 x 1024 (4 MB) 16 and 10, 1 x 16 x 1024 (63 MB) 19 and 19, 16 x 4 x 256 (50 MB) 28 and 23,
//                         4 x 16 x 256 (63 MB) 19 and 23, 1 x 16 x 4032 (248 MB) 29 and 42, 16 x 4 x 1024 (201 MB) 41 and 47
//     windows: 4 x 2 x 1024 under 512 (17 MB) 28 and 11; 1 x 64 x 4096 + up to 300 under 8192 (all share) 44 and 141, under
//     4200 (a third do; 1 GB) 132 and 140; 16 x 4 x 1024 + up to 300 under 1200 (half do; 236 MB) 65 and 50
//   64 channels           1 x 4 x 16000 (98 MB) 27 and 27, 16 x 4 x 1024 (101 MB) 32 and 31, 4 x 2 x 16000 (131 MB) 61 and 46
//   256 channels          1 x 4 x 4032 (99 MB) 23 and 34, 12 / 1 heads 1 x 16 x 16000 (246 MB) 38 and 65, 4 x 16 x 1024 (63 MB) 28 and 28
constexpr int64_t kSharedBytes = 96 << 20;
// Float32 works on its rows as long as on its bytes: with more query heads a key
// head, or 256 channels, the sequences alone already do, and sharing saves little.
//   32 / 8 heads of 64    4 x 16 x 1024 (252 MB) 46 and 55, 16 x 2 x 4032 (264 MB) 78 and 93, 16 x 16 x 256 (252 MB) 86 and 71
//   32 / 8 of 128         4 x 6 x 1024 (168 MB) 43 and 40, 1 x 16 x 4032 (496 MB) 56 and 83, 16 x 2 x 1024 (134 MB) 50 and 53
//   16 / 16 of 128        1 x 6 x 4032 (330 MB) 43 and 53, 4 x 16 x 256 (252 MB) 49 and 51, 16 x 6 x 256 (336 MB) 66 and 74
//   32 / 2 of 128         4 x 16 x 4032 (496 MB) 137 and 126, 16 x 16 x 1024 (503 MB) 183 and 145
//   256 channels          32 / 8 4 x 6 x 1024 (336 MB) 94 and 79, 16 / 16 16 x 2 x 1024 (537 MB) 216 and 165
constexpr int64_t kSharedBytesF32 = 256 << 20;
constexpr int kSharedHeadsF32 = 4;

// Whether any call of such heads shares.
bool may_share(int32_t G, int32_t D, int32_t dtype) {
  return dtype != KDA_DT_F32 || (G <= kSharedHeadsF32 && D <= 128);
}

bool shares(const AttendArgs& a) {
  int64_t most = (int64_t)a.table_cols * a.page_size;  // common positions that a sequence may have
  if (a.window > 0) most = std::min<int64_t>(most, a.window);
  const bool f32 = a.dtype == KDA_DT_F32;
  const double saved = (a.N - (double)a.num_groups) * most * a.Hkv * a.D * (f32 ? 8 : 4);
  return may_share(a.Hq / a.Hkv, a.D, a.dtype) && a.vec16 && saved >= (f32 ? kSharedBytesF32 : kSharedBytes);
}

}  // namespace

int64_t prefix_floats(int64_t N, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype, int32_t sms) {
  const int64_t alone = attend_floats(Hq, Hkv, D, dtype, sms);
  if (!may_share(Hq / Hkv, D, dtype)) return alone;
  return std::max(alone, prefix_plan(nullptr, N, Hq, Hkv, D, dtype, sms, 0).floats);
}

cudaError_t launch_prefix_attention(const AttendArgs& given, int32_t sms, cudaStream_t s) {
  AttendArgs a = given;
  if (!shares(a)) return launch_paged_attention(a, sms, s);
  const bool f32 = a.dtype == KDA_DT_F32;
  const PrefixPlan p = prefix_plan(a.work, a.N, a.Hq, a.Hkv, a.D, a.dtype, sms, a.num_groups);
  a.parts = p.pre_parts;
  const bool two = p.pre.heads > kRows;
  cudaError_t e = cudaErrorInvalidValue;
  if (f32) e = launch_attend_tf32_groups(a, p.pre, s);
  else if (a.D == 64) e = two ? launch_prefix<64, 2>(a, sms, s) : launch_prefix<64, 1>(a, sms, s);
  else if (a.D == 128) e = two ? launch_prefix<128, 2>(a, sms, s) : launch_prefix<128, 1>(a, sms, s);
  else if (a.D == 256) e = launch_prefix<256, 1>(a, sms, s);
  if (e != cudaSuccess) return e;
  a.parts = p.own_parts;
  a.own = 1;
  e = f32 ? launch_attend_tf32_own(a, p.own, s) : launch_attend_mma(a, p.own, s);
  if (e != cudaSuccess) return e;
  if (a.D == 64) return launch_prefix_join<64>(a, p, sms, s);
  if (a.D == 128) return launch_prefix_join<128>(a, p, sms, s);
  return launch_prefix_join<256>(a, p, sms, s);
}

cudaError_t read_prefix_error(unsigned int* flags, bool clear) {
  cudaError_t e = cudaMemcpyFromSymbol(flags, g_kda_prefix_error, sizeof(unsigned int));
  if (e != cudaSuccess || !clear) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_kda_prefix_error, &zero, sizeof(unsigned int));
}

}  // namespace kda
