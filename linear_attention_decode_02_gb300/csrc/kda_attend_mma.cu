// Attention of one new token per sequence over a paged bfloat16 cache, on the
// tensor cores' warp instructions.
//
// Bound by memory: a key or value byte is used for at most 16 query heads, so
// the kernel is built around its loads.  At full DRAM bandwidth these warp
// instructions keep the tensor pipe 17 % busy; tcgen05 would raise a peak that
// is not reached, and would put its 128-row operands, a transposing pass over
// the weights and a barrier a tile between the load and its use.  Each warp is a
// pipeline of its own: it copies 16 positions a stage into shared memory,
// several stages ahead, and meets the block's other warps only at the end of a
// unit.  Nothing between two units waits: the copies run on into the next
// sequence.
//
// Measured (32 query / 8 key heads of 128, pages of 64): 64 sequences of up to
// 8192 positions, 1.27 GB, 189 to 199 us; 2 of up to 131072, 1.0 GB, 150 to 156
// us: 95 to 100 % of the copy bandwidth.  0.4 GB of 256-channel heads 85 us (73 %),
// of 64-channel ones 75 us (79 %), of 128-channel ones 70 us (85 %), with 12 query
// heads a key head 75 us (77 %).  One sequence of 1000 positions 9 to 11 us with the
// join: two launches and four dependent loads (length, page, keys, partials).
//
// Every warp with a piece of its own, instead of four that share a tile: 64
// sequences of up to 8192 199 -> 210 us, 32 of 2000 39 -> 44, 64 of 100 15 -> 22,
// since it leaves more partial results to join; 512 of 64 47 -> 45 and, float32
// with 256 channels, 100 of 50 46 -> 27 were better for it.
//
// S = Q K^T with query heads as rows (16 of them) and positions as columns, so
// that a score's lane already is the one the second product wants its weight
// in; keys come by ldmatrix, values by its transposing form, both from rows
// whose 16-byte chunks are XORed with the row so that no two banks meet.
//
// The weights p enter the second product as two bfloat16 pieces, p = hi + lo
// to 2^-17 (hi alone would put 2^-8 of rounding into the output, as much as
// its own type has).  With up to 8 heads hi takes rows 0..7 and lo rows 8..15,
// which would be empty, at no cost; with 16 heads lo is a second product.  A third
// piece left the outputs as far from 64 bits and from a float32 computation as they
// are, and took 256 channels from 150 to 168 us, 12 heads from 46 to 48.
//
// With PARTS sequences begin behind a prefix that they share, and results go as parts
// to another kernel's join.  Up to 128 channels each warp has a piece of its own, so
// that it ends a quarter of the units and leaves a quarter of the parts: 256 sequences
// of up to 600 such positions, 0.32 GB, 65 us (73 % of the copy bandwidth), with the
// join 77; 74 and 90 us where a block shared its units and each warp left its part, 94
// where the block joined them first.  What is left are the starts and ends of 2048
// short units.
#include <type_traits>

#include "kda_attend_rows.cuh"

namespace kda {
namespace {

constexpr int kWarps = kAttendWarps, kThreads = 32 * kWarps;
constexpr int kKeys = 16;  // positions of a stage
static_assert(kWarps * kKeys == kTile, "a tile is one stage of every warp");

// Blocks a SM and stages a warp: about 192 KB of rings a SM in any case.  For
// D = 64, 48 x 6000 positions x 8 key heads (0.39 GB) took 74 us with 2 blocks of 6
// stages, 82 us with 3 of 4 and 80 us with 4 of 3, and 16 query heads a key head
// 83, 82 and 113 us.
constexpr int blocks_per_sm(int D) { return D == 256 ? 1 : 2; }
template <int D, int HG>
struct Shape {
  static constexpr int CTAS = blocks_per_sm(D);
  static constexpr int STAGES = D == 64 ? 6 : 3;
  static constexpr bool QS = D == 256;  // no registers are left for the queries: they lie in shared memory
  // Sequences' own positions are short units: a warp takes them alone, so that it ends a quarter of them.
  static constexpr bool ALONE = own_warps_alone(D) > 1;
  static_assert(ALONE != QS, "shared queries are the block's");
  // A lone warp's pieces are cut between stages, where 16 x 4 sequences of up to 300 positions take 16.5 us, by tiles of 64
  // positions 20; but with 64 channels, whose rings hold a tile, by tiles: 7 x 20 of up to 500 31 us a call, with its join of
  // fewer parts, 33 between stages.
  static constexpr int CUT = ALONE && D == 128 ? kKeys : kTile;
  template <bool PARTS>
  using PartOf = std::conditional_t<PARTS, Own<CUT>, Whole>;
  template <bool PARTS>
  using CopiesOf = PageCopies<__nv_bfloat16, D, kKeys, STAGES, PARTS && ALONE ? 1 : kWarps, true, WalkOf<PartOf<PARTS>>>;
  using Copies = CopiesOf<false>;
};
template <int D, int HG>
constexpr int smem_bytes() {
  return kWarps * Shape<D, HG>::Copies::RING + (kWarps - 1) * 8 * D * 4 + (Shape<D, HG>::QS ? HG * D * 2 : 0);
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix2(uint32_t& r0, uint32_t& r1, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r0), "=r"(r1) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int D, int HG, bool PARTS>
__global__ void __launch_bounds__(kThreads, Shape<D, HG>::CTAS) kda_attend_mma_kernel(const __grid_constant__ AttendArgs a) {
  using Part = typename Shape<D, HG>::template PartOf<PARTS>;
  using Copies = typename Shape<D, HG>::template CopiesOf<PARTS>;
  constexpr bool ALONE = PARTS && Shape<D, HG>::ALONE;
  constexpr int STAGES = Shape<D, HG>::STAGES, ROW = Copies::ROW;
  constexpr int KSTEPS = D / 16, NT = D / 8;
  constexpr bool PAIR = HG == 8;  // rows 8..15 carry lo
  static_assert(HG == 8 || HG == 16, "16 rows of queries");
  extern __shared__ __align__(128) char smem[];
  __shared__ typename Copies::Notes s_notes[kWarps];
  __shared__ float s_m[2][kWarps][HG], s_l[2][kWarps][HG];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int G = a.Hq / a.Hkv, groups = (G + HG - 1) / HG, units = a.Hkv * groups;
  const int C = ALONE ? gridDim.x * kWarps : gridDim.x, c = ALONE ? blockIdx.x * kWarps + warp : blockIdx.x;
  // Parts go where the kernel before writes nothing, and nothing that it writes is read: that kernel has waited for all
  // before it when this one begins, and is waited for at the end.
  if (!PARTS) pdl_wait();
  pdl_launch_dependents();
  const Place place = find_place<kThreads, Part, ALONE>(a, units, c, C);
  const Workspace ws(a.work, C, HG, D);
  if (place.start == place.stop) {
    if (PARTS) pdl_wait();
    else if (threadIdx.x == 0) ws.note[c].n = -1;
    return;
  }

  WalkOf<Part> walk;
  walk.start(a, place);
  int stage = 0, parity = 0;
  // Queries of the next unit, on their way while this one is worked on: the
  // first product's operand itself, or (QS) the thread's share of HG rows of
  // 16-byte chunks for shared memory, swizzled like the keys.
  constexpr bool QS = Shape<D, HG>::QS;
  constexpr int QN = PAIR ? 2 : 4, SHARE = HG * D / 8 / kThreads;
  uint32_t q_next[QS ? 1 : KSTEPS][QN];
  uint4 q_share[QS ? SHARE : 1];
  const auto load_q = [&](const WalkOf<Part>& w) {
    const int hk = w.group / groups, g0 = (w.group - hk * groups) * HG, heads = min(HG, G - g0);
    const __nv_bfloat16* qh = static_cast<const __nv_bfloat16*>(a.q) + w.n * a.q_rs + (hk * G + g0) * a.q_hs;
    if constexpr (QS) {
#pragma unroll
      for (int i = 0; i < SHARE; ++i) {
        const int row = (i * kThreads + threadIdx.x) / (D / 8), chunk = (i * kThreads + threadIdx.x) % (D / 8);
        q_share[i] = row < heads ? __ldg(reinterpret_cast<const uint4*>(qh + row * a.q_hs) + chunk) : make_uint4(0, 0, 0, 0);
      }
    } else {
#pragma unroll
      for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int col = k * 16 + half * 8 + 2 * t4;
          const auto word = [&](int h) {
            return h < heads ? __ldg(reinterpret_cast<const uint32_t*>(qh + h * a.q_hs + col)) : 0u;
          };
          if constexpr (PAIR) {
            q_next[k][half] = word(g);
          } else {
            q_next[k][2 * half] = word(g);
            q_next[k][2 * half + 1] = word(g + 8);
          }
        }
    }
  };
  char* shared_q = smem + kWarps * Copies::RING + (kWarps - 1) * 8 * D * 4;
  const auto place_q = [&]() {
    if (PARTS) __syncthreads();  // no unit's end held the warps together: all are done with the last one's queries
#pragma unroll
    for (int i = 0; i < SHARE; ++i) {
      const int row = (i * kThreads + threadIdx.x) / (D / 8), chunk = (i * kThreads + threadIdx.x) % (D / 8);
      *reinterpret_cast<uint4*>(shared_q + row * ROW + ((chunk ^ (row & 7)) << 4)) = q_share[i];
    }
    __syncthreads();
  };
  load_q(walk);
  Copies copies(a, place, s_notes[warp], smem + warp * Copies::RING, units, groups, ALONE ? 0 : warp, lane);
  // This lane's address for step k within keys, or values: offset[k % 4] + k / 4 * 128.
  uint32_t key_at[4], value_at[4], query_at[4];
  {
    const int qrow = PAIR ? lane & 7 : lane & 15, qhalf = PAIR ? (lane >> 3) & 1 : lane >> 4;
    const int krow = ((lane >> 4) << 3) + (lane & 7), khalf = (lane >> 3) & 1, vrow = lane & 15, vhalf = lane >> 4;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      key_at[k] = krow * ROW + (((2 * k + khalf) ^ (krow & 7)) << 4);
      value_at[k] = Copies::TENSOR + vrow * ROW + (((2 * k + vhalf) ^ (vrow & 7)) << 4);
      query_at[k] = static_cast<uint32_t>(__cvta_generic_to_shared(shared_q)) + qrow * ROW +
                    (((2 * k + qhalf) ^ (qrow & 7)) << 4);
    }
  }
#pragma unroll 1
  for (int s = 0; s < STAGES - 1; ++s) copies.copy(s);

  while (walk.tile < place.stop) {
    uint32_t q[QS ? 1 : KSTEPS][QN];
    if constexpr (QS) {
      place_q();
    } else {
#pragma unroll
      for (int k = 0; k < KSTEPS; ++k)
#pragma unroll
        for (int i = 0; i < QN; ++i) q[k][i] = q_next[k][i];
    }
    WalkOf<Part> after = walk;
    if (walk.unit_end < place.stop) {
      after.next_unit(a, units);
      load_q(after);
    }
    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
    constexpr int RS = PAIR ? 1 : 2;  // rows of heads per lane
    float m[RS], l[RS];
#pragma unroll
    for (int r = 0; r < RS; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.f;
    }

    const int64_t stop = min(walk.unit_end, place.stop);
#pragma unroll 1
    for (; walk.tile < stop; ++walk.tile) {
#pragma unroll 1
      for (int sub = 0; sub < Copies::SUBS; ++sub) {
        copy_wait<STAGES - 2>();
        __syncwarp();  // every lane's copies of this stage; and all are done with the stage copied to next
        const uint32_t live = s_notes[warp].live[stage];
        copies.copy(stage == 0 ? STAGES - 1 : stage - 1);
        const uint32_t base = copies.ring + stage * Copies::STAGE;
        stage = stage + 1 == STAGES ? 0 : stage + 1;
        if (Copies::SUBS > 1 && live == 0) continue;

        float s[2][2][4] = {};  // [even / odd step][positions 0..7 / 8..15]
        {
#pragma unroll
          for (int k = 0; k < KSTEPS; ++k) {
            uint32_t b[4];
            ldmatrix4(b, base + key_at[k % 4] + k / 4 * 128);
            uint32_t x[4];
            if constexpr (QS && PAIR) ldmatrix2(x[0], x[1], query_at[k % 4] + k / 4 * 128);
            if constexpr (QS && !PAIR) ldmatrix4(x, query_at[k % 4] + k / 4 * 128);
            if constexpr (!QS) {
#pragma unroll
              for (int i = 0; i < QN; ++i) x[i] = q[k][i];
            }
            if constexpr (PAIR) {
              mma(s[k & 1][0], x[0], 0u, x[1], 0u, b[0], b[1]);
              mma(s[k & 1][1], x[0], 0u, x[1], 0u, b[2], b[3]);
            } else {
              mma(s[k & 1][0], x[0], x[1], x[2], x[3], b[0], b[1]);
              mma(s[k & 1][1], x[0], x[1], x[2], x[3], b[2], b[3]);
            }
          }
        }
        float p[RS][4];  // this lane's positions 2 t4, + 1, + 8, + 9
        bool rises = false;
        float ref[RS], fall[RS];
#pragma unroll
        for (int r = 0; r < RS; ++r) {
#pragma unroll
          for (int j = 0; j < 4; ++j) p[r][j] = (s[0][j >> 1][2 * r + (j & 1)] + s[1][j >> 1][2 * r + (j & 1)]) * a.scale_log2;
          if (live != 0xffffu) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (!(live >> ((j >> 1) * 8 + 2 * t4 + (j & 1)) & 1)) p[r][j] = -INFINITY;
          }
          float top = fmaxf(fmaxf(p[r][0], p[r][1]), fmaxf(p[r][2], p[r][3]));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
          top = fmaxf(top, m[r]);
          ref[r] = top == -INFINITY ? 0.f : top;
          fall[r] = ex2(m[r] - ref[r]);
          rises = rises || top > m[r];
          m[r] = top;
        }
        if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
          for (int r = 0; r < RS; ++r) l[r] *= fall[r];
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            o[i][0] *= fall[0];
            o[i][1] *= fall[0];
            o[i][2] *= fall[RS - 1];
            o[i][3] *= fall[RS - 1];
          }
        }
        uint32_t hi[RS][2], lo[RS][2];
#pragma unroll
        for (int r = 0; r < RS; ++r) {
#pragma unroll
          for (int j = 0; j < 4; ++j) p[r][j] = ex2(p[r][j] - ref[r]);
          l[r] += (p[r][0] + p[r][1]) + (p[r][2] + p[r][3]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            hi[r][j] = pack_bf2(p[r][2 * j], p[r][2 * j + 1]);
            lo[r][j] = pack_bf2(p[r][2 * j] - bf_lo(hi[r][j]), p[r][2 * j + 1] - bf_hi(hi[r][j]));
          }
        }
        {
#pragma unroll
          for (int k = 0; k < KSTEPS; ++k) {
            uint32_t b[4];
            ldmatrix4_trans(b, base + value_at[k % 4] + k / 4 * 128);
            if constexpr (PAIR) {
              mma(o[2 * k], hi[0][0], lo[0][0], hi[0][1], lo[0][1], b[0], b[1]);
              mma(o[2 * k + 1], hi[0][0], lo[0][0], hi[0][1], lo[0][1], b[2], b[3]);
            } else {
              mma(o[2 * k], hi[0][0], hi[RS - 1][0], hi[0][1], hi[RS - 1][1], b[0], b[1]);
              mma(o[2 * k + 1], hi[0][0], hi[RS - 1][0], hi[0][1], hi[RS - 1][1], b[2], b[3]);
              mma(o[2 * k], lo[0][0], lo[RS - 1][0], lo[0][1], lo[RS - 1][1], b[0], b[1]);
              mma(o[2 * k + 1], lo[0][0], lo[RS - 1][0], lo[0][1], lo[RS - 1][1], b[2], b[3]);
            }
          }
        }
      }
    }

    if constexpr (PARTS) {
      const int hk = walk.group / groups, g0 = (walk.group - hk * groups) * HG;
      leave_parts<D, HG, ALONE ? 1 : kWarps, RS>(
          a, walk, place, [&](int h) { return (int64_t)walk.n * a.Hq + hk * G + g0 + h; }, min(HG, G - g0), o, m, l,
          ALONE ? 0 : warp, g, t4, c, C);
    } else {
      finish_unit<D, HG, kWarps, RS>(a, walk, place, ws, reinterpret_cast<float*>(smem + kWarps * Copies::RING),
                                     s_m[parity], s_l[parity], o, m, l, groups, warp, g, t4, c);
    }
    parity ^= 1;
    after.tile = walk.tile;
    walk = after;
  }
  copy_wait<0>();
  if (PARTS) pdl_wait();
}

template <int D, int HG, bool PARTS>
cudaError_t launch_parts(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  constexpr int bytes = smem_bytes<D, HG>();
  static std::atomic<bool> set[64];
  const cudaError_t e = allow_shared(kda_attend_mma_kernel<D, HG, PARTS>, bytes, set);
  if (e != cudaSuccess) return e;
  return launch_pdl(kda_attend_mma_kernel<D, HG, PARTS>, dim3(p.ctas), dim3(kThreads), bytes, s, 1, a);
}
template <int D, int HG>
cudaError_t launch(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  return a.own != 0 ? launch_parts<D, HG, true>(a, p, s) : launch_parts<D, HG, false>(a, p, s);
}

}  // namespace

AttendPlan attend_mma_plan(int32_t G, int32_t D, int32_t sms) {
  AttendPlan p;
  p.heads = G <= 8 ? 8 : 16;
  p.ctas = blocks_per_sm(D) * sms;
  p.floats = (int64_t)p.ctas * kNoteFloats + 2LL * p.ctas * p.heads * (2 + D);
  return p;
}

cudaError_t launch_attend_mma(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  switch (a.D * 16 + p.heads - 1) {
    case 64 * 16 + 7: return launch<64, 8>(a, p, s);
    case 64 * 16 + 15: return launch<64, 16>(a, p, s);
    case 128 * 16 + 7: return launch<128, 8>(a, p, s);
    case 128 * 16 + 15: return launch<128, 16>(a, p, s);
    case 256 * 16 + 7: return launch<256, 8>(a, p, s);
    case 256 * 16 + 15: return launch<256, 16>(a, p, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kda
