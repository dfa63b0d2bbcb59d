// Attention of one new token per sequence over a paged cache, float32 with many
// query heads a key head: matrix instructions of a warp, 16 x 8 x 8.
//
// A key or value of up to 16 query heads enters 32 multiply-adds for each of
// its 4 bytes, and the CUDA-core kernel needs an instruction for each of them
// and exchanges for the sums; here the work is a warp's matrix instructions,
// as in the bfloat16 kernel, and the copies are the same rings.
//
// The instructions take 11 significant bits of an operand.  Each is split in
// two, x = hi + lo to 2^-23 (queries and keys, hi rounded) or 2^-21 (weights and
// values, hi cut), and the products hi hi, lo hi and hi lo are added in float32; lo
// lo is below 2^-22 of a score's product, 2^-20 of an output's.  Together that is
// below 7 and 28 half steps of float32, where a float32 sum of that many products
// may be off by more.  With up to 8 heads hi takes rows 0..7 and lo rows 8..15, one
// instruction for two products.  A split loses infinities (inf - inf in lo), so
// scores that come out as NaN are computed once more without it; an infinite value
// makes its row non-finite either way.
//
// Bound by the latency of each warp's steps: 0.37 GB of 12 / 1 heads of 128 take
// 99 us, 57 % of the copy bandwidth (CUDA cores 165), of 64 111 (226), 32 / 2 heads of
// 256 154 (272); keys cut instead of rounded took 98, 110 and 151.  The issue slots
// are 31 % used, the tensor pipe 30 % and shared memory 46 %, with two warps a
// scheduler and all registers taken.  Sums kept
// apart for every kind of product, four outputs in turn, a rolled first product
// and queries laid out without bank conflicts changed that by 2 % or made it
// slower.
//
// Keys and values are read from shared memory a word a lane: rows are XORed
// into the 16-byte chunks, and the second product takes its positions in the
// order in which the first leaves the weights (2 t, 2 t + 1 for lane t of four).
// Both meet every bank once.
#include "kda_attend_rows.cuh"

namespace kda {
namespace {

constexpr int kKeys = 8;  // positions of a stage

// One block a SM, 192 KB of rings in any case; with 256 channels a stage is
// 16 KB and there are only four warps of three.
template <int D>
struct Shape {
  static constexpr int WARPS = D == 256 ? 4 : 8, THREADS = 32 * WARPS;
  static constexpr int STAGES = D == 64 ? 6 : 3;
  using Copies = PageCopies<float, D, kKeys, STAGES, WARPS, true>;
};
// Queries of a unit (both parts), then, when they are done with, the outputs that its warps exchange.
template <int D, int HG>
constexpr int tail_bytes() {
  constexpr int q = 2 * HG * D * 4, o = (Shape<D>::WARPS - 1) * 8 * D * 4;
  return q > o ? q : o;
}
template <int D, int HG>
constexpr int smem_bytes() {
  return Shape<D>::WARPS * Shape<D>::Copies::RING + tail_bytes<D, HG>();
}

__device__ __forceinline__ uint32_t round_tf32(float x) {
  uint32_t r;
  asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
  return r;
}
// x = hi + lo in 11 bits each, less up to 2^-23 of x.  Of keys hi is the nearest
// one: what lo then cuts off is as often above as below, and leans to no side (cut
// in both parts, scores came out 2^-24 too small on average).  It can pass the
// largest float, where hi and lo become opposite infinities and the score NaN.
__device__ __forceinline__ void split_nearest(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}
// The same with hi cut, for weights and values, whose products are not computed
// again: a finite one stays finite, and the 2^-24 that it is short of on average
// is far below a bfloat16 output's step.
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, "
      "%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int HG>
__global__ void __launch_bounds__(Shape<D>::THREADS, 1) kda_attend_tf32_kernel(const __grid_constant__ AttendArgs a) {
  using Copies = typename Shape<D>::Copies;
  constexpr int WARPS = Shape<D>::WARPS, THREADS = Shape<D>::THREADS, STAGES = Shape<D>::STAGES, ROW = Copies::ROW;
  constexpr int KSTEPS = D / 8, NT = D / 8;
  constexpr bool PAIR = HG == 8;  // rows 8..15 carry lo
  constexpr int RS = HG / 8;      // rows of heads per lane
  static_assert(HG == 8 || HG == 16, "16 rows of queries");
  extern __shared__ __align__(128) char smem[];
  __shared__ typename Copies::Notes s_notes[WARPS];
  __shared__ float s_m[2][WARPS][HG], s_l[2][WARPS][HG];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t4 = lane & 3;
  const int G = a.Hq / a.Hkv, groups = (G + HG - 1) / HG, units = a.Hkv * groups;
  const int C = gridDim.x, c = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const Place place = find_place<THREADS>(a, units, c, C);
  const Workspace ws(a.work, C, HG, D);
  if (place.start == place.stop) {
    if (threadIdx.x == 0) ws.note[c].n = -1;
    return;
  }

  Walk walk;
  walk.start(a, place);
  int stage = 0, parity = 0;
  // Queries of the next unit, on their way while this one is worked on; in
  // shared memory the first product's operands, four words a lane and step:
  // rows g and g + 8 of column t4, then of t4 + 4 (hi, then all of lo), or with up
  // to 8 heads hi and lo of row g in their places.
  constexpr int SHARE = (HG * D / 4 + THREADS - 1) / THREADS;
  float4 q_next[SHARE];
  char* const tail = smem + WARPS * Copies::RING;
  const auto q_row = [&](const Walk& w) {
    const int hk = w.group / groups;
    return static_cast<const float*>(a.q) + w.n * a.q_rs + (hk * G + (w.group - hk * groups) * HG) * a.q_hs;
  };
  const auto heads_of = [&](const Walk& w) { return min(HG, G - w.group % groups * HG); };
  const auto load_q = [&](const Walk& w) {
    const float* q = q_row(w);
    const int heads = heads_of(w);
#pragma unroll
    for (int i = 0; i < SHARE; ++i) {
      const int h = (i * THREADS + threadIdx.x) / (D / 4), chunk = (i * THREADS + threadIdx.x) % (D / 4);
      q_next[i] = h < heads ? __ldg(reinterpret_cast<const float4*>(q + h * a.q_hs) + chunk) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  };
  const auto place_q = [&]() {
#pragma unroll
    for (int i = 0; i < SHARE; ++i) {
      const int h = (i * THREADS + threadIdx.x) / (D / 4), chunk = (i * THREADS + threadIdx.x) % (D / 4);
      if (h >= HG) break;
      const float x[4] = {q_next[i].x, q_next[i].y, q_next[i].z, q_next[i].w};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const uint32_t hi = round_tf32(x[t]), lo = round_tf32(x[t] - __uint_as_float(hi));
        uint32_t* at = reinterpret_cast<uint32_t*>(tail) + (chunk / 2 * 32 + (h % 8) * 4 + t) * 4 + chunk % 2 * 2;
        if constexpr (PAIR) {
          at[0] = hi;
          at[1] = lo;
        } else {
          at[h / 8] = hi;
          at[HG * D + h / 8] = lo;
        }
      }
    }
    __syncthreads();
  };
  load_q(walk);
  char* const ring = smem + warp * Copies::RING;
  Copies copies(a, place, s_notes[warp], ring, units, groups, warp, lane);
  // This lane's words of step k: at[k % 4] + k / 4 * 128, of the step's first and second four columns of keys, and of
  // its even and odd position among the values.
  int key_at[2][4], value_at[2][4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      key_at[i][k] = g * ROW + (((2 * k + i) ^ g) << 4) + t4 * 4;
      value_at[i][k] = Copies::TENSOR + (2 * t4 + i) * ROW + (((2 * k + (g >> 2)) ^ (2 * t4 + i)) << 4) + (g & 3) * 4;
    }
  const auto word = [](const char* p) { return *reinterpret_cast<const float*>(p); };
#pragma unroll 1
  for (int s = 0; s < STAGES - 1; ++s) copies.copy(s);

  while (walk.tile < place.stop) {
    __syncthreads();  // all have taken the last unit's outputs
    place_q();
    Walk after = walk;
    if (walk.unit_end < place.stop) {
      after.next_unit(a, units);
      load_q(after);
    }
    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i][j] = 0.f;
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
        const char* base = ring + stage * Copies::STAGE;
        stage = stage + 1 == STAGES ? 0 : stage + 1;

        float s[2][4] = {}, rest[4] = {};  // hi hi of even and odd steps; the products with lo
#pragma unroll
        for (int k = 0; k < KSTEPS; ++k) {
          uint32_t kh[2], kl[2], qh[4];
#pragma unroll
          for (int i = 0; i < 2; ++i) split_nearest(word(base + key_at[i][k % 4] + k / 4 * 128), kh[i], kl[i]);
          const uint4 x = *reinterpret_cast<const uint4*>(tail + (k * 32 + lane) * 16);
          qh[0] = x.x; qh[1] = x.y; qh[2] = x.z; qh[3] = x.w;
          mma(s[k & 1], qh, kh[0], kh[1]);
          mma(rest, qh, kl[0], kl[1]);
          if constexpr (!PAIR) {
            const uint4 y = *reinterpret_cast<const uint4*>(tail + (KSTEPS * 32 + k * 32 + lane) * 16);
            const uint32_t ql[4] = {y.x, y.y, y.z, y.w};
            mma(rest, ql, kh[0], kh[1]);
          }
        }
        float p[RS][2];  // this lane's positions 2 t4 and 2 t4 + 1
        bool lost = false;
#pragma unroll
        for (int r = 0; r < RS; ++r)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int i = 2 * r + j;
            p[r][j] = rest[i] + (s[0][i] + s[1][i]);
            if constexpr (PAIR) p[r][j] += rest[i + 2] + (s[0][i + 2] + s[1][i + 2]);
            lost = lost || p[r][j] != p[r][j];
          }
        if (__any_sync(0xffffffffu, lost)) {
          const float* q = q_row(walk);
#pragma unroll
          for (int r = 0; r < RS; ++r)
#pragma unroll 1
            for (int j = 0; j < 2; ++j) {
              float sum = 0.f;
              const float had = j == 0 ? p[r][0] : p[r][1];
              if (had == had) continue;  // other heads and positions keep their bits
              if (g + 8 * r < heads_of(walk)) {
#pragma unroll 1
                for (int d = 0; d < D; ++d)
                  sum = fmaf(__ldg(q + (g + 8 * r) * a.q_hs + d),
                             word(base + (2 * t4 + j) * ROW + (((d >> 2) ^ (2 * t4 + j)) << 4) + (d & 3) * 4), sum);
              }
              (j == 0 ? p[r][0] : p[r][1]) = sum;
            }
        }
        bool rises = false;
        float ref[RS], fall[RS];
#pragma unroll
        for (int r = 0; r < RS; ++r) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            p[r][j] *= a.scale_log2;
            if (!(live >> (2 * t4 + j) & 1)) p[r][j] = -INFINITY;
          }
          float top = fmaxf(p[r][0], p[r][1]);
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
        uint32_t ph[RS][2], pl[RS][2];
#pragma unroll
        for (int r = 0; r < RS; ++r) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            p[r][j] = ex2(p[r][j] - ref[r]);
            split(p[r][j], ph[r][j], pl[r][j]);
          }
          l[r] += p[r][0] + p[r][1];
        }
        uint32_t w[4], wl[4];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          w[2 * j] = ph[0][j];
          w[2 * j + 1] = PAIR ? pl[0][j] : ph[RS - 1][j];
          wl[2 * j] = pl[0][j];
          wl[2 * j + 1] = pl[RS - 1][j];
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          uint32_t vh[2], vl[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) split(word(base + value_at[j][i % 4] + i / 4 * 128), vh[j], vl[j]);
          mma(o[i], w, vh[0], vh[1]);
          if constexpr (!PAIR) mma(o[i], wl, vh[0], vh[1]);
          mma(o[i], w, vl[0], vl[1]);
        }
      }
    }
    finish_unit<D, HG, WARPS, RS>(a, walk, place, ws, reinterpret_cast<float*>(tail), s_m[parity], s_l[parity], o, m, l,
                                  groups, warp, g, t4, c);
    parity ^= 1;
    after.tile = walk.tile;
    walk = after;
  }
  copy_wait<0>();
}

template <int D, int HG>
cudaError_t launch(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  constexpr int bytes = smem_bytes<D, HG>();
  static std::atomic<bool> set[64];
  const cudaError_t e = allow_shared(kda_attend_tf32_kernel<D, HG>, bytes, set);
  if (e != cudaSuccess) return e;
  return launch_pdl(kda_attend_tf32_kernel<D, HG>, dim3(p.ctas), dim3(Shape<D>::THREADS), bytes, s, 1, a);
}

}  // namespace

AttendPlan attend_tf32_plan(int32_t G, int32_t D, int32_t sms) {
  AttendPlan p;
  p.heads = G <= 8 ? 8 : 16;
  p.ctas = sms;
  p.floats = (int64_t)p.ctas * kNoteFloats + 2LL * p.ctas * p.heads * (2 + D);
  return p;
}

cudaError_t launch_attend_tf32(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
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
