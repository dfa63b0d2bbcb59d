// Attention of one new token per sequence over a paged cache: the CUDA-core
// kernel, and the join of partial results.
//
// softmax_t(scale q . k_t) v_t over one pass: each warp keeps, per query head,
// the running maximum m, the sum l of 2^(s - m) and the output o scaled alike;
// a larger maximum rescales both.  Scores are in units of log2, q carrying
// scale * log2(e).
//
// A warp takes KB positions at a time.  Its lanes hold D/32 channels each, so
// a key or value vector is one coalesced access, reused by HG query heads from
// registers; KB * HG partial dot products are reduced by halving exchanges
// (NV - 1 shuffles for NV values), which leaves each lane one score to
// exponentiate.
//
// float32: each warp copies its positions into a ring of shared-memory stages
// ahead of their use, as the tensor-core kernel does (loads straight to
// registers took 165 us in the first case below).  Bound by memory up to 4 query
// heads a key head: 48 sequences, window 2048, 16 heads of 64, 0.79 GB, 122 to 130
// us, 91 to 97 % of the copy bandwidth; 32 / 8 heads of 128 83 %.  With more by the
// exchanges and products themselves, 12 / 1 heads of 128 165 us for 0.37 GB, so
// those come here only where there is little to attend to (kda_attend_tf32.cu).
// bfloat16 comes here only with vectors off the 16-byte boundaries those
// copies need, and is loaded straight to registers.
#include <algorithm>

#include "kda_attend.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kWarpKeys = kTile / kWarps;  // positions of a tile per warp

template <typename T, int VEC>
__device__ __forceinline__ void load_lane(const T* p, float (&x)[VEC]) {
  if constexpr (sizeof(T) == 4) {
    if constexpr (VEC == 2) {
      const float2 r = __ldg(reinterpret_cast<const float2*>(p));
      x[0] = r.x; x[1] = r.y;
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const float4 r = __ldg(reinterpret_cast<const float4*>(p + i));
        x[i] = r.x; x[i + 1] = r.y; x[i + 2] = r.z; x[i + 3] = r.w;
      }
    }
  } else {
    if constexpr (VEC == 2) {
      const uint32_t r = __ldg(reinterpret_cast<const uint32_t*>(p));
      x[0] = bf_lo(r); x[1] = bf_hi(r);
    } else {
#pragma unroll
      for (int i = 0; i < VEC; i += 4) {
        const uint2 r = __ldg(reinterpret_cast<const uint2*>(p + i));
        x[i] = bf_lo(r.x); x[i + 1] = bf_hi(r.x); x[i + 2] = bf_lo(r.y); x[i + 3] = bf_hi(r.y);
      }
    }
  }
}

template <int VEC>
__device__ __forceinline__ void read_lane(const float* p, float (&x)[VEC]) {
  if constexpr (VEC == 2) {
    const float2 r = *reinterpret_cast<const float2*>(p);
    x[0] = r.x; x[1] = r.y;
  } else {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 r = *reinterpret_cast<const float4*>(p + i);
      x[i] = r.x; x[i + 1] = r.y; x[i + 2] = r.z; x[i + 3] = r.w;
    }
  }
}

// Sums NV values over the warp; lane l returns value l / (32 / NV).
template <int NV>
__device__ __forceinline__ float reduce_scatter(float (&x)[NV], int lane) {
  int o = 16;
#pragma unroll
  for (int n = NV / 2; n >= 1; n /= 2, o /= 2) {
    const bool upper = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = upper ? x[i] : x[i + n];
      const float keep = upper ? x[i + n] : x[i];
      x[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
    }
  }
  float r = x[0];
#pragma unroll
  for (; o >= 1; o /= 2) r += __shfl_xor_sync(0xffffffffu, r, o);
  return r;
}

// Blocks a SM: two, where their rings and the joining of their warps fit in shared memory.
constexpr int blocks_per_sm(bool ring, int D, int heads) { return ring && (D > 64 || heads == 8) ? 1 : 2; }

template <typename T, int D, int HG>
struct Stage {
  static constexpr bool RING = sizeof(T) == 4;
  static constexpr int KEYS = RING && D == 256 ? 4 : kWarpKeys;  // positions of a stage
  static constexpr int CTAS = blocks_per_sm(RING, D, HG);
  static constexpr int STAGES = CTAS == 1 && D == 64 ? 6 : 3;    // 192 KB a SM
  using Copies = PageCopies<T, D, KEYS, STAGES, kWarps, false>;
  static constexpr int BYTES = RING ? kWarps * Copies::RING : 0;
};

template <typename T, int D, int HG, int KB>
__global__ void __launch_bounds__(kThreads, Stage<T, D, HG>::CTAS) kda_attend_kernel(const __grid_constant__ AttendArgs a) {
  using St = Stage<T, D, HG>;
  using Copies = typename St::Copies;
  constexpr int VEC = D / 32, NV = HG * KB, REP = 32 / NV;
  static_assert(NV <= 32 && St::KEYS % KB == 0, "bad shape");
  extern __shared__ __align__(128) char smem[];
  __shared__ float s_p[kWarps][32];
  __shared__ float s_m[kWarps][HG], s_l[kWarps][HG];
  __shared__ float s_o[kWarps][HG * D];
  __shared__ typename Copies::Notes s_notes[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int G = a.Hq / a.Hkv, groups = (G + HG - 1) / HG, units = a.Hkv * groups;
  const int C = gridDim.x, c = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const Place place = find_place<kThreads>(a, units, c, C);
  const Workspace ws(a.work, C, HG, D);
  if (place.start == place.stop) {
    if (threadIdx.x == 0) ws.note[c].n = -1;
    return;
  }
  char* ring = smem + warp * Copies::RING;
  Copies copies(a, place, s_notes[warp], ring, units, groups, warp, lane);
  if constexpr (St::RING) {
#pragma unroll 1
    for (int s = 0; s < St::STAGES - 1; ++s) copies.copy(s);
  }
  Walk walk;
  walk.start(a, place);
  int stage = 0;

  while (walk.tile < place.stop) {
    const int n = walk.n, hk = walk.group / groups, g0 = (walk.group - hk * groups) * HG, heads = min(HG, G - g0);
    const int64_t stop = min(walk.unit_end, place.stop);
    float q[HG][VEC], o[HG][VEC];
#pragma unroll
    for (int h = 0; h < HG; ++h) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) o[h][i] = q[h][i] = 0.f;
      if (h < heads) {
        load_lane<T, VEC>(static_cast<const T*>(a.q) + n * a.q_rs + (hk * G + g0 + h) * a.q_hs + lane * VEC, q[h]);
#pragma unroll
        for (int i = 0; i < VEC; ++i) q[h][i] *= a.scale_log2;
      }
    }
    float m = -INFINITY, l = 0.f;  // of this lane's head (lane / REP) % HG

    // KB positions whose keys and values `fetch(j, k, v)` gives, those in `live` attended to.
    const auto attend = [&](uint32_t live, const auto& fetch) {
      float k[KB][VEC], v[KB][VEC], s[NV];
#pragma unroll
      for (int j = 0; j < KB; ++j) fetch(j, k[j], v[j]);
#pragma unroll
      for (int j = 0; j < KB; ++j)
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          float d = 0.f;
#pragma unroll
          for (int i = 0; i < VEC; ++i) d = fmaf(q[h][i], k[j][i], d);
          s[j * HG + h] = d;
        }
      float score = reduce_scatter<NV>(s, lane);
      if (!(live >> (lane / REP / HG) & 1)) score = -INFINITY;
      float top = fmaxf(m, score);
#pragma unroll
      for (int x = HG * REP; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
      const float ref = top == -INFINITY ? 0.f : top;
      const float p = exp2f(score - ref);
      if (__any_sync(0xffffffffu, top > m)) {
        const float fall = exp2f(m - ref);
        l *= fall;
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          const float f = __shfl_sync(0xffffffffu, fall, h * REP);
#pragma unroll
          for (int i = 0; i < VEC; ++i) o[h][i] *= f;
        }
        m = top;
      }
      l += p;
      if (lane % REP == 0) s_p[warp][lane / REP] = p;
      __syncwarp();
#pragma unroll
      for (int j = 0; j < KB; ++j)
#pragma unroll
        for (int h = 0; h < HG; ++h) {
          const float w = s_p[warp][j * HG + h];
#pragma unroll
          for (int i = 0; i < VEC; ++i) o[h][i] = fmaf(w, v[j][i], o[h][i]);
        }
      __syncwarp();
    };

    if constexpr (St::RING) {
#pragma unroll 1
      for (; walk.tile < stop; ++walk.tile) {
#pragma unroll 1
        for (int sub = 0; sub < Copies::SUBS; ++sub) {
          copy_wait<St::STAGES - 2>();
          __syncwarp();  // every lane's copies of this stage; and all are done with the stage copied to next
          const uint32_t live = s_notes[warp].live[stage];
          copies.copy(stage == 0 ? St::STAGES - 1 : stage - 1);
          const T* keys = reinterpret_cast<const T*>(ring + stage * Copies::STAGE) + lane * VEC;
          const T* values = keys + Copies::TENSOR / sizeof(T);
          stage = stage + 1 == St::STAGES ? 0 : stage + 1;
#pragma unroll
          for (int b = 0; b < St::KEYS; b += KB)
            attend(live >> b, [&](int j, float(&k)[VEC], float(&v)[VEC]) {
              read_lane<VEC>(keys + (b + j) * D, k);
              read_lane<VEC>(values + (b + j) * D, v);
            });
        }
      }
    } else {
#pragma unroll 1
      for (; walk.tile < stop; ++walk.tile) {
        // Lanes 0 .. kWarpKeys-1 look up one position each.
        const int t0 = (walk.sp.tile0 + (int)(walk.tile - walk.unit_start)) * kTile + warp * kWarpKeys;
        int64_t ko = 0, vo = 0;
        bool found = false;
        if (lane < kWarpKeys) {
          const int t = t0 + lane;
          if (t >= walk.sp.first && t < walk.sp.end) {
            const int col = t / a.page_size, at = t - col * a.page_size;
            const int page = __ldg(a.table + (int64_t)n * a.table_rs + col);
            if (page > 0 && page < a.num_pages) {
              ko = page * a.kp.page + at * a.kp.token + hk * a.kp.head;
              vo = page * a.vp.page + at * a.vp.token + hk * a.vp.head;
              found = true;
            }
          }
        }
        const uint32_t live = __ballot_sync(0xffffffffu, found);
#pragma unroll
        for (int b = 0; b < kWarpKeys; b += KB)
          attend(live >> b, [&](int j, float(&k)[VEC], float(&v)[VEC]) {
            const int64_t kj = __shfl_sync(0xffffffffu, ko, b + j), vj = __shfl_sync(0xffffffffu, vo, b + j);
#pragma unroll
            for (int i = 0; i < VEC; ++i) k[i] = v[i] = 0.f;
            if (live >> (b + j) & 1) {
              load_lane<T, VEC>(static_cast<const T*>(a.kp.data) + kj + lane * VEC, k);
              load_lane<T, VEC>(static_cast<const T*>(a.vp.data) + vj + lane * VEC, v);
            }
          });
      }
    }
#pragma unroll
    for (int x = HG * REP; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
    if (lane % REP == 0 && lane / REP < HG) {
      s_m[warp][lane / REP] = m;
      s_l[warp][lane / REP] = l;
    }
#pragma unroll
    for (int h = 0; h < HG; ++h)
#pragma unroll
      for (int i = 0; i < VEC; ++i) s_o[warp][h * D + lane * VEC + i] = o[h][i];
    __syncthreads();

    const bool whole = walk.unit_start >= place.start && walk.unit_end <= place.stop;
    const bool at_start = walk.unit_start <= place.start;
    const int64_t slot = 2 * (int64_t)c + (at_start ? 0 : 1);
    for (int i = threadIdx.x; i < heads * D; i += kThreads) {
      const int h = i / D, d = i - h * D;
      float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][h]);
      const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = exp2f(s_m[w][h] - ref);
        L = fmaf(f, s_l[w][h], L);
        O = fmaf(f, s_o[w][i], O);
      }
      const int64_t head = (int64_t)n * a.Hq + hk * G + g0 + h;
      if (whole) {
        static_cast<__nv_bfloat16*>(a.out)[head * D + d] = __float2bfloat16_rn(finished(O, L));
        if (a.lse != nullptr && d == 0) a.lse[head] = log_sum(ref, L);
      } else {
        ws.o_of(slot, h)[d] = O;
        if (d == 0) {
          ws.ml_of(slot, h)[0] = M;
          ws.ml_of(slot, h)[1] = L;
        }
      }
    }
    if (threadIdx.x == 0 && at_start) ws.note[c] = note_of(walk, place);
    __syncthreads();
    if (walk.tile == walk.unit_end) walk.next_unit(a, units);
  }
  copy_wait<0>();
}

// Joins the partials of one query head of a unit that lies in several pieces.
// BY_CUT: block (c, h) of 4 warps looks at the cut before piece c and works if
// it is the first that crosses its unit, which any number of units allows.
// Otherwise block (u, h) of 16 warps finds unit u itself: for few units, cut
// into many pieces each.  The block's warps share the pieces, each lane D/32
// channels.
template <int D, int HG, bool BY_CUT>
__global__ void __launch_bounds__(BY_CUT ? 128 : 512) kda_attend_join_kernel(const __grid_constant__ AttendArgs a, int C) {
  constexpr int VEC = D / 32, AHEAD = 4, WARPS = BY_CUT ? 4 : 16;
  __shared__ float s_m[WARPS], s_l[WARPS], s_o[WARPS][D];
  const int h = blockIdx.y;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  pdl_launch_dependents();
  const Workspace ws(a.work, C, HG, D);
  const int G = a.Hq / a.Hkv, groups = (G + HG - 1) / HG;
  PieceNote note;
  if constexpr (BY_CUT) {
    note = ws.note[blockIdx.x];
    if (note.n < 0) return;
  } else {
    const int units = a.Hkv * groups;
    note.n = blockIdx.x / units;
    note.group = blockIdx.x - note.n * units;
    int64_t before = 0, all = 0;
    for (int n = lane; n < a.N; n += 32) {
      const int tiles = span_of(a, n).tiles;
      all += tiles;
      before += n < note.n ? tiles : 0;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      all += __shfl_xor_sync(0xffffffffu, all, o);
      before += __shfl_xor_sync(0xffffffffu, before, o);
    }
    const int tiles = span_of(a, note.n).tiles;
    note.tiles = all * units;
    note.unit_start = before * units + (int64_t)note.group * tiles;
    note.unit_end = note.unit_start + tiles;
  }
  const int hk = note.group / groups, g0 = (note.group - hk * groups) * HG;
  if (h >= min(HG, G - g0)) return;
  const int64_t T = note.tiles;
  const int pieces = pieces_of(T, C);
  const int first = (int)piece_of(BY_CUT ? piece_start(blockIdx.x, T, pieces) - 1 : note.unit_start, T, pieces);
  const int64_t first_start = piece_start(first, T, pieces);
  if (BY_CUT && first_start > note.unit_start) return;  // an earlier cut crosses this unit too
  const int last = (int)piece_of(note.unit_end - 1, T, pieces);
  if (!BY_CUT && first == last) return;  // finished by its piece

  // The first piece may hold another unit before this one.
  const auto slot_of = [&](int i) { return 2 * (int64_t)i + (i == first && first_start < note.unit_start ? 1 : 0); };
  float m = -INFINITY, l = 0.f, o[VEC] = {};
#pragma unroll 1
  for (int i = first + warp; i <= last; i += WARPS * AHEAD) {
    float pm[AHEAD], pl[AHEAD], po[AHEAD][VEC];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      pm[k] = -INFINITY;
      pl[k] = 0.f;
#pragma unroll
      for (int j = 0; j < VEC; ++j) po[k][j] = 0.f;
      if (i + k * WARPS <= last) {
        const int64_t slot = slot_of(i + k * WARPS);
        const float2 ml = *reinterpret_cast<const float2*>(ws.ml_of(slot, h));
        pm[k] = ml.x;
        pl[k] = ml.y;
        read_lane<VEC>(ws.o_of(slot, h) + lane * VEC, po[k]);
      }
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) top = fmaxf(top, pm[k]);
    const float ref = top == -INFINITY ? 0.f : top, f = exp2f(m - ref);
    l *= f;
#pragma unroll
    for (int j = 0; j < VEC; ++j) o[j] *= f;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const float w = exp2f(pm[k] - ref);
      l = fmaf(pl[k], w, l);
#pragma unroll
      for (int j = 0; j < VEC; ++j) o[j] = fmaf(po[k][j], w, o[j]);
    }
    m = top;
  }
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
  for (int j = 0; j < VEC; ++j) s_o[warp][lane * VEC + j] = o[j];
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += 32 * WARPS) {
    float M = -INFINITY, L = 0.f, O = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) M = fmaxf(M, s_m[w]);
    const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      const float f = exp2f(s_m[w] - ref);
      L = fmaf(f, s_l[w], L);
      O = fmaf(f, s_o[w][d], O);
    }
    const int64_t head = (int64_t)note.n * a.Hq + hk * G + g0 + h;
    static_cast<__nv_bfloat16*>(a.out)[head * D + d] = __float2bfloat16_rn(finished(O, L));
    if (a.lse != nullptr && d == 0) a.lse[head] = log_sum(ref, L);
  }
}

// Query heads a worker carries: all of the key head's up to 8 (4 where D = 256
// would not leave the registers for more).
int heads_class(int G, int D) {
  const int most = D == 256 ? 4 : 8;
  int h = 1;
  while (h < G && h < most) h *= 2;
  return h;
}

template <typename T, int D, int HG>
cudaError_t launch_attend(const AttendArgs& a, int ctas, cudaStream_t s) {
  constexpr int KB = 32 / HG < 8 ? 32 / HG : (D == 256 ? 4 : 8);
  constexpr int bytes = Stage<T, D, HG>::BYTES;
  static std::atomic<bool> set[64];
  const cudaError_t e = allow_shared(kda_attend_kernel<T, D, HG, KB>, bytes, set);
  if (e != cudaSuccess) return e;
  return launch_pdl(kda_attend_kernel<T, D, HG, KB>, dim3(ctas), dim3(kThreads), bytes, s, 1, a);
}

template <typename T>
cudaError_t launch_attend_d(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  switch (a.D * 16 + p.heads) {
    case 64 * 16 + 1: return launch_attend<T, 64, 1>(a, p.ctas, s);
    case 64 * 16 + 2: return launch_attend<T, 64, 2>(a, p.ctas, s);
    case 64 * 16 + 4: return launch_attend<T, 64, 4>(a, p.ctas, s);
    case 64 * 16 + 8: return launch_attend<T, 64, 8>(a, p.ctas, s);
    case 128 * 16 + 1: return launch_attend<T, 128, 1>(a, p.ctas, s);
    case 128 * 16 + 2: return launch_attend<T, 128, 2>(a, p.ctas, s);
    case 128 * 16 + 4: return launch_attend<T, 128, 4>(a, p.ctas, s);
    case 128 * 16 + 8: return launch_attend<T, 128, 8>(a, p.ctas, s);
    case 256 * 16 + 1: return launch_attend<T, 256, 1>(a, p.ctas, s);
    case 256 * 16 + 2: return launch_attend<T, 256, 2>(a, p.ctas, s);
    case 256 * 16 + 4: return launch_attend<T, 256, 4>(a, p.ctas, s);
    default: return cudaErrorInvalidValue;
  }
}

// Who finds the units to join.  Measured by cut and by unit, us a call with its
// attention, bf16: 16 heads of a unit, 128 channels, units x positions 1 x 500 9.9
// and 9.3, 1 x 16000 21.0 and 14.6, 16 x 2000 15.7 and 13.8, 32 x 500 11.9 and 12.7,
// 64 x 2000 21.2 and 25.5; 256 channels, half the blocks, 8 x 2000 15.9 and 13.2,
// 16 x 2000 20.1 and 20.5; 4 heads, 8 x 500 8.2 and 9.0, 8 x 16000 17.8 and 16.9,
// 32 x 2000 13.0 and 13.4.  So by unit where a unit has 16 heads and there is at
// most one unit for 16 blocks.
template <int D, int HG>
cudaError_t launch_join_heads(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  const int G = a.Hq / a.Hkv, heads = std::min(G, HG);
  const int64_t units = (int64_t)a.N * a.Hkv * ((G + HG - 1) / HG);
  if constexpr (HG == 16)
    if (16 * units <= p.ctas)
      return launch_pdl(kda_attend_join_kernel<D, HG, false>, dim3((unsigned)units, heads), dim3(512), 0, s, 1, a, p.ctas);
  return launch_pdl(kda_attend_join_kernel<D, HG, true>, dim3(p.ctas, heads), dim3(128), 0, s, 1, a, p.ctas);
}

template <int D>
cudaError_t launch_join(const AttendArgs& a, const AttendPlan& p, cudaStream_t s) {
  switch (p.heads) {
    case 1: return launch_join_heads<D, 1>(a, p, s);
    case 2: return launch_join_heads<D, 2>(a, p, s);
    case 4: return launch_join_heads<D, 4>(a, p, s);
    case 8: return launch_join_heads<D, 8>(a, p, s);
    default: return launch_join_heads<D, 16>(a, p, s);
  }
}

// Float32 in matrix instructions: from five query heads a key head, where the
// positions that the call may attend to, over sequences and key heads, are 256 a
// channel or more.  The host knows only how many the table or the window allows;
// short sequences in a roomy table are slower for it, by 2 us at 64 and 128
// channels, 8 us at 256.  Measured in matrix instructions (a form up to 10 %
// slower than the one there now) and on CUDA cores, us:
//   64 channels   12 heads, 8000 positions 10 and 11, 32000 17 and 23, 1.2 million 112 and 226; 8 heads 97 and 118
//   128 channels  12 heads, 8000 13 and 13, 16000 18 and 17, 32000 21 and 22, 0.6 million 102 and 165; 8 heads 78 and 85
//   256 channels  12 heads, 16000 28 and 21, 64000 57 and 58, 0.3 million 167 and 193; 16 heads 175 and 272
// With four heads or fewer CUDA cores are faster: 32 / 8 heads of 64 71 and 100 us.
constexpr int kTensorHeads = 5;
constexpr int64_t kTensorPositions = 256;
bool tensor_path(const AttendArgs& a) {
  if (a.dtype != KDA_DT_F32) return a.vec16;
  int64_t most = (int64_t)a.table_cols * a.page_size;
  if (a.window > 0) most = std::min<int64_t>(most, a.window);
  return a.Hq / a.Hkv >= kTensorHeads && (double)a.N * a.Hkv * most >= (double)kTensorPositions * a.D;
}

AttendPlan plan_of(int32_t G, int32_t D, int32_t dtype, int32_t sms, bool tensor) {
  if (tensor) return dtype == KDA_DT_F32 ? attend_tf32_plan(G, D, sms) : attend_mma_plan(G, D, sms);
  AttendPlan p;
  p.heads = heads_class(G, D);
  p.ctas = blocks_per_sm(dtype == KDA_DT_F32, D, p.heads) * sms;
  p.floats = (int64_t)p.ctas * kNoteFloats + 2LL * p.ctas * p.heads * (2 + D);
  return p;
}

}  // namespace

int64_t attend_floats(int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype, int32_t sms) {
  return std::max(plan_of(Hq / Hkv, D, dtype, sms, false).floats, plan_of(Hq / Hkv, D, dtype, sms, true).floats);
}

cudaError_t launch_paged_attention(const AttendArgs& a, int32_t sms, cudaStream_t s) {
  const bool tensor = tensor_path(a);
  const AttendPlan p = plan_of(a.Hq / a.Hkv, a.D, a.dtype, sms, tensor);
  const cudaError_t e = a.dtype == KDA_DT_F32 ? (tensor ? launch_attend_tf32(a, p, s) : launch_attend_d<float>(a, p, s))
                                              : (tensor ? launch_attend_mma(a, p, s) : launch_attend_d<__nv_bfloat16>(a, p, s));
  if (e != cudaSuccess) return e;
  return a.D == 64 ? launch_join<64>(a, p, s) : (a.D == 128 ? launch_join<128>(a, p, s) : launch_join<256>(a, p, s));
}

}  // namespace kda
