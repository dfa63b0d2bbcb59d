// Beam selection: the best M of all beams' continuations, by
// score_b + x_bt - log sum exp x_b, ties to the lowest beam and token.
//
// Within a beam the order is that of the logits alone, so one pass over them
// finds both the log-sum and the beam's M best; only those enter the
// comparison between beams.  A block reads one piece of one beam's logits into
// registers, takes their maximum and the sum of exponentials, and keeps the M
// best: the M-th largest of the threads' own maxima bounds them from below, so
// few elements pass into the list that one warp then orders.  A second kernel
// joins the pieces' sums and merges their sorted lists.
//
// Which beam wins decides the tokens, so beams are compared in float64: the
// pieces' sums are accumulated in it from float32 exponentials, whose random
// errors average out, and a logit enters unrounded.
//
// Bound by memory: every logit is read once.
#include "kda_cache.h"
#include "kda_device.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kList = 1024;  // elements that may pass the bound

struct PieceSum {
  double sum;   // of exp(x - top)
  float top;    // largest logit, -inf if none
  int32_t next; // the join's place in the piece's list
};
static_assert(sizeof(PieceSum) == 16, "workspace layout");

// Order of the values as unsigned integers; -0 counts as +0.
__device__ __forceinline__ uint32_t sortable(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unsortable(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
constexpr uint32_t kNoKey = 0x007fffffu;  // of -inf: never a candidate

// A candidate: larger is better, ties to the lower index.
__device__ __forceinline__ uint64_t candidate(uint32_t key, int index) {
  return ((uint64_t)key << 32) | (uint32_t)~index;
}

__device__ __forceinline__ uint64_t warp_max64(uint64_t x) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(x >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(x >> 32) == hi ? (uint32_t)x : 0u);
  return ((uint64_t)hi << 32) | lo;
}

// A live beam reads its logits: its score is finite and it is not finished.
__device__ __forceinline__ bool reads_logits(const BeamArgs& a, int64_t beam) {
  return isfinite(__ldg(a.scores + beam)) && (a.finished == nullptr || __ldg(a.finished + beam) == 0);
}

struct Lists {
  PieceSum* sum;
  float* value;
  int32_t* index;
  __device__ __forceinline__ Lists(const BeamArgs& a, int splits) {
    const int64_t pieces = (int64_t)a.N * a.B * splits;
    sum = reinterpret_cast<PieceSum*>(a.work);
    value = a.work + pieces * 4;
    index = reinterpret_cast<int32_t*>(value + pieces * a.M);
  }
};

template <typename T, int E>
__global__ void __launch_bounds__(kThreads) kda_beam_scan_kernel(const BeamArgs a, int splits) {
  constexpr int VEC = 16 / sizeof(T), LOADS = E / VEC;
  static_assert(LOADS * VEC == E && LOADS >= 1, "bad shape");
  __shared__ float s_top[kThreads / 32];
  __shared__ double s_sum[kThreads / 32];
  __shared__ uint32_t s_key[kThreads];
  __shared__ uint64_t s_list[kList];
  __shared__ uint32_t s_bound;
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int split = blockIdx.x % splits;
  const int64_t beam = blockIdx.x / splits;
  pdl_wait();
  pdl_launch_dependents();
  if (!reads_logits(a, beam)) return;

  // The piece's vectors lie on 16-byte boundaries; the row may start and end inside one.
  const T* row = static_cast<const T*>(a.logits) + beam / a.B * a.ns + beam % a.B * a.bs;
  const int lead = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  float x[E];
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    const int64_t i0 = ((int64_t)(split * LOADS + j) * kThreads + tid) * VEC - lead;
    if (i0 >= 0 && i0 + VEC <= a.V) {
      if constexpr (sizeof(T) == 4) {
        const float4 r = __ldcs(reinterpret_cast<const float4*>(row + i0));
        x[j * VEC] = r.x; x[j * VEC + 1] = r.y; x[j * VEC + 2] = r.z; x[j * VEC + 3] = r.w;
      } else {
        const uint4 r = __ldcs(reinterpret_cast<const uint4*>(row + i0));
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          x[j * VEC + 2 * i] = bf_lo(w[i]);
          x[j * VEC + 2 * i + 1] = bf_hi(w[i]);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int64_t at = i0 + i;
        x[j * VEC + i] = -INFINITY;
        if (at >= 0 && at < a.V) {
          if constexpr (sizeof(T) == 4) x[j * VEC + i] = __ldg(row + at);
          else x[j * VEC + i] = __bfloat162float(__ldg(row + at));
        }
      }
    }
  }

  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < E; ++i) top = fmaxf(top, x[i]);
  s_key[tid] = sortable(top);
  float wtop = top;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) wtop = fmaxf(wtop, __shfl_xor_sync(0xffffffffu, wtop, o));
  if (lane == 0) s_top[warp] = wtop;
  if (tid == 0) s_count = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) wtop = fmaxf(wtop, s_top[w]);
  const float ref = wtop == -INFINITY ? 0.f : wtop;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) sum += expf(x[i] - ref);
  double total = sum;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  if (lane == 0) s_sum[warp] = total;

  if (warp == 0) {  // the M-th largest of the threads' maxima
    uint32_t k[kThreads / 32];
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) k[w] = s_key[w * 32 + lane];
    uint32_t bound = 0;
    for (int m = 0; m < a.M; ++m) {
      uint32_t mine = 0;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) mine = max(mine, k[w]);
      bound = __reduce_max_sync(0xffffffffu, mine);
      const int owner = __ffs(__ballot_sync(0xffffffffu, mine == bound)) - 1;
      bool gone = lane != owner;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w)
        if (!gone && k[w] == bound) { k[w] = 0; gone = true; }
    }
    if (lane == 0) s_bound = max(bound, kNoKey + 1);
  }
  __syncthreads();
  const uint32_t bound = s_bound;
  const Lists lists(a, splits);
  const int64_t piece = beam * splits + split;
  if (tid == 0) {
    double all = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) all += s_sum[w];
    lists.sum[piece].sum = all;
    lists.sum[piece].top = wtop;
  }
  if (sortable(top) >= bound) {
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const uint32_t key = sortable(x[i]);
      if (key >= bound) {
        const int at = atomicAdd(&s_count, 1);
        const int64_t index = ((int64_t)(split * LOADS + i / VEC) * kThreads + tid) * VEC - lead + i % VEC;
        if (at < kList) s_list[at] = candidate(key, (int)index);
      }
    }
  }
  __syncthreads();
  const int count = s_count;
  float* value = lists.value + piece * a.M;
  int32_t* index = lists.index + piece * a.M;
  if (count <= kList) {
    if (warp != 0) return;
    uint64_t last = ~0ull;
    for (int m = 0; m < a.M; ++m) {
      uint64_t best = 0;
      for (int i = lane; i < count; i += 32)
        if (s_list[i] < last && s_list[i] > best) best = s_list[i];
      last = best = warp_max64(best);
      if (lane == 0) {
        value[m] = best == 0 ? -INFINITY : unsortable((uint32_t)(best >> 32));
        index[m] = best == 0 ? -1 : (int)~(uint32_t)best;
      }
    }
    return;
  }
  // Too many equal values at the bound: take the best below the last one, M times, from the registers.
  __shared__ uint64_t s_best[kThreads / 32];
  uint64_t last = ~0ull;
  for (int m = 0; m < a.M; ++m) {
    uint64_t best = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const uint32_t key = sortable(x[i]);
      const int64_t at = ((int64_t)(split * LOADS + i / VEC) * kThreads + tid) * VEC - lead + i % VEC;
      const uint64_t c = candidate(key, (int)at);
      if (key >= bound && c < last && c > best) best = c;
    }
    best = warp_max64(best);
    if (lane == 0) s_best[warp] = best;
    __syncthreads();
    best = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) best = max(best, s_best[w]);
    last = best;
    if (tid == 0) {
      value[m] = best == 0 ? -INFINITY : unsortable((uint32_t)(best >> 32));
      index[m] = best == 0 ? -1 : (int)~(uint32_t)best;
    }
    __syncthreads();
  }
}

// One request: the beams' offsets score - log sum exp, then the merge of the
// pieces' sorted lists, one best candidate of the block a round.
__global__ void __launch_bounds__(kThreads) kda_beam_join_kernel(const BeamArgs a, int splits) {
  // A candidate is worth (x - top) + offset, offset = score - log sum exp(x - top): near the best, no large numbers cancel.
  __shared__ double s_offset[kBeamMax];
  __shared__ float s_top[kBeamMax];
  __shared__ int s_kind[kBeamMax];  // 0: nothing, 1: lists, 2: finished
  __shared__ double s_value[kThreads / 32];
  __shared__ int64_t s_flat[kThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t n = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const Lists lists(a, splits);

  for (int b = warp; b < a.B; b += kThreads / 32) {
    const int64_t beam = n * a.B + b;
    const float score = __ldg(a.scores + beam);
    int kind = 0;
    double offset = 0.0;
    float top = -INFINITY;
    if (isfinite(score)) {
      if (a.finished != nullptr && __ldg(a.finished + beam) != 0) {
        kind = 2;
        offset = score;
      } else {
        const PieceSum* p = lists.sum + beam * splits;
        for (int s = lane; s < splits; s += 32) top = fmaxf(top, p[s].top);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        double sum = 0.0;
        for (int s = lane; s < splits; s += 32) {
          const double part = p[s].sum;  // NaN if the piece holds one
          sum += part == 0.0 ? 0.0 : part * exp((double)p[s].top - (double)top);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        offset = (double)score - log(sum);
        kind = isfinite(offset) && isfinite(top) ? 1 : 0;
      }
    }
    if (lane == 0) {
      s_offset[b] = offset;
      s_top[b] = top;
      s_kind[b] = kind;
    }
  }
  __syncthreads();

  // Thread t owns the lists t, t + kThreads, ...: it alone moves their `next`
  // forward.  `head` is the best candidate its lists still hold.
  const int count = a.B * splits;
  PieceSum* piece = lists.sum + n * count;
  for (int l = tid; l < count; l += kThreads) piece[l].next = 0;
  double head = -INFINITY;
  int64_t head_flat = INT64_MAX;
  int head_list = -1;
  bool stale = true;
  for (int m = 0; m < a.M; ++m) {
    if (stale) {
      head = -INFINITY;
      head_flat = INT64_MAX;
      for (int l = tid; l < count; l += kThreads) {
        const int b = l / splits, next = piece[l].next;
        if (s_kind[b] == 0 || next == a.M) continue;
        int token = -1;
        double v = s_offset[b];
        if (s_kind[b] == 1) {
          token = lists.index[(n * count + l) * a.M + next];
          v += (double)lists.value[(n * count + l) * a.M + next] - (double)s_top[b];
        } else if (l == b * splits && next == 0) {
          token = a.eos;  // the one continuation of a finished beam
        }
        const int64_t flat = (int64_t)b * a.V + token;
        if (token >= 0 && (v > head || (v == head && flat < head_flat))) {
          head = v;
          head_flat = flat;
          head_list = l;
        }
      }
      stale = false;
    }
    double best = head;
    int64_t flat = head_flat;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double v = __shfl_xor_sync(0xffffffffu, best, o);
      const int64_t f = __shfl_xor_sync(0xffffffffu, flat, o);
      if (v > best || (v == best && f < flat)) {
        best = v;
        flat = f;
      }
    }
    if (lane == 0) {
      s_value[warp] = best;
      s_flat[warp] = flat;
    }
    __syncthreads();
    best = s_value[0];
    flat = s_flat[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w)
      if (s_value[w] > best || (s_value[w] == best && s_flat[w] < flat)) {
        best = s_value[w];
        flat = s_flat[w];
      }
    const bool none = flat == INT64_MAX;
    if (tid == 0) {
      const int64_t at = n * a.M + m;
      a.out_scores[at] = none ? -INFINITY : (float)best;
      a.out_parents[at] = none ? -1 : (int)(flat / a.V);
      a.out_tokens[at] = none ? -1 : (int)(flat % a.V);
    }
    if (!none && flat == head_flat) {
      ++piece[head_list].next;
      stale = true;
    }
    __syncthreads();
  }
}

template <typename T>
cudaError_t launch_scan(const BeamArgs& a, const BeamPlan& p, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.N * a.B * p.splits)), threads(kThreads);
  switch (p.per_thread) {
    case 8: return launch_pdl(kda_beam_scan_kernel<T, 8>, grid, threads, 0, s, 1, a, p.splits);
    case 16: return launch_pdl(kda_beam_scan_kernel<T, 16>, grid, threads, 0, s, 1, a, p.splits);
    default: return launch_pdl(kda_beam_scan_kernel<T, 32>, grid, threads, 0, s, 1, a, p.splits);
  }
}

}  // namespace

// Logits per thread: as many as still give every SM two blocks.
BeamPlan beam_plan(int64_t N, int32_t B, int32_t V, int32_t M, int32_t dtype, int32_t sms) {
  BeamPlan p;
  p.per_thread = 32;
  const int vec = dtype == KDA_DT_F32 ? 4 : 8;
  // A row that starts inside a vector reaches up to vec - 1 elements further.
  const auto splits = [&](int e) { return (int32_t)((V + vec - 1 + kThreads * (int64_t)e - 1) / (kThreads * (int64_t)e)); };
  while (p.per_thread > 8 && N * B * splits(p.per_thread) < 2 * sms) p.per_thread /= 2;
  p.splits = splits(p.per_thread);
  p.floats = N * B * p.splits * (4 + 2 * (int64_t)M);
  return p;
}

cudaError_t launch_beam_select(const BeamArgs& a, const BeamPlan& p, cudaStream_t s) {
  const cudaError_t e = a.dtype == KDA_DT_F32 ? launch_scan<float>(a, p, s) : launch_scan<__nv_bfloat16>(a, p, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(kda_beam_join_kernel, dim3((unsigned)a.N), dim3(kThreads), 0, s, 1, a, p.splits);
}

}  // namespace kda
