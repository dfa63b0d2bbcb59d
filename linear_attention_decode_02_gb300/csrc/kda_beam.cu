// Beam selection: the best M of all beams' continuations, by
// score_b + x_bt - log sum exp x_b, ties to the lowest beam and token.
//
// Within a beam the order is that of the logits alone, so one pass over them
// finds both the log-sum and the beam's M best; only those enter the
// comparison between beams.  A block holds one piece of one beam's logits in
// registers as they were loaded.  Its threads' maxima give the piece's largest
// logit and a bound: the least maximum of at least M disjoint groups of
// threads, above which at least M elements lie and, on unordered data, about
// M ln M.  Those few go to a list, where each finds its place by counting the
// larger ones.  A second kernel joins the pieces' sums and orders the pieces'
// candidates of all beams in the same way.
//
// Which beam wins decides the tokens, so the log-sums have to be better than
// float32 gives: a piece's exponentials are 2^((x - top) log2(e) + c), with c
// such that top log2(e) - c is an integer, so that pieces are rescaled by exact
// powers of two; log2(e) enters in two parts; batches, lanes and
// pieces are added with the rounding carried along; and logarithms and
// candidates are unrounded sums of two float32 (float64 runs at a hundredth of
// float32's rate here: a logarithm in it alone took 1.8 us).  What is left,
// relative to the sum: 2^-22 of the exponential's approximation; two roundings of
// its argument, 4.4e-7 at worst, where a thread's 256 logits are all 8 ln 2 below
// its largest; and six of a batch's additions, 3.6e-7.  Measured: 1.6e-7 on rows
// of one or two values (3.1e-7 with a thread's terms added one after another, in
// 0.5 us less for the large case below); on 65536 normal logits 5e-8, all but 5e-9 of
// it common to all beams, since the approximation errs a little to one side.
//
// Every logit is read once, 64 bytes a thread on their way while 64 are summed.
// 32 requests of 8 beams, a tenth of them finished, over 131072 tokens in bf16,
// 61 MB, which a copy would read in 9 us, take 20 to 22 us a call.  Alone the scan
// takes 18 to 19 us and the join 6, which starts under the scan's end.  The scan
// uses 40 % of the DRAM's peak: after the last logit come the bound, the list
// and the order, behind barriers, and all pieces reach them at the same time.
// Shorter pieces made more of that: 1024 blocks instead of 512 took 22 to 25 us,
// 2048 26 to 28, beside 19 to 21 then.  Both kernels run their code once a block, so
// what is unrolled counts: one thread that read a marked batch again, all four
// vectors of it, and a join unrolled over 32 beams took 21 us instead of 19.
// 12 x 6 float32 rows of 50257 take 13 to 15 us, 4 rows of 32000 bf16 9 to 11.
#include <float.h>

#include "kda_cache.h"
#include "kda_device.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kList = 1024;   // elements that may pass the bound
constexpr int kJoin = 4096;
constexpr float kLog2e = 1.44269502f, kLog2eLow = 1.92596299e-8f;  // log2(e) to 2^-50
constexpr float kLn2 = 0.693147182f, kLn2Low = -1.90465421e-9f;  // ln 2 to 2^-50
constexpr double kLog2eDouble = 1.4426950408889634;

// Sum of 2^((x - top) log2(e) + c) over a piece, as hi + lo.
struct PieceSum {
  float hi, lo;
  float top;    // largest logit
  float pad;
};
static_assert(sizeof(PieceSum) == 16, "workspace layout");

// hi + lo += x, the rounding of the first kept in the second (Knuth's two-sum).
__device__ __forceinline__ void add_carried(float& hi, float& lo, float x, float xlo) {
  const float s = hi + x, t = s - hi;
  lo += xlo + ((hi - (s - t)) + (x - t));
  hi = s;
}
__device__ __forceinline__ void warp_sum_carried(float& hi, float& lo) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float x = __shfl_xor_sync(0xffffffffu, hi, o), y = __shfl_xor_sync(0xffffffffu, lo, o);
    add_carried(hi, lo, x, y);
  }
}

// Natural logarithm of hi + lo, normal and positive, as hi + lo, to 2^-32 and a
// few 2^-46 of it: with m in [0.7, 1.4) and s = (m - 1) / (m + 1), log m =
// 2 (s + s^3 / 3 + s^5 / 5 + ...), |s| < 0.172; only s itself needs two floats.
__device__ __forceinline__ void log_carried(float& hi, float& lo) {
  int e = ((__float_as_int(hi) >> 23) & 255) - 127;
  float m = __int_as_float((__float_as_int(hi) & 0x7fffff) | 0x3f800000);
  if (m > 1.41421354f) {
    m *= 0.5f;
    ++e;
  }
  const float ml = lo * __int_as_float((127 - max(e, -126)) << 23);
  const float num = m - 1.f, den = m + 1.f, dl = (1.f - (den - m)) + ml;
  const float q = num / den;
  const float ql = (fmaf(-q, den, num) + ml - q * dl) / den;
  const float z = q * q;
  float tail = 1.f / 13.f;
  tail = fmaf(tail, z, 1.f / 11.f);
  tail = fmaf(tail, z, 1.f / 9.f);
  tail = fmaf(tail, z, 1.f / 7.f);
  tail = fmaf(tail, z, 1.f / 5.f);
  tail = fmaf(tail, z, 1.f / 3.f);
  const float fe = (float)e, p = fe * kLn2;
  hi = p;
  lo = fmaf(fe, kLn2, -p) + fe * kLn2Low;
  add_carried(hi, lo, 2.f * q, 2.f * (ql + q * z * tail));
}

// A piece with the largest logit `top` is summed relative to 2^r, r the integer
// next above top log2(e).  Its float32 product rounds to 2^-4 before kNear, so r
// can be one off there; all that counts is that a piece's r, and the scaling of
// its sum, follow from its own top alone: in float32 where near() holds,
// in float64 beyond.
constexpr float kNear = 1048576.f;  // float32 holds r exactly, with room for c
__device__ __forceinline__ bool near(float top) { return fabsf(top * kLog2e) < kNear; }
__device__ __forceinline__ double reference(float top) {
  return near(top) ? (double)ceilf(top * kLog2e) : ceil(top * kLog2eDouble);
}
// c = top log2(e) - r of a top that is not near, to float32.
__device__ __forceinline__ float far_fraction(float top) {
  const double x = top * kLog2eDouble;
  return (float)(x - ceil(x));
}
// r of `own` minus r of `top`, at most 0 for own <= top; below -1000 it is -1000.
__device__ __forceinline__ int reference_shift(float own, float top) {
  if (near(own) && near(top)) return (int)fmaxf(ceilf(own * kLog2e) - ceilf(top * kLog2e), -1000.f);
  return (int)fmax(reference(own) - reference(top), -1000.0);
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Order of the values as unsigned integers; -0 counts as +0.
__device__ __forceinline__ uint32_t sortable(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float unsortable(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// A logit and its place: larger is better, ties to the lower index.  0 is none.
__device__ __forceinline__ uint64_t candidate(float x, int index) {
  return ((uint64_t)sortable(x) << 32) | (uint32_t)~index;
}

// Workspace: the pieces' sums, then their M best (0 past the last), best first.
struct Lists {
  PieceSum* sum;
  uint64_t* best;
  __device__ __forceinline__ Lists(const BeamArgs& a, int splits) {
    sum = reinterpret_cast<PieceSum*>(a.work);
    best = reinterpret_cast<uint64_t*>(a.work + (int64_t)a.N * a.B * splits * 4);
  }
};

// Every warp alone, from the threads' maxima: the largest, and the least maximum
// of `groups` (8 .. 64, a power of two) groups of threads, thread t in group
// t % groups, so that a few threads with data already fill all groups.
__device__ __forceinline__ void block_bound(const uint32_t (&keys)[kThreads], int groups, int lane, uint32_t& highest,
                                            uint32_t& lowest) {
  uint32_t even = keys[lane], odd = keys[32 + lane];
#pragma unroll
  for (int w = 2; w < kWarps; w += 2) {
    even = max(even, keys[w * 32 + lane]);
    odd = max(odd, keys[(w + 1) * 32 + lane]);
  }
  uint32_t m = max(even, odd);
  highest = __reduce_max_sync(0xffffffffu, m);
  if (groups == 64) m = min(even, odd);
  for (int o = groups; o < 32; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  lowest = __reduce_min_sync(0xffffffffu, m);
}
__device__ __forceinline__ uint64_t warp_max64(uint64_t x) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, (uint32_t)(x >> 32));
  const uint32_t lo = __reduce_max_sync(0xffffffffu, (uint32_t)(x >> 32) == hi ? (uint32_t)x : 0u);
  return ((uint64_t)hi << 32) | lo;
}

// Calls put(rank, list[i]) for the i below `count` whose rank, the number of
// larger entries, is below M.  Four lanes share an entry's comparisons.
template <typename E, typename Larger, typename Put>
__device__ __forceinline__ void place(const E* list, int count, int M, const Larger& larger, const Put& put) {
  const int part = threadIdx.x & 3;
  for (int base = 0; base < count; base += kThreads / 4) {
    const int i = base + (threadIdx.x >> 2);
    const E mine = list[min(i, count - 1)];
    int rank = 0;
#pragma unroll 8
    for (int j = part; j < count; j += 4) rank += larger(list[j], mine) ? 1 : 0;
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    if (i < count && part == 0 && rank < M) put(rank, mine);
  }
}

template <typename T>
struct Raw;  // 16 bytes of logits as loaded
template <>
struct Raw<float> {
  static constexpr int VEC = 4;
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void set(int i, const float* p) {
    const float x = p != nullptr ? __ldg(p) : -INFINITY;
    (i == 0 ? v.x : (i == 1 ? v.y : (i == 2 ? v.z : v.w))) = x;
  }
  __device__ __forceinline__ float2 pair(int i) const { return i == 0 ? make_float2(v.x, v.y) : make_float2(v.z, v.w); }
  __device__ __forceinline__ float top() const { return fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)); }
};
template <>
struct Raw<__nv_bfloat16> {
  static constexpr int VEC = 8;
  uint32_t w[4];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    const uint4 r = __ldcs(reinterpret_cast<const uint4*>(p));
    w[0] = r.x; w[1] = r.y; w[2] = r.z; w[3] = r.w;
  }
  __device__ __forceinline__ void set(int i, const __nv_bfloat16* p) {
    const uint32_t x = p != nullptr ? __ldg(reinterpret_cast<const unsigned short*>(p)) : 0xff80u;
    w[i / 2] = i % 2 == 0 ? (w[i / 2] & 0xffff0000u) | x : (w[i / 2] & 0xffffu) | (x << 16);
  }
  __device__ __forceinline__ float2 pair(int i) const { return make_float2(bf_lo(w[i]), bf_hi(w[i])); }
  __device__ __forceinline__ float top() const {
    __nv_bfloat162 m = __hmax2(__hmax2(h(0), h(1)), __hmax2(h(2), h(3)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  __device__ __forceinline__ __nv_bfloat162 h(int i) const { return *reinterpret_cast<const __nv_bfloat162*>(&w[i]); }
};

// A thread's vector of a batch on its way.  Rows that all start on 16-byte
// boundaries: neighbouring elements in one load.  Others: elements kThreads apart,
// loaded one by one, so that which of them a thread adds, and in what order, does
// not depend on where a row starts: equal rows have equal log-sums, and tie.
// Elements past the row are -infinity.
//
// Measured, kernels alone, against 16-byte loads from each row's own boundary on,
// whose sums depend on it: bfloat16 32 x 8 rows of 131071 27.0 and 23.7 us, 64 x 4 of
// 50257 17.0 and 14.6, 16 x 8 of 50257 13.1 and 12.0, 4 x 16 15.7 and 16.5; float32
// 12 x 6 of 50257 12.8 and 12.4.  Others that do not depend on it: pairs of bfloat16
// in one load where a row allows it 27.9, 18.0 and 14.5 us for the first three;
// vectors put together from two lanes' 16 bytes 28.2 and 15.5 for the first and third;
// four vectors instead of two on their way, at three blocks a SM, 27.1, 20.2 and 12.7.
template <typename T, bool ALIGNED>
struct Ahead;
template <typename T>
struct Ahead<T, true> {
  static constexpr int STEP = 1;
  Raw<T> v;
  __device__ __forceinline__ void load(const T* row, int i, int V) {
    constexpr int VEC = Raw<T>::VEC;
    if (i + VEC <= V) {
      v.load(row + i);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v.set(e, i + e < V ? row + i + e : nullptr);
    }
  }
  __device__ __forceinline__ Raw<T> get() const { return v; }
};
template <>
struct Ahead<float, false> {
  static constexpr int STEP = kThreads;
  Raw<float> v;
  __device__ __forceinline__ void load(const float* row, int i, int V) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v.set(e, i + e * STEP < V ? row + i + e * STEP : nullptr);
  }
  __device__ __forceinline__ Raw<float> get() const { return v; }
};
template <>
struct Ahead<__nv_bfloat16, false> {
  static constexpr int STEP = kThreads;
  unsigned short u[8];  // a register each until they are used
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int i, int V) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      u[e] = i + e * STEP < V ? __ldg(reinterpret_cast<const unsigned short*>(row) + i + e * STEP) : (unsigned short)0xff80;
  }
  __device__ __forceinline__ Raw<__nv_bfloat16> get() const {
    Raw<__nv_bfloat16> v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v.w[e] = u[2 * e] | (uint32_t)u[2 * e + 1] << 16;
    return v;
  }
};

// Groups of threads for the bound.
__device__ __forceinline__ int bound_groups(int M) {
  int g = kWarps;
  while (g < M) g *= 2;
  return g;
}

// Batches that a block may take: pieces have up to 32 vectors a thread, 2 where a batch has one.
__host__ __device__ constexpr int most_batches(int loads) { return loads == 1 ? 2 : 32 / loads; }

// Thread's sum of 2^(x log2(e) - r) for one batch of loads, r at least every
// exponent.  Added in a tree: at most six roundings in a row, and next to none
// where all terms are equal.
template <typename T, int LOADS>
__device__ __forceinline__ float batch_sum(const Raw<T> (&x)[LOADS], float r) {
  constexpr int PAIRS = Raw<T>::VEC / 2;
  const float2 hi2 = dup2(kLog2e), lo2 = dup2(kLog2eLow), r2 = dup2(-r);
  float2 sum;
#pragma unroll
  for (int j = 0; j < LOADS; ++j) {
    float2 e[PAIRS];
#pragma unroll
    for (int i = 0; i < PAIRS; ++i) {
      const float2 v = x[j].pair(i);
      e[i] = fma2(v, lo2, fma2(v, hi2, r2));
      e[i] = make_float2(ex2(e[i].x), ex2(e[i].y));
    }
#pragma unroll
    for (int o = 1; o < PAIRS; o *= 2)
#pragma unroll
      for (int i = 0; i < PAIRS; i += 2 * o) e[i] = add2(e[i], e[i + o]);
    sum = j == 0 ? e[0] : add2(sum, e[0]);
  }
  return sum.x + sum.y;
}

template <typename T, int LOADS, bool ALIGNED>
__global__ void __launch_bounds__(kThreads, 4) kda_beam_scan_kernel(const BeamArgs a, int splits, int batches) {
  using Vector = Ahead<T, ALIGNED>;
  constexpr int VEC = Raw<T>::VEC, BATCH = LOADS * kThreads * VEC, STEP = Vector::STEP;
  constexpr int MOST = most_batches(LOADS);
  __shared__ uint32_t s_key[kThreads];
  __shared__ float s_hi[kThreads], s_lo[kThreads], s_tops[MOST][kThreads];
  __shared__ uint64_t s_list[kList];
  __shared__ uint16_t s_hot[MOST * kThreads];
  __shared__ int s_count, s_hots;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t beam = blockIdx.x / (uint32_t)splits;
  const int split = blockIdx.x - beam * splits;
  if (tid == 0) s_count = s_hots = 0;

  const uint32_t n = beam / (uint32_t)a.B;
  const T* row = static_cast<const T*>(a.logits) + n * a.ns + (beam - n * a.B) * a.bs;
  const int first = split * batches * BATCH;  // of the piece
  // Where vector j of thread t's batch starts; its elements are STEP apart.
  const auto place_of = [&](int batch, int j, int t) {
    return first + batch * BATCH + j * kThreads * VEC + (ALIGNED ? t * VEC : t);
  };
  const auto load = [&](int batch, Vector(&x)[LOADS]) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) x[j].load(row, place_of(batch, j, tid), a.V);
  };
  pdl_wait();
  pdl_launch_dependents();
  Raw<T> x[LOADS];
  Vector ahead[LOADS];
  load(0, ahead);
  // A live beam's score is finite and it is not finished; of others the first batch is read for nothing.
  const int done = a.finished != nullptr ? __ldg(a.finished + beam) : 0;
  if (!isfinite(__ldg(a.scores + beam)) || done != 0) return;

  // One batch is summed while the next is on its way.  The thread's reference
  // r moves in whole steps, so rescaling its sum is exact.
  float top = -INFINITY, r = -kNear, sum = 0.f, rest = 0.f;
#pragma unroll 1
  for (int k = 0; k < batches; ++k) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) x[j] = ahead[j].get();
    if (k + 1 < batches) load(k + 1, ahead);
    float t = x[0].top();
#pragma unroll
    for (int j = 1; j < LOADS; ++j) t = fmaxf(t, x[j].top());
    s_tops[k][tid] = t;
    top = fmaxf(top, t);
    const float up = ceilf(t * kLog2e);
    if (up > r) {
      const float down = __int_as_float(max((int)fmaxf(r - up, -126.f) + 127, 0) << 23);
      sum *= down;
      rest *= down;
      r = up;
    }
    add_carried(sum, rest, batch_sum<T, LOADS>(x, r), 0.f);
  }

  s_key[tid] = sortable(top);
  __syncthreads();
  uint32_t lowest, highest;
  block_bound(s_key, bound_groups(a.M), lane, highest, lowest);
  const float bound = unsortable(lowest), all = unsortable(highest);
  const int end = (int)min((int64_t)a.V, (int64_t)first + (int64_t)batches * BATCH);

  // Elements at or above the bound go to the list.  One batch is still in
  // registers; of several, the threads' batches that hold one are noted first
  // and read again, a vector a thread, so that one memory latency serves all.
  const auto push = [&](const Raw<T>& v, int i) {
    if (!(v.top() >= bound)) return;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float2 p = v.pair(e / 2);
      const float w = e % 2 == 0 ? p.x : p.y;
      if (w >= bound && w > -INFINITY) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kList) s_list[at] = candidate(w, i + e * STEP);
      }
    }
  };
  if (batches == 1) {
#pragma unroll
    for (int j = 0; j < LOADS; ++j) push(x[j], place_of(0, j, tid));
  } else if (top >= bound) {
#pragma unroll 1
    for (int k = 0; k < batches; ++k)
      if (s_tops[k][tid] >= bound) s_hot[atomicAdd(&s_hots, 1)] = (uint16_t)(k * kThreads + tid);
  }
  float hi, lo = 0.f;
  if (near(all)) {
    const int shift = (int)fmaxf(r - ceilf(all * kLog2e), -127.f);  // r is at most the block's
    const float down = __int_as_float((shift + 127) << 23);
    hi = sum * down;
    lo = rest * down;
  } else if (all > -INFINITY) {
    // Logits of 10^6 and more: once more, by their distance from the largest.
    const float c = far_fraction(all);
    hi = 0.f;
    for (int i = first + tid; i < end; i += kThreads)
      add_carried(hi, lo, ex2(fmaf(static_cast<float>(row[i]) - all, kLog2e, c)), 0.f);
  } else {
    hi = sum;  // nothing above -infinity: 0, or NaN
  }
  s_hi[tid] = hi;
  s_lo[tid] = lo;
  __syncthreads();
  if (batches > 1) {
    for (int h = tid; h < s_hots * LOADS; h += kThreads) {
      const int entry = s_hot[h / LOADS];
      const int at = place_of(entry / kThreads, h % LOADS, entry % kThreads);
      Vector v;
      v.load(row, at, a.V);
      push(v.get(), at);
    }
    __syncthreads();
  }
  const int count = s_count;
  const Lists lists(a, splits);
  const int64_t piece = blockIdx.x;
  uint64_t* best = lists.best + piece * a.M;
  if (warp == kWarps - 1) {  // the last to have a candidate to place
    hi = s_hi[lane];
    lo = s_lo[lane];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) add_carried(hi, lo, s_hi[w * 32 + lane], s_lo[w * 32 + lane]);
    warp_sum_carried(hi, lo);
    if (lane == 0) {
      PieceSum p;
      p.hi = hi; p.lo = lo; p.top = all; p.pad = 0.f;
      lists.sum[piece] = p;
    }
  }
  const auto above = [](uint64_t x, uint64_t y) { return x > y; };
  const auto keep = [&](int rank, uint64_t x) { best[rank] = x; };
  if (count <= kList) {
    place(s_list, count, a.M, above, keep);
    for (int i = count + tid; i < a.M; i += kThreads) best[i] = 0;
    return;
  }
  // Too many at the bound.  On masked or constant logits they equal it; of
  // those only the first in the row matter.  The larger ones are counted again,
  // in the row's own order: 16 bytes at a time from the boundary before the piece,
  // what is not the piece's left out.
  const int from = first - (int)((reinterpret_cast<uintptr_t>(row + first) & 15) / sizeof(T));
  const auto load_run = [&](int i, Raw<T>& v) {
    if (i >= first && i + VEC <= end) {
      v.load(row + i);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v.set(e, i + e >= first && i + e < end ? row + i + e : nullptr);
    }
  };
  __syncthreads();
  if (tid == 0) s_count = 0;
  __syncthreads();
  const int vectors = (end - from + VEC - 1) / VEC;
  for (int h = tid; h < vectors; h += kThreads) {
    Raw<T> v;
    load_run(from + h * VEC, v);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float2 p = v.pair(e / 2);
      const float w = e % 2 == 0 ? p.x : p.y;
      if (w > bound) {
        const int at = atomicAdd(&s_count, 1);
        if (at < kList) s_list[at] = candidate(w, from + h * VEC + e);
      }
    }
  }
  __syncthreads();
  const int larger = s_count;
  if (larger <= kList) {
    place(s_list, larger, a.M, above, keep);
    int next = larger;  // place of the next equal one
    for (int h0 = 0; h0 < vectors && next < a.M && bound > -INFINITY; h0 += kThreads) {
      Raw<T> v;
      load_run(from + (h0 + tid) * VEC, v);
      int equal = 0;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float2 p = v.pair(e / 2);
        equal |= (e % 2 == 0 ? p.x : p.y) == bound ? 1 << e : 0;
      }
      if (h0 + tid >= vectors) equal = 0;
      int scan = __popc(equal);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o) scan += up;
      }
      __syncthreads();  // the last step's readers
      if (lane == 31) s_key[warp] = scan;
      __syncthreads();
      int at = next + scan - __popc(equal);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) at += s_key[w];
        next += s_key[w];
      }
      for (int left = equal; left != 0 && at < a.M; left &= left - 1, ++at)
        best[at] = candidate(bound, from + (h0 + tid) * VEC + __ffs(left) - 1);
    }
    for (int i = next + tid; i < a.M; i += kThreads) best[i] = 0;
    return;
  }
  // Neither: M times the best below the last one, from memory.
  uint64_t last = ~0ull;
  for (int m = 0; m < a.M; ++m) {
    uint64_t mine = 0;
    for (int i = first + tid; i < end; i += kThreads) {
      const float v = static_cast<float>(row[i]);
      const uint64_t at = candidate(v, i);
      if (v >= bound && v > -INFINITY && at < last && at > mine) mine = at;
    }
    mine = warp_max64(mine);
    __syncthreads();  // the list's last readers
    if (lane == 0) s_list[warp] = mine;
    __syncthreads();
    mine = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mine = max(mine, s_list[w]);
    last = mine;
    if (tid == 0) best[m] = mine;
  }
}

// (x - top) + (hi + lo) to about 48 bits.
__device__ __forceinline__ uint64_t value_key(float x, float top, float hi, float lo) {
  float s = x, rest = 0.f;
  add_carried(s, rest, -top, 0.f);
  add_carried(s, rest, hi, lo);
  if (!(s >= -FLT_MAX)) return 1;  // beyond float32: the last of all
  const float value = s + rest;
  return ((uint64_t)sortable(value) << 32) | sortable(rest - (value - s));
}

// A continuation of any beam: larger value, then lower flat index.
struct __align__(16) Choice {
  uint64_t key;  // sortable(hi) and sortable(lo) of the value hi + lo, hi its float32 rounding; 0: none
  int32_t flat;  // beam * V + token
};
__device__ __forceinline__ bool before(const Choice& a, const Choice& b) {
  return (a.key > b.key) | ((a.key == b.key) & (a.flat < b.flat));
}

// One request.  List l is the one of piece l % splits of beam l / splits; a
// finished beam has one candidate, in its first list.  The bound comes from the
// first entries of the lists, kJoin in all, dealt to its groups by a hash: the
// best may all be of one beam, and of the first places of a few lists.  The
// lists are sorted, so each is then followed only as far as the bound lets it.
constexpr int kStep = 8;  // entries of a list that one thread follows
constexpr int kHeld = 4;  // entries a thread keeps from the bound to the list
__global__ void __launch_bounds__(kThreads) kda_beam_join_kernel(const BeamArgs a, int splits) {
  // A candidate is worth (x - top) + offset, offset = score - log sum exp(x - top): no large numbers cancel.
  __shared__ float s_hi[kBeamMax], s_lo[kBeamMax];  // the sum, then the offset
  __shared__ float s_top[kBeamMax];
  __shared__ int s_kind[kBeamMax];                  // 0: nothing, 1: lists, 2: finished
  __shared__ uint32_t s_group[64];
  __shared__ Choice s_list[kList];
  __shared__ int s_count;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t n = blockIdx.x;
  if (tid == 0) s_count = 0;
  if (tid < 64) s_group[tid] = 0;
  pdl_wait();
  pdl_launch_dependents();
  const Lists lists(a, splits);
  const int pieces = a.B * splits;
  const uint64_t* best = lists.best + n * pieces * a.M;
  const auto fetch = [&](int l, int m) { return best[(int64_t)l * a.M + m]; };
  const int heads = min(a.M, max(1, kJoin / pieces)), count = heads * pieces;
  uint64_t held[kHeld];  // on their way while the sums are joined; without meaning for a beam whose logits were not read
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int e = tid + k * kThreads;
    held[k] = e < count ? fetch(e / heads, e % heads) : 0;
  }

  // Warp w joins the sums of the beams w, w + kWarps, ..., the next one's loads on their way.
  struct Loads {
    float score;
    int done;
    PieceSum part;
  };
  const auto load_beam = [&](int b) {
    Loads x;
    x.score = 0.f;
    x.done = 0;
    x.part.hi = x.part.lo = 0.f;
    x.part.top = -INFINITY;
    if (b < a.B) {
      x.score = __ldg(a.scores + n * a.B + b);
      if (a.finished != nullptr) x.done = __ldg(a.finished + n * a.B + b);
      if (lane < splits) x.part = lists.sum[n * pieces + b * splits + lane];  // of a beam not read: not used
    }
    return x;
  };
  Loads next = load_beam(warp);
#pragma unroll 1
  for (int b = warp; b < a.B; b += kWarps) {
    const Loads x = next;
    next = load_beam(b + kWarps);
    const bool reads = isfinite(x.score) && x.done == 0;
    float hi = 0.f, lo = 0.f, top = -INFINITY;
    if (reads) {
      const PieceSum* p = lists.sum + n * pieces + b * splits;
      top = x.part.top;
      for (int s = lane + 32; s < splits; s += 32) top = fmaxf(top, p[s].top);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 1
      for (int s = lane; s < splits; s += 32) {
        // Times 2^(r_s - r), exact; below 2^-126 it adds nothing.  A NaN in the piece is in hi.
        const PieceSum q = s == lane ? x.part : p[s];
        const int shift = q.top > -INFINITY ? reference_shift(q.top, top) : 0;
        const float scale = shift < -126 ? 0.f : __int_as_float((127 + min(shift, 0)) << 23);
        add_carried(hi, lo, q.hi * scale, q.lo * scale);
      }
      warp_sum_carried(hi, lo);
    }
    if (lane == 0) {
      s_hi[b] = hi;
      s_lo[b] = lo;
      s_top[b] = top;
      s_kind[b] = reads ? (isfinite(top) ? 1 : 0) : (isfinite(x.score) ? 2 : 0);
    }
  }
  __syncthreads();
  if (tid < a.B && s_kind[tid] != 0) {
    const float score = __ldg(a.scores + n * a.B + tid);
    float hi = score, lo = 0.f;
    if (s_kind[tid] == 1) {
      // log sum exp(x - top) = log(1 + (S - E) / 2^c), with S the pieces' sum, c = top log2(e) - r, and E = 2^c as the
      // scan rounded it: E's own error, `off` relative to it, is not in the result, which is 0 where nothing but
      // the largest logit weighs anything, so that a beam's only token is worth its score to the bit.
      const float top = s_top[tid], all = s_hi[tid], up = ceilf(top * kLog2e);
      const float c = near(top) ? fmaf(top, kLog2eLow, fmaf(top, kLog2e, -up)) : far_fraction(top), e = ex2(c);
      float base = e, basel = 0.f;
      log_carried(base, basel);
      const float of = near(top) ? -up : c, p = of * kLn2;  // c ln 2 as two floats
      float exact = near(top) ? top : 0.f, exactl = 0.f;
      add_carried(exact, exactl, p, fmaf(of, kLn2, -p) + of * kLn2Low);
      add_carried(exact, exactl, -base, -basel);
      const float off = exact + exactl;
      float ln = all, lnl = s_lo[tid], rest = ln, restl = lnl;
      add_carried(rest, restl, -e, 0.f);
      add_carried(ln, lnl, -(rest + restl) * off, 0.f);
      log_carried(ln, lnl);
      add_carried(base, basel, -ln, -lnl);
      add_carried(hi, lo, base, basel);
      if (!(all > 0.f && isfinite(all))) hi = NAN;
      if (!isfinite(hi)) s_kind[tid] = 0;
    }
    s_hi[tid] = hi;
    s_lo[tid] = lo;
  }
  __syncthreads();

  const auto choice = [&](int l, int m, uint64_t x) {
    Choice c;
    c.key = 0;
    c.flat = INT32_MAX;
    const int b = l / splits, kind = s_kind[b];
    if (kind == 1) {
      if (x != 0) {
        c.flat = b * a.V + (int)~(uint32_t)x;
        c.key = value_key(unsortable((uint32_t)(x >> 32)), s_top[b], s_hi[b], s_lo[b]);
      }
    } else if (kind == 2 && l == b * splits && m == 0) {
      c.flat = b * a.V + a.eos;
      c.key = value_key(0.f, 0.f, s_hi[b], 0.f);
    }
    return c;
  };
  const int groups = bound_groups(a.M);
  const auto enter = [&](int e, const Choice& c) {
    atomicMax(&s_group[((uint32_t)e * 2654435761u >> 26) & (groups - 1)], (uint32_t)(c.key >> 32));
  };
  Choice own[kHeld];
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int e = tid + k * kThreads;
    own[k].key = 0;
    if (e < count) {
      own[k] = choice(e / heads, e % heads, held[k]);
      enter(e, own[k]);
    }
  }
  for (int e = tid + kHeld * kThreads; e < count; e += kThreads) enter(e, choice(e / heads, e % heads, fetch(e / heads, e % heads)));
  __syncthreads();
  uint32_t least = min(s_group[lane & (groups - 1)], s_group[(lane + 32) & (groups - 1)]);
  least = __reduce_min_sync(0xffffffffu, least);
  const uint64_t bound = max((uint64_t)least << 32, (uint64_t)1);
  const auto push = [&](const Choice& c) {
    const int at = atomicAdd(&s_count, 1);
    if (at < kList) s_list[at] = c;
  };
  if (heads == a.M && count <= kHeld * kThreads) {  // all of them are at hand
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (own[k].key >= bound) push(own[k]);
  }
  const int steps = heads == a.M && count <= kHeld * kThreads ? 0 : (a.M + kStep - 1) / kStep;
  for (int u = tid; u < pieces * steps; u += kThreads) {
    const int l = u / steps, step = u - l * steps;
    for (int m = step * kStep; m < min(a.M, (step + 1) * kStep); ++m) {
      const Choice c = choice(l, m, fetch(l, m));
      if (c.key < bound) break;
      push(c);
    }
  }
  __syncthreads();
  const int found = s_count;
  const auto put = [&](int m, const Choice& c) {
    const int64_t at = n * a.M + m;
    a.out_scores[at] = c.key <= 1 ? -INFINITY : unsortable((uint32_t)(c.key >> 32));
    a.out_parents[at] = c.key == 0 ? -1 : c.flat / a.V;
    a.out_tokens[at] = c.key == 0 ? -1 : c.flat % a.V;
  };
  if (found <= kList) {
    place(s_list, found, a.M, before, put);
    for (int i = found + tid; i < a.M; i += kThreads) put(i, Choice{0, 0});
    return;
  }
  // Too many equal values at the bound: M times the best after the last one.
  Choice last{~0ull, -1};
  for (int m = 0; m < a.M; ++m) {
    Choice c{0, INT32_MAX};
    for (int i = tid; i < pieces * a.M; i += kThreads) {
      const Choice x = choice(i / a.M, i % a.M, fetch(i / a.M, i % a.M));
      if (x.key >= bound && before(last, x) && before(x, c)) c = x;
    }
    const uint64_t key = warp_max64(c.key);
    const int32_t flat = (int32_t)__reduce_min_sync(0xffffffffu, c.key == key ? (unsigned)c.flat : 0xffffffffu);
    __syncthreads();
    if (lane == 0) s_list[warp] = Choice{key, flat};
    __syncthreads();
    c = s_list[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w)
      if (before(s_list[w], c)) c = s_list[w];
    last = c;
    if (tid == 0) put(m, c);
  }
}

template <typename T, int LOADS, bool ALIGNED>
cudaError_t launch_scan(const BeamArgs& a, const BeamPlan& p, cudaStream_t s) {
  const dim3 grid((unsigned)((int64_t)a.N * a.B * p.splits)), threads(kThreads);
  return launch_pdl(kda_beam_scan_kernel<T, LOADS, ALIGNED>, grid, threads, 0, s, 1, a, p.splits, p.batches);
}

// Vectors of a batch.  Elements loaded one by one take a register each, so
// there bfloat16 has half as many on their way.
int batch_loads(int vectors, int32_t dtype, bool aligned) {
  if (vectors < 4) return 1;
  return aligned || dtype == KDA_DT_F32 ? 4 : 2;
}

}  // namespace

// The longest pieces (32 vectors a thread) that still give every SM
// two blocks, down to one vector, and not so short that the join, one
// block a request, would have more than kJoin candidates to look at.
BeamPlan beam_plan(int64_t N, int32_t B, int32_t V, int32_t M, int32_t dtype, bool aligned, int32_t sms) {
  BeamPlan p;
  const int64_t vec = dtype == KDA_DT_F32 ? 4 : 8;
  const auto splits = [&](int vectors) { return (int32_t)((V + kThreads * vec * vectors - 1) / (kThreads * vec * vectors)); };
  int vectors = 32;
  while (vectors > 1 && (splits(vectors / 2) == 1 || (N * B * splits(vectors) < 2 * sms &&
                                                      (int64_t)B * splits(vectors / 2) * M <= kJoin)))
    vectors /= 2;
  p.aligned = aligned;
  p.loads = batch_loads(vectors, dtype, aligned);
  p.splits = splits(vectors);
  const int64_t batch = kThreads * vec * p.loads * (int64_t)p.splits;  // the splits share the row evenly
  p.batches = (int32_t)((V + batch - 1) / batch);
  p.floats = N * B * p.splits * (4 + 2 * (int64_t)M);
  return p;
}

cudaError_t launch_beam_select(const BeamArgs& a, const BeamPlan& p, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  cudaError_t e;
  if (a.dtype == KDA_DT_F32) {
    e = p.aligned ? (p.loads == 1 ? launch_scan<float, 1, true>(a, p, s) : launch_scan<float, 4, true>(a, p, s))
                  : (p.loads == 1 ? launch_scan<float, 1, false>(a, p, s) : launch_scan<float, 4, false>(a, p, s));
  } else {
    e = p.aligned ? (p.loads == 1 ? launch_scan<bf16, 1, true>(a, p, s) : launch_scan<bf16, 4, true>(a, p, s))
                  : (p.loads == 1 ? launch_scan<bf16, 1, false>(a, p, s) : launch_scan<bf16, 2, false>(a, p, s));
  }
  if (e != cudaSuccess) return e;
  return launch_pdl(kda_beam_join_kernel, dim3((unsigned)a.N), dim3(kThreads), 0, s, 1, a, p.splits);
}

}  // namespace kda
