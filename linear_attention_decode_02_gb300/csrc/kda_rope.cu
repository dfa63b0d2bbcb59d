// Rotary positions of new tokens' queries and keys, and the write of their
// keys and values into the pages of a KV cache.
//
// Pair i of a head turns by the angle 2 pi pos s_i, with s_i turns per
// position held as a 64-bit binary fraction.  The product pos * s_i modulo
// 2^64 is exact in integers, so a far position loses no more of the angle
// than position 1 does (a float32 product would lose 0.06 rad at 10^6).  Of its
// top 32 bits the nearest quarter turn is taken off as an integer and the rest, at
// most an eighth of a turn, goes to sincospif as a float32, whose rounding is then
// within pi 2^-27 of the angle (pi 2^-25 for a half turn, more than a float32 cosine's
// own).  The rotation is float32 and each output is rounded once.
//
// Bound by memory: every input is read once and every output written once.
// A block takes ROWS token rows, or where they are few a part of their heads.
// Sines and cosines are computed once into shared memory and reused by the
// rows' heads; then each thread walks the vectors of a row and moves each for
// all the rows at once, so that 2 * ROWS loads are in flight and the way from
// the row to its position and page (three dependent loads) is paid once for
// them.
#include <algorithm>

#include "kda_cache.h"
#include "kda_device.cuh"

namespace kda {
namespace {

constexpr int kMaxPairs = 256;  // head_dim <= 512
// Small blocks, so that some load while others wait for positions: 23119 rows
// of 48 heads of 128 bf16 channels take 86 us (6.6 TB/s) with 128 threads, 97 us
// with 256 and 112 us with 512.
constexpr int kThreads = 128;
// Rows from which a block takes four of them.  Measured at four rows and at one
// (40 heads, 128 bf16 / 256 float32 channels): 128 rows 4.0 and 3.3 / 4.9 and 5.5
// us, 256 rows 4.3 and 4.0 / 7.0 and 7.9, 384 rows 4.2 and 4.5 / 7.2 and 10.5,
// 1536 rows 8.4 and 9.9 / 26.6 and 40.2, 23119 rows 86 and 99 us.
constexpr int kManyRows = 320;

// Index of the sequence owning `row`: the number of entries of cu[1..N] that
// are <= row, by a 32-way search of the whole warp (N <= 32: one load).
__device__ __forceinline__ int find_sequence(const int32_t* cu, int N, int row, int lane) {
  int lo = 0, hi = N;
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int64_t p = lo + (int64_t)(lane + 1) * step - 1;
    const bool le = p < hi && __ldg(cu + 1 + p) <= row;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    lo += c * step;
    hi = min(hi, lo + step - 1);
  }
  return lo;
}

// VEC elements as loaded, as floats, and rounded to nearest even for the store.
template <typename T, int VEC>
struct Vec;
template <>
struct Vec<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = __ldcs(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void get(float (&x)[4]) const { x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w; }
  __device__ __forceinline__ static void store(float* p, const float (&x)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};
template <>
struct Vec<__nv_bfloat16, 4> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldcs(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = bf_lo(v.x); x[1] = bf_hi(v.x); x[2] = bf_lo(v.y); x[3] = bf_hi(v.y);
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&x)[4]) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]));
  }
};
template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = bf_lo(v.x); x[1] = bf_hi(v.x); x[2] = bf_lo(v.y); x[3] = bf_hi(v.y);
    x[4] = bf_lo(v.z); x[5] = bf_hi(v.z); x[6] = bf_lo(v.w); x[7] = bf_hi(v.w);
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&x)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]),
                                              pack_bf2(x[6], x[7]));
  }
};

// A thread's place among heads x tasks, moved on by the row's blocks without dividing.
struct Slot {
  int h, t, dh, dt, tasks;
  __device__ __forceinline__ explicit Slot(int tasks_) : tasks(tasks_) {
    const int at = blockIdx.y * kThreads + threadIdx.x, step = gridDim.y * kThreads;
    h = at / tasks;
    t = at - h * tasks;
    dh = step / tasks;
    dt = step - dh * tasks;
  }
  __device__ __forceinline__ void next() {
    h += dh;
    t += dt;
    if (t >= tasks) {
      t -= tasks;
      ++h;
    }
  }
};

template <typename In, typename Out, int VEC, bool INTERLEAVED, int ROWS>
__global__ void __launch_bounds__(kThreads, 6) kda_rope_append_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 s_cs[ROWS][kMaxPairs];
  __shared__ int s_pos[ROWS];           // -1: zero output
  __shared__ int64_t s_k[ROWS], s_v[ROWS];  // element offsets of the row's place in its page, or -1
  const int row0 = blockIdx.x * ROWS;
  pdl_wait();
  pdl_launch_dependents();

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp < ROWS) {
    const int row = row0 + warp;
    int n = row, end = row + 1;
    bool live = row < a.R;
    if (a.cu != nullptr) {
      n = find_sequence(a.cu, a.N, row, lane);
      live = live && n < a.N && row >= __ldg(a.cu + n);
      end = live ? min(__ldg(a.cu + n + 1), a.R) : 0;
    }
    if (lane == 0) {
      const int64_t pos = live ? (int64_t)__ldg(a.lens + n) - end + row : -1;
      int64_t ko = -1, vo = -1;
      if (pos >= 0) {
        const int64_t col = pos / a.page_size;
        if (col < a.table_cols) {
          const int page = __ldg(a.table + (int64_t)n * a.table_rs + col);
          if (page > 0 && page < a.num_pages) {
            const int64_t t = pos - col * a.page_size;
            ko = page * a.kp.page + t * a.kp.token;
            vo = page * a.vp.page + t * a.vp.token;
          }
        }
      }
      s_pos[warp] = pos < 0 ? -1 : (int)pos;
      s_k[warp] = ko;
      s_v[warp] = vo;
    }
  }
  __syncthreads();
  // Tasks of a rotated head: its pair vectors, then its unrotated tail.  The
  // half layout's pair vectors hold VEC elements of either half.  Pair j of
  // task t lies at j * pair_tasks + t, so that neighbouring tasks meet no bank.
  constexpr int PAIRS = INTERLEAVED ? VEC / 2 : VEC;
  const int pair_tasks = a.rot / (2 * PAIRS);
  for (int i = threadIdx.x; i < ROWS * (a.rot / 2); i += blockDim.x) {
    const int r = i / (a.rot / 2), pair = i - r * (a.rot / 2);
    const uint64_t phase = (uint64_t)(uint32_t)max(s_pos[r], 0) * __ldg(a.steps + pair);
    float sn, cs;
    const uint32_t turn = (uint32_t)((phase + 0x80000000u) >> 32), quarter = (turn + 0x20000000u) >> 30;
    sincospif((float)(int32_t)(turn - (quarter << 30)) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31: half turns
    if (quarter & 1) {
      const float x = cs;
      cs = -sn;
      sn = x;
    }
    const float amplitude = quarter & 2 ? -a.amplitude : a.amplitude;
    s_cs[r][(pair % PAIRS) * pair_tasks + pair / PAIRS] = make_float2(cs * amplitude, sn * amplitude);
  }
  __syncthreads();

  Slot s(pair_tasks + (a.D - a.rot) / VEC);
  for (; s.h < a.Hq + a.Hkv; s.next()) {
    const bool is_q = s.h < a.Hq;
    const int h = is_q ? s.h : s.h - a.Hq;
    const In* src = is_q ? static_cast<const In*>(a.q) + h * a.q_hs : static_cast<const In*>(a.k) + h * a.k_hs;
    const int64_t src_rs = is_q ? a.q_rs : a.k_rs;
    const bool turns = s.t < pair_tasks;
    const bool two = turns && !INTERLEAVED;
    const int c = turns ? s.t * VEC : a.rot + (s.t - pair_tasks) * VEC;
    Vec<In, VEC> vx[ROWS], vy[ROWS];
    bool go[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      go[r] = row0 + r < a.R && (is_q || s_k[r] >= 0);
      if (go[r]) {
        const In* p = src + (row0 + r) * src_rs + c;
        vx[r].load(p);
        if (two) vy[r].load(p + a.rot / 2);
      }
    }
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (!go[r]) continue;
      Out* dst = (is_q ? static_cast<Out*>(a.q_out) + (row0 + r) * a.o_rs + h * a.o_hs
                       : static_cast<Out*>(a.kp.data) + s_k[r] + h * a.kp.head) + c;
      float x[VEC], y[VEC];
      vx[r].get(x);
      if (two) {
        vy[r].get(y);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float2 cs = s_cs[r][j * pair_tasks + s.t];
          const float u = x[j], w = y[j];
          x[j] = u * cs.x - w * cs.y;
          y[j] = u * cs.y + w * cs.x;
        }
      } else if (turns) {
#pragma unroll
        for (int j = 0; j < VEC; j += 2) {
          const float2 cs = s_cs[r][j / 2 * pair_tasks + s.t];
          const float u = x[j], w = x[j + 1];
          x[j] = u * cs.x - w * cs.y;
          x[j + 1] = u * cs.y + w * cs.x;
        }
      }
      if (s_pos[r] < 0) {  // padding row or null sequence (queries only)
#pragma unroll
        for (int j = 0; j < VEC; ++j) x[j] = y[j] = 0.f;
      }
      Vec<Out, VEC>::store(dst, x);
      if (two) Vec<Out, VEC>::store(dst + a.rot / 2, y);
    }
  }
  for (Slot s(a.D / VEC); s.h < a.Hkv; s.next()) {
    const int c = s.t * VEC;
    const In* src = static_cast<const In*>(a.v) + s.h * a.v_hs + c;
    Vec<In, VEC> vx[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r)
      if (s_v[r] >= 0) vx[r].load(src + (row0 + r) * a.v_rs);
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
      if (s_v[r] < 0) continue;
      float x[VEC];
      vx[r].get(x);
      Vec<Out, VEC>::store(static_cast<Out*>(a.vp.data) + s_v[r] + s.h * a.vp.head + c, x);
    }
  }
}

template <typename In, typename Out, int VEC, int ROWS>
cudaError_t launch_rope_rows(const RopeArgs& a, cudaStream_t s) {
  auto kernel = a.interleaved ? kda_rope_append_kernel<In, Out, VEC, true, ROWS>
                              : kda_rope_append_kernel<In, Out, VEC, false, ROWS>;
  // Few rows: several blocks share each, down to one vector a thread, until every SM has its six.
  const int64_t blocks = (a.R + (int64_t)ROWS - 1) / ROWS;
  const int pairs = a.interleaved ? a.rot / VEC : a.rot / (2 * VEC);
  const int64_t tasks = (int64_t)(a.Hq + a.Hkv) * (pairs + (a.D - a.rot) / VEC);
  const int64_t parts = std::max<int64_t>(1, std::min<int64_t>((tasks + kThreads - 1) / kThreads, 6 * a.sms / blocks));
  return launch_pdl(kernel, dim3((unsigned)blocks, (unsigned)parts), dim3(kThreads), 0, s, 1, a);
}

template <typename In, typename Out, int VEC>
cudaError_t launch_rope_variant(const RopeArgs& a, cudaStream_t s) {
  return a.R >= kManyRows ? launch_rope_rows<In, Out, VEC, 4>(a, s) : launch_rope_rows<In, Out, VEC, 1>(a, s);
}

}  // namespace

cudaError_t launch_rope_append(const RopeArgs& a, cudaStream_t s) {
  using bf16 = __nv_bfloat16;
  if (a.in_dtype == KDA_DT_BF16 && a.page_dtype == KDA_DT_BF16)
    return a.vec == 8 ? launch_rope_variant<bf16, bf16, 8>(a, s) : launch_rope_variant<bf16, bf16, 4>(a, s);
  if (a.in_dtype == KDA_DT_BF16) return launch_rope_variant<bf16, float, 4>(a, s);
  if (a.page_dtype == KDA_DT_BF16) return launch_rope_variant<float, bf16, 4>(a, s);
  return launch_rope_variant<float, float, 4>(a, s);
}

}  // namespace kda
