// Rotary positions of new tokens' queries and keys, and the write of their
// keys and values into the pages of a KV cache.
//
// Pair i of a head turns by the angle 2 pi pos s_i, with s_i turns per
// position held as a 64-bit binary fraction.  The product pos * s_i modulo
// 2^64 is exact in integers, so a far position loses no more of the angle
// than position 1 does (a float32 product would lose 0.06 rad at 10^6); its
// top 32 bits, taken as a signed fraction of a turn, go to sincospif.  The
// rotation is float32 and each output is rounded once.
//
// Bound by memory: every input is read once and every output written once.
// One CTA per token row: its rot/2 sines and cosines are computed once into
// shared memory and reused by the row's Hq + Hkv heads, then the threads walk
// the row's vectors.
#include "kda_cache.h"
#include "kda_device.cuh"

namespace kda {
namespace {

constexpr int kMaxPairs = 256;  // head_dim <= 512

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

// VEC elements of type T as floats, and back (round to nearest even).
template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&x)[VEC]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 r = __ldcs(reinterpret_cast<const float4*>(p + i));
      x[i] = r.x; x[i + 1] = r.y; x[i + 2] = r.z; x[i + 3] = r.w;
    }
  } else if constexpr (VEC == 8) {
    const uint4 r = __ldcs(reinterpret_cast<const uint4*>(p));
    x[0] = bf_lo(r.x); x[1] = bf_hi(r.x); x[2] = bf_lo(r.y); x[3] = bf_hi(r.y);
    x[4] = bf_lo(r.z); x[5] = bf_hi(r.z); x[6] = bf_lo(r.w); x[7] = bf_hi(r.w);
  } else {
    const uint2 r = __ldcs(reinterpret_cast<const uint2*>(p));
    x[0] = bf_lo(r.x); x[1] = bf_hi(r.x); x[2] = bf_lo(r.y); x[3] = bf_hi(r.y);
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&x)[VEC]) {
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
  } else if constexpr (VEC == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]),
                                              pack_bf2(x[6], x[7]));
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]));
  }
}

template <typename In, typename Out, int VEC, bool INTERLEAVED>
__global__ void __launch_bounds__(256) kda_rope_append_kernel(const RopeArgs a) {
  __shared__ float2 s_cs[kMaxPairs];
  __shared__ int s_pos;
  __shared__ int64_t s_k, s_v;
  __shared__ int s_write;
  const int row = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();

  if (threadIdx.x < 32) {
    int n = row, end = row + 1;
    bool live = true;
    if (a.cu != nullptr) {
      n = find_sequence(a.cu, a.N, row, threadIdx.x);
      live = n < a.N && row >= __ldg(a.cu + n);
      end = live ? min(__ldg(a.cu + n + 1), a.R) : 0;
    }
    if (threadIdx.x == 0) {
      int64_t pos = live ? (int64_t)__ldg(a.lens + n) - end + row : -1;
      int write = 0;
      if (pos >= 0) {
        const int64_t col = pos / a.page_size;
        if (col < a.table_cols) {
          const int page = __ldg(a.table + (int64_t)n * a.table_rs + col);
          if (page > 0 && page < a.num_pages) {
            const int64_t t = pos - col * a.page_size;
            s_k = page * a.kp.page + t * a.kp.token;
            s_v = page * a.vp.page + t * a.vp.token;
            write = 1;
          }
        }
      }
      s_pos = pos < 0 ? -1 : (int)pos;
      s_write = write;
    }
  }
  __syncthreads();
  const int pos = s_pos;
  const bool write = s_write != 0;
  for (int i = threadIdx.x; i < a.rot / 2; i += blockDim.x) {
    const uint64_t phase = (uint64_t)(uint32_t)max(pos, 0) * __ldg(a.steps + i);
    float sn, cs;
    sincospif((float)(int32_t)(phase >> 32) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31: half turns
    s_cs[i] = make_float2(cs * a.amplitude, sn * a.amplitude);
  }
  __syncthreads();

  // Tasks of a rotated head: its pair vectors, then its unrotated tail.  The
  // half layout's pair vectors hold VEC elements of either half.
  const int pair_tasks = INTERLEAVED ? a.rot / VEC : a.rot / (2 * VEC);
  const int tasks = pair_tasks + (a.D - a.rot) / VEC;
  const int rotated = a.Hq + a.Hkv;
  for (int i = threadIdx.x; i < rotated * tasks; i += blockDim.x) {
    const int h = i / tasks, t = i - h * tasks;
    const bool is_q = h < a.Hq;
    if (!is_q && !write) break;  // only keys follow
    const In* src = is_q ? static_cast<const In*>(a.q) + row * a.q_rs + h * a.q_hs
                         : static_cast<const In*>(a.k) + row * a.k_rs + (h - a.Hq) * a.k_hs;
    Out* dst = is_q ? static_cast<Out*>(a.q_out) + row * a.o_rs + h * a.o_hs
                    : static_cast<Out*>(a.kp.data) + s_k + (h - a.Hq) * a.kp.head;
    if (pos < 0) {  // padding row or null sequence (queries only)
      float z[VEC] = {};
      if (t < pair_tasks) {
        store_vec<Out, VEC>(dst + t * VEC, z);
        if (!INTERLEAVED) store_vec<Out, VEC>(dst + a.rot / 2 + t * VEC, z);
      } else {
        store_vec<Out, VEC>(dst + a.rot + (t - pair_tasks) * VEC, z);
      }
      continue;
    }
    float x[VEC];
    if (t >= pair_tasks) {
      const int c = a.rot + (t - pair_tasks) * VEC;
      load_vec<In, VEC>(src + c, x);
      store_vec<Out, VEC>(dst + c, x);
    } else if (INTERLEAVED) {
      load_vec<In, VEC>(src + t * VEC, x);
#pragma unroll
      for (int j = 0; j < VEC; j += 2) {
        const float2 cs = s_cs[(t * VEC + j) / 2];
        const float p = x[j], r = x[j + 1];
        x[j] = p * cs.x - r * cs.y;
        x[j + 1] = p * cs.y + r * cs.x;
      }
      store_vec<Out, VEC>(dst + t * VEC, x);
    } else {
      float y[VEC];
      load_vec<In, VEC>(src + t * VEC, x);
      load_vec<In, VEC>(src + a.rot / 2 + t * VEC, y);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float2 cs = s_cs[t * VEC + j];
        const float p = x[j], r = y[j];
        x[j] = p * cs.x - r * cs.y;
        y[j] = p * cs.y + r * cs.x;
      }
      store_vec<Out, VEC>(dst + t * VEC, x);
      store_vec<Out, VEC>(dst + a.rot / 2 + t * VEC, y);
    }
  }
  if (!write) return;
  const int vt = a.D / VEC;
  for (int i = threadIdx.x; i < a.Hkv * vt; i += blockDim.x) {
    const int h = i / vt, c = (i - h * vt) * VEC;
    float x[VEC];
    load_vec<In, VEC>(static_cast<const In*>(a.v) + row * a.v_rs + h * a.v_hs + c, x);
    store_vec<Out, VEC>(static_cast<Out*>(a.vp.data) + s_v + h * a.vp.head + c, x);
  }
}

template <typename In, typename Out, int VEC>
cudaError_t launch_rope_variant(const RopeArgs& a, cudaStream_t s) {
  auto kernel = a.interleaved ? kda_rope_append_kernel<In, Out, VEC, true> : kda_rope_append_kernel<In, Out, VEC, false>;
  return launch_pdl(kernel, dim3((unsigned)a.R), dim3(256), 0, s, 1, a);
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
