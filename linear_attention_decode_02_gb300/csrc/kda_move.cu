// Copies of whole slots within pools: forks, compaction, clearing, and the
// in-place reorder of the beams of each request.
//
// Row n of the call moves, for every j at once, slot src[n, parent[n, j]] to
// slot dst[n, j]; within a row a slot may be the source of several moves and
// the destination of another.  Each thread owns a byte column (the same bytes
// of every slot of its row) and reads all its row's sources there before it
// writes any destination, so the in-place permutation needs neither a staging
// copy nor a barrier.
//
// Bound by memory.  A block covers one row, one pool and kThreads * U vectors
// of the slot; a thread keeps K * U independent 16-byte loads in flight.  64
// beams' float32 states of 32 heads and conv caches in four layers, 0.85 GB read
// and written, take 125 us, the copy bandwidth; 256 forks of 12-head bf16 states
// 32 us (97 %), 128 states of 32 beams a row 138 us for 0.86 GB (92 %).
#include "kda_cache.h"
#include "kda_device.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;

// Vectors of the slot per thread: 8 loads in flight, fewer where K alone gives them.
__host__ __device__ constexpr int unroll(int KMAX) { return KMAX >= 8 ? 1 : 8 / KMAX; }

template <typename V, int KMAX>
__global__ void __launch_bounds__(kThreads) kda_pool_move_kernel(const __grid_constant__ MoveArgs a) {
  constexpr int U = unroll(KMAX);
  __shared__ int s_src[KMAX], s_dst[KMAX];  // dst 0: nothing to do; src 0: clear
  int64_t block = blockIdx.x;
  int p = 0;
  while (p + 1 < a.pools && block >= a.pool[p + 1].first) ++p;
  block -= a.pool[p].first;
  const int64_t vectors = a.pool[p].bytes / (int64_t)sizeof(V);
  const int64_t chunks = (vectors + kThreads * U - 1) / (kThreads * U);
  const int64_t n = block / chunks;
  const int64_t v0 = (block - n * chunks) * (kThreads * U) + threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();

  if (threadIdx.x < KMAX) {
    const int j = threadIdx.x;
    int s = 0, d = 0;
    if (j < a.K) {
      d = __ldg(a.dst + n * a.dst_rs + j);
      const int par = a.parents != nullptr ? __ldg(a.parents + n * a.par_rs + j) : j;
      if (d <= 0 || d >= a.num_slots || par < 0 || par >= a.K) {
        d = 0;
      } else {
        s = __ldg(a.src + n * a.src_rs + par);
        if (s <= 0 || s >= a.num_slots) s = 0;
        if (s == d) d = 0;
      }
    }
    s_src[j] = s;
    s_dst[j] = d;
  }
  __syncthreads();
  char* base = a.pool[p].base;
  const int64_t stride = a.pool[p].stride;
  V x[KMAX][U];
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    const int s = s_src[j];
    const bool load = s_dst[j] != 0 && s != 0;
    const V* src = reinterpret_cast<const V*>(base + s * stride);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = v0 + u * kThreads;
      x[j][u] = V{};
      if (load && v < vectors) x[j][u] = __ldcs(src + v);
    }
  }
#pragma unroll
  for (int j = 0; j < KMAX; ++j) {
    const int d = s_dst[j];
    if (d == 0) continue;
    V* dst = reinterpret_cast<V*>(base + d * stride);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t v = v0 + u * kThreads;
      if (v < vectors) __stcs(dst + v, x[j][u]);
    }
  }
}

int beams_class(int K) {
  int k = 1;
  while (k < K) k *= 2;
  return k;
}

template <typename V>
cudaError_t launch_move(const MoveArgs& a, int64_t blocks, cudaStream_t s) {
  const dim3 grid((unsigned)blocks), threads(kThreads);
  switch (beams_class(a.K)) {
    case 1: return launch_pdl(kda_pool_move_kernel<V, 1>, grid, threads, 0, s, 1, a);
    case 2: return launch_pdl(kda_pool_move_kernel<V, 2>, grid, threads, 0, s, 1, a);
    case 4: return launch_pdl(kda_pool_move_kernel<V, 4>, grid, threads, 0, s, 1, a);
    case 8: return launch_pdl(kda_pool_move_kernel<V, 8>, grid, threads, 0, s, 1, a);
    case 16: return launch_pdl(kda_pool_move_kernel<V, 16>, grid, threads, 0, s, 1, a);
    default: return launch_pdl(kda_pool_move_kernel<V, 32>, grid, threads, 0, s, 1, a);
  }
}

}  // namespace

bool plan_pool_move(MoveArgs& a, int64_t* blocks) {
  const int64_t per = (int64_t)kThreads * unroll(beams_class(a.K));
  int64_t total = 0;
  for (int i = 0; i < a.pools; ++i) {
    const int64_t chunks = (a.pool[i].bytes / a.align + per - 1) / per;
    a.pool[i].first = total;
    if (chunks > INT32_MAX / (int64_t)a.N) return false;
    total += chunks * a.N;
    if (total >= INT32_MAX) return false;
  }
  *blocks = total;
  return true;
}

cudaError_t launch_pool_move(const MoveArgs& a, int64_t blocks, cudaStream_t s) {
  if (a.align == 16) return launch_move<uint4>(a, blocks, s);
  if (a.align == 4) return launch_move<uint32_t>(a, blocks, s);
  return launch_move<unsigned short>(a, blocks, s);
}

}  // namespace kda
