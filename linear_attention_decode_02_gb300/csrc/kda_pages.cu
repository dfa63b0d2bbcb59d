// Pages for the sequences of a step, from their lengths: page tables grown from
// and shrunk into a ring of free pages, and the slot of every new token row.
//
// With held_n = ceil(old_n / page_size) and want_n = ceil(new_n / page_size) the
// pages taken are sums over the sequences before n, so three prefix sums (pages
// asked for, to decide who is served; then pages taken, rows and pages given
// back) say where everything goes, and all writes are independent.  Free pages
// are taken from the ring's head and given back behind its tail: no place of the
// ring is both read and written in a call.
//
// Bound by latency: the widest call moves a few MB.  So it is one launch of one
// thread-block cluster: every CTA makes the sums for itself in shared memory,
// only the count of the pages given back, which has to read the table, is shared
// out and exchanged over distributed shared memory, and one cluster barrier
// separates the last read of the lengths and the ring's state from the first
// write, so both may be updated in place.  Small calls are one CTA.
//
// Measured, one call after another: 8 sequences of a step 5.6 us (7.1 with the host's
// part, through the binding); 512 sequences, a few ended, 47,515 rows 12.4 us; 48
// prompts of up to 16,384 tokens, 486,830 rows, 12.1 us.  With 8 CTAs 19.8 and 19.5
// us, with 512 threads a CTA 17.1 and 13.1; rows taken 4 at a time 28.8 us for the
// prompts (8 CTAs), 16 at a time 13.0, 32 at a time 12.1.
#include <cooperative_groups.h>

#include <algorithm>

#include "kda_attend.cuh"
#include "kda_cache.h"
#include "kda_device.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kMostThreads = 1024;
constexpr int kCluster = 16, kPortableCluster = 8;  // CTAs; more than 8 a device need not grant

__device__ __forceinline__ int ceil_div(int a, int b) { return a / b + (a % b != 0); }

// Exclusive prefix sums of V values a thread over the block; `total` their sums.
// `scratch` holds [warps][V] and may be used again after the next __syncthreads.
template <int V>
__device__ __forceinline__ void block_scan(int64_t (&x)[V], int64_t (&total)[V], int64_t (*scratch)[V]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t own[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    own[v] = x[v];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, x[v], o);
      if (lane >= o) x[v] += up;
    }
    if (lane == 31) scratch[warp][v] = x[v];
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int64_t w = lane < warps ? scratch[lane][v] : 0;
    int64_t before = lane < warp ? w : 0, all = w;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      before += __shfl_xor_sync(0xffffffffu, before, o);
      all += __shfl_xor_sync(0xffffffffu, all, o);
    }
    x[v] += before - own[v];
    total[v] = all;
  }
}

// The last n of [0, N) with first[n] <= i, first rising and first[0] = 0.
__device__ __forceinline__ int owner_of(const int* first, int N, int i) {
  int lo = 0, hi = N;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kMostThreads) kda_page_assign_kernel(const __grid_constant__ PagesArgs a) {
  extern __shared__ int smem[];
  __shared__ int64_t s_asked[kMostThreads / 32][1], s_sums[kMostThreads / 32][3];
  const int N = a.N, page_size = a.page_size, threads = blockDim.x, tid = threadIdx.x, lane = tid & 31;
  int* s_old = smem;            // [N] length before
  int* s_new = s_old + N;       // [N] length wanted, then the one given; -1: more than the table holds
  int* s_take = s_new + N;      // [N] first page taken, counted over the call
  int* s_rel = s_take + N;      // [N] pages given back, then the first of them
  int* s_cu = s_rel + N;        // [N + 1] first row
  const cg::cluster_group cluster = cg::this_cluster();
  const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  if (ctas > 1) cluster.sync();  // every CTA runs, so its shared memory can be written
  pdl_wait();
  pdl_launch_dependents();

  const uint32_t C = (uint32_t)a.capacity;
  int head = a.state[0], count = a.state[1];
  if (head < 0 || (uint32_t)head >= C || count < 0) head = count = 0;
  count = min(count, (int)C);
  const int cap = (int)min((int64_t)a.table_cols * page_size, (int64_t)INT32_MAX);
  const int per = (N + threads - 1) / threads;
  const int n0 = min(N, tid * per), n1 = min(N, n0 + per);
  for (int n = n0; n < n1; ++n) {
    s_old[n] = min(max(a.old_lens[n], 0), cap);
    const int to = max(a.new_lens[n], 0);
    s_new[n] = to > cap ? -1 : to;
  }
  __syncthreads();

  // Pages given back, a warp a sequence: those of the table's columns past the
  // new length that are real and not of the shared beginning.
  const int warps = threads >> 5;
  const auto released = [&](int n, int& lo, int& hi) {
    const int to = s_new[n];
    hi = ceil_div(s_old[n], page_size);
    lo = to < 0 ? hi : ceil_div(to, page_size);
    if (lo < hi && a.shared_lens != nullptr) lo = max(lo, max(__ldg(a.shared_lens + n), 0) / page_size);
  };
  constexpr int AHEAD = 8;
  for (int n = rank * warps + (tid >> 5); n < N; n += ctas * warps) {
    int lo, hi, found = 0;
    released(n, lo, hi);
    for (int col = lo; col < hi; col += 32 * AHEAD) {
      int page[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) page[j] = hi - col > j * 32 + lane ? a.table[n * a.table_rs + col + j * 32 + lane] : 0;
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) found += page[j] > 0 && (uint32_t)page[j] <= C;
    }
    if (lo < hi) found = __reduce_add_sync(0xffffffffu, found);
    if (lane < ctas) *cluster.map_shared_rank(s_rel + n, lane) = found;
  }
  if (ctas > 1) cluster.sync();  // all counts are here, and every CTA has read the lengths and the state
  else __syncthreads();

  // Who is served: those that ask for no page, and those whose pages, counted
  // with all asked for before them, are there.
  int64_t asked[1] = {0}, all_asked[1];
  for (int n = n0; n < n1; ++n)
    if (s_new[n] >= 0) asked[0] += max(0, ceil_div(s_new[n], page_size) - ceil_div(s_old[n], page_size));
  block_scan<1>(asked, all_asked, s_asked);
  int64_t sums[3] = {0, 0, 0}, all[3];  // pages taken, rows, pages given back
  for (int n = n0; n < n1; ++n) {
    const int old = s_old[n];
    int to = s_new[n], take = 0;
    if (to >= 0) take = max(0, ceil_div(to, page_size) - ceil_div(old, page_size));
    asked[0] += take;
    if (to < 0 || (take > 0 && asked[0] > count)) {
      to = old;
      take = 0;
    }
    s_new[n] = to;
    s_take[n] = take;
    sums[0] += take;
    sums[1] += max(0, to - old);
    sums[2] += s_rel[n];
  }
  block_scan<3>(sums, all, s_sums);
  for (int n = n0; n < n1; ++n) {
    const int take = s_take[n], rel = s_rel[n];
    s_take[n] = (int)sums[0];
    s_rel[n] = (int)min(sums[2], (int64_t)INT32_MAX);
    s_cu[n] = (int)min(sums[1], (int64_t)INT32_MAX);
    sums[0] += take;
    sums[1] += max(0, s_new[n] - s_old[n]);
    sums[2] += rel;
  }
  if (tid == 0) s_cu[N] = (int)min(all[1], (int64_t)INT32_MAX);
  __syncthreads();

  const int takes = (int)all[0], rows = s_cu[N];
  const auto ring = [&](uint32_t i) {  // place i <= C behind the head
    i += (uint32_t)head;
    return i >= C ? i - C : i;
  };
  if (rank == 0) {
    for (int n = tid; n < N; n += threads) {
      a.lens_out[n] = s_new[n];
      a.cu[n] = s_cu[n];
    }
    if (tid == 0) {
      a.cu[N] = rows;
      a.state_out[0] = (int)ring((uint32_t)takes);
      a.state_out[1] = (int)(count - takes + min(all[2], (int64_t)C - count));
    }
  }
  for (int64_t i = (int64_t)rank * threads + tid; i < takes; i += (int64_t)ctas * threads) {
    const int n = owner_of(s_take, N, (int)i);
    a.table[n * a.table_rs + ceil_div(s_old[n], page_size) + ((int)i - s_take[n])] = a.ring[ring((uint32_t)i)];
  }
  for (int n = rank * warps + (tid >> 5); n < N; n += ctas * warps) {
    int lo, hi;
    released(n, lo, hi);
    int64_t at = s_rel[n];
    for (int col = lo; col < hi; col += 32 * AHEAD) {
      int page[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) page[j] = hi - col > j * 32 + lane ? a.table[n * a.table_rs + col + j * 32 + lane] : 0;
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        const bool real = page[j] > 0 && (uint32_t)page[j] <= C;
        const uint32_t mask = __ballot_sync(0xffffffffu, real);
        const int64_t k = at + __popc(mask & ((1u << lane) - 1));
        if (real && k < (int64_t)C - count) a.ring[ring((uint32_t)(count + k))] = page[j];
        at += __popc(mask);
      }
    }
  }

  // Slots.  A thread takes a.run rows, found by one search, one look-up a page.
  const bool wide = reinterpret_cast<uintptr_t>(a.slots) % 16 == 0;
  for (int64_t r0 = (int64_t)a.run * ((int64_t)rank * threads + tid); r0 < a.R; r0 += (int64_t)a.run * ctas * threads) {
    int n = 0, stop = 0, col = 0, off = 0, held = 0, page = 0;
    bool enter = true;  // a sequence's first row here
    if (r0 < rows) {
      n = owner_of(s_cu, N, (int)r0);
      stop = s_cu[n + 1];
    }
    for (int64_t r = r0; r < min(r0 + a.run, a.R); r += 4) {
      int slot[4] = {-1, -1, -1, -1};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (r + j >= rows) break;
        if (r + j >= stop) {
          do stop = s_cu[++n + 1];
          while (r + j >= stop);
          enter = true;
        }
        bool turn = enter;
        if (enter) {
          const int pos = s_old[n] + ((int)r + j - s_cu[n]);
          col = pos / page_size;
          off = pos - col * page_size;
          held = ceil_div(s_old[n], page_size);
          enter = false;
        } else if (++off == page_size) {
          ++col;
          off = 0;
          turn = true;
        }
        if (turn)
          page = col < held ? a.table[n * a.table_rs + col] : a.ring[ring((uint32_t)(s_take[n] + (col - held)))];
        if (page > 0 && (uint32_t)page <= C) slot[j] = page * page_size + off;
      }
      if (wide && r + 4 <= a.R) {
        *reinterpret_cast<int4*>(a.slots + r) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (r + j < a.R) a.slots[r + j] = slot[j];
      }
    }
  }
}

}  // namespace

cudaError_t launch_page_assign(const PagesArgs& given, cudaStream_t s) {
  PagesArgs a = given;
  const int bytes = (5 * a.N + 1) * (int)sizeof(int), most_bytes = (5 * kPageSequences + 1) * (int)sizeof(int);
  static std::atomic<bool> set[64];
  static std::atomic<int> granted[64];  // CTAs of a cluster, 0: not asked yet
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = allow_shared(kda_page_assign_kernel, most_bytes, set);
  if (e != cudaSuccess) return e;
  int cluster = a.R + 16LL * a.N > 2048 ? granted[dev].load(std::memory_order_acquire) : 1;
  if (cluster == 0) {
    cluster = kPortableCluster;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCluster);
    cfg.blockDim = dim3(kMostThreads);
    cfg.dynamicSmemBytes = most_bytes;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = kCluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    if (cudaFuncSetAttribute(kda_page_assign_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
        cudaOccupancyMaxActiveClusters(&clusters, kda_page_assign_kernel, &cfg) == cudaSuccess && clusters > 0)
      cluster = kCluster;
    else
      cudaGetLastError();  // a refusal here is no error of the call
    granted[dev].store(cluster, std::memory_order_release);
  }
  const int threads = cluster > 1 ? kMostThreads : 256;
  const int64_t each = (a.R + 4LL * cluster * threads - 1) / (4LL * cluster * threads);
  a.run = 4 * (int)std::max<int64_t>(1, std::min<int64_t>(each, 8));
  return launch_pdl(kda_page_assign_kernel, dim3(cluster), dim3(threads), bytes, s, cluster, a);
}

}  // namespace kda
