// Pages for the sequences of a step, from their lengths: page tables grown from
// and shrunk into a ring of free pages, and the slot of every new token row.
//
// With held_n = ceil(old_n / page_size) and want_n = ceil(new_n / page_size) the
// pages taken are sums over the sequences before n, so prefix sums (pages taken,
// rows, pieces, pages given back) say where everything goes, and all writes are
// independent.  They are made as if all were served; where that takes more pages than
// are free, the first of them says who is, and they are made again.  Free pages are
// taken from the ring's head and given back behind its tail: no place of the ring
// is both read and written in a call.
//
// Slots come in pieces, the new rows of a sequence that lie on one page: a lane
// searches a piece's sequence and loads its page once, then lanes write its rows.
//
// Bound by latency: the widest call moves a few MB.  So it is one launch of one
// thread-block cluster: every CTA makes the sums for itself in shared memory,
// only the count of the pages given back, which has to read the table, is shared
// out and exchanged over distributed shared memory, and one cluster barrier
// separates the last read of the lengths and the ring's state from the first
// write, so both may be updated in place.  Small calls are one CTA.  Every
// instruction runs a few times at most, so that fewer of them count: sums in 32 bits
// that saturate, by the warps that have sequences, and division by a factor.
//
// Measured in a graph, one call after another: 8 sequences of a step 3.8 us (6.6 to 7.1
// with the host's part, through the binding; 5.7 with 64-bit sums and divisions); 512
// sequences, a few ended, 47,515 rows 8.8 us (12.2); 48 prompts of up to 16,384
// tokens, 486,830 rows, 8.4 us (12.0): half of that is writing 2 MB from 16 SMs, which
// took as long with 15 pieces a warp, all warps at work, and longer with four or
// eight rows a lane that searches for itself (10.9 us; 512 sequences 12.3).  With 8 CTAs
// instead of 16, before these steps, 19.8 and 19.5 us, with 512 threads a CTA 17.1 and 13.1.
#include <cooperative_groups.h>

#include <algorithm>

#include "kda_attend.cuh"
#include "kda_cache.h"
#include "kda_device.cuh"

namespace cg = cooperative_groups;

namespace kda {
namespace {

constexpr int kMostThreads = 1024;
constexpr int kPiece = 256;  // most rows of a piece
constexpr int kCluster = 16, kPortableCluster = 8;  // CTAs; more than 8 a device need not grant

// a + b, or the largest int32 where that is less; so sums of what is not negative saturate in any order.
__device__ __forceinline__ int saturated(int a, int b) {
  return (int)min((uint32_t)a + (uint32_t)b, (uint32_t)INT32_MAX);
}

// Exclusive saturating prefix sums of V values a thread over the first `warps`
// warps of the block; `total` their sums.  The other warps only pass the barrier.
template <int V>
__device__ __forceinline__ void block_scan(int (&x)[V], int (&total)[V], int (*scratch)[V], int warps) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (warp < warps) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, x[v], o);
        if (lane >= o) x[v] = saturated(x[v], up);
      }
      if (lane == 31) scratch[warp][v] = x[v];
      const int before = __shfl_up_sync(0xffffffffu, x[v], 1);
      x[v] = lane > 0 ? before : 0;
    }
  }
  __syncthreads();
  if (warp < warps) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      int w = lane < warps ? scratch[lane][v] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w = saturated(w, up);
      }
      total[v] = __shfl_sync(0xffffffffu, w, 31);
      const int before = __shfl_sync(0xffffffffu, w, max(warp, 1) - 1);
      if (warp > 0) x[v] = saturated(x[v], before);
    }
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
  __shared__ int s_sums[kMostThreads / 32][4], s_takes, s_given, s_pieces;
  const int N = a.N, page_size = a.page_size, threads = blockDim.x, tid = threadIdx.x, lane = tid & 31;
  int* s_old = smem;            // [N] length before
  int* s_new = s_old + N;       // [N] length wanted, then the one given; -1: more than the table holds
  int* s_take = s_new + N;      // [N] first page taken, counted over the call
  int* s_rel = s_take + N;      // [N] pages given back, then the first of them
  int* s_piece = s_rel + N;     // [N] first piece
  int* s_cu = s_piece + N;      // [N + 1] first row
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
  const auto page_of = [&](int place) { return (int)(((uint64_t)(uint32_t)place * a.page_factor) >> a.page_shift); };
  const auto pages_of = [&](int places) { return places > 0 ? page_of(places - 1) + 1 : 0; };
  const auto old_of = [&](int n) { return min(max(a.old_lens[n], 0), cap); };
  const auto new_of = [&](int n) {  // -1: more than the table holds
    const int to = max(a.new_lens[n], 0);
    return to > cap ? -1 : to;
  };
  for (int n = n0; n < n1; ++n) {
    s_old[n] = old_of(n);
    s_new[n] = new_of(n);
  }

  // Pages given back, a warp a sequence: those of the table's columns past the
  // new length that are real and not of the shared beginning.
  const int warps = threads >> 5;
  const auto released = [&](int n, int old, int to, int& lo, int& hi) {
    hi = pages_of(old);
    lo = to < 0 ? hi : pages_of(to);
    if (lo < hi && a.shared_lens != nullptr) lo = max(lo, page_of(max(__ldg(a.shared_lens + n), 0)));
  };
  constexpr int AHEAD = 8;
  for (int n = rank * warps + (tid >> 5); n < N; n += ctas * warps) {
    int lo, hi, found = 0;
    released(n, old_of(n), new_of(n), lo, hi);  // not those in shared memory, which would be waited for
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

  // A sequence's new rows come in pieces: what lies on one page, or, of pages of more than kPiece, that many rows, which
  // lie on two at most.
  const int piece = min(page_size, kPiece);
  const auto piece0 = [&](int old) { return page_size <= kPiece ? page_of(old) * page_size : old; };  // where the first would begin
  // Who is served: those that ask for no page, and those whose pages, counted
  // with all asked for before them, are there.  Mostly that is everybody, and the
  // sums for everybody are the ones wanted; else they are made once more.
  const int scanning = N == 0 ? 0 : ((N + per - 1) / per + 31) / 32;  // warps that have sequences
#pragma unroll 1
  for (bool scarce = false;; scarce = true) {
    int sums[4] = {0, 0, 0, 0}, all[4] = {0, 0, 0, 0};  // pages taken, rows, pieces, pages given back
    for (int n = n0; n < n1; ++n) {
      const int old = s_old[n];
      int to = s_new[n], take = to < 0 ? 0 : max(0, pages_of(to) - pages_of(old));
      if (to < 0 || (scarce && take > 0 && saturated(s_take[n], take) > count)) {
        s_new[n] = to = old;
        take = 0;
      }
      const int last = to - 1 - piece0(old);  // from where the first piece would begin to the last row
      const int pieces = to <= old ? 0 : (page_size <= kPiece ? page_of(last) : last / kPiece) + 1;
      s_take[n] = take;
      s_piece[n] = pieces;
      sums[0] = saturated(sums[0], take);
      sums[1] = saturated(sums[1], max(0, to - old));
      sums[2] = saturated(sums[2], pieces);
      if (!scarce) sums[3] = saturated(sums[3], s_rel[n]);  // who grows gives none back
    }
    block_scan<4>(sums, all, s_sums, scanning);
    for (int n = n0; n < n1; ++n) {
      const int take = s_take[n], pieces = s_piece[n], rel = s_rel[n];
      s_take[n] = sums[0];
      s_cu[n] = sums[1];
      s_piece[n] = sums[2];
      sums[0] = saturated(sums[0], take);
      sums[1] = saturated(sums[1], max(0, s_new[n] - s_old[n]));
      sums[2] = saturated(sums[2], pieces);
      if (!scarce) {
        s_rel[n] = sums[3];
        sums[3] = saturated(sums[3], rel);
      }
    }
    if (tid == 0) {
      s_takes = all[0];
      s_cu[N] = all[1];
      s_pieces = all[2];
      if (!scarce) s_given = all[3];
    }
    __syncthreads();
    if (scarce || s_takes <= count) break;
  }

  const int takes = s_takes, rows = s_cu[N];
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
      a.state_out[1] = count - takes + min(s_given, (int)C - count);
    }
  }
  for (int64_t i = (int64_t)rank * threads + tid; i < takes; i += (int64_t)ctas * threads) {
    const int n = owner_of(s_take, N, (int)i);
    a.table[n * a.table_rs + pages_of(s_old[n]) + ((int)i - s_take[n])] = a.ring[ring((uint32_t)i)];
  }
  for (int n = rank * warps + (tid >> 5); n < N; n += ctas * warps) {
    int lo, hi;
    released(n, s_old[n], s_new[n], lo, hi);
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

  // Slots, 32 pieces a warp: a lane finds one, then all write each, or, where all are short, every lane its own.
  const auto page_at = [&](int n, int held, int col) {
    return col < held ? a.table[n * a.table_rs + col] : a.ring[ring((uint32_t)(s_take[n] + (col - held)))];
  };
  const auto slot_of = [&](int page, int off) { return page > 0 && (uint32_t)page <= C ? page * page_size + off : -1; };
  const int pieces = s_pieces;
  // Lanes that write a piece together.
  const int share = piece <= 8 ? 8 : (piece <= 16 ? 16 : 32), x0 = lane & (share - 1);
  for (int64_t i0 = 32LL * ((tid >> 5) * ctas + rank); i0 < pieces; i0 += 32LL * warps * ctas) {
    int row = 0, len = 0, left = 0;  // the piece's first row, its rows, those on its first page
    int first = -1, second = -1;     // slots of its first place and of the next page's
    if (i0 + lane < pieces) {
      const int n = owner_of(s_piece, N, (int)i0 + lane), old = s_old[n], held = pages_of(old);
      const int64_t start = piece0(old) + (int64_t)((int)i0 + lane - s_piece[n]) * piece;
      const int from = (int)max(start, (int64_t)old), to = (int)min(start + piece, (int64_t)s_new[n]);
      const int col = page_of(from), off = from - col * page_size;
      row = saturated(s_cu[n], from - old);
      len = (int)min((int64_t)(to - from), a.R - row);
      left = page_size - off;
      if (len > 0) first = slot_of(page_at(n, held, col), off);
      if (left < len) second = slot_of(page_at(n, held, col + 1), 0);
    }
    if (__shfl_sync(0xffffffffu, row, 0) >= a.R) break;  // nor are later ones wanted
    if (__all_sync(0xffffffffu, len <= 4 && len <= left)) {
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (x < len) a.slots[row + x] = first < 0 ? -1 : first + x;
    } else if (page_size <= kPiece) {  // one page each
#pragma unroll 4
      for (int k = 0; k < 32; k += 32 / share) {
        const int from = k + lane / share;
        const int n = __shfl_sync(0xffffffffu, len, from), at = __shfl_sync(0xffffffffu, first, from);
        int32_t* const to = a.slots + __shfl_sync(0xffffffffu, row, from);
        for (int x = x0; x < n; x += share) to[x] = at < 0 ? -1 : at + x;
      }
    } else {
#pragma unroll 1
      for (int k = 0; k < 32; ++k) {
        const int n = __shfl_sync(0xffffffffu, len, k), here = __shfl_sync(0xffffffffu, left, k);
        const int at = __shfl_sync(0xffffffffu, first, k), after = __shfl_sync(0xffffffffu, second, k);
        int32_t* const to = a.slots + __shfl_sync(0xffffffffu, row, k);
        for (int x = lane; x < n; x += 32) {
          const int page = x < here ? at : after;
          to[x] = page < 0 ? -1 : page + (x < here ? x : x - here);
        }
      }
    }
  }
  for (int64_t r = rows + (int64_t)rank * threads + tid; r < a.R; r += (int64_t)ctas * threads) a.slots[r] = -1;
}

}  // namespace

cudaError_t launch_page_assign(const PagesArgs& given, cudaStream_t s) {
  PagesArgs a = given;
  // Division by an invariant (Granlund and Montgomery, 1994): with 2^(k-1) < d <= 2^k and f = floor(2^(31+k) / d) + 1,
  // f d - 2^(31+k) is 1 to d, at most 2^k, so that floor(n f / 2^(31+k)) = floor(n / d) for n < 2^31.
  int k = 0;
  while ((int64_t{1} << k) < a.page_size) ++k;
  a.page_shift = 31 + k;
  a.page_factor = (uint32_t)((uint64_t{1} << a.page_shift) / (uint32_t)a.page_size + 1);
  const int bytes = (6 * a.N + 1) * (int)sizeof(int), most_bytes = (6 * kPageSequences + 1) * (int)sizeof(int);
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
  return launch_pdl(kda_page_assign_kernel, dim3(cluster), dim3(threads), bytes, s, cluster, a);
}

}  // namespace kda
