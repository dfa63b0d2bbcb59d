// What the matrix-instruction attention kernels share: the end of a unit, with
// outputs and row statistics in the layout of a 16 x 8 accumulator.
#pragma once

#include "kda_attend.cuh"

namespace kda {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Joins the warps of a block at a unit's end in its piece and writes the
// result, or the piece's partial.  Lane (g, t4) holds channels 8 i + 2 t4 and + 1
// of rows g (o[i][0], o[i][1]) and g + 8 (o[i][2], o[i][3]): two heads with HG =
// 16, two parts of one head to be added with HG = 8.  m and l are the warp's
// row maxima and this lane's sums.  shared_o: (WARPS - 1) * 8 * D floats; stats:
// [WARPS][HG] maxima and sums, other ones than the last unit's.
template <int D, int HG, int WARPS, int RS>
__device__ __forceinline__ void finish_unit(const AttendArgs& a, const Walk& walk, const Place& place, const Workspace& ws,
                                            float* shared_o, float (&s_m)[WARPS][HG], float (&s_l)[WARPS][HG],
                                            float (&o)[D / 8][4], float (&m)[RS], float (&l)[RS], int groups, int warp,
                                            int g, int t4, int c) {
  constexpr bool PAIR = HG == 8;
  constexpr int NT = D / 8;
  static_assert(RS == HG / 8 && NT % WARPS == 0, "bad shape");
  const int G = a.Hq / a.Hkv, hk = walk.group / groups, g0 = (walk.group - hk * groups) * HG, heads = min(HG, G - g0);
#pragma unroll
  for (int r = 0; r < RS; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
    if (t4 == 0) {
      s_m[warp][g + 8 * r] = m[r];
      s_l[warp][g + 8 * r] = l[r];
    }
  }
  __syncthreads();  // all have left the last unit's outputs too
  float M[RS], f[RS];
#pragma unroll
  for (int r = 0; r < RS; ++r) {
    M[r] = s_m[0][g + 8 * r];
#pragma unroll
    for (int w = 1; w < WARPS; ++w) M[r] = fmaxf(M[r], s_m[w][g + 8 * r]);
    f[r] = ex2(m[r] - (M[r] == -INFINITY ? 0.f : M[r]));
  }
  // Warp w finishes the w-th share of the channels: it keeps its own part
  // of that and hands over the rest, to place (its warp, as the owner counts),
  // 8 heads at a time.
  constexpr int PART = NT / WARPS, PD = D / WARPS;
  const auto part = [&](int owner, int from) {
    return shared_o + (owner * (WARPS - 1) + (from - owner - 1 + WARPS) % WARPS) * 8 * PD;
  };
  const bool whole = walk.unit_start >= place.start && walk.unit_end <= place.stop;
  const bool at_start = walk.unit_start <= place.start;
  const int64_t slot = 2 * (int64_t)c + (at_start ? 0 : 1);
#pragma unroll
  for (int r = 0; r < RS; ++r) {
    if (r > 0) __syncthreads();  // all have taken the first heads
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int owner = i / PART;
      o[i][2 * r] = (PAIR ? o[i][0] + o[i][2] : o[i][2 * r]) * f[r];
      o[i][2 * r + 1] = (PAIR ? o[i][1] + o[i][3] : o[i][2 * r + 1]) * f[r];
      if (owner != warp)
        *reinterpret_cast<float2*>(part(owner, warp) + g * PD + (i % PART) * 8 + 2 * t4) =
            make_float2(o[i][2 * r], o[i][2 * r + 1]);
    }
    __syncthreads();
    const int h = g + 8 * r;
    if (h >= heads) continue;
    const float ref = M[r] == -INFINITY ? 0.f : M[r];
    float L = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) L = fmaf(ex2(s_m[w][h] - ref), s_l[w][h], L);
    const int64_t head = (int64_t)walk.n * a.Hq + hk * G + g0 + h;
    const float scale = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      if (i / PART != warp) continue;
      const int d = i * 8 + 2 * t4;
      float x = o[i][2 * r], y = o[i][2 * r + 1];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) {
        const float2 v = *reinterpret_cast<const float2*>(shared_o + (warp * (WARPS - 1) + w - 1) * 8 * PD + g * PD +
                                                          (i % PART) * 8 + 2 * t4);
        x += v.x;
        y += v.y;
      }
      if (whole) {
        *reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.out) + head * D + d) = pack_bf2(x * scale, y * scale);
      } else {
        *reinterpret_cast<float2*>(ws.o_of(slot, h) + d) = make_float2(x, y);
      }
    }
    if (t4 == 0 && warp == 0) {
      if (!whole) {
        ws.ml_of(slot, h)[0] = M[r];
        ws.ml_of(slot, h)[1] = L;
      } else if (a.lse != nullptr) {
        a.lse[head] = log_sum(ref, L);
      }
    }
  }
  if (threadIdx.x == 0 && at_start) ws.note[c] = note_of(walk, place);
}

}  // namespace kda
