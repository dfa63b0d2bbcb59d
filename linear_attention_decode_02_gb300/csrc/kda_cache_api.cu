// libkda C ABI: the paged KV cache, beam selection and slot copies around the
// recurrent layers.  Contract checks on the host, then the launch; no device
// reads, no allocation, no synchronisation.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kda_cache.h"
#include "kda_host.h"
#include "kda_launch.h"

using namespace kda::host;

namespace {

// No byte is shared although the byte ranges cross: views that interleave
// along one axis, as keys and values of one allocation do.  For a stride s of
// `a` with every larger stride of both views a multiple of s, addresses modulo
// s lie in [0, ea) and [r, r + eb), ea and eb the extents below that axis and
// r the offset modulo s, which are disjoint where ea <= r and r + eb <= s.
bool interleaved(const View& a, const View& b) {
  const int64_t ba = esize(a.dtype), bb = esize(b.dtype);
  for (int i = 0; i < a.ndim; ++i) {
    if (a.shape[i] <= 1) continue;
    const int64_t s = a.stride[i] * ba;
    int64_t ext[2] = {0, 0};
    bool nested = true;
    for (int w = 0; w < 2; ++w) {
      const View& v = w == 0 ? a : b;
      const int64_t es = w == 0 ? ba : bb;
      ext[w] = es;
      for (int j = 0; j < v.ndim; ++j) {
        if (v.shape[j] <= 1) continue;
        const int64_t st = v.stride[j] * es;
        if (st < s) ext[w] += (v.shape[j] - 1) * st;
        else if (st % s != 0) nested = false;
      }
    }
    if (!nested) continue;
    const int64_t d = b.data - a.data;
    const int64_t r = ((d % s) + s) % s;
    if (ext[0] <= r && r + ext[1] <= s) return true;
  }
  return false;
}

kda_status no_shared_bytes(const View& w, std::initializer_list<const View*> others) {
  for (const View* o : others)
    KDA_CHECK(!overlap(w, *o) || interleaved(w, *o) || interleaved(*o, w), KDA_ERR_ALIAS, "%s overlaps %s", w.name,
              o->name);
  return KDA_OK;
}

bool same_view(const View& a, const View& b) {
  if (a.data != b.data || a.dtype != b.dtype || a.ndim != b.ndim) return false;
  for (int i = 0; i < a.ndim; ++i)
    if (a.shape[i] != b.shape[i] || (a.shape[i] > 1 && a.stride[i] != b.stride[i])) return false;
  return true;
}

// Every vector of the last axis starts on a `bytes` boundary.
bool vectors_aligned(const View& v, int64_t bytes) {
  if (reinterpret_cast<uintptr_t>(v.data) % bytes != 0) return false;
  for (int i = 0; i < v.ndim - 1; ++i)
    if (v.shape[i] > 1 && (v.stride[i] * esize(v.dtype)) % bytes != 0) return false;
  return true;
}

// No two elements of a view that is written share an address: every stride
// spans the axes of smaller strides.
kda_status need_distinct(const View& v) {
  for (int i = 0; i < v.ndim; ++i) {
    if (v.shape[i] <= 1) continue;
    int64_t inner = 1;
    for (int j = 0; j < v.ndim; ++j)
      if (j != i && v.shape[j] > 1 && (v.stride[j] < v.stride[i] || (v.stride[j] == v.stride[i] && j < i)))
        inner += (v.shape[j] - 1) * v.stride[j];
    KDA_CHECK(v.stride[i] >= inner, KDA_ERR_INVALID_ARG, "%s: elements overlap along axis %d", v.name, i);
  }
  return KDA_OK;
}

// Key and value pages [num_pages, page_size, Hkv, D] of one dtype and shape.
kda_status need_pages(const View& K, const View& V, int64_t Hkv, int64_t D) {
  KDA_TRY(need_dtype(K, KDA_F32, KDA_BF16));
  KDA_CHECK(V.dtype == K.dtype, KDA_ERR_INVALID_ARG, "v_pages: dtype must match k_pages");
  for (const View* p : {&K, &V}) {
    KDA_CHECK(p->shape[0] >= 1 && p->shape[0] <= INT32_MAX, KDA_ERR_INVALID_ARG, "%s: num_pages %lld out of range",
              p->name, (long long)p->shape[0]);
    KDA_CHECK(p->shape[1] >= 1 && p->shape[1] <= INT32_MAX, KDA_ERR_INVALID_ARG, "%s: page size %lld out of range",
              p->name, (long long)p->shape[1]);
    KDA_TRY(need_shape(*p, 0, K.shape[0]));
    KDA_TRY(need_shape(*p, 1, K.shape[1]));
    KDA_TRY(need_shape(*p, 2, Hkv));
    KDA_TRY(need_shape(*p, 3, D));
    KDA_TRY(need_vec_layout(*p));
  }
  return KDA_OK;
}

kda_status need_table(const View& T, int64_t N) {
  KDA_TRY(need_dtype(T, KDA_I32));
  KDA_TRY(need_shape(T, 0, N));
  KDA_CHECK(T.shape[1] <= INT32_MAX, KDA_ERR_INVALID_ARG, "%s: too many pages a sequence", T.name);
  KDA_CHECK(T.shape[1] <= 1 || T.stride[1] == 1, KDA_ERR_INVALID_ARG, "%s: column stride must be 1", T.name);
  return KDA_OK;
}

constexpr int32_t kMaxPools = 256;

kda_status check_attention_heads(int64_t Hq, int64_t Hkv, int64_t D) {
  KDA_CHECK(Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0, KDA_ERR_INVALID_ARG,
            "%lld query heads cannot share %lld key heads evenly", (long long)Hq, (long long)Hkv);
  KDA_CHECK(Hq <= 4096, KDA_ERR_UNSUPPORTED, "%lld query heads, at most 4096", (long long)Hq);
  KDA_CHECK(D == 64 || D == 128 || D == 256, KDA_ERR_UNSUPPORTED, "head dimension %lld: 64, 128 and 256 are served",
            (long long)D);
  return KDA_OK;
}

kda_status check_beam_sizes(int64_t N, int64_t B, int64_t V, int64_t M) {
  KDA_CHECK(N >= 0 && N < (1 << 24), KDA_ERR_UNSUPPORTED, "%lld requests, fewer than 2^24 are served", (long long)N);
  KDA_CHECK(B >= 1 && B <= kda::kBeamMax, KDA_ERR_UNSUPPORTED, "%lld beams, 1 to %d are served", (long long)B,
            kda::kBeamMax);
  KDA_CHECK(V >= 1 && V <= (1 << 24), KDA_ERR_UNSUPPORTED, "vocabulary of %lld, 1 to 2^24 are served", (long long)V);
  KDA_CHECK(M >= 1 && M <= kda::kBeamOutMax, KDA_ERR_UNSUPPORTED, "%lld candidates, 1 to %d are served", (long long)M,
            kda::kBeamOutMax);
  return KDA_OK;
}

kda::PageView page_view(const View& v) { return {v.data, v.stride[0], v.stride[1], v.stride[2]}; }

}  // namespace

extern "C" {

kda_status kda_rope_phase_steps(int32_t rot_dim, double base, double factor, double original_len, double low,
                                double high, uint64_t* steps) {
  KDA_CHECK(rot_dim >= 0 && rot_dim % 2 == 0 && rot_dim <= 512, KDA_ERR_INVALID_ARG,
            "rot_dim %d must be even and in 0..512", rot_dim);
  KDA_CHECK(std::isfinite(base) && base > 1.0, KDA_ERR_INVALID_ARG, "base must be finite and above 1");
  KDA_CHECK(std::isfinite(factor) && factor >= 1.0, KDA_ERR_INVALID_ARG, "factor must be finite and at least 1");
  KDA_CHECK(std::isfinite(original_len) && original_len >= 0.0, KDA_ERR_INVALID_ARG,
            "original_len must be finite and not negative");
  KDA_CHECK(original_len == 0.0 || (std::isfinite(low) && std::isfinite(high) && low < high), KDA_ERR_INVALID_ARG,
            "low must be below high");
  KDA_CHECK(steps != nullptr || rot_dim == 0, KDA_ERR_INVALID_ARG, "steps: null pointer");
  const double two_pi = 6.283185307179586;
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double turns = std::pow(base, -2.0 * i / rot_dim) / two_pi;  // a position
    double keep = 0.0;
    if (original_len > 0.0) keep = std::min(1.0, std::max(0.0, (original_len * turns - low) / (high - low)));
    const double scaled = turns * (keep + (1.0 - keep) / factor);
    steps[i] = static_cast<uint64_t>(std::llround(std::ldexp(scaled, 64)));  // at most 2^64 / 2 pi
  }
  return KDA_OK;
}

kda_status kda_rope_append(const kda_tensor* q, const kda_tensor* k, const kda_tensor* v, const kda_tensor* phase_steps,
                           const kda_tensor* cu_seqlens, const kda_tensor* seq_lens, const kda_tensor* page_table,
                           const kda_tensor* k_pages, const kda_tensor* v_pages, const kda_tensor* q_out,
                           int32_t is_interleaved, float amplitude, void* stream) {
  View Q, K, V, P, CU, L, T, KP, VP, O;
  KDA_TRY(ranked_view(q, "q", 3, -1, &Q));
  KDA_TRY(ranked_view(k, "k", 3, -1, &K));
  KDA_TRY(ranked_view(v, "v", 3, -1, &V));
  KDA_TRY(ranked_view(phase_steps, "phase_steps", 2, -1, &P));
  if (cu_seqlens != nullptr) KDA_TRY(raw_view(cu_seqlens, "cu_seqlens", &CU));
  KDA_TRY(raw_view(seq_lens, "seq_lens", &L));
  KDA_TRY(ranked_view(page_table, "page_table", 2, -1, &T));
  KDA_TRY(ranked_view(k_pages, "k_pages", 4, -1, &KP));
  KDA_TRY(ranked_view(v_pages, "v_pages", 4, -1, &VP));
  KDA_TRY(ranked_view(q_out, "q_out", 3, -1, &O));

  const int64_t R = Q.shape[0], Hq = Q.shape[1], D = Q.shape[2], Hkv = K.shape[1];
  KDA_TRY(need_dtype(Q, KDA_F32, KDA_BF16));
  KDA_CHECK(R <= INT32_MAX, KDA_ERR_INVALID_ARG, "q: too many token rows");
  KDA_CHECK(Hq >= 1 && Hkv >= 1, KDA_ERR_INVALID_ARG, "q, k: need at least one head");
  KDA_CHECK((Hq + 2 * Hkv) * D <= (1 << 24), KDA_ERR_UNSUPPORTED, "q, k: too many heads");
  KDA_CHECK(D >= 4 && D % 4 == 0 && D <= 512, KDA_ERR_UNSUPPORTED, "q: head dimension %lld must be a multiple of 4 in 4..512",
            (long long)D);
  for (View* t : {&K, &V}) {
    KDA_CHECK(t->dtype == Q.dtype, KDA_ERR_INVALID_ARG, "%s: dtype must match q", t->name);
    KDA_TRY(need_shape(*t, 0, R));
    KDA_TRY(need_shape(*t, 1, Hkv));
    KDA_TRY(need_shape(*t, 2, D));
  }
  for (View* t : {&Q, &K, &V}) KDA_TRY(need_vec_layout(*t));
  KDA_TRY(need_dtype(P, KDA_I32));
  KDA_TRY(need_shape(P, 1, 2));
  KDA_TRY(need_contiguous(P));
  const int64_t rot = 2 * P.shape[0];
  KDA_CHECK(rot <= D && rot % 8 == 0, KDA_ERR_INVALID_ARG,
            "phase_steps: %lld pairs; the rotated part must be a multiple of 8 and at most the head dimension",
            (long long)P.shape[0]);
  KDA_CHECK(reinterpret_cast<uintptr_t>(P.data) % 8 == 0, KDA_ERR_INVALID_ARG, "phase_steps: data must be 8-byte aligned");
  KDA_CHECK(L.ndim == 1, KDA_ERR_INVALID_ARG, "seq_lens: expected rank 1");
  const int64_t N = L.shape[0];
  KDA_CHECK(N <= INT32_MAX - 1, KDA_ERR_INVALID_ARG, "seq_lens: too many sequences");
  KDA_TRY(need_indices(L, N));
  if (cu_seqlens != nullptr) {
    KDA_TRY(need_indices(CU, N + 1));
  } else {
    KDA_CHECK(R == N, KDA_ERR_INVALID_ARG, "q: without cu_seqlens each of the %lld sequences has one row, not %lld",
              (long long)N, (long long)R);
  }
  KDA_TRY(need_table(T, N));
  KDA_TRY(need_pages(KP, VP, Hkv, D));
  KDA_CHECK(O.dtype == KP.dtype, KDA_ERR_INVALID_ARG, "q_out: dtype must match the pages");
  KDA_TRY(need_shape(O, 0, R));
  KDA_TRY(need_shape(O, 1, Hq));
  KDA_TRY(need_shape(O, 2, D));
  KDA_TRY(need_vec_layout(O));
  KDA_CHECK(is_interleaved == 0 || is_interleaved == 1, KDA_ERR_INVALID_ARG, "interleaved must be 0 or 1");
  KDA_CHECK(std::isfinite(amplitude), KDA_ERR_INVALID_ARG, "amplitude must be finite");
  for (const View* w : {&O, &KP, &VP}) KDA_TRY(need_distinct(*w));
  if (!same_view(O, Q)) KDA_TRY(no_shared_bytes(O, {&Q}));
  KDA_TRY(no_shared_bytes(O, {&K, &V, &P, &CU, &L, &T, &KP, &VP}));
  KDA_TRY(no_shared_bytes(KP, {&Q, &K, &V, &P, &CU, &L, &T, &VP}));
  KDA_TRY(no_shared_bytes(VP, {&Q, &K, &V, &P, &CU, &L, &T}));
  if (R == 0) return KDA_OK;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  KDA_TRY(current_device(st, &dev));
  kda::RopeArgs a{};
  a.q = Q.data; a.k = K.data; a.v = V.data;
  a.q_rs = Q.stride[0]; a.q_hs = Q.stride[1];
  a.k_rs = K.stride[0]; a.k_hs = K.stride[1];
  a.v_rs = V.stride[0]; a.v_hs = V.stride[1];
  a.steps = reinterpret_cast<const uint64_t*>(P.data);
  a.cu = cu_seqlens != nullptr ? reinterpret_cast<const int32_t*>(CU.data) : nullptr;
  a.lens = reinterpret_cast<const int32_t*>(L.data);
  a.table = reinterpret_cast<const int32_t*>(T.data); a.table_rs = T.stride[0]; a.table_cols = (int32_t)T.shape[1];
  a.kp = page_view(KP); a.vp = page_view(VP);
  a.num_pages = (int32_t)KP.shape[0]; a.page_size = (int32_t)KP.shape[1];
  a.q_out = O.data; a.o_rs = O.stride[0]; a.o_hs = O.stride[1];
  a.R = (int32_t)R; a.N = (int32_t)N; a.Hq = (int32_t)Hq; a.Hkv = (int32_t)Hkv; a.D = (int32_t)D; a.rot = (int32_t)rot;
  a.interleaved = is_interleaved; a.amplitude = amplitude;
  a.in_dtype = Q.dtype; a.page_dtype = KP.dtype;
  a.vec = 4; a.sms = dev.sms;
  if (Q.dtype == KDA_BF16 && KP.dtype == KDA_BF16 && D % 8 == 0 && (is_interleaved || rot % 16 == 0)) {
    bool wide = true;
    for (const View* t : {&Q, &K, &V, &KP, &VP, &O}) wide = wide && vectors_aligned(*t, 16);
    if (wide) a.vec = 8;
  }
  return check_launch(kda::launch_rope_append(a, st));
}

kda_status kda_pool_move(const kda_tensor* const* pools, int32_t n_pools, const kda_tensor* src_slots,
                         const kda_tensor* dst_slots, const kda_tensor* parents, void* stream) {
  View S, D, P;
  KDA_CHECK(n_pools >= 1, KDA_ERR_INVALID_ARG, "pools: need at least one pool");
  KDA_CHECK(pools != nullptr, KDA_ERR_INVALID_ARG, "pools: null pointer");
  KDA_TRY(ranked_view(src_slots, "src_slots", 2, -1, &S));
  KDA_TRY(ranked_view(dst_slots, "dst_slots", 2, -1, &D));
  const int64_t N = S.shape[0], K = S.shape[1];
  KDA_CHECK(N <= INT32_MAX, KDA_ERR_INVALID_ARG, "src_slots: too many rows");
  KDA_CHECK(K <= kda::kMoveBeams, KDA_ERR_UNSUPPORTED, "src_slots: %lld slots a row, at most %d", (long long)K,
            kda::kMoveBeams);
  KDA_TRY(need_table(S, N));
  KDA_TRY(need_table(D, N));
  KDA_TRY(need_shape(D, 1, K));
  if (parents != nullptr) {
    KDA_TRY(ranked_view(parents, "parents", 2, -1, &P));
    KDA_TRY(need_table(P, N));
    KDA_TRY(need_shape(P, 1, K));
  }
  KDA_CHECK(n_pools <= kMaxPools, KDA_ERR_UNSUPPORTED, "pools: %d pools, at most %d a call", n_pools, kMaxPools);
  View V[kMaxPools];
  kda::MovePool M[kMaxPools];
  uintptr_t lo[kMaxPools], hi[kMaxPools];
  for (int32_t i = 0; i < n_pools; ++i) {
    View& v = V[i];
    KDA_TRY(raw_view(pools[i], "pool", &v));
    KDA_CHECK(v.shape[0] >= 1 && v.shape[0] <= INT32_MAX, KDA_ERR_INVALID_ARG, "pool %d: num_slots %lld out of range", i,
              (long long)v.shape[0]);
    KDA_CHECK(v.shape[0] == V[0].shape[0], KDA_ERR_INVALID_ARG, "pool %d: %lld slots, pool 0 has %lld", i,
              (long long)v.shape[0], (long long)V[0].shape[0]);
    // The axes of a slot, smallest stride first, must follow one another without gaps.
    int64_t size = 1;
    bool used[4] = {false, false, false, false};
    for (int step = 1; step < v.ndim; ++step) {
      int at = -1;
      for (int j = 1; j < v.ndim; ++j)
        if (!used[j] && (at < 0 || v.shape[j] <= 1 || (v.shape[at] > 1 && v.stride[j] < v.stride[at]))) at = j;
      used[at] = true;
      KDA_CHECK(v.shape[at] <= 1 || v.stride[at] == size, KDA_ERR_INVALID_ARG, "pool %d: a slot must be dense", i);
      size *= v.shape[at];
    }
    KDA_CHECK(v.shape[0] <= 1 || v.stride[0] >= size, KDA_ERR_INVALID_ARG, "pool %d: slot stride %lld overlaps slots", i,
              (long long)v.stride[0]);
    M[i] = {v.data, v.shape[0] <= 1 ? 0 : v.stride[0] * esize(v.dtype), size * esize(v.dtype), 0};
    KDA_TRY(no_alias(v, {&S, &D, &P}));
    v.range(&lo[i], &hi[i]);
    for (int32_t j = 0; j < i; ++j)
      KDA_CHECK(hi[i] <= lo[j] || hi[j] <= lo[i] || !overlap(v, V[j]) || interleaved(v, V[j]) || interleaved(V[j], v),
                KDA_ERR_ALIAS, "pool %d overlaps pool %d", i, j);
  }
  if (N == 0 || K == 0) return KDA_OK;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  KDA_TRY(current_device(st, &dev));
  kda::MoveArgs a{};
  a.src = reinterpret_cast<const int32_t*>(S.data); a.src_rs = S.stride[0];
  a.dst = reinterpret_cast<const int32_t*>(D.data); a.dst_rs = D.stride[0];
  if (parents != nullptr) { a.parents = reinterpret_cast<const int32_t*>(P.data); a.par_rs = P.stride[0]; }
  a.N = (int32_t)N; a.K = (int32_t)K; a.num_slots = (int32_t)V[0].shape[0];
  // All launches are planned before the first, so that a refusal moves nothing.
  for (int pass = 0; pass < 2; ++pass) {
    for (int32_t i = 0; i < n_pools; i += kda::kMovePools) {
      a.pools = std::min(kda::kMovePools, n_pools - i);
      uintptr_t bits = 0;
      for (int j = 0; j < a.pools; ++j) {
        a.pool[j] = M[i + j];
        bits |= reinterpret_cast<uintptr_t>(M[i + j].base) | (uintptr_t)M[i + j].stride | (uintptr_t)M[i + j].bytes;
      }
      a.align = bits % 16 == 0 ? 16 : (bits % 4 == 0 ? 4 : 2);
      int64_t blocks = 0;
      KDA_CHECK(kda::plan_pool_move(a, &blocks), KDA_ERR_UNSUPPORTED, "pools: too much to move in one call");
      if (pass == 1 && blocks > 0) KDA_TRY(check_launch(kda::launch_pool_move(a, blocks, st)));
    }
  }
  return KDA_OK;
}

kda_status kda_paged_attention_workspace(int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t dtype,
                                         int32_t sm_count, int64_t* floats) {
  KDA_CHECK(floats != nullptr, KDA_ERR_INVALID_ARG, "floats: null pointer");
  KDA_TRY(check_attention_heads(q_heads, kv_heads, head_dim));
  KDA_CHECK(dtype == KDA_F32 || dtype == KDA_BF16, KDA_ERR_INVALID_ARG, "dtype %s not accepted", dtname(dtype));
  KDA_CHECK(sm_count >= 1 && sm_count <= 4096, KDA_ERR_INVALID_ARG, "sm_count %d out of range", sm_count);
  *floats = kda::attend_floats(q_heads, kv_heads, head_dim, dtype, sm_count);
  return KDA_OK;
}

kda_status kda_paged_attention_decode(const kda_tensor* q, const kda_tensor* k_pages, const kda_tensor* v_pages,
                                      const kda_tensor* page_table, const kda_tensor* seq_lens,
                                      const kda_tensor* workspace, int32_t window, float scale, const kda_tensor* out,
                                      const kda_tensor* lse, void* stream) {
  View Q, KP, VP, T, L, W, O, E;
  KDA_TRY(ranked_view(q, "q", 3, -1, &Q));
  KDA_TRY(ranked_view(k_pages, "k_pages", 4, -1, &KP));
  KDA_TRY(ranked_view(v_pages, "v_pages", 4, -1, &VP));
  KDA_TRY(ranked_view(page_table, "page_table", 2, -1, &T));
  KDA_TRY(raw_view(seq_lens, "seq_lens", &L));
  KDA_TRY(ranked_view(workspace, "workspace", 1, -1, &W));
  KDA_TRY(ranked_view(out, "out", 3, -1, &O));
  const int64_t N = Q.shape[0], Hq = Q.shape[1], D = Q.shape[2], Hkv = KP.shape[2];
  KDA_TRY(need_dtype(Q, KDA_F32, KDA_BF16));
  KDA_CHECK(N <= INT32_MAX, KDA_ERR_INVALID_ARG, "q: too many sequences");
  KDA_TRY(check_attention_heads(Hq, Hkv, D));
  KDA_TRY(need_vec_layout(Q));
  KDA_TRY(need_pages(KP, VP, Hkv, D));
  KDA_CHECK(KP.dtype == Q.dtype, KDA_ERR_INVALID_ARG, "k_pages: dtype must match q");
  KDA_TRY(need_table(T, N));
  KDA_CHECK(T.shape[1] <= (1 << 30) / KP.shape[1], KDA_ERR_UNSUPPORTED,
            "page_table: %lld pages of %lld positions, more than 2^30 positions a sequence", (long long)T.shape[1],
            (long long)KP.shape[1]);
  KDA_TRY(need_indices(L, N));
  KDA_TRY(need_out(O));
  KDA_TRY(need_shape(O, 0, N));
  KDA_TRY(need_shape(O, 1, Hq));
  KDA_TRY(need_shape(O, 2, D));
  if (lse != nullptr) {
    KDA_TRY(ranked_view(lse, "lse", 2, -1, &E));
    KDA_TRY(need_dtype(E, KDA_F32));
    KDA_TRY(need_shape(E, 0, N));
    KDA_TRY(need_shape(E, 1, Hq));
    KDA_TRY(need_contiguous(E));
  }
  KDA_TRY(need_dtype(W, KDA_F32));
  KDA_TRY(need_contiguous(W));
  KDA_CHECK(reinterpret_cast<uintptr_t>(W.data) % 16 == 0, KDA_ERR_INVALID_ARG, "workspace: data must be 16-byte aligned");
  KDA_CHECK(window >= 0, KDA_ERR_INVALID_ARG, "window must not be negative (0: all positions)");
  const float scale_log2 = scale * 1.4426950408889634f;  // scores are taken in units of log 2
  KDA_CHECK(scale > 0.f && std::isfinite(scale_log2), KDA_ERR_INVALID_ARG, "scale must be positive and at most 2.3e38");
  KDA_TRY(no_shared_bytes(O, {&Q, &KP, &VP, &T, &L, &W, &E}));
  KDA_TRY(no_shared_bytes(W, {&Q, &KP, &VP, &T, &L, &E}));
  KDA_TRY(no_shared_bytes(E, {&Q, &KP, &VP, &T, &L}));
  if (N == 0) return KDA_OK;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  KDA_TRY(current_device(st, &dev));
  const int64_t floats = kda::attend_floats((int32_t)Hq, (int32_t)Hkv, (int32_t)D, KP.dtype, dev.sms);
  KDA_CHECK(W.shape[0] >= floats, KDA_ERR_INVALID_ARG, "workspace: %lld floats, this call needs %lld",
            (long long)W.shape[0], (long long)floats);
  kda::AttendArgs a{};
  a.q = Q.data; a.q_rs = Q.stride[0]; a.q_hs = Q.stride[1];
  a.kp = page_view(KP); a.vp = page_view(VP);
  a.num_pages = (int32_t)KP.shape[0]; a.page_size = (int32_t)KP.shape[1];
  a.table = reinterpret_cast<const int32_t*>(T.data); a.table_rs = T.stride[0]; a.table_cols = (int32_t)T.shape[1];
  a.lens = reinterpret_cast<const int32_t*>(L.data);
  a.out = O.data;
  a.lse = lse != nullptr ? reinterpret_cast<float*>(E.data) : nullptr;
  a.work = reinterpret_cast<float*>(W.data);
  a.N = (int32_t)N; a.Hq = (int32_t)Hq; a.Hkv = (int32_t)Hkv; a.D = (int32_t)D; a.dtype = KP.dtype;
  a.window = window;
  a.scale_log2 = scale_log2;
  a.vec16 = vectors_aligned(Q, 16) && vectors_aligned(KP, 16) && vectors_aligned(VP, 16);
  return check_launch(kda::launch_paged_attention(a, dev.sms, st));
}

kda_status kda_beam_select_workspace(int64_t requests, int32_t beams, int64_t vocab, int32_t num_out, int32_t dtype,
                                     int32_t sm_count, int64_t* floats) {
  KDA_CHECK(floats != nullptr, KDA_ERR_INVALID_ARG, "floats: null pointer");
  KDA_TRY(check_beam_sizes(requests, beams, vocab, num_out));
  KDA_CHECK(dtype == KDA_F32 || dtype == KDA_BF16, KDA_ERR_INVALID_ARG, "dtype %s not accepted", dtname(dtype));
  KDA_CHECK(sm_count >= 1 && sm_count <= 4096, KDA_ERR_INVALID_ARG, "sm_count %d out of range", sm_count);
  *floats = requests == 0 ? 0 : kda::beam_plan(requests, beams, (int32_t)vocab, num_out, dtype, false, sm_count).floats;
  return KDA_OK;
}

kda_status kda_beam_select(const kda_tensor* logits, const kda_tensor* scores, const kda_tensor* finished,
                           int32_t eos_token, const kda_tensor* workspace, const kda_tensor* out_scores,
                           const kda_tensor* out_parents, const kda_tensor* out_tokens, void* stream) {
  View X, S, F, W, OS, OP, OT;
  KDA_TRY(ranked_view(logits, "logits", 3, -1, &X));
  KDA_TRY(ranked_view(scores, "scores", 2, -1, &S));
  if (finished != nullptr) KDA_TRY(ranked_view(finished, "finished", 2, -1, &F));
  KDA_TRY(ranked_view(workspace, "workspace", 1, -1, &W));
  KDA_TRY(ranked_view(out_scores, "out_scores", 2, -1, &OS));
  KDA_TRY(ranked_view(out_parents, "out_parents", 2, -1, &OP));
  KDA_TRY(ranked_view(out_tokens, "out_tokens", 2, -1, &OT));
  const int64_t N = X.shape[0], B = X.shape[1], V = X.shape[2], M = OS.shape[1];
  KDA_TRY(need_dtype(X, KDA_F32, KDA_BF16));
  KDA_CHECK(V <= 1 || X.stride[2] == 1, KDA_ERR_INVALID_ARG, "logits: vocabulary axis must have stride 1");
  KDA_TRY(check_beam_sizes(N, B, V, M));
  KDA_TRY(need_dtype(S, KDA_F32));
  KDA_TRY(need_shape(S, 0, N));
  KDA_TRY(need_shape(S, 1, B));
  KDA_TRY(need_contiguous(S));
  if (finished != nullptr) {
    KDA_TRY(need_dtype(F, KDA_I32));
    KDA_TRY(need_shape(F, 0, N));
    KDA_TRY(need_shape(F, 1, B));
    KDA_TRY(need_contiguous(F));
    KDA_CHECK(eos_token >= 0 && eos_token < V, KDA_ERR_INVALID_ARG, "eos_token %d outside the vocabulary", eos_token);
  }
  KDA_TRY(need_dtype(OS, KDA_F32));
  for (const View* o : {&OP, &OT}) KDA_TRY(need_dtype(*o, KDA_I32));
  for (const View* o : {&OS, &OP, &OT}) {
    KDA_TRY(need_shape(*o, 0, N));
    KDA_TRY(need_shape(*o, 1, M));
    KDA_TRY(need_contiguous(*o));
  }
  KDA_TRY(need_dtype(W, KDA_F32));
  KDA_TRY(need_contiguous(W));
  KDA_CHECK(reinterpret_cast<uintptr_t>(W.data) % 16 == 0, KDA_ERR_INVALID_ARG, "workspace: data must be 16-byte aligned");
  KDA_TRY(no_alias(W, {&X, &S, &F, &OS, &OP, &OT}));
  KDA_TRY(no_alias(OS, {&X, &S, &F, &OP, &OT}));
  KDA_TRY(no_alias(OP, {&X, &S, &F, &OT}));
  KDA_TRY(no_alias(OT, {&X, &S, &F}));
  if (N == 0) return KDA_OK;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  KDA_TRY(current_device(st, &dev));
  const kda::BeamPlan plan =
      kda::beam_plan(N, (int32_t)B, (int32_t)V, (int32_t)M, X.dtype, vectors_aligned(X, 16), dev.sms);
  KDA_TRY(check_grid(N * B * plan.splits));
  KDA_CHECK(W.shape[0] >= plan.floats, KDA_ERR_INVALID_ARG, "workspace: %lld floats, this call needs %lld",
            (long long)W.shape[0], (long long)plan.floats);
  kda::BeamArgs a{};
  a.logits = X.data; a.ns = X.stride[0]; a.bs = X.stride[1];
  a.scores = reinterpret_cast<const float*>(S.data);
  a.finished = finished != nullptr ? reinterpret_cast<const int32_t*>(F.data) : nullptr;
  a.out_scores = reinterpret_cast<float*>(OS.data);
  a.out_parents = reinterpret_cast<int32_t*>(OP.data);
  a.out_tokens = reinterpret_cast<int32_t*>(OT.data);
  a.work = reinterpret_cast<float*>(W.data);
  a.N = (int32_t)N; a.B = (int32_t)B; a.V = (int32_t)V; a.M = (int32_t)M; a.eos = eos_token; a.dtype = X.dtype;
  return check_launch(kda::launch_beam_select(a, plan, st));
}

}  // extern "C"
