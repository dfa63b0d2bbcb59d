// Contract checks shared by the entry points over the paged cache: views that
// interleave, element alignment, page and table shapes.  Host only.
#pragma once

#include <cmath>

#include "kda_cache.h"
#include "kda_host.h"

namespace kda {
namespace host {

// No byte is shared although the byte ranges cross: views that interleave
// along one axis, as keys and values of one allocation do.  For a stride s of
// `a` with every larger stride of both views a multiple of s, addresses modulo
// s lie in [0, ea) and [r, r + eb), ea and eb the extents below that axis and
// r the offset modulo s, which are disjoint where ea <= r and r + eb <= s.
inline bool interleaved(const View& a, const View& b) {
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

inline kda_status no_shared_bytes(const View& w, std::initializer_list<const View*> others) {
  for (const View* o : others)
    KDA_CHECK(!overlap(w, *o) || interleaved(w, *o) || interleaved(*o, w), KDA_ERR_ALIAS, "%s overlaps %s", w.name,
              o->name);
  return KDA_OK;
}

inline bool same_view(const View& a, const View& b) {
  if (a.data != b.data || a.dtype != b.dtype || a.ndim != b.ndim) return false;
  for (int i = 0; i < a.ndim; ++i)
    if (a.shape[i] != b.shape[i] || (a.shape[i] > 1 && a.stride[i] != b.stride[i])) return false;
  return true;
}

// Every vector of the last axis starts on a `bytes` boundary.
inline bool vectors_aligned(const View& v, int64_t bytes) {
  if (reinterpret_cast<uintptr_t>(v.data) % bytes != 0) return false;
  for (int i = 0; i < v.ndim - 1; ++i)
    if (v.shape[i] > 1 && (v.stride[i] * esize(v.dtype)) % bytes != 0) return false;
  return true;
}

// No two elements of a view that is written share an address: every stride
// spans the axes of smaller strides.
inline kda_status need_distinct(const View& v) {
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
inline kda_status need_pages(const View& K, const View& V, int64_t Hkv, int64_t D) {
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

inline kda_status need_table(const View& T, int64_t N) {
  KDA_TRY(need_dtype(T, KDA_I32));
  KDA_TRY(need_shape(T, 0, N));
  KDA_CHECK(T.shape[1] <= INT32_MAX, KDA_ERR_INVALID_ARG, "%s: too many pages a sequence", T.name);
  KDA_CHECK(T.shape[1] <= 1 || T.stride[1] == 1, KDA_ERR_INVALID_ARG, "%s: column stride must be 1", T.name);
  return KDA_OK;
}

inline kda_status check_attention_heads(int64_t Hq, int64_t Hkv, int64_t D) {
  KDA_CHECK(Hq >= 1 && Hkv >= 1 && Hq % Hkv == 0, KDA_ERR_INVALID_ARG,
            "%lld query heads cannot share %lld key heads evenly", (long long)Hq, (long long)Hkv);
  KDA_CHECK(Hq <= 4096, KDA_ERR_UNSUPPORTED, "%lld query heads, at most 4096", (long long)Hq);
  KDA_CHECK(D == 64 || D == 128 || D == 256, KDA_ERR_UNSUPPORTED, "head dimension %lld: 64, 128 and 256 are served",
            (long long)D);
  return KDA_OK;
}

inline kda::PageView page_view(const View& v) { return {v.data, v.stride[0], v.stride[1], v.stride[2]}; }

// Rows, steps, pages and outputs of the rotary entry points: checked, and the arguments that they share filled in.
inline kda_status check_rope(const View& Q, const View& K, const View& V, const View& P, const View& KP, const View& VP,
                             const View& O, int32_t is_interleaved, float amplitude, kda::RopeArgs* a) {
  const int64_t R = Q.shape[0], Hq = Q.shape[1], D = Q.shape[2], Hkv = K.shape[1];
  KDA_TRY(need_dtype(Q, KDA_F32, KDA_BF16));
  KDA_CHECK(R <= INT32_MAX, KDA_ERR_INVALID_ARG, "q: too many token rows");
  KDA_CHECK(Hq >= 1 && Hkv >= 1, KDA_ERR_INVALID_ARG, "q, k: need at least one head");
  KDA_CHECK((Hq + 2 * Hkv) * D <= (1 << 24), KDA_ERR_UNSUPPORTED, "q, k: too many heads");
  KDA_CHECK(D >= 4 && D % 4 == 0 && D <= 512, KDA_ERR_UNSUPPORTED, "q: head dimension %lld must be a multiple of 4 in 4..512",
            (long long)D);
  for (const View* t : {&K, &V}) {
    KDA_CHECK(t->dtype == Q.dtype, KDA_ERR_INVALID_ARG, "%s: dtype must match q", t->name);
    KDA_TRY(need_shape(*t, 0, R));
    KDA_TRY(need_shape(*t, 1, Hkv));
    KDA_TRY(need_shape(*t, 2, D));
  }
  for (const View* t : {&Q, &K, &V}) KDA_TRY(need_vec_layout(*t));
  KDA_TRY(need_dtype(P, KDA_I32));
  KDA_TRY(need_shape(P, 1, 2));
  KDA_TRY(need_contiguous(P));
  const int64_t rot = 2 * P.shape[0];
  KDA_CHECK(rot <= D && rot % 8 == 0, KDA_ERR_INVALID_ARG,
            "phase_steps: %lld pairs; the rotated part must be a multiple of 8 and at most the head dimension",
            (long long)P.shape[0]);
  KDA_CHECK(reinterpret_cast<uintptr_t>(P.data) % 8 == 0, KDA_ERR_INVALID_ARG, "phase_steps: data must be 8-byte aligned");
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
  a->q = Q.data; a->k = K.data; a->v = V.data;
  a->q_rs = Q.stride[0]; a->q_hs = Q.stride[1];
  a->k_rs = K.stride[0]; a->k_hs = K.stride[1];
  a->v_rs = V.stride[0]; a->v_hs = V.stride[1];
  a->steps = reinterpret_cast<const uint64_t*>(P.data);
  a->kp = page_view(KP); a->vp = page_view(VP);
  a->num_pages = (int32_t)KP.shape[0]; a->page_size = (int32_t)KP.shape[1];
  a->q_out = O.data; a->o_rs = O.stride[0]; a->o_hs = O.stride[1];
  a->R = (int32_t)R; a->Hq = (int32_t)Hq; a->Hkv = (int32_t)Hkv; a->D = (int32_t)D; a->rot = (int32_t)rot;
  a->interleaved = is_interleaved; a->amplitude = amplitude;
  a->in_dtype = Q.dtype; a->page_dtype = KP.dtype;
  a->vec = 4;
  if (Q.dtype == KDA_BF16 && KP.dtype == KDA_BF16 && D % 8 == 0 && (is_interleaved || rot % 16 == 0)) {
    bool wide = true;
    for (const View* t : {&Q, &K, &V, &KP, &VP, &O}) wide = wide && vectors_aligned(*t, 16);
    if (wide) a->vec = 8;
  }
  return KDA_OK;
}

// Tensors of the attention entry points: checked, and the launch arguments that they share filled in.
struct AttentionViews {
  View Q, KP, VP, T, L, W, O, E;
};
inline kda_status check_attention(const kda_tensor* q, const kda_tensor* k_pages, const kda_tensor* v_pages,
                                  const kda_tensor* page_table, const kda_tensor* seq_lens, const kda_tensor* workspace,
                                  int32_t window, float scale, const kda_tensor* out, const kda_tensor* lse,
                                  AttentionViews* views, kda::AttendArgs* args) {
  View &Q = views->Q, &KP = views->KP, &VP = views->VP, &T = views->T, &L = views->L, &W = views->W, &O = views->O,
       &E = views->E;
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
  kda::AttendArgs& a = *args;
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
  return KDA_OK;
}

}  // namespace host
}  // namespace kda
