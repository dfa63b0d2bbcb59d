// libkda C ABI: pages of a step's sequences, rotary positions with several axes,
// and attention of sequences that share prefixes.  Contract checks on the host,
// then the launch; no device reads, no allocation, no synchronisation.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "kda_cache_host.h"
#include "kda_launch.h"

using namespace kda::host;

namespace {

kda_status check_prefix_sequences(int64_t N) {
  KDA_CHECK(N >= 0 && N < (1 << 24), KDA_ERR_UNSUPPORTED, "%lld sequences, fewer than 2^24 are served", (long long)N);
  return KDA_OK;
}

}  // namespace

extern "C" {

kda_status kda_page_assign(const kda_tensor* seq_lens, const kda_tensor* new_lens, const kda_tensor* shared_lens,
                           const kda_tensor* page_table, const kda_tensor* free_pages, const kda_tensor* free_state,
                           int32_t page_size, const kda_tensor* lens_out, const kda_tensor* state_out,
                           const kda_tensor* cu_seqlens, const kda_tensor* slots, void* stream) {
  View L, W, H, T, F, S, LO, SO, CU, X;
  KDA_TRY(raw_view(seq_lens, "seq_lens", &L));
  KDA_TRY(raw_view(new_lens, "new_lens", &W));
  if (shared_lens != nullptr) KDA_TRY(raw_view(shared_lens, "shared_lens", &H));
  KDA_TRY(ranked_view(page_table, "page_table", 2, -1, &T));
  KDA_TRY(raw_view(free_pages, "free_pages", &F));
  KDA_TRY(raw_view(free_state, "free_state", &S));
  KDA_TRY(raw_view(lens_out, "lens_out", &LO));
  KDA_TRY(raw_view(state_out, "state_out", &SO));
  KDA_TRY(raw_view(cu_seqlens, "cu_seqlens", &CU));
  KDA_TRY(raw_view(slots, "slots", &X));
  KDA_CHECK(L.ndim == 1, KDA_ERR_INVALID_ARG, "seq_lens: expected rank 1");
  const int64_t N = L.shape[0];
  KDA_CHECK(N <= kda::kPageSequences, KDA_ERR_UNSUPPORTED, "seq_lens: %lld sequences, at most %d a call", (long long)N,
            kda::kPageSequences);
  KDA_TRY(need_indices(L, N));
  KDA_TRY(need_indices(W, N));
  if (shared_lens != nullptr) KDA_TRY(need_indices(H, N));
  KDA_TRY(need_table(T, N));
  KDA_TRY(need_distinct(T));
  KDA_CHECK(F.ndim == 1, KDA_ERR_INVALID_ARG, "free_pages: expected rank 1");
  const int64_t C = F.shape[0];
  KDA_TRY(need_indices(F, C));
  KDA_CHECK(C >= 1, KDA_ERR_INVALID_ARG, "free_pages: no place for a page");
  KDA_CHECK(page_size >= 1, KDA_ERR_INVALID_ARG, "page_size %d must be positive", page_size);
  KDA_CHECK(C < INT32_MAX && (C + 1) * page_size <= INT32_MAX, KDA_ERR_UNSUPPORTED,
            "free_pages: the slots of %lld pages of %d positions pass 2^31", (long long)C + 1, page_size);
  KDA_TRY(need_indices(S, 2));
  KDA_TRY(need_indices(LO, N));
  KDA_TRY(need_indices(SO, 2));
  KDA_TRY(need_indices(CU, N + 1));
  KDA_CHECK(X.ndim == 1, KDA_ERR_INVALID_ARG, "slots: expected rank 1");
  KDA_CHECK(X.shape[0] <= INT32_MAX, KDA_ERR_INVALID_ARG, "slots: too many rows");
  KDA_TRY(need_indices(X, X.shape[0]));
  KDA_TRY(no_alias(T, {&L, &W, &H, &F, &S, &LO, &SO, &CU, &X}));
  KDA_TRY(no_alias(F, {&L, &W, &H, &S, &LO, &SO, &CU, &X}));
  KDA_TRY(no_alias(CU, {&L, &W, &H, &S, &LO, &SO, &X}));
  KDA_TRY(no_alias(X, {&L, &W, &H, &S, &LO, &SO}));
  KDA_TRY(no_alias(LO, {&H, &S, &SO}));
  for (const View* in : {&L, &W})
    if (!same_view(LO, *in)) KDA_TRY(no_alias(LO, {in}));
  KDA_TRY(no_alias(SO, {&L, &W, &H}));
  if (!same_view(SO, S)) KDA_TRY(no_alias(SO, {&S}));

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  KDA_TRY(current_device(st, &dev));
  kda::PagesArgs a{};
  const auto i32 = [](const View& v) { return reinterpret_cast<int32_t*>(v.data); };
  a.old_lens = i32(L); a.new_lens = i32(W); a.shared_lens = shared_lens != nullptr ? i32(H) : nullptr;
  a.table = i32(T); a.table_rs = T.stride[0]; a.table_cols = (int32_t)T.shape[1];
  a.ring = i32(F); a.capacity = (int32_t)C; a.state = i32(S);
  a.lens_out = i32(LO); a.state_out = i32(SO); a.cu = i32(CU); a.slots = i32(X);
  a.N = (int32_t)N; a.page_size = page_size; a.R = X.shape[0];
  return check_launch(kda::launch_page_assign(a, st));
}

kda_status kda_rope_pair_axes(const int32_t* sections, int32_t num_axes, int32_t cyclic, int32_t* pair_axes) {
  KDA_CHECK(sections != nullptr, KDA_ERR_INVALID_ARG, "sections: null pointer");
  KDA_CHECK(num_axes >= 1 && num_axes <= kda::kRopeAxes, KDA_ERR_UNSUPPORTED, "%d axes, 1 to %d are served", num_axes,
            kda::kRopeAxes);
  KDA_CHECK(cyclic == 0 || cyclic == 1, KDA_ERR_INVALID_ARG, "cyclic must be 0 or 1");
  int64_t pairs = 0, left[kda::kRopeAxes];
  for (int a = 0; a < num_axes; ++a) {
    KDA_CHECK(sections[a] >= 0, KDA_ERR_INVALID_ARG, "section %d is negative", a);
    left[a] = sections[a];
    pairs += sections[a];
  }
  KDA_CHECK(pairs <= 256, KDA_ERR_INVALID_ARG, "sections of %lld pairs, a head has at most 256", (long long)pairs);
  KDA_CHECK(pair_axes != nullptr || pairs == 0, KDA_ERR_INVALID_ARG, "pair_axes: null pointer");
  for (int64_t i = 0; i < pairs;)
    for (int a = 0; a < num_axes; ++a) {
      int64_t n = cyclic ? std::min<int64_t>(left[a], 1) : left[a];
      left[a] -= n;
      while (n-- > 0) pair_axes[i++] = a;
    }
  return KDA_OK;
}

kda_status kda_rope_axes_append(const kda_tensor* q, const kda_tensor* k, const kda_tensor* v,
                                const kda_tensor* phase_steps, const kda_tensor* pair_axes, const kda_tensor* positions,
                                const kda_tensor* slots, const kda_tensor* k_pages, const kda_tensor* v_pages,
                                const kda_tensor* q_out, int32_t is_interleaved, float amplitude, void* stream) {
  View Q, K, V, P, A, X, S, KP, VP, O;
  KDA_TRY(ranked_view(q, "q", 3, -1, &Q));
  KDA_TRY(ranked_view(k, "k", 3, -1, &K));
  KDA_TRY(ranked_view(v, "v", 3, -1, &V));
  KDA_TRY(ranked_view(phase_steps, "phase_steps", 2, -1, &P));
  KDA_TRY(raw_view(pair_axes, "pair_axes", &A));
  KDA_TRY(ranked_view(positions, "positions", 2, -1, &X));
  KDA_TRY(raw_view(slots, "slots", &S));
  KDA_TRY(ranked_view(k_pages, "k_pages", 4, -1, &KP));
  KDA_TRY(ranked_view(v_pages, "v_pages", 4, -1, &VP));
  KDA_TRY(ranked_view(q_out, "q_out", 3, -1, &O));

  kda::RopeArgs a{};
  KDA_TRY(check_rope(Q, K, V, P, KP, VP, O, is_interleaved, amplitude, &a));
  const int64_t R = Q.shape[0];
  KDA_TRY(need_indices(A, P.shape[0]));
  KDA_TRY(need_dtype(X, KDA_I32));
  KDA_TRY(need_shape(X, 0, R));
  KDA_CHECK(X.shape[1] >= 1 && X.shape[1] <= kda::kRopeAxes, KDA_ERR_UNSUPPORTED, "positions: %lld axes, 1 to %d are served",
            (long long)X.shape[1], kda::kRopeAxes);
  KDA_TRY(need_indices(S, R));
  KDA_TRY(no_shared_bytes(O, {&K, &V, &P, &A, &X, &S, &KP, &VP}));
  KDA_TRY(no_shared_bytes(KP, {&Q, &K, &V, &P, &A, &X, &S, &VP}));
  KDA_TRY(no_shared_bytes(VP, {&Q, &K, &V, &P, &A, &X, &S}));
  if (R == 0) return KDA_OK;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  KDA_TRY(current_device(st, &dev));
  a.sms = dev.sms;
  a.positions = reinterpret_cast<const int32_t*>(X.data); a.p_rs = X.stride[0]; a.p_as = X.stride[1];
  a.slots = reinterpret_cast<const int32_t*>(S.data);
  a.pair_axes = reinterpret_cast<const int32_t*>(A.data);
  a.num_axes = (int32_t)X.shape[1];
  return check_launch(kda::launch_rope_append(a, st));
}

kda_status kda_prefix_attention_workspace(int64_t sequences, int32_t q_heads, int32_t kv_heads, int32_t head_dim,
                                          int32_t dtype, int32_t sm_count, int64_t* floats) {
  KDA_CHECK(floats != nullptr, KDA_ERR_INVALID_ARG, "floats: null pointer");
  KDA_TRY(check_attention_heads(q_heads, kv_heads, head_dim));
  KDA_TRY(check_prefix_sequences(sequences));
  KDA_CHECK(dtype == KDA_F32 || dtype == KDA_BF16, KDA_ERR_INVALID_ARG, "dtype %s not accepted", dtname(dtype));
  KDA_CHECK(sm_count >= 1 && sm_count <= 4096, KDA_ERR_INVALID_ARG, "sm_count %d out of range", sm_count);
  *floats = kda::prefix_floats(sequences, q_heads, kv_heads, head_dim, dtype, sm_count);
  return KDA_OK;
}

kda_status kda_prefix_attention_decode(const kda_tensor* q, const kda_tensor* k_pages, const kda_tensor* v_pages,
                                       const kda_tensor* page_table, const kda_tensor* seq_lens,
                                       const kda_tensor* group_starts, const kda_tensor* prefix_lens,
                                       const kda_tensor* workspace, int32_t window, float scale, const kda_tensor* out,
                                       const kda_tensor* lse, void* stream) {
  AttentionViews v;
  View S, P;
  kda::AttendArgs a{};
  KDA_TRY(check_attention(q, k_pages, v_pages, page_table, seq_lens, workspace, window, scale, out, lse, &v, &a));
  KDA_TRY(check_prefix_sequences(v.Q.shape[0]));
  KDA_TRY(raw_view(group_starts, "group_starts", &S));
  KDA_TRY(raw_view(prefix_lens, "prefix_lens", &P));
  KDA_CHECK(P.ndim == 1, KDA_ERR_INVALID_ARG, "prefix_lens: expected rank 1");
  const int64_t G = P.shape[0];
  KDA_CHECK(G <= INT32_MAX - 1, KDA_ERR_INVALID_ARG, "prefix_lens: too many groups");
  KDA_TRY(need_indices(P, G));
  KDA_TRY(need_indices(S, G + 1));
  KDA_TRY(no_shared_bytes(v.O, {&S, &P}));
  KDA_TRY(no_shared_bytes(v.W, {&S, &P}));
  KDA_TRY(no_shared_bytes(v.E, {&S, &P}));
  if (a.N == 0) return KDA_OK;

  cudaStream_t st = static_cast<cudaStream_t>(stream);
  DeviceInfo dev;
  KDA_TRY(current_device(st, &dev));
  const int64_t floats = kda::prefix_floats(a.N, a.Hq, a.Hkv, a.D, a.dtype, dev.sms);
  KDA_CHECK(v.W.shape[0] >= floats, KDA_ERR_INVALID_ARG, "workspace: %lld floats, this call needs %lld",
            (long long)v.W.shape[0], (long long)floats);
  a.starts = reinterpret_cast<const int32_t*>(S.data);
  a.prefix_lens = reinterpret_cast<const int32_t*>(P.data);
  a.num_groups = (int32_t)G;
  return check_launch(kda::launch_prefix_attention(a, dev.sms, st));
}

}  // extern "C"
