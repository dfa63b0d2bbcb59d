// Host side of the C ABI shared by its translation units: error messages,
// tensor views, the contract checks every entry point is made of, and the
// device query.  Nothing here reads device memory.
#pragma once

#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <initializer_list>
#include <mutex>
#include <string>

#include "../../include/kda.h"

namespace kda {
namespace host {

constexpr int64_t kD = 128;
constexpr int64_t kUnit = kD * kD;  // elements of one (slot, head) state block

// One message per thread and one device table per process, shared by the translation units of the C ABI.
inline thread_local std::string g_last_error;

inline kda_status fail(kda_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return st;
}

#define KDA_CHECK(cond, st, ...)          \
  do {                                    \
    if (!(cond)) return fail(st, __VA_ARGS__); \
  } while (0)

#define KDA_TRY(expr)                \
  do {                               \
    kda_status s__ = (expr);         \
    if (s__ != KDA_OK) return s__;   \
  } while (0)

inline int64_t esize(int32_t dtype) { return dtype == KDA_BF16 ? 2 : 4; }

inline const char* dtname(int32_t d) {
  switch (d) {
    case KDA_F32: return "float32";
    case KDA_BF16: return "bfloat16";
    case KDA_I32: return "int32";
    default: return "unknown";
  }
}

// A tensor viewed with a fixed rank after dropping a leading/inner unit axis.
struct View {
  const char* name = nullptr;
  char* data = nullptr;
  int32_t dtype = -1;
  int ndim = 0;
  int64_t shape[4] = {0, 0, 0, 0};
  int64_t stride[4] = {0, 0, 0, 0};
  int64_t numel() const {
    int64_t n = 1;
    for (int i = 0; i < ndim; ++i) n *= shape[i];
    return n;
  }
  // Byte range [lo, hi) touched by the view (all strides are positive).
  void range(uintptr_t* lo, uintptr_t* hi) const {
    if (numel() == 0) { *lo = *hi = 0; return; }
    int64_t ext = 1;
    for (int i = 0; i < ndim; ++i) ext += (shape[i] - 1) * stride[i];
    *lo = reinterpret_cast<uintptr_t>(data);
    *hi = *lo + static_cast<uintptr_t>(ext * esize(dtype));
  }
};

inline kda_status raw_view(const kda_tensor* t, const char* name, View* v) {
  KDA_CHECK(t != nullptr, KDA_ERR_INVALID_ARG, "%s: null tensor descriptor", name);
  KDA_CHECK(t->ndim >= 1 && t->ndim <= 4, KDA_ERR_INVALID_ARG, "%s: ndim %d not in 1..4", name, t->ndim);
  KDA_CHECK(t->dtype == KDA_F32 || t->dtype == KDA_BF16 || t->dtype == KDA_I32, KDA_ERR_INVALID_ARG,
            "%s: unknown dtype %d", name, t->dtype);
  v->name = name;
  v->data = static_cast<char*>(t->data);
  v->dtype = t->dtype;
  v->ndim = t->ndim;
  for (int i = 0; i < t->ndim; ++i) {
    KDA_CHECK(t->shape[i] >= 0, KDA_ERR_INVALID_ARG, "%s: negative extent %lld on axis %d", name,
              (long long)t->shape[i], i);
    KDA_CHECK(t->stride[i] > 0 || t->shape[i] <= 1, KDA_ERR_INVALID_ARG,
              "%s: stride %lld on axis %d must be positive", name, (long long)t->stride[i], i);
    v->shape[i] = t->shape[i];
    v->stride[i] = t->shape[i] <= 1 && t->stride[i] <= 0 ? 1 : t->stride[i];
  }
  if (v->numel() == 0) return KDA_OK;
  KDA_CHECK(v->data != nullptr, KDA_ERR_INVALID_ARG, "%s: null data pointer", name);
  KDA_CHECK(reinterpret_cast<uintptr_t>(v->data) % esize(v->dtype) == 0, KDA_ERR_INVALID_ARG,
            "%s: data must be %lld-byte aligned", name, (long long)esize(v->dtype));
  return KDA_OK;
}

// Accepts rank `want`, or rank want+1 with a unit axis at `unit_axis` (dropped).
inline kda_status ranked_view(const kda_tensor* t, const char* name, int want, int unit_axis, View* v) {
  KDA_TRY(raw_view(t, name, v));
  if (v->ndim == want + 1 && unit_axis >= 0 && v->shape[unit_axis] == 1) {
    for (int i = unit_axis; i < v->ndim - 1; ++i) {
      v->shape[i] = v->shape[i + 1];
      v->stride[i] = v->stride[i + 1];
    }
    v->ndim = want;
  }
  KDA_CHECK(v->ndim == want, KDA_ERR_INVALID_ARG, "%s: expected rank %d, got %d", name, want, t->ndim);
  return KDA_OK;
}

inline kda_status need_dtype(const View& v, int32_t a, int32_t b = -1) {
  KDA_CHECK(v.dtype == a || v.dtype == b, KDA_ERR_INVALID_ARG, "%s: dtype %s not accepted", v.name,
            dtname(v.dtype));
  return KDA_OK;
}

inline kda_status need_shape(const View& v, int axis, int64_t want) {
  KDA_CHECK(v.shape[axis] == want, KDA_ERR_INVALID_ARG, "%s: axis %d is %lld, expected %lld", v.name, axis,
            (long long)v.shape[axis], (long long)want);
  return KDA_OK;
}

inline kda_status need_contiguous(const View& v) {
  int64_t expect = 1;
  for (int i = v.ndim - 1; i >= 0; --i) {
    KDA_CHECK(v.shape[i] <= 1 || v.stride[i] == expect, KDA_ERR_INVALID_ARG, "%s: must be contiguous", v.name);
    expect *= v.shape[i];
  }
  return KDA_OK;
}

// Activation vectors [rows, heads, 128]: channel stride 1, 4-element aligned
// rows and heads so lanes can read 4 channels with one 8/16-byte load.
inline kda_status need_vec_layout(const View& v) {
  KDA_CHECK(v.stride[v.ndim - 1] == 1, KDA_ERR_INVALID_ARG, "%s: channel axis must have stride 1", v.name);
  for (int i = 0; i < v.ndim - 1; ++i)
    KDA_CHECK(v.shape[i] <= 1 || v.stride[i] % 4 == 0, KDA_ERR_INVALID_ARG,
              "%s: stride %lld on axis %d must be a multiple of 4 elements", v.name, (long long)v.stride[i], i);
  KDA_CHECK(reinterpret_cast<uintptr_t>(v.data) % (4 * esize(v.dtype)) == 0, KDA_ERR_INVALID_ARG,
            "%s: data must be %lld-byte aligned", v.name, (long long)(4 * esize(v.dtype)));
  return KDA_OK;
}

// State pool [num_slots, H, 128, 128]: per-slot block contiguous, slot stride
// >= H*128*128 and 16-byte aligned.
inline kda_status need_state_layout(const View& v, int64_t H) {
  KDA_TRY(need_dtype(v, KDA_F32, KDA_BF16));
  KDA_CHECK(v.ndim == 4, KDA_ERR_INVALID_ARG, "state: expected rank 4");
  KDA_TRY(need_shape(v, 1, H));
  KDA_TRY(need_shape(v, 2, kD));
  KDA_TRY(need_shape(v, 3, kD));
  KDA_CHECK(v.shape[0] >= 1 && v.shape[0] <= INT32_MAX, KDA_ERR_INVALID_ARG, "state: num_slots %lld out of range",
            (long long)v.shape[0]);
  KDA_CHECK(v.stride[3] == 1 && v.stride[2] == kD && (H <= 1 || v.stride[1] == kUnit), KDA_ERR_INVALID_ARG,
            "state: each slot's [H, 128, 128] block must be contiguous");
  KDA_CHECK(v.shape[0] <= 1 || v.stride[0] >= H * kUnit, KDA_ERR_INVALID_ARG,
            "state: slot stride %lld overlaps slots (needs >= %lld)", (long long)v.stride[0], (long long)(H * kUnit));
  KDA_CHECK((v.stride[0] * esize(v.dtype)) % 16 == 0 || v.shape[0] <= 1, KDA_ERR_INVALID_ARG,
            "state: slot stride must keep 16-byte alignment");
  KDA_CHECK(reinterpret_cast<uintptr_t>(v.data) % 16 == 0, KDA_ERR_INVALID_ARG, "state: data must be 16-byte aligned");
  return KDA_OK;
}

inline kda_status need_indices(const View& v, int64_t n) {
  KDA_TRY(need_dtype(v, KDA_I32));
  KDA_CHECK(v.ndim == 1, KDA_ERR_INVALID_ARG, "%s: expected rank 1", v.name);
  KDA_TRY(need_shape(v, 0, n));
  KDA_CHECK(v.shape[0] <= 1 || v.stride[0] == 1, KDA_ERR_INVALID_ARG, "%s: must be contiguous", v.name);
  return KDA_OK;
}

inline kda_status need_f32_vector(const View& v, int64_t n) {
  KDA_TRY(need_dtype(v, KDA_F32));
  KDA_CHECK(v.numel() == n, KDA_ERR_INVALID_ARG, "%s: expected %lld elements, got %lld", v.name, (long long)n,
            (long long)v.numel());
  KDA_TRY(need_contiguous(v));
  KDA_CHECK(reinterpret_cast<uintptr_t>(v.data) % 16 == 0, KDA_ERR_INVALID_ARG, "%s: data must be 16-byte aligned",
            v.name);
  return KDA_OK;
}

inline kda_status need_out(const View& v) {
  KDA_TRY(need_dtype(v, KDA_BF16));
  KDA_TRY(need_contiguous(v));
  KDA_CHECK(reinterpret_cast<uintptr_t>(v.data) % 16 == 0, KDA_ERR_INVALID_ARG, "%s: data must be 16-byte aligned",
            v.name);
  return KDA_OK;
}

inline bool overlap(const View& a, const View& b) {
  uintptr_t alo, ahi, blo, bhi;
  a.range(&alo, &ahi);
  b.range(&blo, &bhi);
  if (alo == ahi || blo == bhi) return false;
  return alo < bhi && blo < ahi;
}

// `w` is written: it must not share bytes with any other argument.
inline kda_status no_alias(const View& w, std::initializer_list<const View*> others) {
  for (const View* o : others)
    KDA_CHECK(!overlap(w, *o), KDA_ERR_ALIAS, "%s overlaps %s", w.name, o->name);
  return KDA_OK;
}

// ---- device properties (cached per device) ------------------------------------

struct DeviceInfo {
  int cc_major = 0, cc_minor = 0, sms = 0;
  bool valid = false;
};
inline std::mutex g_dev_mu;
inline DeviceInfo g_dev[64];

inline kda_status current_device(cudaStream_t stream, DeviceInfo* info) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  KDA_CHECK(e == cudaSuccess, KDA_ERR_CUDA, "cudaGetDevice: %s", cudaGetErrorString(e));
  KDA_CHECK(dev >= 0 && dev < 64, KDA_ERR_UNSUPPORTED, "device ordinal %d out of range", dev);
  {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (!g_dev[dev].valid) {
      DeviceInfo d;
      e = cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev);
      if (e == cudaSuccess) e = cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev);
      KDA_CHECK(e == cudaSuccess, KDA_ERR_CUDA, "cudaDeviceGetAttribute: %s", cudaGetErrorString(e));
      d.valid = true;
      g_dev[dev] = d;
    }
    *info = g_dev[dev];
  }
  KDA_CHECK(info->cc_major == 10 && info->cc_minor == 3, KDA_ERR_UNSUPPORTED,
            "device %d is compute capability %d.%d; this library is built for sm_103a (GB300) only", dev,
            info->cc_major, info->cc_minor);
  // The stream's device is checked outside graph capture only: the query is
  // not permitted on a capturing stream (a capture on a stream of another
  // device fails at launch instead).
  cudaStreamCaptureStatus cap = cudaStreamCaptureStatusNone;
  if (stream != nullptr) {
    e = cudaStreamIsCapturing(stream, &cap);
    KDA_CHECK(e == cudaSuccess, KDA_ERR_INVALID_ARG, "stream: %s", cudaGetErrorString(e));
  }
  if (stream != nullptr && cap == cudaStreamCaptureStatusNone) {
    int sdev = -1;
    e = cudaStreamGetDevice(stream, &sdev);
    KDA_CHECK(e == cudaSuccess, KDA_ERR_INVALID_ARG, "stream: %s", cudaGetErrorString(e));
    KDA_CHECK(sdev == dev, KDA_ERR_INVALID_ARG, "stream belongs to device %d, current device is %d", sdev, dev);
  }
  return KDA_OK;
}

// Every head vector of the view starts on a 16-byte boundary (bulk copies).
inline bool rows_aligned16(const View& v) {
  if (reinterpret_cast<uintptr_t>(v.data) % 16 != 0) return false;
  for (int i = 0; i < v.ndim - 1; ++i)
    if (v.shape[i] > 1 && (v.stride[i] * esize(v.dtype)) % 16 != 0) return false;
  return true;
}

inline kda_status check_launch(cudaError_t e) {
  KDA_CHECK(e == cudaSuccess, KDA_ERR_CUDA, "kernel launch: %s", cudaGetErrorString(e));
  return KDA_OK;
}

inline kda_status check_grid(int64_t blocks) {
  KDA_CHECK(blocks < (int64_t)INT32_MAX, KDA_ERR_UNSUPPORTED, "grid of %lld CTAs too large", (long long)blocks);
  return KDA_OK;
}

}  // namespace host
}  // namespace kda
