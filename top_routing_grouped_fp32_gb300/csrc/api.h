// api.h -- what the translation units of the C ABI (api.cu, api_mx.cu) share:
// the experts' handle, the error message of a thread, argument checks and
// workspace cursors.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <string>

#include "common.cuh"
#include "internal.h"

struct moe_experts {
  const void* gate;
  const void* up;
  const void* down;
  moe_dtype dt;
  int64_t E, I, H;
  int device;
  int num_sms;
  moe::TcWeights* tc;  // null when the tcgen05 path does not apply (FP32, odd sizes)
};

namespace moe {
namespace api {

using moe::align_up;
using moe::dtype_size;
using moe::kWsHeader;

inline thread_local std::string g_error;  // of this thread's last failing call

inline moe_status fail(moe_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_error = buf;
  return st;
}

inline moe_status ok() {
  g_error.clear();
  return MOE_OK;
}

inline moe_status cuda_fail(cudaError_t e, const char* what) {
  return fail(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

#define MOE_TRY_CUDA(expr, what)                   \
  do {                                             \
    cudaError_t _e = (expr);                       \
    if (_e != cudaSuccess) return cuda_fail(_e, what); \
  } while (0)

constexpr int64_t kMaxE = 1024, kMaxK = 64, kMaxDim = int64_t(1) << 20;
constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1;

inline bool valid_dtype(moe_dtype d) { return d == MOE_F32 || d == MOE_F16 || d == MOE_BF16; }
inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
inline bool aligned256(const void* p) { return reinterpret_cast<uintptr_t>(p) % 256 == 0; }

// Whether na bytes from a and nb bytes from b share any.
inline bool overlap(const void* a, uint64_t na, const void* b, uint64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < na : x - y < nb;
}

struct Range {
  const void* p;
  uint64_t n;
};
// Whether no range of a shares bytes with one of b, or with another of a.
template <int NA, int NB>
bool apart(const Range (&a)[NA], const Range (&b)[NB]) {
  for (const Range& x : a)
    for (const Range& y : b)
      if (overlap(x.p, x.n, y.p, y.n)) return false;
  return true;
}
template <int N>
bool apart(const Range (&a)[N]) {
  for (int i = 0; i < N; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(a[i].p, a[i].n, a[j].p, a[j].n)) return false;
  return true;
}

// Checks shared by the calls that take (T, E, top_k).
inline moe_status check_tek(int64_t T, int64_t E, int32_t k) {
  if (T < 0) return fail(MOE_ERR_SHAPE, "T must be >= 0 (got %lld)", (long long)T);
  if (E < 1) return fail(MOE_ERR_SHAPE, "E must be >= 1 (got %lld)", (long long)E);
  if (k < 1 || k > E)
    return fail(MOE_ERR_INVALID_ARG, "top_k must satisfy 1 <= top_k <= E (top_k=%d, E=%lld)", k,
                (long long)E);
  if (E > kMaxE) return fail(MOE_ERR_UNSUPPORTED, "E=%lld exceeds the supported 1024", (long long)E);
  if (k > kMaxK) return fail(MOE_ERR_UNSUPPORTED, "top_k=%d exceeds the supported 64", k);
  if (T > kMaxRows / k)
    return fail(MOE_ERR_UNSUPPORTED, "T*top_k=%lld exceeds 2^31-1", (long long)T * k);
  return MOE_OK;
}

// GroupRoutingOptions rules of the user guide, section 10.
inline moe_status check_group_options(int64_t T, int64_t E, const moe_group_routing_options* o) {
  if (!o) return fail(MOE_ERR_INVALID_ARG, "group routing options are NULL");
  if (T < 0) return fail(MOE_ERR_SHAPE, "T must be >= 0 (got %lld)", (long long)T);
  if (E < 1 || E > kMaxE)
    return fail(E < 1 ? MOE_ERR_SHAPE : MOE_ERR_UNSUPPORTED, "expert count must be in 1..=1024 (got %lld)",
                (long long)E);
  if (o->groups < 1 || o->groups > 128)
    return fail(MOE_ERR_INVALID_ARG, "group count must be in 1..=128 (got %d)", o->groups);
  if (E % o->groups != 0)
    return fail(MOE_ERR_INVALID_ARG, "expert count %lld is not divisible by %d groups", (long long)E, o->groups);
  if (o->selected_groups < 1 || o->selected_groups > o->groups)
    return fail(MOE_ERR_INVALID_ARG, "selected_groups must be in 1..=groups (got %d of %d)",
                o->selected_groups, o->groups);
  const int64_t per = E / o->groups;
  if (o->top_k < 1 || o->top_k > 64)
    return fail(MOE_ERR_INVALID_ARG, "top_k must be in 1..=64 (got %d)", o->top_k);
  if (o->top_k > o->selected_groups * per)
    return fail(MOE_ERR_INVALID_ARG, "top_k=%d exceeds the %lld experts of the selected groups", o->top_k,
                (long long)(o->selected_groups * per));
  if (o->group_top_two && per < 2)
    return fail(MOE_ERR_INVALID_ARG, "group_top_two needs at least two experts per group");
  if (!(o->scale > 0.f) || !std::isfinite(o->scale))
    return fail(MOE_ERR_INVALID_ARG, "scale must be finite and positive");
  if (T > kMaxRows / o->top_k) return fail(MOE_ERR_UNSUPPORTED, "T*top_k exceeds 2^31-1");
  return MOE_OK;
}

inline moe_status check_dim(int64_t v, const char* name) {
  if (v < 1) return fail(MOE_ERR_SHAPE, "%s must be >= 1 (got %lld)", name, (long long)v);
  if (v > kMaxDim) return fail(MOE_ERR_UNSUPPORTED, "%s=%lld exceeds 2^20", name, (long long)v);
  return MOE_OK;
}

inline moe_status check_ws(const void* ws, size_t have, size_t need) {
  if (!ws) return fail(MOE_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned256(ws)) return fail(MOE_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  if (have < need)
    return fail(MOE_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed", have, need);
  return MOE_OK;
}

inline moe_status check_handle(const moe_experts* x) {
  if (!x) return fail(MOE_ERR_INVALID_ARG, "experts handle is NULL");
  int dev = -1;
  MOE_TRY_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev != x->device)
    return fail(MOE_ERR_INVALID_ARG, "experts live on device %d but device %d is current", x->device,
                dev);
  return MOE_OK;
}

// ---- workspace layouts -----------------------------------------------------
struct Cursor {
  size_t off = kWsHeader;
  size_t take(size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 1024);
    return at;
  }
};

template <typename P>
P* at(void* base, size_t off) {
  return reinterpret_cast<P*>(static_cast<char*>(base) + off);
}

inline uint32_t* status_word(void* ws) { return static_cast<uint32_t*>(ws); }

}  // namespace api
}  // namespace moe
