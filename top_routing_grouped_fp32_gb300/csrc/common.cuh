// common.cuh -- small device helpers shared by the kernels of this library.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

constexpr uint32_t kInvalid = 0xFFFFFFFFu;

// Every workspace starts with this header; word 0 is the device status.
constexpr size_t kWsHeader = 256;

__host__ __device__ inline size_t align_up(size_t v, size_t a) { return (v + a - 1) / a * a; }

inline size_t dtype_size(moe_dtype d) { return d == MOE_F32 ? 4 : 2; }

// ---- element conversions --------------------------------------------------
template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}

template <typename T> __device__ __forceinline__ T from_f32(float v);
template <> __device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <> __device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// ---- programmatic dependent launch ------------------------------------------
// Kernels of a call sequence are launched with programmatic stream
// serialisation: a kernel may be launched (and run its prologue) before its
// predecessor in the stream has finished.  pdl_wait() blocks until every
// predecessor grid has completed and its memory is visible, so each kernel
// calls it before its first read of anything a predecessor wrote;
// pdl_trigger() lets the successor be launched once every CTA of this grid has
// started.  Without the launch attribute both are no-ops.
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// Reads element i of a weights array whose dtype is only known at run time.
__device__ __forceinline__ float load_dyn(const void* p, int dtype, size_t i) {
  if (dtype == MOE_F32) return static_cast<const float*>(p)[i];
  if (dtype == MOE_F16) return __half2float(static_cast<const __half*>(p)[i]);
  return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// Packs 8 floats to 8 16-bit values (one 16-byte store).
template <typename T> __device__ __forceinline__ uint4 pack8(const float* f);
template <> __device__ __forceinline__ uint4 pack8<__nv_bfloat16>(const float* f) {
  uint4 r;
  __nv_bfloat162 v0 = __floats2bfloat162_rn(f[0], f[1]);
  __nv_bfloat162 v1 = __floats2bfloat162_rn(f[2], f[3]);
  __nv_bfloat162 v2 = __floats2bfloat162_rn(f[4], f[5]);
  __nv_bfloat162 v3 = __floats2bfloat162_rn(f[6], f[7]);
  r.x = *reinterpret_cast<uint32_t*>(&v0);
  r.y = *reinterpret_cast<uint32_t*>(&v1);
  r.z = *reinterpret_cast<uint32_t*>(&v2);
  r.w = *reinterpret_cast<uint32_t*>(&v3);
  return r;
}
template <> __device__ __forceinline__ uint4 pack8<__half>(const float* f) {
  uint4 r;
  __half2 v0 = __floats2half2_rn(f[0], f[1]);
  __half2 v1 = __floats2half2_rn(f[2], f[3]);
  __half2 v2 = __floats2half2_rn(f[4], f[5]);
  __half2 v3 = __floats2half2_rn(f[6], f[7]);
  r.x = *reinterpret_cast<uint32_t*>(&v0);
  r.y = *reinterpret_cast<uint32_t*>(&v1);
  r.z = *reinterpret_cast<uint32_t*>(&v2);
  r.w = *reinterpret_cast<uint32_t*>(&v3);
  return r;
}

// Two floats as two 16-bit values.
template <typename T> __device__ __forceinline__ uint32_t pack2(float2 f);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float2 f) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float2 f) {
  const __half2 v = __floats2half2_rn(f.x, f.y);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Unpacks 8 16-bit values from a 16-byte vector.
template <typename T> __device__ __forceinline__ void unpack8(uint4 v, float* f) {
  const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = to_f32<T>(e[i]);
}

// ---- FP32 arithmetic ---------------------------------------------------------
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^x, 1 / x and log2(x), within 2 ulp, 1 ulp and 2^-22; subnormals are zero.
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float log2_fast(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two FP32 operations an instruction (x[n], x[n + 1] in a register pair).
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 a, b, c, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 d, a, b, c;\n mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n add.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 a, b, d;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 d, a, b;\n"
      " mov.b64 {%0, %1}, d;\n}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// ---- places in a table of running sums ------------------------------------------
// The last e < n with table[e] <= v (table[0] <= v; entries do not decrease;
// n <= 1024), by a converged warp: two rounds of one load and a vote.
__device__ __forceinline__ int warp_search(const uint32_t* table, int n, uint32_t v) {
  const int lane = threadIdx.x & 31;
  const int c = lane * 32;
  const uint32_t coarse = __ballot_sync(0xffffffffu, c < n && table[c] <= v);  // a run of low bits
  const int base = (31 - __clz(coarse)) * 32;
  const int f = base + lane;
  const uint32_t fine = __ballot_sync(0xffffffffu, f < n && table[f] <= v);
  return base + 31 - __clz(fine);
}
// a / b for a < 2^31, b >= 1: an FP32 quotient (off by one part in 2^21), then
// single steps (none or one for quotients below 2^20)
__device__ __forceinline__ uint32_t small_div(uint32_t a, uint32_t b) {
  uint32_t q = (uint32_t)__fdividef((float)a, (float)b);
  int32_t r = (int32_t)(a - q * b);
  while (r < 0) --q, r += (int32_t)b;
  while (r >= (int32_t)b) ++q, r -= (int32_t)b;
  return q;
}

// A caller's offsets [E+1] as kernels read them, by one warp: each clamped to
// [previous, N], so that no segment runs backwards or past the N rows of the
// buffers.  Returns whether an entry was clamped (the same in every lane).
__device__ __forceinline__ bool clamp_offsets(const uint32_t* __restrict__ in, int E, int64_t N, uint32_t* out) {
  const int lane = threadIdx.x & 31;
  const int n = E + 1;
  const int per = (n + 31) / 32;
  const uint32_t cap = N < (int64_t)0xFFFFFFFFu ? (uint32_t)N : 0xFFFFFFFEu;
  uint32_t run = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < n) {
      const uint32_t v = in[e];
      run = max(run, v < cap ? v : cap);
    }
  }
  uint32_t incl = run;  // max over this lane's entries and every earlier lane's
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl = max(incl, o);
  }
  uint32_t prev = __shfl_up_sync(0xffffffffu, incl, 1);
  if (lane == 0) prev = 0;
  bool bad = false;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < n) {
      const uint32_t v = in[e];
      const uint32_t c = max(prev, v < cap ? v : cap);
      out[e] = c;
      bad |= c != v;
      prev = c;
    }
  }
  return __any_sync(0xffffffffu, bad);
}

// Records the first device-side error in a workspace status word.
__device__ __forceinline__ void set_status(uint32_t* status, uint32_t code) {
  if (status) atomicCAS(status, 0u, code);
}

}  // namespace moe
