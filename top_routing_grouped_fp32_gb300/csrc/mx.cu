// mx.cu -- rows to microscaled (MX) form and back (the format: mx.cuh), and the
// re-ordering of scale bytes for the block-scaled products (gemm_mx4.cu).
//
// Each of these kernels is bound by memory: every input is read once and every
// output written once, a few operations a value between.  Where rows are whole
// blocks and the pointers are aligned, blocks lie one behind the other in all
// three tensors and rows do not matter: four lanes share a block (8 values
// each), a warp holds 32 blocks.  Other rows take a lane per value.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace moe {
namespace {

// 8 consecutive values as FP32 (16-byte aligned)
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* v) {
  if constexpr (sizeof(T) == 4) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    unpack8<T>(*reinterpret_cast<const uint4*>(p), v);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* v) {
  if constexpr (sizeof(T) == 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(p) = pack8<T>(v);
  }
}

__device__ __forceinline__ uint32_t max8(const float* v) {
  uint32_t a = mx::abs_bits(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) a = max(a, mx::abs_bits(v[i]));
  return a;
}
// 8 values over the scale of byte b, as elements (uint32 for e2m1, uint2 for e4m3)
template <int FMT>
__device__ __forceinline__ uint2 encode8(const float* v, uint32_t b) {
  const float inv = mx::inverse_scale(b);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = b == 255u ? 0.f : v[i] * inv;
  if constexpr (FMT == MOE_MXFP4) return make_uint2(mx::to_e2m1x8(q), 0u);
  else return make_uint2(mx::to_e4m3x4(q), mx::to_e4m3x4(q + 4));
}

// N blocks with a lane per value (v[u] of block u): each largest magnitude goes to
// a lane of its own, so that the scales are worked out once for all of them; put(u,
// byte) stores this lane's element of block u (of e2m1 its pair with the next
// lane's).  Returns the scale byte of block `lane`.
template <int FMT, int N, typename Put>
__device__ __forceinline__ uint32_t encode_blocks(float* v, int lane, Put put) {
  uint32_t a = 0;
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, mx::abs_bits(v[u]));
    if (lane == u) a = m;
  }
  const uint32_t sb = mx::scale_byte<FMT>(a);
  const float inv = mx::inverse_scale(sb);
  if (__any_sync(0xffffffffu, sb == 255u)) {
#pragma unroll
    for (int u = 0; u < N; ++u)
      if (__shfl_sync(0xffffffffu, sb, u) == 255u) v[u] = 0.f;
  }
#pragma unroll
  for (int u = 0; u < N; u += 2) {
    const float q0 = v[u] * __shfl_sync(0xffffffffu, inv, u), q1 = v[u + 1] * __shfl_sync(0xffffffffu, inv, u + 1);
    if constexpr (FMT == MOE_MXFP8) {
      uint32_t two;
      asm("{\n\t.reg .b16 a;\n\tcvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\tcvt.u32.u16 %0, a;\n\t}" : "=r"(two) : "f"(q0), "f"(q1));
      put(u, two & 0xFFu);
      put(u + 1, two >> 8);
    } else {
      const float n0 = __shfl_down_sync(0xffffffffu, q0, 1), n1 = __shfl_down_sync(0xffffffffu, q1, 1);
      uint32_t two;
      asm("{\n\t.reg .b8 a, b, z;\n\tcvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
          "mov.b32 %0, {a, b, a, b};\n\t}"
          : "=r"(two)
          : "f"(q0), "f"(n0), "f"(q1), "f"(n1));
      put(u, two & 0xFFu);
      put(u + 1, two >> 8 & 0xFFu);
    }
  }
  return sb;
}
// The values of two blocks: q0, q1 the bytes that hold this lane's elements
template <int FMT>
__device__ __forceinline__ float2 decode_pair(uint32_t q0, uint32_t q1, int lane) {
  uint32_t h;
  if constexpr (FMT == MOE_MXFP8) {
    asm("{\n\t.reg .b16 a;\n\tcvt.u16.u32 a, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(h) : "r"(q0 | q1 << 8));
  } else {
    const int s = 4 * (lane & 1);
    const uint32_t both4 = (q0 >> s & 15u) | (q1 >> s & 15u) << 4;
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h) : "r"(both4));
  }
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The bits of the largest magnitude, as FP32, of a block that four lanes hold 8
// 16-bit values of each: two values an instruction; NaN wins.
template <typename T>
__device__ __forceinline__ uint32_t block_max(uint4 raw) {
  using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
  auto two = [](uint32_t w) {
    w &= 0x7FFF7FFFu;
    return *reinterpret_cast<T2*>(&w);
  };
  T2 m = __hmax2_nan(__hmax2_nan(two(raw.x), two(raw.y)), __hmax2_nan(two(raw.z), two(raw.w)));
  m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = __hmax2_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
  return max(mx::abs_bits(to_f32<T>(m.x)), mx::abs_bits(to_f32<T>(m.y)));
}

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// whole blocks: warp w takes blocks 32 w .. 32 w + 31 (1024 values), four loads
// of 8 values a lane in flight
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads)
mx_quantize_blocks(const T* __restrict__ x, int64_t blocks, uint8_t* __restrict__ values,
                   uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int64_t b0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * 32;
  if (b0 >= blocks) return;
  const int64_t n8 = blocks * 4;        // groups of 8 values
  const int64_t g0 = b0 * 4 + lane;
  float v[4][8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t g = g0 + 32 * j;
    if (g < n8) load8(x + g * 8, v[j]);
    else
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
  }
  uint32_t mine = 0;  // the byte of block b0 + lane
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t a = max8(v[j]);
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    const uint32_t b = mx::scale_byte<FMT>(a);
    const int64_t g = g0 + 32 * j;
    const uint2 q = encode8<FMT>(v[j], b);
    if (g < n8) {
      if constexpr (FMT == MOE_MXFP4) reinterpret_cast<uint32_t*>(values)[g] = q.x;
      else reinterpret_cast<uint2*>(values)[g] = q;
    }
    const uint32_t o = __shfl_sync(0xffffffffu, b, (lane & 7) * 4);
    if (lane >> 3 == j) mine = o;
  }
  if (b0 + lane < blocks) scales[b0 + lane] = (uint8_t)mine;
}

// Any row length and alignment, long rows: a warp per row and kSegment columns, a
// lane per value of a block, all blocks in flight.
constexpr int kSegBlocks = 16, kSegment = 32 * kSegBlocks;
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads)
mx_quantize_segments(const T* __restrict__ x, int64_t R, int64_t C, int segs, uint8_t* __restrict__ values,
                 uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t r = w / segs;
  if (r >= R) return;
  const int64_t c0 = (w - r * segs) * kSegment;
  const int64_t nb = (C + 31) / 32;
  const T* xr = x + r * C + c0;
  uint8_t* sr = scales + r * nb + c0 / 32;
  uint8_t* vr = values + (FMT == MOE_MXFP4 ? r * ((C + 1) / 2) + c0 / 2 : r * C + c0);
  const int left = (int)min((int64_t)kSegment, C - c0);
  float v[kSegBlocks];
#pragma unroll
  for (int u = 0; u < kSegBlocks; ++u) v[u] = u * 32 + lane < left ? to_f32<T>(xr[u * 32 + lane]) : 0.f;
  const uint32_t mine = encode_blocks<FMT, kSegBlocks>(v, lane, [&](int u, uint32_t byte) {
    const int c = u * 32 + lane;
    if constexpr (FMT == MOE_MXFP8) {
      if (c < left) vr[c] = (uint8_t)byte;
    } else {
      if (c < left && (lane & 1) == 0) vr[c >> 1] = (uint8_t)byte;
    }
  });
  if (lane < kSegBlocks && lane * 32 < left) sr[lane] = (uint8_t)mine;
}

// Any row length and alignment, short rows: a warp takes kRun blocks, one behind
// the other through the rows, a lane per value, all blocks in flight.  Lane u
// looks block u up.
constexpr int kRun = 16;
// Segments that are mostly full are faster (4097 rows of 1001 FP16 values to 8
// bits and back in 8194 rows: 15 against 21 us), short rows leave most of one empty
// (1027166 rows of 102 FP32 values to 4 bits and back: 594 against 384 us, both
// before the scales of a run were worked out together; 304 us now).
__host__ inline bool long_rows(int64_t C) { return C > kSegment * 5 / 8; }
__device__ __forceinline__ int64_t shfl64(int64_t v, int u) {
  return __shfl_sync(0xffffffffu, (long long)v, u);
}
// row and block-in-row of block i of rows of nb blocks
__device__ __forceinline__ void place_of(int64_t i, int64_t nb, int64_t* row, int64_t* blk) {
  *row = i < ((int64_t)1 << 32) ? (int64_t)((uint32_t)i / (uint32_t)nb) : i / nb;
  *blk = i - *row * nb;
}

template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads)
mx_quantize_rows(const T* __restrict__ x, int64_t blocks, int64_t C, uint8_t* __restrict__ values,
                 uint8_t* __restrict__ scales) {
  const int lane = threadIdx.x & 31;
  const int64_t b0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRun;
  if (b0 >= blocks) return;
  const int64_t nb = (C + 31) / 32;
  int64_t r, b;
  place_of(min(b0 + (lane & (kRun - 1)), blocks - 1), nb, &r, &b);
  const int64_t in = r * C + b * 32;
  const int64_t at = FMT == MOE_MXFP4 ? r * ((C + 1) / 2) + b * 16 : in;
  const int left = (int)min(C - b * 32, (int64_t)32);
  const int n = (int)min((int64_t)kRun, blocks - b0);
  float v[kRun];
#pragma unroll
  for (int u = 0; u < kRun; ++u) {
    const int64_t p = shfl64(in, u);
    const int l = __shfl_sync(0xffffffffu, left, u);
    v[u] = u < n && lane < l ? to_f32<T>(x[p + lane]) : 0.f;
  }
  const uint32_t mine = encode_blocks<FMT, kRun>(v, lane, [&](int u, uint32_t byte) {
    const int64_t p = shfl64(at, u);
    const int l = __shfl_sync(0xffffffffu, left, u);
    if constexpr (FMT == MOE_MXFP8) {
      if (u < n && lane < l) values[p + lane] = (uint8_t)byte;
    } else {
      if (u < n && lane < l && (lane & 1) == 0) values[p + (lane >> 1)] = (uint8_t)byte;
    }
  });
  if (lane < n) scales[b0 + lane] = (uint8_t)mine;
}

template <int FMT>
__device__ __forceinline__ void decode8(const uint8_t* values, int64_t g, uint32_t b, float* v) {
  if constexpr (FMT == MOE_MXFP4) {
    mx::from_e2m1x8(__ldg(reinterpret_cast<const uint32_t*>(values) + g), v);
  } else {
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(values) + g);
    mx::from_e4m3x4(q.x, v);
    mx::from_e4m3x4(q.y, v + 4);
  }
  const float s = mx::scale_value(b);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= s;
}

// whole blocks, in order: four groups of 8 values a lane
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads)
mx_dequantize_blocks(const uint8_t* __restrict__ values, const uint8_t* __restrict__ scales, int64_t blocks,
                     T* __restrict__ out) {
  const int64_t n8 = blocks * 4;
  const int64_t g0 = (int64_t)blockIdx.x * kThreads * 4 + threadIdx.x;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int64_t g = g0 + (int64_t)kThreads * j;
    if (g < n8) {
      float v[8];
      decode8<FMT>(values, g, __ldg(scales + (g >> 2)), v);
      store8(out + g * 8, v);
    }
  }
}

// rows of whole blocks through a dispatch map: output row r is row perm[r] / k,
// zero where perm[r] names none
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads)
mx_dequantize_gather(const uint8_t* __restrict__ values, const uint8_t* __restrict__ scales, int64_t R, int64_t C,
                     const uint32_t* __restrict__ perm, uint32_t k, int64_t n, T* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const int64_t r = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (r >= n) return;
  const int64_t src = (int64_t)(__ldg(perm + r) / k);
  const int64_t g8 = C / 8;
  T* o = out + r * C;
  if (src >= R) {
    const float z[8] = {};
    for (int64_t g = lane; g < g8; g += 32) store8(o + g * 8, z);
    return;
  }
#pragma unroll 4
  for (int64_t g = lane; g < g8; g += 32) {
    float v[8];
    decode8<FMT>(values, src * g8 + g, __ldg(scales + src * (C / 32) + (g >> 2)), v);
    store8(o + g * 8, v);
  }
}

// any row length and alignment, with or without a map: as mx_quantize_rows
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads)
mx_dequantize_rows(const uint8_t* __restrict__ values, const uint8_t* __restrict__ scales, int64_t R, int64_t C,
                   const uint32_t* __restrict__ perm, uint32_t k, int64_t blocks, T* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const int64_t b0 = ((int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRun;
  if (b0 >= blocks) return;
  const int64_t nb = (C + 31) / 32;
  int64_t r, b;
  place_of(min(b0 + (lane & (kRun - 1)), blocks - 1), nb, &r, &b);
  const int64_t src = perm ? (int64_t)(__ldg(perm + r) / k) : r;
  const int left = (int)min(C - b * 32, (int64_t)32);
  const int held = src < R ? left : 0;  // values to read
  const int64_t at = FMT == MOE_MXFP4 ? src * ((C + 1) / 2) + b * 16 : src * C + b * 32;
  const int64_t to = r * C + b * 32;
  const float mine = mx::scale_value(src < R ? (uint32_t)__ldg(scales + src * nb + b) : 0u);
  const int n = (int)min((int64_t)kRun, blocks - b0);
  uint32_t q[kRun];
#pragma unroll
  for (int u = 0; u < kRun; ++u) {
    const int64_t p = shfl64(at, u);
    const int l = __shfl_sync(0xffffffffu, held, u);
    q[u] = u < n && lane < l ? (uint32_t)__ldg(values + p + (FMT == MOE_MXFP4 ? lane >> 1 : lane)) : 0u;
  }
#pragma unroll
  for (int u = 0; u < kRun; u += 2) {
    const float2 v = decode_pair<FMT>(q[u], q[u + 1], lane);
    const float f[2] = {v.x, v.y};
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float s = __shfl_sync(0xffffffffu, mine, u + w);
      const int64_t p = shfl64(to, u + w);
      const int l = __shfl_sync(0xffffffffu, left, u + w);
      if (u + w < n && lane < l) out[p + lane] = from_f32<T>(f[w] * s);
    }
  }
}

// the same of long rows, as mx_quantize_segments
template <typename T, int FMT>
__global__ void __launch_bounds__(kThreads)
mx_dequantize_segments(const uint8_t* __restrict__ values, const uint8_t* __restrict__ scales, int64_t R, int64_t C,
                   int segs, const uint32_t* __restrict__ perm, uint32_t k, int64_t n, T* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t r = w / segs;
  if (r >= n) return;
  const int64_t c0 = (w - r * segs) * kSegment;
  const int64_t src = perm ? (int64_t)(__ldg(perm + r) / k) : r;
  const int left = src < R ? (int)min((int64_t)kSegment, C - c0) : 0;  // values to read
  const int64_t nb = (C + 31) / 32;
  const uint8_t* vr = values + (FMT == MOE_MXFP4 ? src * ((C + 1) / 2) + c0 / 2 : src * C + c0);
  uint32_t q[kSegBlocks];
#pragma unroll
  for (int u = 0; u < kSegBlocks; ++u) {
    const int c = u * 32 + lane;
    q[u] = c < left ? (uint32_t)__ldg(vr + (FMT == MOE_MXFP4 ? c >> 1 : c)) : 0u;
  }
  // lane u: the scale of block u
  const float mine = mx::scale_value(lane * 32 < left ? (uint32_t)__ldg(scales + src * nb + c0 / 32 + lane) : 0u);
  T* o = out + r * C + c0;
  const int end = (int)min((int64_t)kSegment, C - c0);
#pragma unroll
  for (int u = 0; u < kSegBlocks; u += 2) {
    const float2 v = decode_pair<FMT>(q[u], q[u + 1], lane);
    const float s0 = __shfl_sync(0xffffffffu, mine, u), s1 = __shfl_sync(0xffffffffu, mine, u + 1);
    if (u * 32 + lane < end) o[u * 32 + lane] = from_f32<T>(v.x * s0);
    if (u * 32 + 32 + lane < end) o[u * 32 + 32 + lane] = from_f32<T>(v.y * s1);
  }
}

// ---- activations of the 4-bit products ---------------------------------------
// 256-row units of experts < e (ceil per expert): where expert e's scales begin.
// One block; s_off [E+1] is filled, s_unit [E+1] written.
__device__ __forceinline__ void unit_starts(const uint32_t* s_off, int E, uint32_t* s_unit) {
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x, per = (E + 31) / 32;
    uint32_t loc = 0;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < E) loc += (s_off[e + 1] - s_off[e] + 255u) >> 8;
    }
    uint32_t incl = loc;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    uint32_t run = incl - loc;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < E) {
        s_unit[e] = run;
        run += (s_off[e + 1] - s_off[e] + 255u) >> 8;
      }
    }
    if (lane == 31) s_unit[E] = incl;
  }
}

constexpr int kSmallSlots = 256;

// Rows of C values (C a multiple of 32) to e2m1 in dispatch order, scales in
// the order of the products.  A warp takes 1024 columns of a source row at a
// time, 8 values a lane, and asks for its next ones before these are rounded;
// neighbouring warps take a row's neighbouring columns, so that a few long rows
// spread over the SMs too.  A block makes its table of expert starts once and takes
// many rows.  With slot_row, source row t goes to the dispatch rows
// slot_row[t k + j]: a token is read and rounded once however many experts it
// goes to.
// kDispatch: dispatch too, for batches of at most kSmallSlots slots: every block
// sorts the slots idx [rows, k] itself (a count, a scan, and for each slot the
// number of equal experts before it, so in the order of moe_dispatch) and the
// first one writes offsets and perm.  A decode step is a chain of short
// kernels; this takes two out of it (27.5 -> 23.6 us for one token over 64
// experts of 2048 x 1408, replayed from a graph).
// kOrder: rows in order, the caller's offsets checked by every block for itself.
enum Rows { kSlots = 0, kOrder = 1, kDispatch = 2 };
struct RowsArgs {
  const uint32_t* idx;  // kDispatch
  uint32_t* offsets;    // kDispatch, kOrder: written
  uint32_t* perm;       // kDispatch
  uint32_t* status;     // kDispatch, kOrder
};
template <typename T, int ROWS>
__global__ void __launch_bounds__(kThreads, 4)
mx4_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t C, const uint32_t* __restrict__ slot_row, int k,
                const uint32_t* __restrict__ offsets, int E, uint8_t* __restrict__ values,
                uint8_t* __restrict__ scales, const RowsArgs ra) {
  extern __shared__ uint32_t s_mem[];
  uint32_t* s_off = s_mem;
  uint32_t* s_unit = s_mem + E + 1;
  uint32_t* s_expert = s_unit + E + 1;     // kDispatch
  uint32_t* s_row = s_expert + kSmallSlots;
  const int lane = threadIdx.x & 31;
  const int64_t vb = C / 2;
  const int chunks = (int)((C + 1023) / 1024);
  // this warp's row and part of it, and the step to its next ones
  const uint32_t warps = gridDim.x * kWarps, w0 = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t step_row = warps / (uint32_t)chunks;
  const int step_chunk = (int)(warps % (uint32_t)chunks);
  int64_t src = w0 / (uint32_t)chunks;
  int chunk = (int)(w0 % (uint32_t)chunks);
  uint4 raw[4];
  auto load = [&](int64_t row, int chunk) {
    const T* p = x + row * C + (int64_t)chunk * 1024;
    const int left = (int)(C - (int64_t)chunk * 1024);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int c = u * 256 + lane * 8;
      raw[u] = c < left ? *reinterpret_cast<const uint4*>(p + c) : make_uint4(0u, 0u, 0u, 0u);
    }
  };
  pdl_wait();
  pdl_trigger();
  if (src < rows) load(src, chunk);
  if constexpr (ROWS == kDispatch) {
    static_assert(kSmallSlots <= kThreads, "a thread per slot");
    const int n = (int)rows * k, i = threadIdx.x;
    // counts one place up, so that their running sum is the offsets
    for (int e = i; e <= E; e += kThreads) s_off[e] = 0;
    const uint32_t mine = i < n ? min(ra.idx[i], (uint32_t)(E - 1)) : 0u;
    if (i < n) s_expert[i] = mine;
    __syncthreads();
    if (i < n) atomicAdd(&s_off[mine + 1], 1u);
    uint32_t before = 0;
    for (int j = 0; j < i && i < n; ++j) before += s_expert[j] == mine ? 1u : 0u;
    __syncthreads();
    if (i < 32) {  // running sum of the counts, in runs of consecutive experts a lane
      const int per = (E + 32) / 32;
      uint32_t loc = 0;
      for (int q = 0; q < per; ++q)
        if (i * per + q <= E) loc += s_off[i * per + q];
      uint32_t incl = loc;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
        if (i >= d) incl += o;
      }
      uint32_t run = incl - loc;
      for (int q = 0; q < per; ++q) {
        const int e = i * per + q;
        if (e <= E) {
          run += s_off[e];
          s_off[e] = run;
        }
      }
    }
    __syncthreads();
    if (i < n) s_row[i] = s_off[mine] + before;
    if (blockIdx.x == 0) {
      for (int e = i; e <= E; e += kThreads) ra.offsets[e] = s_off[e];
      if (i < n) ra.perm[s_off[mine] + before] = (uint32_t)i;
      if (i == 0) *ra.status = 0u;
    }
  } else if constexpr (ROWS == kOrder) {
    if (threadIdx.x < 32) {
      const bool bad = clamp_offsets(offsets, E, rows, s_off);
      if (blockIdx.x == 0 && lane == 0) *ra.status = bad ? (uint32_t)MOE_ERR_INVALID_INDEX : 0u;
    }
    __syncthreads();
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i <= E; i += kThreads) ra.offsets[i] = s_off[i];
  } else {
    for (int i = threadIdx.x; i <= E; i += kThreads) s_off[i] = offsets[i];
    __syncthreads();
  }
  unit_starts(s_off, E, s_unit);
  __syncthreads();
  const uint32_t first = s_off[0], last = s_off[E];
  const int64_t spans = mx::spans(C);
  while (src < rows) {
    uint4 cur[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) cur[u] = raw[u];
    int64_t next = src + step_row;
    int next_chunk = chunk + step_chunk;
    if (next_chunk >= chunks) {
      next_chunk -= chunks;
      ++next;
    }
    if (next < rows) load(next, next_chunk);
    uint32_t q[4], w[8];  // w: the chunk's two spans of scales
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t b = mx::scale_byte<MOE_MXFP4>(block_max<T>(cur[u]));
      // (a block with a NaN has scale NaN; its elements then do not matter)
      const float2 inv = both(mx::inverse_scale(b));
      float v[8];
      unpack8<T>(cur[u], v);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = mul2(make_float2(v[2 * i], v[2 * i + 1]), inv);
        v[2 * i] = y.x;
        v[2 * i + 1] = y.y;
      }
      q[u] = mx::to_e2m1x8(v);
      uint32_t word = b << (8 * ((lane >> 2) & 3));  // four blocks of 16 lanes in one word
      word |= __shfl_xor_sync(0xffffffffu, word, 4);
      word |= __shfl_xor_sync(0xffffffffu, word, 8);
      w[2 * u] = word;
      w[2 * u + 1] = __shfl_xor_sync(0xffffffffu, word, 16);
    }
    const int left = (int)(C - (int64_t)chunk * 1024);
    for (int j = 0; j < k; ++j) {
      uint32_t r;
      int e;
      if constexpr (ROWS == kDispatch) {
        r = s_row[src * k + j];
        e = (int)s_expert[src * k + j];
      } else {
        r = ROWS == kSlots ? __ldg(slot_row + src * k + j) : (uint32_t)src;
        if (r < first || r >= last) continue;
        e = warp_search(s_off, E, r);
      }
      const uint32_t local = r - s_off[e];
      uint8_t* vr = values + (int64_t)r * vb + (int64_t)chunk * 512;
      uint8_t* sr = scales +
                    (((int64_t)(s_unit[e] + (local >> 8)) * spans + 2 * chunk) * mx::kUnitGroups + (local >> 5 & 7u)) *
                        mx::kGroupBytes +
                    (local & 31u) * 16;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = u * 256 + lane * 8;
        if (c < left) *reinterpret_cast<uint32_t*>(vr + c / 2) = q[u];
      }
      if (lane == 0) {
        *reinterpret_cast<uint4*>(sr) = make_uint4(w[0], w[1], w[2], w[3]);
        if (left > 512)
          *reinterpret_cast<uint4*>(sr + mx::kUnitGroups * mx::kGroupBytes) = make_uint4(w[4], w[5], w[6], w[7]);
      }
    }
    src = next;
    chunk = next_chunk;
  }
}

// Weight scales [E, rows, C/32] in the order of the products (rows a multiple
// of 32): a thread per row and span.
__global__ void __launch_bounds__(kThreads)
mx4_weight_scales_kernel(const uint8_t* __restrict__ scales, int64_t E, int64_t rows, int64_t nb, int64_t spans,
                         uint4* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= E * rows * spans) return;
  const int64_t r = i % rows, span = i / rows % spans, e = i / rows / spans;
  const uint8_t* s = scales + (e * rows + r) * nb;
  uint32_t w[4] = {};
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    const uint32_t b = span * 16 + c < nb ? s[span * 16 + c] : 127u;
    w[c >> 2] |= b << (8 * (c & 3));
  }
  out[i] = make_uint4(w[0], w[1], w[2], w[3]);
}

// y[t] = sum_j slots[t k + j] (FP32, ascending j), rounded once
template <typename T>
__global__ void __launch_bounds__(kThreads)
slot_sum_f32_kernel(const float* __restrict__ slots, int64_t T_, int k, int64_t H, T* __restrict__ y) {
  pdl_wait();
  pdl_trigger();
  const int64_t g8 = H / 8;
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= T_ * g8) return;
  const int64_t t = i / g8, c = (i - t * g8) * 8;
  float acc[8] = {};
  const float* s = slots + t * k * H + c;
#pragma unroll 4
  for (int j = 0; j < k; ++j, s += H) {
    float v[8];
    load8(s, v);
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] += v[q];
  }
  store8(y + t * H + c, acc);
}

template <typename T, int FMT>
cudaError_t quantize_t(const void* x, int64_t R, int64_t C, uint8_t* values, uint8_t* scales, cudaStream_t s) {
  const T* xp = static_cast<const T*>(x);
  if (C % 32 == 0 && (reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(values)) % 16 == 0) {
    const int64_t blocks = R * (C / 32);
    const int64_t grid = (blocks + 32 * kWarps - 1) / (32 * kWarps);
    mx_quantize_blocks<T, FMT><<<(unsigned)grid, kThreads, 0, s>>>(xp, blocks, values, scales);
  } else {
    const int segs = (int)((C + kSegment - 1) / kSegment);
    if (long_rows(C)) {
      mx_quantize_segments<T, FMT><<<(unsigned)((R * segs + kWarps - 1) / kWarps), kThreads, 0, s>>>(xp, R, C, segs,
                                                                                                   values, scales);
      return cudaGetLastError();
    }
    const int64_t blocks = R * ((C + 31) / 32), per = kWarps * kRun;
    mx_quantize_rows<T, FMT><<<(unsigned)((blocks + per - 1) / per), kThreads, 0, s>>>(xp, blocks, C, values, scales);
  }
  return cudaGetLastError();
}

template <typename T, int FMT>
cudaError_t dequantize_t(const uint8_t* values, const uint8_t* scales, int64_t R, int64_t C, const uint32_t* perm,
                         int k, int64_t n, void* out, cudaStream_t s) {
  T* o = static_cast<T*>(out);
  const unsigned by_row = (unsigned)((n + kWarps - 1) / kWarps);
  const bool whole = C % 32 == 0 && (reinterpret_cast<uintptr_t>(out) | reinterpret_cast<uintptr_t>(values)) % 16 == 0;
  if (whole && !perm) {
    const int64_t blocks = R * (C / 32), per = kThreads;  // 4 groups a thread, 4 groups a block
    mx_dequantize_blocks<T, FMT><<<(unsigned)((blocks + per - 1) / per), kThreads, 0, s>>>(values, scales, blocks, o);
  } else if (whole) {
    mx_dequantize_gather<T, FMT><<<by_row, kThreads, 0, s>>>(values, scales, R, C, perm, (uint32_t)k, n, o);
  } else {
    const int segs = (int)((C + kSegment - 1) / kSegment);
    if (long_rows(C)) {
      mx_dequantize_segments<T, FMT><<<(unsigned)((n * segs + kWarps - 1) / kWarps), kThreads, 0, s>>>(
          values, scales, R, C, segs, perm, (uint32_t)k, n, o);
      return cudaGetLastError();
    }
    const int64_t blocks = n * ((C + 31) / 32), per = kWarps * kRun;
    mx_dequantize_rows<T, FMT><<<(unsigned)((blocks + per - 1) / per), kThreads, 0, s>>>(values, scales, R, C, perm,
                                                                                         (uint32_t)k, blocks, o);
  }
  return cudaGetLastError();
}

}  // namespace

#define MOE_MX_DISPATCH(fn, ...)                                                                             \
  (dt == MOE_F32 ? (fmt == MOE_MXFP4 ? fn<float, MOE_MXFP4>(__VA_ARGS__) : fn<float, MOE_MXFP8>(__VA_ARGS__)) \
   : dt == MOE_F16                                                                                           \
       ? (fmt == MOE_MXFP4 ? fn<__half, MOE_MXFP4>(__VA_ARGS__) : fn<__half, MOE_MXFP8>(__VA_ARGS__))        \
       : (fmt == MOE_MXFP4 ? fn<__nv_bfloat16, MOE_MXFP4>(__VA_ARGS__) : fn<__nv_bfloat16, MOE_MXFP8>(__VA_ARGS__)))

cudaError_t launch_mx_quantize(const void* x, moe_dtype dt, int64_t R, int64_t C, moe_mx_format fmt,
                               uint8_t* values, uint8_t* scales, cudaStream_t s) {
  return MOE_MX_DISPATCH(quantize_t, x, R, C, values, scales, s);
}

cudaError_t launch_mx_dequantize(const uint8_t* values, const uint8_t* scales, moe_mx_format fmt, int64_t R,
                                 int64_t C, const uint32_t* perm, int k, int64_t n, void* out, moe_dtype dt,
                                 cudaStream_t s) {
  return MOE_MX_DISPATCH(dequantize_t, values, scales, R, C, perm, k, n, out, s);
}
#undef MOE_MX_DISPATCH

template <typename T, int ROWS>
static cudaError_t rows_t(const void* x, int64_t rows, int64_t C, const uint32_t* slot_row, int k,
                          const uint32_t* offsets, int E, uint8_t* values, uint8_t* scales, const RowsArgs& ra,
                          int num_sms, cudaStream_t s) {
  // four blocks stay on an SM
  const int64_t items = rows * ((C + 1023) / 1024);
  const unsigned grid = (unsigned)std::min<int64_t>((items + kWarps - 1) / kWarps, (int64_t)num_sms * 4);
  const size_t smem = 4 * (2 * (size_t)(E + 1) + (ROWS == kDispatch ? 2 * kSmallSlots : 0));
  return launch_pdl(mx4_rows_kernel<T, ROWS>, dim3(grid), dim3(kThreads), smem, s, static_cast<const T*>(x), rows, C,
                    slot_row, k, offsets, E, values, scales, ra);
}

cudaError_t launch_mx4_rows(const void* x, moe_dtype dt, int64_t rows, int64_t C, const uint32_t* slot_row, int k,
                            const uint32_t* offsets, int E, uint32_t* off_ok, uint32_t* status, uint8_t* values,
                            uint8_t* scales, int num_sms, cudaStream_t s) {
  const RowsArgs ra{nullptr, off_ok, nullptr, status};
  if (slot_row)
    return dt == MOE_BF16
               ? rows_t<__nv_bfloat16, kSlots>(x, rows, C, slot_row, k, offsets, E, values, scales, ra, num_sms, s)
               : rows_t<__half, kSlots>(x, rows, C, slot_row, k, offsets, E, values, scales, ra, num_sms, s);
  return dt == MOE_BF16 ? rows_t<__nv_bfloat16, kOrder>(x, rows, C, nullptr, 1, offsets, E, values, scales, ra, num_sms, s)
                        : rows_t<__half, kOrder>(x, rows, C, nullptr, 1, offsets, E, values, scales, ra, num_sms, s);
}

int64_t mx4_small_slots() { return kSmallSlots; }

cudaError_t launch_mx4_dispatch_rows(const void* x, moe_dtype dt, int64_t T, int64_t C, const uint32_t* idx, int k,
                                     int E, uint32_t* offsets, uint32_t* perm, uint32_t* status, uint8_t* values,
                                     uint8_t* scales, int num_sms, cudaStream_t s) {
  if (T * k > kSmallSlots) return cudaErrorInvalidValue;
  const RowsArgs ra{idx, offsets, perm, status};
  return dt == MOE_BF16 ? rows_t<__nv_bfloat16, kDispatch>(x, T, C, nullptr, k, nullptr, E, values, scales, ra, num_sms, s)
                        : rows_t<__half, kDispatch>(x, T, C, nullptr, k, nullptr, E, values, scales, ra, num_sms, s);
}

cudaError_t launch_mx4_weight_scales(const uint8_t* scales, int64_t E, int64_t rows, int64_t C, uint8_t* out,
                                     cudaStream_t s) {
  const int64_t spans = mx::spans(C), n = E * rows * spans;
  mx4_weight_scales_kernel<<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, s>>>(scales, E, rows, C / 32, spans,
                                                                                         reinterpret_cast<uint4*>(out));
  return cudaGetLastError();
}

cudaError_t launch_slot_sum_f32(const float* slots, int64_t T, int k, int64_t H, void* y, moe_dtype dt,
                                cudaStream_t s) {
  const unsigned grid = (unsigned)((T * (H / 8) + kThreads - 1) / kThreads);
  return dt == MOE_BF16 ? launch_pdl(slot_sum_f32_kernel<__nv_bfloat16>, dim3(grid), dim3(kThreads), 0, s, slots, T,
                                     k, H, static_cast<__nv_bfloat16*>(y))
                        : launch_pdl(slot_sum_f32_kernel<__half>, dim3(grid), dim3(kThreads), 0, s, slots, T, k, H,
                                     static_cast<__half*>(y));
}

}  // namespace moe
