// rowpad.cu -- the 64-padded row space of the tensor-core expert backward
// (ExpertTrainingCache::backward in src/moe/experts.rs), and the check of the
// offsets a caller passes to the staged expert calls.
//
// The weight gradients are per-expert sums over that expert's dispatched
// rows.  The tcgen05 engine reads them 64 rows per k-block; if each expert's
// rows start on a multiple of 64 and are followed by zero rows up to the next
// multiple, no k-block mixes two experts and the zero rows add nothing:
//
//  * pad_offsets: pad[e] = sum_{e' < e} roundup(count_e', 64), pad[E] the total;
//  * pad_rows: dst row pad[e] + j = src row offsets[e] + j for j < count_e,
//    zero for count_e <= j < pad[e+1] - pad[e]  (rows of C 16-bit elements,
//    C a multiple of 8, copied in 16-byte vectors: one warp per row).
#include "common.cuh"
#include "internal.h"
#include "mx.cuh"

namespace moe {
namespace {

__device__ __forceinline__ void pad_starts(const uint32_t* offsets, int E, uint32_t* pad) {
  // one warp: per-lane serial sums, then a warp scan (E <= 1024)
  const int lane = threadIdx.x;
  const int per = (E + 31) / 32;
  uint32_t loc = 0;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < E) loc += (offsets[e + 1] - offsets[e] + 63u) & ~63u;
  }
  uint32_t incl = loc;
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  uint32_t run = incl - loc;
  for (int i = 0; i < per; ++i) {
    const int e = lane * per + i;
    if (e < E) {
      pad[e] = run;
      run += (offsets[e + 1] - offsets[e] + 63u) & ~63u;
    }
  }
  if (lane == 31) pad[E] = incl;
}
__global__ void pad_offsets_kernel(const uint32_t* __restrict__ offsets, int E, uint32_t* __restrict__ pad) {
  pad_starts(offsets, E, pad);
}

// The offsets of a staged expert call as its kernels read them (clamp_offsets);
// a clamped entry marks the status word MOE_ERR_INVALID_INDEX.  One warp.
__global__ void sanitize_offsets_kernel(const uint32_t* __restrict__ in, int E, int64_t N,
                                        uint32_t* __restrict__ out, uint32_t* __restrict__ status) {
  if (clamp_offsets(in, E, N, out) && threadIdx.x == 0) set_status(status, (uint32_t)MOE_ERR_INVALID_INDEX);
}

// The same, the status word's first value and, with pad, where each expert's
// rows begin in the 64-padded row space, in one launch.
__global__ void check_offsets_kernel(const uint32_t* __restrict__ in, int E, int64_t N, uint32_t* __restrict__ out,
                                     uint32_t* __restrict__ status, uint32_t* __restrict__ pad) {
  const bool bad = clamp_offsets(in, E, N, out);
  if (threadIdx.x == 0) *status = bad ? (uint32_t)MOE_ERR_INVALID_INDEX : 0u;
  __syncwarp();
  if (pad) pad_starts(out, E, pad);
}

constexpr int kRowsPerBlock = 8;  // one warp per row

__global__ void __launch_bounds__(32 * kRowsPerBlock)
pad_rows_kernel(const uint4* __restrict__ src, int64_t vecs, const uint32_t* __restrict__ offsets,
                const uint32_t* __restrict__ pad, int E, uint4* __restrict__ dst) {
  const int64_t j = (int64_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5);  // padded row
  const int lane = threadIdx.x & 31;
  if (j >= (int64_t)pad[E]) return;
  int lo = 0, hi = E;  // pad[lo] <= j < pad[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)pad[mid] <= j) lo = mid; else hi = mid;
  }
  const int64_t r = (int64_t)offsets[lo] + (j - (int64_t)pad[lo]);
  uint4* d = dst + j * vecs;
  if (r < (int64_t)offsets[lo + 1]) {
    const uint4* s = src + r * vecs;
    for (int64_t v = lane; v < vecs; v += 32) d[v] = __ldg(s + v);
  } else {
    for (int64_t v = lane; v < vecs; v += 32) d[v] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// The last count_e % 64 rows of every expert's segment: dst row 64 e + j, zeros
// behind them (rows of C 16-bit elements, one warp per row).
__global__ void __launch_bounds__(32 * kRowsPerBlock)
tail_rows_kernel(const uint4* __restrict__ src, int64_t vecs, const uint32_t* __restrict__ offsets, int E,
                 uint4* __restrict__ dst) {
  const int row = blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, e = row >> 6, j = row & 63;
  if (e >= E) return;
  const uint32_t end = offsets[e + 1];
  const int tail = (int)((end - offsets[e]) & 63u);
  if (tail == 0) return;  // not read
  uint4* d = dst + (int64_t)row * vecs;
  if (j < tail) {
    const uint4* s = src + ((int64_t)end - tail + j) * vecs;
    for (int64_t v = lane; v < vecs; v += 32) d[v] = __ldg(s + v);
  } else {
    for (int64_t v = lane; v < vecs; v += 32) d[v] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// pad_rows of 8-bit tokens (e4m3, a scale a 32-column block), read through the
// dispatch map and written as T: a warp per row, 8 values a lane.
template <typename T>
__global__ void __launch_bounds__(32 * kRowsPerBlock)
pad_rows_mx8_kernel(const uint2* __restrict__ x, const uint8_t* __restrict__ scales, int64_t tokens, int64_t vecs,
                    const uint32_t* __restrict__ perm, uint32_t k, const uint32_t* __restrict__ offsets,
                    const uint32_t* __restrict__ pad, int E, uint4* __restrict__ dst) {
  const int64_t j = (int64_t)blockIdx.x * kRowsPerBlock + (threadIdx.x >> 5);  // padded row
  const int lane = threadIdx.x & 31;
  if (j >= (int64_t)pad[E]) return;
  int lo = 0, hi = E;  // pad[lo] <= j < pad[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((int64_t)pad[mid] <= j) lo = mid; else hi = mid;
  }
  const int64_t r = (int64_t)offsets[lo] + (j - (int64_t)pad[lo]);
  uint4* d = dst + j * vecs;
  int64_t t = tokens;
  if (r < (int64_t)offsets[lo + 1]) t = (int64_t)(__ldg(perm + r) / k);
  if (t < tokens) {
    const uint2* s = x + t * vecs;
    const uint8_t* sc = scales + t * ((vecs + 3) / 4);
#pragma unroll 4
    for (int64_t v = lane; v < vecs; v += 32) {
      const uint2 q = __ldg(s + v);
      const float f = mx::scale_value(__ldg(sc + (v >> 2)));
      float o[8];
      mx::from_e4m3x4(q.x, o);
      mx::from_e4m3x4(q.y, o + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] *= f;
      d[v] = pack8<T>(o);
    }
  } else {
    for (int64_t v = lane; v < vecs; v += 32) d[v] = make_uint4(0u, 0u, 0u, 0u);
  }
}

// out[e, i] = sum over the parts of parts[e, part, i], in order, rounded once.
// With offsets (E = 1: rows of row_vecs vectors) only rows inside the segments.
template <typename T>
__global__ void __launch_bounds__(256)
join_parts_kernel(const float4* __restrict__ parts, int k, int64_t vecs, int64_t total,
                  const uint32_t* __restrict__ offsets, int last, int64_t row_vecs, uint4* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // 8 values
  if (i >= total) return;
  if (offsets) {
    const int64_t row = i / row_vecs;
    if (row < (int64_t)offsets[0] || row >= (int64_t)offsets[last]) return;
  }
  const int64_t e = i / vecs, v = i - e * vecs;
  const float4* s = parts + ((e * k) * vecs + v) * 2;
  float acc[8] = {};
#pragma unroll 4
  for (int j = 0; j < k; ++j, s += 2 * vecs) {
    const float4 a = __ldg(s), b = __ldg(s + 1);
    acc[0] += a.x; acc[1] += a.y; acc[2] += a.z; acc[3] += a.w;
    acc[4] += b.x; acc[5] += b.y; acc[6] += b.z; acc[7] += b.w;
  }
  out[i] = pack8<T>(acc);
}

}  // namespace

static cudaError_t join(const float* parts, int E, int k, int64_t n, const uint32_t* offsets, int last,
                        int64_t row_vecs, void* out, moe_dtype dt, cudaStream_t s) {
  const int64_t total = E * (n / 8);
  const unsigned blocks = (unsigned)((total + 255) / 256);
  const float4* p = reinterpret_cast<const float4*>(parts);
  uint4* o = static_cast<uint4*>(out);
  if (dt == MOE_BF16) join_parts_kernel<__nv_bfloat16><<<blocks, 256, 0, s>>>(p, k, n / 8, total, offsets, last, row_vecs, o);
  else join_parts_kernel<__half><<<blocks, 256, 0, s>>>(p, k, n / 8, total, offsets, last, row_vecs, o);
  return cudaGetLastError();
}

cudaError_t launch_join_parts(const float* parts, int E, int k, int64_t n, void* out, moe_dtype dt, cudaStream_t s) {
  return join(parts, E, k, n, nullptr, 0, 1, out, dt, s);
}

cudaError_t launch_join_rows(const float* parts, int k, int64_t N, int64_t H, const uint32_t* offsets, int E, void* out,
                             moe_dtype dt, cudaStream_t s) {
  return join(parts, 1, k, N * H, offsets, E, H / 8, out, dt, s);
}

cudaError_t launch_tail_rows(const void* src, int64_t C, const uint32_t* offsets, int E, void* dst, cudaStream_t s) {
  tail_rows_kernel<<<(unsigned)(E * 64 / kRowsPerBlock), 32 * kRowsPerBlock, 0, s>>>(
      static_cast<const uint4*>(src), C / 8, offsets, E, static_cast<uint4*>(dst));
  return cudaGetLastError();
}

cudaError_t launch_pad_rows_mx8(const uint8_t* x, const uint8_t* scales, int64_t T, int64_t C, const uint32_t* perm,
                                int k, const uint32_t* offsets, const uint32_t* pad, int E, int64_t npad_max,
                                void* dst, moe_dtype dt, cudaStream_t s) {
  const unsigned blocks = (unsigned)((npad_max + kRowsPerBlock - 1) / kRowsPerBlock);
  const uint2* xp = reinterpret_cast<const uint2*>(x);
  uint4* dp = static_cast<uint4*>(dst);
  if (dt == MOE_BF16)
    pad_rows_mx8_kernel<__nv_bfloat16><<<blocks, 32 * kRowsPerBlock, 0, s>>>(xp, scales, T, C / 8, perm, (uint32_t)k,
                                                                            offsets, pad, E, dp);
  else
    pad_rows_mx8_kernel<__half><<<blocks, 32 * kRowsPerBlock, 0, s>>>(xp, scales, T, C / 8, perm, (uint32_t)k, offsets,
                                                                     pad, E, dp);
  return cudaGetLastError();
}

cudaError_t launch_sanitize_offsets(const uint32_t* offsets, int E, int64_t N, uint32_t* out,
                                   uint32_t* status, cudaStream_t s) {
  sanitize_offsets_kernel<<<1, 32, 0, s>>>(offsets, E, N, out, status);
  return cudaGetLastError();
}

cudaError_t launch_check_offsets(const uint32_t* offsets, int E, int64_t N, uint32_t* out, uint32_t* status,
                                 uint32_t* pad, cudaStream_t s) {
  check_offsets_kernel<<<1, 32, 0, s>>>(offsets, E, N, out, status, pad);
  return cudaGetLastError();
}

cudaError_t launch_pad_offsets(const uint32_t* offsets, int E, uint32_t* pad, cudaStream_t s) {
  pad_offsets_kernel<<<1, 32, 0, s>>>(offsets, E, pad);
  return cudaGetLastError();
}

cudaError_t launch_pad_rows(const void* src, int64_t C, const uint32_t* offsets, const uint32_t* pad,
                            int E, int64_t npad_max, void* dst, cudaStream_t s) {
  const int64_t blocks = (npad_max + kRowsPerBlock - 1) / kRowsPerBlock;
  pad_rows_kernel<<<(unsigned)blocks, 32 * kRowsPerBlock, 0, s>>>(
      static_cast<const uint4*>(src), C / 8, offsets, pad, E, static_cast<uint4*>(dst));
  return cudaGetLastError();
}

}  // namespace moe
