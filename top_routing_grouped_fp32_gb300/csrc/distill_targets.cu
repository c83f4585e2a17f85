// distill_targets.cu -- a teacher router's top logits, with the logit of all other
// experts together, rest = tau log sum_{e not in top} exp(t_e / tau).
//
// 32 of 256 BF16 logits, 524288 rows: 213 us (268 MB read, 79 MB written).  Bound by
// issue: sorting and merging take 321 instructions a row, 2.5 a cycle of a SM.
#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

struct TargetArgs {
  const void* logits;
  int E, m, lpr;
  int64_t T;
  float tau, c;
  uint32_t* idx;
  void* top;
  float* rest;
  bool vec_out;  // rows of idx and top are whole 16- and 8-byte vectors
};

// A logit and its expert as one unsigned key: larger logit first, then the lower
// id; keys of a row differ.  Adding +0 makes -0 a +0 and a NaN the positive one,
// which lies above +inf: a row is broken where its largest key is not below +inf's.
template <typename T>
struct SortKey {  // 16-bit logits: order-preserving bits above 0xffff - id
  using Key = uint32_t;
  static constexpr uint32_t kInf = (std::is_same<T, __half>::value ? 0xfc00u : 0xff80u) << 16;
  static __device__ __forceinline__ Key make(T x, int id) {
    uint32_t b;
    if constexpr (std::is_same<T, __half>::value) b = __half_as_ushort(__hadd(x, __ushort_as_half(0)));
    else b = __float_as_uint(__bfloat162float(x) + 0.f) >> 16;
    const uint32_t o = b ^ ((b & 0x8000u) ? 0xffffu : 0x8000u);
    return (o << 16) | (0xffffu - (uint32_t)id);
  }
  static __device__ __forceinline__ bool broken(Key k) { return k >= kInf; }
  // The keys of a lane's elements: their order-preserving bits, two a word, are
  // made and joined with the ids a word at a time.
  template <int VEC, int NV>
  struct Keys {
    static constexpr int N = VEC * NV;
    uint32_t o[N > 1 ? N / 2 : 1], ids;
    int lpr, sub;
    __device__ __forceinline__ Keys(const RowRegs<T, VEC, NV>& r, int lpr_, int sub_) : lpr(lpr_), sub(sub_) {
      ids = 0u;
      if constexpr (VEC == 8) {
        ids = 0xfffeffffu - (uint32_t)(sub * VEC) * 0x10001u;  // of elements 0 and 1
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
          uint32_t w = reinterpret_cast<const uint32_t*>(r.raw)[i];
          if constexpr (std::is_same<T, __half>::value) {
            const __half2 z = __hadd2(*reinterpret_cast<__half2*>(&w), __half2(__ushort_as_half(0), __ushort_as_half(0)));
            w = *reinterpret_cast<const uint32_t*>(&z);
          } else {
            const __nv_bfloat162 z = __hadd2(*reinterpret_cast<__nv_bfloat162*>(&w),
                                             __nv_bfloat162(__ushort_as_bfloat16(0), __ushort_as_bfloat16(0)));
            w = *reinterpret_cast<const uint32_t*>(&z);
          }
          o[i] = w ^ ((w >> 15 & 0x10001u) * 0x7fffu) ^ 0x80008000u;
        }
      } else {
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const uint32_t b = make(r.raw[n], 0) >> 16;
          if (n % 2) o[n / 2] |= b << 16;
          else o[n / 2] = b;
        }
      }
    }
    __device__ __forceinline__ Key operator[](int n) const {
      if constexpr (VEC == 8)
        return __byte_perm(ids - (uint32_t)(n / 8 * lpr * 8 + n % 8 / 2 * 2) * 0x10001u, o[n / 2],
                           n % 2 ? 0x7632 : 0x5410);
      return (n % 2 ? o[n / 2] & 0xffff0000u : o[n / 2] << 16) |
             (0xffffu - (uint32_t)RowRegs<T, VEC, NV>::elem(n, lpr, sub));
    }
  };
  static __device__ __forceinline__ uint32_t id(Key k) { return 0xffffu - (k & 0xffffu); }
  static __device__ __forceinline__ T logit(Key k) {
    const uint16_t b = (uint16_t)((k >> 16) ^ ((k & 0x80000000u) ? 0x8000u : 0xffffu));
    if constexpr (std::is_same<T, __half>::value) return __ushort_as_half(b);
    else return __ushort_as_bfloat16(b);
  }
};
template <>
struct SortKey<float> {
  using Key = uint64_t;
  static __device__ __forceinline__ Key make(float x, int id) {
    const uint32_t b = __float_as_uint(x + 0.f);
    const uint32_t o = b ^ ((b & 0x80000000u) ? 0xffffffffu : 0x80000000u);
    return ((uint64_t)o << 32) | (0xffffffffu - (uint32_t)id);
  }
  static __device__ __forceinline__ bool broken(Key k) { return (uint32_t)(k >> 32) >= 0xff800000u; }
  template <int VEC, int NV>
  struct Keys {
    const RowRegs<float, VEC, NV>& r;
    int lpr, sub;
    __device__ __forceinline__ Keys(const RowRegs<float, VEC, NV>& r_, int lpr_, int sub_) : r(r_), lpr(lpr_), sub(sub_) {}
    __device__ __forceinline__ Key operator[](int n) const { return make(r.raw[n], RowRegs<float, VEC, NV>::elem(n, lpr, sub)); }
  };
  static __device__ __forceinline__ uint32_t id(Key k) { return 0xffffffffu - (uint32_t)k; }
  static __device__ __forceinline__ float logit(Key k) {
    const uint32_t o = (uint32_t)(k >> 32);
    return __uint_as_float(o ^ ((o & 0x80000000u) ? 0x80000000u : 0xffffffffu));
  }
};

// Descending order of N = 2^i keys: Batcher's odd-even merge network.
template <typename Key>
__device__ __forceinline__ void order(Key& x, Key& y) {
  const Key a = x, b = y;
  x = a > b ? a : b;
  y = a > b ? b : a;
}
template <int LO, int CNT, int GAP, typename Key, int N>
__device__ __forceinline__ void odd_even_merge(Key (&k)[N]) {
  if constexpr (2 * GAP < CNT) {
    odd_even_merge<LO, CNT, 2 * GAP>(k);
    odd_even_merge<LO + GAP, CNT, 2 * GAP>(k);
#pragma unroll
    for (int i = LO + GAP; i + GAP < LO + CNT; i += 2 * GAP) order(k[i], k[i + GAP]);
  } else {
    order(k[LO], k[LO + GAP]);
  }
}
template <int LO, int CNT, typename Key, int N>
__device__ __forceinline__ void sort_descending(Key (&k)[N]) {
  if constexpr (CNT > 1) {
    sort_descending<LO, CNT / 2>(k);
    sort_descending<LO + CNT / 2, CNT / 2>(k);
    odd_even_merge<LO, CNT, 1>(k);
  }
}

// ---- merging the lanes' lists --------------------------------------------------
// A group of S lanes holds a descending list, P keys a lane: lane a of the group has
// keys a P .. a P + P - 1.  merge() joins the lists of neighbouring groups until a
// group is a row, and keeps the K largest of a list that gets longer: bitonic
// networks over registers and shuffles, with nothing that waits for a result of
// another row.  (Rounds that each take the row's largest head wait for one another:
// 297 us where the networks took 220, for 32 of 256 BF16 logits and 524288 rows.)
template <typename Key>
__device__ __forceinline__ Key shfl_xor(Key k, int mask) { return __shfl_xor_sync(0xffffffffu, k, mask); }
template <typename Key>
__device__ __forceinline__ Key larger(Key a, Key b) { return a > b ? a : b; }
template <typename Key>
__device__ __forceinline__ Key pick(Key a, Key b, bool large) {
  const Key lo = a > b ? b : a, hi = a > b ? a : b;
  return large ? hi : lo;
}

// Descending order of a bitonic sequence over the lanes of a group (lane `a` of it,
// lanes a and a ^ d hold keys P d apart) and the lane's own P keys.
template <int S, int P, typename Key>
__device__ __forceinline__ void clean(Key (&x)[P], int a) {
#pragma unroll
  for (int d = S / 2; d > 0; d /= 2)
#pragma unroll
    for (int p = 0; p < P; ++p) x[p] = pick(x[p], shfl_xor(x[p], d), (a & d) == 0);
#pragma unroll
  for (int d = P / 2; d > 0; d /= 2)
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (!(p & d)) order(x[p], x[p + d]);
}

// `lane`: lane of the warp; `lpr`: lanes of a row.  Calls done(x, P) with the row's
// list; where K lanes hold it with a key each (P = 1), other lanes hold copies.
template <int S, int P, int K, int LPR, typename Key, typename F>
__device__ __forceinline__ void merge(const Key (&x)[P], int lane, int lpr, F done) {
  if constexpr (S == 32 || (LPR && S == LPR)) {
    done(x, lane & (S < K ? S - 1 : K - 1));
  } else {
    if (!LPR && S == lpr) {
      done(x, lane & (S < K ? S - 1 : K - 1));
      return;
    }
    const bool upper = lane & S;
    if constexpr (2 * S * P <= K) {  // the whole of both lists
      Key y[P];
#pragma unroll
      for (int p = 0; p < P; ++p) y[p] = pick(x[p], shfl_xor(x[P - 1 - p], 2 * S - 1), !upper);
      clean<S, P>(y, lane & (S - 1));
      merge<2 * S, P, K, LPR>(y, lane, lpr, done);
    } else if constexpr (P > 1) {
      // The K largest are the larger of x_i and the other's x_(K-1-i), a bitonic
      // sequence.  Lane a of the lower group takes its first P/2 keys, its mirror
      // lane the others, in descending places.
      static_assert(S * P == K, "lists of K keys");
      constexpr int H = P / 2;
      Key y[H], z[H];
#pragma unroll
      for (int p = 0; p < H; ++p) y[p] = larger(x[p], shfl_xor(x[P - 1 - p], 2 * S - 1));
#pragma unroll
      for (int p = 0; p < H; ++p) z[p] = upper ? y[H - 1 - p] : y[p];
      // place of z[p]: a P + p, or a P + H + p on the mirror lane of a
      const int a = (upper ? ~lane : lane) & (S - 1);
#pragma unroll
      for (int d = S / 2; d > 0; d /= 2)
#pragma unroll
        for (int p = 0; p < H; ++p) z[p] = pick(z[p], shfl_xor(z[p], d), (a & d) == 0);
#pragma unroll
      for (int p = 0; p < H; ++p) z[p] = pick(z[p], shfl_xor(z[p], 2 * S - 1), !upper);
#pragma unroll
      for (int d = H / 2; d > 0; d /= 2)
#pragma unroll
        for (int p = 0; p < H; ++p)
          if (!(p & d)) order(z[p], z[p + d]);
      // lane q of the joined group takes the keys from place q H on
      const int q = lane & (2 * S - 1), from = (q & 1) ? 2 * S - 1 - q / 2 : q / 2;
#pragma unroll
      for (int p = 0; p < H; ++p) z[p] = __shfl_sync(0xffffffffu, z[p], (lane & ~(2 * S - 1)) | from);
      merge<2 * S, H, K, LPR>(z, lane, lpr, done);
    } else {
      // a key a lane on K lanes, with copies on the other lanes of the group
      Key y[1] = {larger(x[0], shfl_xor(x[0], S | (K - 1)))};
      clean<K, 1>(y, lane & (K - 1));
      merge<2 * S, 1, K, LPR>(y, lane, lpr, done);
    }
  }
}

// Each lane sorts its share of the row, the lanes' lists are merged, and the rest is
// summed about the last key that was taken.
constexpr int kTargetThreads = 128;
constexpr int kTargetBlocks = 152 * 8;
template <typename T, int VEC, int NV, int LPR, int K>
__global__ void __launch_bounds__(kTargetThreads, VEC * NV * sizeof(T) <= 64 ? 4 : 2) distill_targets_kernel(TargetArgs a) {
  constexpr int W = kTargetThreads / 32;
  using Row = RowRegs<T, VEC, NV>;
  using SK = SortKey<T>;
  using Key = typename SK::Key;
  constexpr int N = Row::N, P0 = N < K ? N : K;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Lanes<LPR> L(a.lpr);
  extern __shared__ __align__(16) unsigned char smem[];
  using Stream = RowStream<T, VEC, NV, LPR>;
  Stream rows(L, smem, a.logits, a.E, a.T);
  T* top = static_cast<T*>(a.top);
  const int64_t step = (int64_t)gridDim.x * W * L.rows;
  int64_t t0 = ((int64_t)blockIdx.x * W + warp) * L.rows;
  rows.start(t0, step);
#pragma unroll
  for (int i = 0; i < Stream::kStages - 1; ++i) rows.issue(t0 + i * step + L.grp < a.T);
  for (; t0 < a.T; t0 += step) {
    Row cur;
    rows.take(cur);
    rows.issue(t0 + (Stream::kStages - 1) * step + L.grp < a.T);
    const int64_t t = t0 + L.grp;
    const bool in = t < a.T;
    typename SK::template Keys<VEC, NV> keys(cur, L.lpr, L.sub);
    Key list[N], best[P0];
#pragma unroll
    for (int n = 0; n < N; ++n) list[n] = keys[n];
    sort_descending<0, N>(list);
#pragma unroll
    for (int p = 0; p < P0; ++p) best[p] = list[p];
    merge<1, P0, K, LPR>(best, lane, L.lpr, [&](const auto& x, int q) {
      constexpr int P = sizeof(x) / sizeof(Key);
      const bool broken = SK::broken(__shfl_sync(0xffffffffu, x[0], L.grp * L.lpr));
      Key last = x[0];
#pragma unroll
      for (int p = 1; p < P; ++p)
        if (p == (a.m - 1) % P) last = x[p];
      last = __shfl_sync(0xffffffffu, last, L.grp * L.lpr + (a.m - 1) / P);
      const float v = to_f32<T>(SK::logit(last));
      const RowExp ex(v, a.c);
      float e[N], s = 0.f, odd = 0.f;
      ex.row(cur, e);
#pragma unroll
      for (int n = 0; n < N; ++n) (n % 2 ? odd : s) += keys[n] < last ? e[n] : 0.f;
      s = L.sum(s + odd) * ex.fix();
      float rest = fmaf(a.tau, logf(s), v);
      // far below it (or nothing, or -inf): about the maximum of what stays
      if (__any_sync(0xffffffffu, !(s >= 1e-30f))) {
        float mr = -INFINITY;
#pragma unroll
        for (int n = 0; n < N; ++n) mr = keys[n] < last ? fmaxf(mr, cur[n]) : mr;
        mr = L.max(mr);
        float sr = 0.f;
#pragma unroll
        for (int n = 0; n < N; ++n) sr += keys[n] < last ? exp2_fast((cur[n] - mr) * a.c) : 0.f;
        sr = L.sum(sr);
        if (!(s >= 1e-30f)) rest = mr == -INFINITY ? -INFINITY : fmaf(a.tau, logf(sr), mr);
      }
      if (!in) return;
      if (L.sub == 0) a.rest[t] = broken ? NAN : rest;
      if (L.sub != q) return;  // a copy
      uint32_t ids[P];
      T tops[P];
#pragma unroll
      for (int p = 0; p < P; ++p) {
        ids[p] = broken ? (uint32_t)(q * P + p) : SK::id(x[p]);
        tops[p] = broken ? from_f32<T>(NAN) : SK::logit(x[p]);
      }
      uint32_t* const to = a.idx + t * a.m + q * P;
      T* const tl = top + t * a.m + q * P;
      if (P >= 4 && a.vec_out && a.m % P == 0) {  // whole vectors
        if (q * P < a.m) {
          if constexpr (P >= 4) {
#pragma unroll
            for (int p = 0; p < P; p += 4) {
              *reinterpret_cast<uint4*>(to + p) = make_uint4(ids[p], ids[p + 1], ids[p + 2], ids[p + 3]);
              if constexpr (sizeof(T) == 4) {
                *reinterpret_cast<float4*>(tl + p) = make_float4(tops[p], tops[p + 1], tops[p + 2], tops[p + 3]);
              } else {
                alignas(8) T h[4] = {tops[p], tops[p + 1], tops[p + 2], tops[p + 3]};
                *reinterpret_cast<uint2*>(tl + p) = *reinterpret_cast<const uint2*>(h);
              }
            }
          }
        }
      } else {
#pragma unroll
        for (int p = 0; p < P; ++p)
          if (q * P + p < a.m) to[p] = ids[p], tl[p] = tops[p];
      }
    });
  }
  rows.drain();
}

struct LaunchTargets {
  TargetArgs a;
  cudaStream_t s;
  template <typename T, int VEC, int NV, int LPR, int K>
  cudaError_t with() {
    const int64_t per = (int64_t)(kTargetThreads / 32) * (32 / a.lpr);
    const int64_t blocks = (a.T + per - 1) / per;
    static std::atomic<uint64_t> asked{0};
    return launch_rows(distill_targets_kernel<T, VEC, NV, LPR, K>,
                       (int)(blocks < kTargetBlocks ? blocks : kTargetBlocks), kTargetThreads,
                       kTargetThreads / 32 * RowStream<T, VEC, NV, LPR>::kWarpBytes, asked, s, a);
  }
  // The shortest kept list that holds m keys.  524288 rows of 256 BF16 logits take
  // 142 us for 8, 214 for 9 to 32 and 291 for 33 keys; of FP32 logits, whose keys are
  // twice as long, 394 for 8 and 1040 to 1050 for 9 to 64 (32 is not among their
  // lengths, and was not measured).
  template <typename T, int VEC, int NV, int LPR>
  cudaError_t run() {
    if (a.m <= 8) return with<T, VEC, NV, LPR, 8>();
    if constexpr (sizeof(T) == 2)
      if (a.m <= 32) return with<T, VEC, NV, LPR, 32>();
    return with<T, VEC, NV, LPR, 64>();
  }
};

}  // namespace

cudaError_t launch_distill_targets(const void* logits, moe_dtype dt, int64_t T, int E, int m, float temperature,
                                   uint32_t* idx, void* top, float* rest, cudaStream_t s) {
  const void* ptrs[] = {logits};
  const RowPlan plan = row_plan(ptrs, 1, dt, E);
  const bool vec_out = m % 4 == 0 && reinterpret_cast<uintptr_t>(idx) % 16 == 0 &&
                       reinterpret_cast<uintptr_t>(top) % (4 * dtype_size(dt)) == 0;
  LaunchTargets f{TargetArgs{logits, E, m, plan.lpr, T, temperature, kLog2e / temperature, idx, top, rest, vec_out},
                  s};
  return with_row_variant(dt, plan, f);
}

}  // namespace moe
