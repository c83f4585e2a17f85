// distill_targets.cu -- a teacher router's top logits, with the logit of all other
// experts together, rest = tau log sum_{e not in top} exp(t_e / tau).
#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kMaxList = 64;

struct TargetArgs {
  const void* logits;
  int E, m, lpr;
  int64_t T;
  float tau, c;
  uint32_t* idx;
  void* top;
  float* rest;
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

template <int LPR>
__device__ __forceinline__ uint32_t row_max(const Lanes<LPR>& L, uint32_t k) {
  if constexpr (LPR == 32) return __reduce_max_sync(0xffffffffu, k);
  return L.all(k, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}
template <int LPR>
__device__ __forceinline__ uint64_t row_max(const Lanes<LPR>& L, uint64_t k) {
  if constexpr (LPR == 32) {
    const uint32_t hi = row_max(L, (uint32_t)(k >> 32));
    const uint32_t lo = row_max(L, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
    return ((uint64_t)hi << 32) | lo;
  } else {
    return L.all(k, [](uint64_t a, uint64_t b) { return a > b ? a : b; });
  }
}

// One round: where this lane's head is the row's largest, it goes to out[j] and
// the next of the lane's list takes its place.  (Written out so that no lane
// branches.)
__device__ __forceinline__ void take(uint32_t best, uint32_t& head, uint32_t& next, uint32_t out) {
  asm volatile("{\n .reg .pred p;\n setp.eq.u32 p, %0, %2;\n @p st.shared.u32 [%3], %0;\n @p ld.shared.u32 %0, [%1];\n"
               " @p add.u32 %1, %1, 128;\n}"
               : "+r"(head), "+r"(next)
               : "r"(best), "r"(out)
               : "memory");
}
__device__ __forceinline__ void take(uint64_t best, uint64_t& head, uint32_t& next, uint32_t out) {
  asm volatile("{\n .reg .pred p;\n setp.eq.u64 p, %0, %2;\n @p st.shared.u64 [%3], %0;\n @p ld.shared.u64 %0, [%1];\n"
               " @p add.u32 %1, %1, 256;\n}"
               : "+l"(head), "+r"(next)
               : "l"(best), "r"(out)
               : "memory");
}

// Each lane sorts its share of the row; then m rounds take the largest head of
// the row's lanes.  A round is one reduction, a compare and the winner's next
// entry from shared memory: its cost does not grow with the row, and with eight
// lanes a row a warp takes four rows' entries in a round.
constexpr int kTargetThreads = 128;
constexpr int kTargetBlocks = 152 * 8;
template <typename T, int VEC, int NV, int LPR>
__global__ void __launch_bounds__(kTargetThreads) distill_targets_kernel(TargetArgs a) {
  constexpr int N = VEC * NV, W = kTargetThreads / 32;
  using Row = RowRegs<T, VEC, NV>;
  using SK = SortKey<T>;
  using Key = typename SK::Key;
  // taken[]: [rows][m] in order; m <= E bounds it where a row has few lanes
  constexpr int kTaken = LPR ? 32 / (LPR ? LPR : 1) * kMaxList : 32 * N;
  __shared__ Key lists[W][N + 1][32];  // entry N ends a list: below every key
  __shared__ Key taken[W][kTaken];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Lanes<LPR> L(a.lpr);
  const int room = a.E - L.sub * VEC;
  T* top = static_cast<T*>(a.top);
  lists[warp][N][lane] = 0;
  const int64_t step = (int64_t)gridDim.x * W * L.rows;
  int64_t t0 = ((int64_t)blockIdx.x * W + warp) * L.rows;
  const T* lp = static_cast<const T*>(a.logits) + (t0 + L.grp) * a.E + L.sub * VEC;
  Row cur, nxt;
  cur.fill(from_f32<T>(-INFINITY));
  nxt.fill(from_f32<T>(-INFINITY));
  cur.load(lp, room, L.lpr, t0 + L.grp < a.T);
  for (; t0 < a.T; t0 += step) {
    lp += step * a.E;
    nxt.load(lp, room, L.lpr, t0 + step + L.grp < a.T);
    const int64_t t = t0 + L.grp;
    const bool in = t < a.T;
    typename SK::template Keys<VEC, NV> keys(cur, L.lpr, L.sub);
    Key head;
    {
      Key list[N];
#pragma unroll
      for (int n = 0; n < N; ++n) list[n] = keys[n];
      sort_descending<0, N>(list);
#pragma unroll
      for (int n = 0; n < N; ++n) lists[warp][n][lane] = list[n];
      head = list[0];
    }
    Key* out = &taken[warp][L.grp * a.m];
    uint32_t next = (uint32_t)__cvta_generic_to_shared(&lists[warp][1][lane]);
    const uint32_t out_at = (uint32_t)__cvta_generic_to_shared(out);
    Key best = row_max(L, head);
    const bool broken = SK::broken(best);
#pragma unroll 4
    for (int j = 0; j < a.m; ++j) {
      take(best, head, next, out_at + j * (int)sizeof(Key));
      best = row_max(L, head);
    }
    __syncwarp();
    // what stays, about the last one taken
    const Key last = out[a.m - 1];
    const float v = to_f32<T>(SK::logit(last));
    const RowExp ex(v, a.c);
    float p[N], part[4] = {0.f, 0.f, 0.f, 0.f};
    ex.row(cur, p);
#pragma unroll
    for (int n = 0; n < N; ++n) part[n % 4] += keys[n] < last ? p[n] : 0.f;
    float s = L.sum((part[0] + part[1]) + (part[2] + part[3])) * ex.fix();
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
    if (in) {
      for (int j = L.sub; j < a.m; j += L.lpr) {
        const Key k = out[j];
        a.idx[t * a.m + j] = broken ? (uint32_t)j : SK::id(k);
        top[t * a.m + j] = broken ? from_f32<T>(NAN) : SK::logit(k);
      }
      if (L.sub == 0) a.rest[t] = broken ? NAN : rest;
    }
    __syncwarp();  // before the next row's lists
    cur = nxt;
  }
}

struct LaunchTargets {
  TargetArgs a;
  cudaStream_t s;
  template <typename T, int VEC, int NV, int LPR>
  cudaError_t run() {
    const int64_t per = (int64_t)(kTargetThreads / 32) * (32 / a.lpr);
    const int64_t blocks = (a.T + per - 1) / per;
    return launch_pdl(distill_targets_kernel<T, VEC, NV, LPR>,
                      dim3((unsigned)(blocks < kTargetBlocks ? blocks : kTargetBlocks)), dim3(kTargetThreads), 0, s, a);
  }
};

}  // namespace

cudaError_t launch_distill_targets(const void* logits, moe_dtype dt, int64_t T, int E, int m, float temperature,
                                   uint32_t* idx, void* top, float* rest, cudaStream_t s) {
  const void* ptrs[] = {logits};
  const RowPlan plan = row_plan(ptrs, 1, dt, E);
  LaunchTargets f{TargetArgs{logits, E, m, plan.lpr, T, temperature, kLog2e / temperature, idx, top, rest}, s};
  return with_row_variant(dt, plan, f);
}

}  // namespace moe
