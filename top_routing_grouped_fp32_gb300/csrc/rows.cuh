// rows.cuh -- rows of router logits in registers, and packed sequences of rows.
//
// Shared by the router's training losses (balance.cu, distill.cu).  A row of
// E <= 1024 logits is held by `lpr` lanes (a power of two), NV vectors of VEC
// elements per lane: vector v of lane `sub` starts at element
// (v * lpr + sub) * VEC, so that one warp load reads a contiguous piece.  With
// fewer than 32 lanes a row (NV == 1) a warp holds 32 / lpr rows at once.
#pragma once

#include <math.h>

#include <type_traits>

#include "common.cuh"

namespace moe {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^x and log2(x), within 2 ulp and 2^-22 absolute; subnormals are zero.
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

// How the lanes of a warp are laid over rows.  FULL: all 32 lanes hold one row.
template <bool FULL>
struct Lanes {
  int lpr, sub, grp, rows;  // lanes per row, lane in its row, row in the warp, rows per warp
  __device__ __forceinline__ explicit Lanes(int lpr_) {
    const int lane = threadIdx.x & 31;
    lpr = FULL ? 32 : lpr_;
    sub = FULL ? lane : lane & (lpr - 1);
    grp = FULL ? 0 : lane / lpr;
    rows = FULL ? 1 : 32 / lpr;
  }
  __device__ __forceinline__ unsigned mask() const {
    return FULL ? 0xffffffffu : (lpr == 32 ? 0xffffffffu : ((1u << lpr) - 1u) << (grp * lpr));
  }
  // Butterflies over the lanes of a row: every lane gets the same bits.  All
  // lanes of the warp take part.
  template <typename F>
  __device__ __forceinline__ float all(float x, F f) const {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      if (FULL || d < lpr) x = f(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
  }
  __device__ __forceinline__ float sum(float x) const {
    return all(x, [](float a, float b) { return a + b; });
  }
  __device__ __forceinline__ float max(float x) const {  // passes over NaN
    if constexpr (FULL) {
      float y;
      asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
      return y;
    } else {
      return all(x, [](float a, float b) { return fmaxf(a, b); });
    }
  }
  // R sums at once.  Two values share one exchange: of x[0] and x[1] a lane
  // keeps one and sends the other, so that R sums over 32 lanes cost about
  // 2 R + 3 shuffles where R butterflies cost 5 R.
  template <int R>
  __device__ __forceinline__ void sums(float (&x)[R]) const {
    if constexpr (FULL && R == 4) {
      const int lane = threadIdx.x & 31;
      const bool h = lane & 16, q = lane & 8;
      float a = (h ? x[1] : x[0]) + __shfl_xor_sync(0xffffffffu, h ? x[0] : x[1], 16);
      const float b = (h ? x[3] : x[2]) + __shfl_xor_sync(0xffffffffu, h ? x[2] : x[3], 16);
      a = (q ? b : a) + __shfl_xor_sync(0xffffffffu, q ? a : b, 8);
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
      x[0] = __shfl_sync(0xffffffffu, a, 0);
      x[1] = __shfl_sync(0xffffffffu, a, 16);
      x[2] = __shfl_sync(0xffffffffu, a, 8);
      x[3] = __shfl_sync(0xffffffffu, a, 24);
    } else if constexpr (FULL && R == 2) {
      const bool h = threadIdx.x & 16;
      float a = (h ? x[1] : x[0]) + __shfl_xor_sync(0xffffffffu, h ? x[0] : x[1], 16);
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) a += __shfl_xor_sync(0xffffffffu, a, d);
      x[0] = __shfl_sync(0xffffffffu, a, 0);
      x[1] = __shfl_sync(0xffffffffu, a, 16);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) x[r] = sum(x[r]);
    }
  }
};

// Rows (of each lane group) that a warp works on at once: enough independent
// loads in flight for HBM, within the registers.
template <int VEC, int NV>
constexpr int rows_at_once() {
  return VEC * NV <= 8 ? 4 : VEC * NV <= 16 ? 2 : 1;
}

// One row's elements of this lane.
template <typename T, int VEC, int NV>
struct RowRegs {
  static constexpr int N = VEC * NV;
  // VEC == 1 rows skip the vectors that lie behind their end
  static __device__ __forceinline__ bool used(int v, int lpr, int E) { return VEC > 1 || v * lpr < E; }
  static __device__ __forceinline__ int elem(int v, int i, int lpr, int sub) { return (v * lpr + sub) * VEC + i; }

  alignas(16) T raw[N];

  __device__ __forceinline__ void load(const T* row, int E, int lpr, int sub, bool ok, T fill) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int e = elem(v, 0, lpr, sub);
      if constexpr (VEC > 1) {
        static_assert(VEC * sizeof(T) == 16, "16-byte vectors");
        if (ok && e < E) {
          *reinterpret_cast<uint4*>(raw + v * VEC) = __ldg(reinterpret_cast<const uint4*>(row + e));
        } else {
#pragma unroll
          for (int i = 0; i < VEC; ++i) raw[v * VEC + i] = fill;
        }
      } else {
        raw[v] = ok && e < E ? __ldg(row + e) : fill;
      }
    }
  }
  __device__ __forceinline__ float operator[](int n) const { return to_f32<T>(raw[n]); }

  // This lane's maximum; passes over NaN.
  __device__ __forceinline__ float lane_max() const {
    if constexpr (sizeof(T) == 2 && VEC == 8) {  // two elements an instruction
      using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      T2 m = reinterpret_cast<const T2*>(raw)[0];
#pragma unroll
      for (int i = 1; i < N / 2; ++i) m = __hmax2(m, reinterpret_cast<const T2*>(raw)[i]);
      return fmaxf(to_f32<T>(m.x), to_f32<T>(m.y));
    } else {
      float m = (*this)[0];
#pragma unroll
      for (int n = 1; n < N; ++n) m = fmaxf(m, (*this)[n]);
      return m;
    }
  }
};

// exp((x - m) / tau) as 2^(x c - m c), c = log2(e) / tau, in one FMA an element.
// mc = m c is rounded, which leaves a factor 2^(m c - mc) on every element of the
// row: `fix` takes it out of their sum (to first order: |m c - mc| < 2^-12).
// Rows that lie farther out (masked with a large negative value, say) form x - m
// first.
struct RowExp {
  float c, mc, m, fix;
  bool wide;
  __device__ __forceinline__ RowExp(float m_, float c_) : c(c_), m(m_) {
    mc = m_ * c_;
    wide = fabsf(mc) > 4096.f && fabsf(m_) < INFINITY;
    fix = fabsf(mc) <= 4096.f ? fmaf(fmaf(m_, c_, -mc), -kLn2, 1.f) : 1.f;
  }
  __device__ __forceinline__ float operator()(float x) const { return exp2_fast(fmaf(x, c, -mc)); }
  __device__ __forceinline__ float far(float x) const { return exp2_fast((x - m) * c); }
};

// Stores N values of a lane at `row` (16-byte vectors or single elements).
template <typename T, int VEC, int NV>
__device__ __forceinline__ void store_row(T* row, int E, int lpr, int sub, const float (&f)[VEC * NV]) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    const int e = (v * lpr + sub) * VEC;
    if (e >= E) continue;
    if constexpr (VEC == 8) {
      *reinterpret_cast<uint4*>(row + e) = pack8<T>(f + v * VEC);
    } else if constexpr (VEC == 4) {
      *reinterpret_cast<float4*>(row + e) = make_float4(f[v * 4], f[v * 4 + 1], f[v * 4 + 2], f[v * 4 + 3]);
    } else {
      row[e] = from_f32<T>(f[v]);
    }
  }
}

// ---- packed sequences --------------------------------------------------------
// Sequence s holds the rows off[s] <= t < off[s+1] of a batch of T rows; a null
// `off` is one sequence of all rows.  Offsets come from the device and are
// clamped where they are used, so that no malformed entry leads outside.
struct Seqs {
  const uint32_t* off;
  int num;
  int64_t T;
  __device__ __forceinline__ int64_t at(int s) const {
    if (!off) return s == 0 ? 0 : T;
    const int64_t o = __ldg(off + s);
    return o < T ? o : T;
  }
  // How many of off[1..num] are <= row: the first sequence that ends behind it.
  // A whole warp searches, 32 entries a step.
  __device__ __forceinline__ int first(int64_t row) const {
    if (!off) return 0;
    int lo = 0, hi = num;  // the answer is in lo..hi
    const int lane = threadIdx.x & 31;
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32;
      const int64_t i = (int64_t)lo + (int64_t)(lane + 1) * step;  // entry i, at most hi
      const bool le = i <= hi && at((int)i) <= row;
      const int n = __popc(__ballot_sync(0xffffffffu, le));
      hi = min(hi, lo + (n + 1) * step - 1);
      lo = min(hi, lo + n * step);
    }
    return lo;
  }
};

// Walks the rows [a, b): calls seq(s, lo, hi) for each piece that lies in a
// sequence and gap(lo, hi) for rows outside every sequence, in order, each row
// once whatever the offsets hold.
template <typename FSeq, typename FGap>
__device__ __forceinline__ void walk_sequences(const Seqs& q, int64_t a, int64_t b, FSeq seq, FGap gap) {
  int64_t cur = a;
  for (int s = q.first(a); cur < b; ++s) {
    if (s >= q.num) {
      gap(cur, b);
      break;
    }
    const int64_t lo = min(max(q.at(s), cur), b);
    const int64_t hi = min(max(q.at(s + 1), lo), b);
    if (lo > cur) gap(cur, lo);
    if (hi > lo) seq(s, lo, hi);
    cur = hi;
  }
}

// ---- variants by row length ------------------------------------------------------
// 16-byte vectors where every row starts on a 16-byte boundary, else single
// elements; the fewest lanes that hold a row in one vector each, else 32 lanes
// and more vectors.
struct RowPlan {
  bool vec;
  int lpr;
  int nv;
};
inline RowPlan row_plan(const void* const* ptrs, int n_ptrs, moe_dtype dt, int E) {
  const int esz = (int)dtype_size(dt);
  bool vec = (E * esz) % 16 == 0;
  for (int i = 0; i < n_ptrs; ++i) vec = vec && reinterpret_cast<uintptr_t>(ptrs[i]) % 16 == 0;
  const int units = vec ? E * esz / 16 : E;
  RowPlan p{vec, 1, 1};
  while (p.lpr < 32 && p.lpr < units) p.lpr *= 2;
  while (p.lpr * p.nv < units) p.nv *= 2;
  return p;
}

// Calls f.template run<T, VEC, NV, FULL>() for a plan.
template <typename T, typename F>
cudaError_t with_row_variant(const RowPlan& p, F&& f) {
  constexpr int V = 16 / sizeof(T);
  if (p.vec) {
    if (p.lpr < 32) return f.template run<T, V, 1, false>();
    switch (p.nv) {
      case 1: return f.template run<T, V, 1, true>();
      case 2: return f.template run<T, V, 2, true>();
      case 4: return f.template run<T, V, 4, true>();
      default:
        if constexpr (V == 4) return f.template run<T, V, 8, true>();
        return cudaErrorInvalidValue;
    }
  }
  if (p.lpr < 32) return f.template run<T, 1, 1, false>();
  switch (p.nv) {
    case 1: return f.template run<T, 1, 1, true>();
    case 2: return f.template run<T, 1, 2, true>();
    case 4: return f.template run<T, 1, 4, true>();
    case 8: return f.template run<T, 1, 8, true>();
    case 16: return f.template run<T, 1, 16, true>();
    default: return f.template run<T, 1, 32, true>();
  }
}
template <typename F>
cudaError_t with_row_variant(moe_dtype dt, const RowPlan& p, F&& f) {
  if (dt == MOE_F32) return with_row_variant<float>(p, f);
  if (dt == MOE_F16) return with_row_variant<__half>(p, f);
  return with_row_variant<__nv_bfloat16>(p, f);
}

// How a batch of rows is cut over blocks: `chunks` blocks of `rows` rows.
struct Chunks {
  int64_t rows;
  int chunks;
};
inline Chunks cut_rows(int64_t T, int64_t step, int64_t max_chunks) {
  int64_t steps = (T + step - 1) / step;
  if (steps < 1) steps = 1;
  const int64_t per = (steps + max_chunks - 1) / max_chunks;
  Chunks c;
  c.rows = per * step;
  c.chunks = (int)((steps + per - 1) / per);
  return c;
}

}  // namespace moe
