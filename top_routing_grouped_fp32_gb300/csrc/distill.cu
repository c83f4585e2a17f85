// distill.cu -- distillation of a router from a teacher's top logits.
//
// A teacher's row is kept as its m largest logits t_j (with their experts
// idx_j) and `rest`, the logit of all its other experts together,
//   rest = tau log sum_{e not in top} exp(t_e / tau).
// With a_j = t_j / tau (and rest / tau), b_e = l_e / tau for the student's row,
//   q = softmax(a_1..a_m, rest / tau),  p = softmax(b),  R = sum_{e not in top} p_e,
//   KL = sum_j q_j (log q_j - log p_idx_j) + q_r (log q_r - log R)
// and without a rest q = softmax(a_1..a_m).  An entry t_j = -inf is absent and its index is not
// read; a row without any entry has no target and does not count.  A sequence's
// loss is the mean KL of its counted rows, and
//   dKL/dl_e = 1/tau (p_e - q_e)                      for e in the list
//            = 1/tau p_e (1 - q_r / R)                otherwise
// The forward leaves what the backward needs of a row: the maxima and sums of
// both sides and q_r / R, so that the backward has no reduction to make.
//
// Both sides sum to one, so KL = sum (q log(q/p) - q + p) over the list and the
// rest (over the mass outside the list, p alone, without a rest).  Every term is
// >= 0 and of second order in log(q/p), so a student near its teacher loses no
// digits and errors of the two normalisers cancel to first order.
#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunks = 1216;  // eight blocks per SM
constexpr int kMaxList = 64;

// Below this share of the row's maximum the student's mass outside the list is
// taken about its own maximum, and -q_r stands in the place of q_r / R.
constexpr float kFarBelow = 1e-30f;

// q log(q/p) - q + p from d = log(q/p); its series where the terms nearly cancel
// (|d| < 1/2: the first term left out is below 2^-24 of the sum).
__device__ __forceinline__ float kl_term(float q, float p, float d) {
  if (!(q > 0.f)) return q == 0.f ? p : q;  // no mass (its limit), or NaN
  if (fabsf(d) < 0.5f) {
    float h = fmaf(d, -1.f / 362880.f, 1.f / 40320.f);
    h = fmaf(-d, h, 1.f / 5040.f);
    h = fmaf(-d, h, 1.f / 720.f);
    h = fmaf(-d, h, 1.f / 120.f);
    h = fmaf(-d, h, 1.f / 24.f);
    h = fmaf(-d, h, 1.f / 6.f);
    h = fmaf(-d, h, 1.f / 2.f);
    return q * d * d * h;
  }
  return fmaf(q, d, p - q);
}

struct FwdArgs {
  const void* logits;
  const uint32_t* t_idx;
  const void* t_logits;
  int t_dt;
  const float* t_rest;
  const uint8_t* mask;
  Seqs seqs;
  int E, m, lpr;
  int64_t T, chunk_rows;
  float inv_tau, c;  // 1 / tau and log2(e) / tau
  float* part_loss;      // [slots]
  uint32_t* part_rows;   // [slots]
  uint32_t* part_bad;    // [slots] lists with an index that is no expert or is there twice
  float* row_loss;
  float* row_stats;
  uint32_t* status;
};

template <typename T, int VEC, int NV, bool FULL>
__global__ void __launch_bounds__(kThreads) distill_fwd_kernel(FwdArgs a) {
  using Row = RowRegs<T, VEC, NV>;
  // one bit per expert and row: is it in the teacher's list
  extern __shared__ uint32_t bits_smem[];
  __shared__ float red_l[kWarps];
  __shared__ uint32_t red_n[kWarps], red_b[kWarps];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0u;
  const Lanes<FULL> L(a.lpr);
  const int words = (a.E + 31) / 32;
  uint32_t* bits = bits_smem + (warp * L.rows + L.grp) * words;
  const T* logits = static_cast<const T*>(a.logits);
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk_rows;
  const int64_t c1 = min(c0 + a.chunk_rows, a.T);

  auto write_row = [&](int64_t t, float kl, float m, float s, float mt, float st, float ratio) {
    a.row_loss[t] = kl;
    a.row_stats[t] = m;
    a.row_stats[a.T + t] = s;
    a.row_stats[2 * a.T + t] = mt;
    a.row_stats[3 * a.T + t] = st;
    a.row_stats[4 * a.T + t] = ratio;
  };
  auto gap = [&](int64_t lo, int64_t hi) {
    for (int64_t t = lo + threadIdx.x; t < hi; t += kThreads) write_row(t, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f);
  };
  auto piece = [&](int seq, int64_t lo, int64_t hi) {
    float loss = 0.f;
    uint32_t counted = 0, broken = 0;
    for (int64_t t0 = lo + warp * L.rows; t0 < hi; t0 += kWarps * L.rows) {
      const int64_t t = t0 + L.grp;
      const bool in = t < hi;
      bool ok = in && (!a.mask || __ldg(a.mask + t));
      const T* row = logits + t * a.E;
      Row r;
      r.load(row, a.E, L.lpr, L.sub, ok, from_f32<T>(-INFINITY));
      for (int w = L.sub; w < words; w += L.lpr) bits[w] = 0u;
      __syncwarp();
      // the teacher's maximum, the list's experts
      const float rest = ok && a.t_rest ? __ldg(a.t_rest + t) : -INFINITY;
      float mt = rest;
      bool bad = false, nan = rest != rest || rest == INFINITY;
      if (ok)
        for (int j = L.sub; j < a.m; j += L.lpr) {
          const float x = load_dyn(a.t_logits, a.t_dt, (size_t)t * a.m + j);
          mt = fmaxf(mt, x);
          nan |= x != x || x == INFINITY;
          if (x == -INFINITY) continue;
          const uint32_t e = __ldg(a.t_idx + t * a.m + j);
          if (e >= (uint32_t)a.E) bad = true;
          else if (atomicOr(bits + (e >> 5), 1u << (e & 31)) >> (e & 31) & 1u) bad = true;
        }
      mt = L.max(mt);
      // a NaN or +inf in the list, a bad index or a NaN or +inf in the row: the row counts as NaN
      const bool any_nan = (__ballot_sync(0xffffffffu, nan) & L.mask()) != 0;
      const bool any_bad = (__ballot_sync(0xffffffffu, bad) & L.mask()) != 0;
      ok = ok && (mt != -INFINITY || any_nan);  // else no target
      // the student's softmax
      float m = -INFINITY;
#pragma unroll
      for (int n = 0; n < Row::N; ++n) m = fmaxf(m, r[n]);
      m = L.max(m);
      __syncwarp();
      float s = 0.f, out = 0.f;
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        if (!Row::used(v, L.lpr, a.E)) continue;
        const int e0 = Row::elem(v, 0, L.lpr, L.sub);
        const uint32_t b = e0 < a.E ? bits[e0 >> 5] >> (e0 & 31) : 0u;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          const float p = exp2_fast((r[v * VEC + i] - m) * a.c);
          s += p;
          out += b >> i & 1u ? 0.f : p;
        }
      }
      s = L.sum(s);
      out = L.sum(out);
      // the teacher's sum
      float st = L.sub == 0 ? exp2_fast((rest - mt) * a.c) : 0.f;
      if (ok)
        for (int j = L.sub; j < a.m; j += L.lpr)
          st += exp2_fast((load_dyn(a.t_logits, a.t_dt, (size_t)t * a.m + j) - mt) * a.c);
      st = L.sum(st);
      // log of the mass outside the list, about its own maximum where it is far below the row's
      float ln_out = logf(out);
      const bool far = ok && a.t_rest && out < kFarBelow;
      if (far) {
        float mo = -INFINITY;
#pragma unroll
        for (int n = 0; n < Row::N; ++n) {
          const int e = Row::elem(n / VEC, n % VEC, L.lpr, L.sub);
          if (e < a.E && !(bits[e >> 5] >> (e & 31) & 1u)) mo = fmaxf(mo, r[n]);
        }
        for (int d = L.lpr / 2; d > 0; d >>= 1) mo = fmaxf(mo, __shfl_xor_sync(L.mask(), mo, d));
        float so = 0.f;
#pragma unroll
        for (int n = 0; n < Row::N; ++n) {
          const int e = Row::elem(n / VEC, n % VEC, L.lpr, L.sub);
          if (e < a.E && !(bits[e >> 5] >> (e & 31) & 1u)) so += exp2_fast((r[n] - mo) * a.c);
        }
        for (int d = L.lpr / 2; d > 0; d >>= 1) so += __shfl_xor_sync(L.mask(), so, d);
        ln_out = mo == -INFINITY ? -INFINITY : (mo - m) * a.inv_tau + logf(so);
      }
      if (any_bad || any_nan) s = NAN;
      const float inv_s = 1.f / s, inv_st = 1.f / st;
      const float dz = logf(s) - logf(st);
      float kl = 0.f, ratio = 0.f;
      if (ok)
        for (int j = L.sub; j < a.m; j += L.lpr) {
          const float x = load_dyn(a.t_logits, a.t_dt, (size_t)t * a.m + j);
          if (x == -INFINITY) continue;
          const uint32_t e = __ldg(a.t_idx + t * a.m + j);
          if (e >= (uint32_t)a.E) continue;
          const float y = to_f32<T>(__ldg(row + e));
          const float q = exp2_fast((x - mt) * a.c) * inv_st;
          const float p = exp2_fast((y - m) * a.c) * inv_s;
          kl += kl_term(q, p, ((x - mt) - (y - m)) * a.inv_tau + dz);
        }
      if (a.t_rest) {
        const float q = exp2_fast((rest - mt) * a.c) * inv_st, p = out * inv_s;
        if (L.sub == 0) kl += kl_term(q, p, (rest - mt) * a.inv_tau - ln_out + dz);
        ratio = far ? -q : q / p;
      } else if (L.sub == 0) {
        kl += out * inv_s;
      }
      kl = L.sum(kl);
      if (L.sub == 0 && in) {
        if (ok) {
          if (s != s || st != st) kl = NAN;
          write_row(t, kl, m, s, mt, st, ratio);
          loss += kl;
          ++counted;
          broken += any_bad;
        } else {
          write_row(t, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f);
        }
      }
      __syncwarp();  // before the next row clears the bits
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      loss += __shfl_xor_sync(0xffffffffu, loss, d);
      counted += __shfl_xor_sync(0xffffffffu, counted, d);
      broken += __shfl_xor_sync(0xffffffffu, broken, d);
    }
    if (lane == 0) red_l[warp] = loss, red_n[warp] = counted, red_b[warp] = broken;
    __syncthreads();
    if (threadIdx.x == 0) {
      float l = 0.f;
      uint32_t n = 0, b = 0;
      for (int w = 0; w < kWarps; ++w) l += red_l[w], n += red_n[w], b += red_b[w];
      const int64_t slot = (int64_t)blockIdx.x + seq;
      a.part_loss[slot] = l;
      a.part_rows[slot] = n;
      a.part_bad[slot] = b;
    }
    __syncthreads();
  };
  walk_sequences(a.seqs, c0, c1, piece, gap);
}

struct FinishArgs {
  const float* part_loss;
  const uint32_t* part_rows;
  const uint32_t* part_bad;
  Seqs seqs;
  int64_t chunk_rows;
  float* loss;
  uint32_t* tokens;
  uint32_t* status;
};

// One warp per sequence adds its slots in a fixed order.
__global__ void __launch_bounds__(kThreads) distill_finish_kernel(FinishArgs a) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (s >= a.seqs.num) return;
  const int64_t lo = a.seqs.at(s), hi = a.seqs.at(s + 1);
  if (lane == 0 && a.seqs.off &&
      (hi < lo || (int64_t)__ldg(a.seqs.off + s) > a.seqs.T || (int64_t)__ldg(a.seqs.off + s + 1) > a.seqs.T))
    set_status(a.status, MOE_ERR_INVALID_INDEX);
  float l = 0.f;
  uint32_t n = 0, b = 0;
  if (hi > lo) {
    const int64_t last = (hi - 1) / a.chunk_rows + s;
    for (int64_t i = lo / a.chunk_rows + s + lane; i <= last; i += 32) {
      l += a.part_loss[i];
      n += a.part_rows[i];
      b += a.part_bad[i];
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, d);
    n += __shfl_xor_sync(0xffffffffu, n, d);
    b += __shfl_xor_sync(0xffffffffu, b, d);
  }
  if (lane == 0) {
    a.loss[s] = n ? l / (float)n : 0.f;
    a.tokens[s] = n;
    if (b) set_status(a.status, MOE_ERR_INVALID_INDEX);
  }
}

struct BwdArgs {
  const void* logits;
  const uint32_t* t_idx;
  const void* t_logits;
  int t_dt;
  const float* row_stats;
  const uint32_t* tokens;
  const float* dloss;
  Seqs seqs;
  int E, m, lpr;
  int64_t T, chunk_rows;
  float inv_tau, c;
  const void* base;
  void* out;
};

// The list's entries differ from p_e (1 - ratio): a row is laid out in shared
// memory in its final type, the lanes of the list overwrite their entries, and
// the row leaves in full vectors.
template <typename T, int VEC, int NV, bool FULL>
__global__ void __launch_bounds__(kThreads) distill_bwd_kernel(BwdArgs a) {
  constexpr int N = VEC * NV;
  using Row = RowRegs<T, VEC, NV>;
  extern __shared__ __align__(16) unsigned char row_smem[];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const Lanes<FULL> L(a.lpr);
  const int pitch = (int)align_up((size_t)a.E * sizeof(T), 16) / (int)sizeof(T);
  T* buf = reinterpret_cast<T*>(row_smem) + (warp * L.rows + L.grp) * pitch;
  const T* logits = static_cast<const T*>(a.logits);
  const T* base = static_cast<const T*>(a.base);
  T* out = static_cast<T*>(a.out);
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk_rows;
  const int64_t c1 = min(c0 + a.chunk_rows, a.T);

  // rows [lo, hi) with gradient scale c; outside every sequence: nothing but the base
  auto rows = [&](bool inside, float c, int64_t lo, int64_t hi) {
    for (int64_t t0 = lo + warp * L.rows; t0 < hi; t0 += kWarps * L.rows) {
      const int64_t t = t0 + L.grp;
      const bool in = t < hi;
      float m = 0.f, s = 0.f, mt = 0.f, st = 0.f, ratio = 0.f;
      if (in && inside) {
        s = __ldg(a.row_stats + a.T + t);
        if (s != 0.f) {
          m = __ldg(a.row_stats + t);
          mt = __ldg(a.row_stats + 2 * a.T + t);
          st = __ldg(a.row_stats + 3 * a.T + t);
          ratio = __ldg(a.row_stats + 4 * a.T + t);
        }
      }
      const bool ok = s != 0.f;  // the row counted; NaN sums leave NaN
      const T* row = logits + t * a.E;
      Row r;
      r.load(row, a.E, L.lpr, L.sub, ok, from_f32<T>(-INFINITY));
      const float ps = ok ? c / s : 0.f;
      const float w = ps * (1.f - ratio);
      float d[N];
#pragma unroll
      for (int n = 0; n < N; ++n) d[n] = ok ? exp2_fast((r[n] - m) * a.c) * w : 0.f;
      if (ratio < 0.f) {  // the shares of the rest about their own maximum
        float mo = -INFINITY;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int e = Row::elem(n / VEC, n % VEC, L.lpr, L.sub);
          bool listed = e >= a.E;
          for (int j = 0; j < a.m && !listed; ++j)
            listed = __ldg(a.t_idx + t * a.m + j) == (uint32_t)e &&
                     load_dyn(a.t_logits, a.t_dt, (size_t)t * a.m + j) != -INFINITY;
          d[n] = listed ? -INFINITY : r[n];
          mo = fmaxf(mo, d[n]);
        }
        for (int k = L.lpr / 2; k > 0; k >>= 1) mo = fmaxf(mo, __shfl_xor_sync(L.mask(), mo, k));
        float so = 0.f;
#pragma unroll
        for (int n = 0; n < N; ++n) {
          d[n] = mo == -INFINITY ? 0.f : exp2_fast((d[n] - mo) * a.c);
          so += d[n];
        }
        for (int k = L.lpr / 2; k > 0; k >>= 1) so += __shfl_xor_sync(L.mask(), so, k);
        const float f = so > 0.f ? c * ratio / so : 0.f;
#pragma unroll
        for (int n = 0; n < N; ++n) d[n] *= f;
      }
      if (in && base) {
        Row b;
        b.load(base + t * a.E, a.E, L.lpr, L.sub, true, from_f32<T>(0.f));
#pragma unroll
        for (int n = 0; n < N; ++n) d[n] += b[n];
      }
      store_row<T, VEC, NV>(buf, a.E, L.lpr, L.sub, d);
      __syncwarp();
      if (ok) {
        const float qs = c / st;
        for (int j = L.sub; j < a.m; j += L.lpr) {
          const float x = load_dyn(a.t_logits, a.t_dt, (size_t)t * a.m + j);
          if (x == -INFINITY) continue;
          const uint32_t e = __ldg(a.t_idx + t * a.m + j);
          if (e >= (uint32_t)a.E) continue;  // the row is NaN already
          float g = exp2_fast((to_f32<T>(__ldg(row + e)) - m) * a.c) * ps - exp2_fast((x - mt) * a.c) * qs;
          if (base) g += to_f32<T>(__ldg(base + t * a.E + e));
          buf[e] = from_f32<T>(g);
        }
      }
      __syncwarp();
      if (in) {
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const int e = Row::elem(v, 0, L.lpr, L.sub);
          if (e >= a.E) continue;
          if constexpr (VEC > 1)
            *reinterpret_cast<uint4*>(out + t * a.E + e) = *reinterpret_cast<const uint4*>(buf + e);
          else
            out[t * a.E + e] = buf[e];
        }
      }
      __syncwarp();  // before the next row is laid out
    }
  };
  walk_sequences(
      a.seqs, c0, c1,
      [&](int seq, int64_t lo, int64_t hi) {
        const uint32_t n = __ldg(a.tokens + seq);
        rows(true, n ? __ldg(a.dloss + seq) * a.inv_tau / (float)n : 0.f, lo, hi);
      },
      [&](int64_t lo, int64_t hi) { rows(false, 0.f, lo, hi); });
}

// ---- a teacher's targets ----------------------------------------------------
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

template <bool FULL>
__device__ __forceinline__ uint32_t row_max(const Lanes<FULL>& L, uint32_t k) {
  if constexpr (FULL) return __reduce_max_sync(0xffffffffu, k);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1)
    if (d < L.lpr) k = max(k, __shfl_xor_sync(0xffffffffu, k, d));
  return k;
}
template <bool FULL>
__device__ __forceinline__ uint64_t row_max(const Lanes<FULL>& L, uint64_t k) {
  const uint32_t hi = row_max(L, (uint32_t)(k >> 32));
  const uint32_t lo = row_max(L, (uint32_t)(k >> 32) == hi ? (uint32_t)k : 0u);
  return ((uint64_t)hi << 32) | lo;
}

// Each lane sorts its share of the row; then m rounds take the largest head of
// the lanes' lists.  A round is one reduction, a compare and the winner's next
// entry from shared memory: its cost does not grow with the row.
constexpr int kTargetThreads = 128;
template <typename T, int VEC, int NV, bool FULL>
__global__ void __launch_bounds__(kTargetThreads) distill_targets_kernel(TargetArgs a) {
  constexpr int N = VEC * NV, W = kTargetThreads / 32;
  using Row = RowRegs<T, VEC, NV>;
  using SK = SortKey<T>;
  using Key = typename SK::Key;
  __shared__ Key lists[W][N + 1][32];               // entry N ends a list: below every key
  __shared__ Key taken[W][FULL ? kMaxList : 32 * N];  // [rows][m], in order
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Lanes<FULL> L(a.lpr);
  const T* logits = static_cast<const T*>(a.logits);
  T* top = static_cast<T*>(a.top);
  lists[warp][N][lane] = 0;
  const int64_t step = (int64_t)gridDim.x * W * L.rows;
  int64_t t0 = ((int64_t)blockIdx.x * W + warp) * L.rows;
  auto load = [&](Row& r, int64_t t) { r.load(logits + t * a.E, a.E, L.lpr, L.sub, t < a.T, from_f32<T>(-INFINITY)); };
  Row cur, nxt;
  load(cur, t0 + L.grp);
  for (; t0 < a.T; t0 += step) {
    load(nxt, t0 + step + L.grp);
    const int64_t t = t0 + L.grp;
    const bool in = t < a.T;
    Key key[N], list[N];
#pragma unroll
    for (int n = 0; n < N; ++n)
      list[n] = key[n] = SK::make(cur.raw[n], Row::elem(n / VEC, n % VEC, L.lpr, L.sub));
    sort_descending<0, N>(list);
#pragma unroll
    for (int n = 0; n < N; ++n) lists[warp][n][lane] = list[n];
    Key head = list[0];
    const Key* next = &lists[warp][1][lane];
    Key* out = &taken[warp][L.grp * a.m];
    const bool broken = SK::broken(row_max(L, head));
#pragma unroll 4
    for (int j = 0; j < a.m; ++j) {
      if (head == row_max(L, head)) {
        out[j] = head;
        head = *next;
        next += 32;
      }
    }
    __syncwarp();
    // what stays, about the last one taken
    const Key last = out[a.m - 1];
    const float v = to_f32<T>(SK::logit(last));
    const RowExp ex(v, a.c);
    float s = 0.f;
    if (ex.wide) {
#pragma unroll
      for (int n = 0; n < N; ++n) s += key[n] < last ? ex.far(cur[n]) : 0.f;
    } else {
#pragma unroll
      for (int n = 0; n < N; ++n) s += key[n] < last ? ex(cur[n]) : 0.f;
    }
    s = L.sum(s) * ex.fix;
    float rest = fmaf(a.tau, logf(s), v);
    // far below it (or nothing, or -inf): about the maximum of what stays
    if (__any_sync(0xffffffffu, !(s >= 1e-30f))) {
      float mr = -INFINITY;
#pragma unroll
      for (int n = 0; n < N; ++n) mr = key[n] < last ? fmaxf(mr, cur[n]) : mr;
      mr = L.max(mr);
      float sr = 0.f;
#pragma unroll
      for (int n = 0; n < N; ++n) sr += key[n] < last ? exp2_fast((cur[n] - mr) * a.c) : 0.f;
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

struct LaunchFwd {
  FwdArgs a;
  int chunks;
  size_t smem;
  cudaStream_t s;
  template <typename T, int VEC, int NV, bool FULL>
  cudaError_t run() {
    return launch_pdl(distill_fwd_kernel<T, VEC, NV, FULL>, dim3((unsigned)chunks), dim3(kThreads), smem, s, a);
  }
};
struct LaunchBwd {
  BwdArgs a;
  int chunks;
  size_t smem;
  cudaStream_t s;
  template <typename T, int VEC, int NV, bool FULL>
  cudaError_t run() {
    return launch_pdl(distill_bwd_kernel<T, VEC, NV, FULL>, dim3((unsigned)chunks), dim3(kThreads), smem, s, a);
  }
};
struct LaunchTargets {
  TargetArgs a;
  cudaStream_t s;
  template <typename T, int VEC, int NV, bool FULL>
  cudaError_t run() {
    const int64_t per = (int64_t)(kTargetThreads / 32) * (32 / a.lpr);
    const int64_t blocks = (a.T + per - 1) / per;
    return launch_pdl(distill_targets_kernel<T, VEC, NV, FULL>,
                      dim3((unsigned)(blocks < kMaxChunks ? blocks : kMaxChunks)), dim3(kTargetThreads), 0, s, a);
  }
};

size_t slot_count(int64_t T, int64_t num_seqs) { return (size_t)(kMaxChunks < T ? kMaxChunks : T) + (size_t)num_seqs; }

}  // namespace

size_t distill_workspace_bytes(int64_t T, int64_t num_seqs) { return align_up(slot_count(T, num_seqs) * 12, 256); }

cudaError_t launch_distill_loss(const DistillArgs& d, void* ws, uint32_t* status, cudaStream_t s) {
  const void* ptrs[] = {d.logits};
  const RowPlan plan = row_plan(ptrs, 1, d.dt, d.E);
  const int rows = kWarps * (32 / plan.lpr);
  const Chunks ch = cut_rows(d.T, rows, kMaxChunks);
  const size_t slots = slot_count(d.T, d.num_seqs);
  FwdArgs a{};
  a.logits = d.logits;
  a.t_idx = d.t_idx;
  a.t_logits = d.t_logits;
  a.t_dt = d.t_dt;
  a.t_rest = d.t_rest;
  a.mask = d.mask;
  a.seqs = Seqs{d.seq_offsets, (int)d.num_seqs, d.T};
  a.E = d.E;
  a.m = d.m;
  a.lpr = plan.lpr;
  a.T = d.T;
  a.chunk_rows = ch.rows;
  a.inv_tau = 1.f / d.temperature;
  a.c = kLog2e / d.temperature;
  a.part_loss = static_cast<float*>(ws);
  a.part_rows = reinterpret_cast<uint32_t*>(a.part_loss + slots);
  a.part_bad = a.part_rows + slots;
  a.row_loss = d.row_loss;
  a.row_stats = d.row_stats;
  a.status = status;
  LaunchFwd f{a, ch.chunks, (size_t)rows * ((d.E + 31) / 32) * 4, s};
  const cudaError_t e = with_row_variant(d.dt, plan, f);
  if (e != cudaSuccess) return e;
  FinishArgs fin{a.part_loss, a.part_rows, a.part_bad, a.seqs, ch.rows, d.loss, d.tokens, status};
  return launch_pdl(distill_finish_kernel, dim3((unsigned)((d.num_seqs + kWarps - 1) / kWarps)), dim3(kThreads), 0,
                    s, fin);
}

cudaError_t launch_distill_loss_backward(const DistillBwdArgs& d, cudaStream_t s) {
  const void* ptrs[] = {d.logits, d.base, d.dlogits};
  const RowPlan plan = row_plan(ptrs, 3, d.dt, d.E);
  const int rows = kWarps * (32 / plan.lpr);
  const Chunks ch = cut_rows(d.T, rows, kMaxChunks);
  BwdArgs a{};
  a.logits = d.logits;
  a.t_idx = d.t_idx;
  a.t_logits = d.t_logits;
  a.t_dt = d.t_dt;
  a.row_stats = d.row_stats;
  a.tokens = d.tokens;
  a.dloss = d.dloss;
  a.seqs = Seqs{d.seq_offsets, (int)d.num_seqs, d.T};
  a.E = d.E;
  a.m = d.m;
  a.lpr = plan.lpr;
  a.T = d.T;
  a.chunk_rows = ch.rows;
  a.inv_tau = 1.f / d.temperature;
  a.c = kLog2e / d.temperature;
  a.base = d.base;
  a.out = d.dlogits;
  LaunchBwd f{a, ch.chunks, (size_t)rows * align_up((size_t)d.E * dtype_size(d.dt), 16), s};
  return with_row_variant(d.dt, plan, f);
}

cudaError_t launch_distill_targets(const void* logits, moe_dtype dt, int64_t T, int E, int m, float temperature,
                                   uint32_t* idx, void* top, float* rest, cudaStream_t s) {
  const void* ptrs[] = {logits};
  const RowPlan plan = row_plan(ptrs, 1, dt, E);
  LaunchTargets f{TargetArgs{logits, E, m, plan.lpr, T, temperature, kLog2e / temperature, idx, top, rest}, s};
  return with_row_variant(dt, plan, f);
}

}  // namespace moe
