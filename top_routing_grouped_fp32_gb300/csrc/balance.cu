// balance.cu -- the router's balance loss with per-expert counts, its z-loss
// and their gradient.
//
// For the valid rows V_s of a sequence s (L_s of them), row scores p_te that sum
// to one over the experts and the routed slots idx [T,k]:
//   n_se   = #{(t, j) : t in V_s, idx_tj = e}
//   P_se   = 1/L_s sum_{t in V_s} p_te
//   loss_s = E sum_e n_se / (k L_s) P_se
//   z_s    = 1/L_s sum_{t in V_s} (log sum_e exp l_te)^2
// The counts are not differentiated.  With g_se = dloss_s E n_se / (k L_s^2),
//   softmax: dl_te = p_te (g_se - sum_i p_ti g_si) + dz_s 2 lse_t p_te / L_s
//   sigmoid: dl_te = p_te (1 - sigmoid(l_te)) (g_se - sum_i p_ti g_si)
//
// Forward: one pass over the logits.  A block owns a range of rows; each lane
// keeps the sum of p for its own experts in registers, the block adds its warps
// in a fixed order and writes one partial per (block, sequence) that it meets,
// at slot block + sequence (unique, since rows and sequences both ascend).  A
// second kernel adds each sequence's slots in a fixed order.  The counts are
// integers, so shared-memory atomics leave them reproducible.
#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunks = 608;    // partials a sequence may have: four blocks per SM
constexpr int kHistWords = 2048;   // copies of the block's histogram share this many words

struct Partials {
  float* p;        // [slots, E] sums of the scores
  uint32_t* n;     // [slots, E] counts
  float* z;        // [slots] sums of squared log-sum-exps
  uint32_t* rows;  // [slots] valid rows
  uint32_t* bad;   // [slots] indices that are no expert
};

struct FwdArgs {
  const void* logits;
  const uint32_t* idx;
  const uint8_t* mask;
  Seqs seqs;
  int E, k, lpr, copies;
  int64_t T, chunk_rows;
  Partials part;
  float2* row_stats;
  uint32_t* status;
  uint32_t k_magic;  // floor(2^32 / k) + 1 (k > 1): i / k = umulhi(i, magic) while i * k < 2^32
};

// Shift and sum of a row, and its normalised scores: softmax about the row's
// maximum; sigmoid about 0, or about the maximum where all scores are so small
// that their FP32 sum would lose them (sigmoid(l) = exp(l) there).
constexpr float kFarBelow = -60.f;

template <typename T, int VEC, int NV, bool FULL, bool SIG>
__device__ __forceinline__ void row_scores(const RowRegs<T, VEC, NV>& r, const Lanes<FULL>& L, int E, bool ok,
                                           float& shift, float& s, float (&p)[VEC * NV]) {
  constexpr int N = VEC * NV;
  float m = -INFINITY;
#pragma unroll
  for (int n = 0; n < N; ++n) m = fmaxf(m, r[n]);
  m = L.max(m);
  if (!ok) m = 0.f;
  s = 0.f;
  if (SIG && m >= kFarBelow) {
    shift = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!RowRegs<T, VEC, NV>::used(v, L.lpr, E)) {
        p[v] = 0.f;
        continue;
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int n = v * VEC + i;
        p[n] = rcp_fast(1.f + exp2_fast(-r[n] * kLog2e));
        s += p[n];
      }
    }
  } else {
    shift = m;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!RowRegs<T, VEC, NV>::used(v, L.lpr, E)) {
        p[v] = 0.f;
        continue;
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        const int n = v * VEC + i;
        p[n] = exp2_fast((r[n] - m) * kLog2e);
        s += p[n];
      }
    }
  }
  s = L.sum(s);
}

template <typename T, int VEC, int NV, bool FULL, bool SIG>
__global__ void __launch_bounds__(kThreads) balance_fwd_kernel(FwdArgs a) {
  extern __shared__ float smem[];
  constexpr int N = VEC * NV;
  using Row = RowRegs<T, VEC, NV>;
  float* red = smem;                                             // [kWarps][E]
  uint32_t* hist = reinterpret_cast<uint32_t*>(smem + kWarps * a.E);  // [E][copies]
  __shared__ float red_z[kWarps];
  __shared__ uint32_t red_rows[kWarps], red_bad[kWarps];

  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0u;
  const Lanes<FULL> L(a.lpr);
  const T* logits = static_cast<const T*>(a.logits);
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk_rows;
  const int64_t c1 = min(c0 + a.chunk_rows, a.T);

  auto gap = [&](int64_t lo, int64_t hi) {
    for (int64_t t = lo + threadIdx.x; t < hi; t += kThreads) a.row_stats[t] = make_float2(0.f, 0.f);
  };
  auto piece = [&](int seq, int64_t lo, int64_t hi) {
    for (int i = threadIdx.x; i < a.E * a.copies; i += kThreads) hist[i] = 0u;
    __syncthreads();
    // counts of the piece's slots; each thread adds to one of the copies
    uint32_t bad = 0, valid = 0;
    {
      const uint32_t* ip = a.idx + lo * a.k;
      const uint32_t n = (uint32_t)(hi - lo) * (uint32_t)a.k;
      const int copy = lane & (a.copies - 1);
      for (uint32_t i = threadIdx.x; i < n; i += kThreads) {
        if (a.mask && !__ldg(a.mask + lo + (a.k == 1 ? i : __umulhi(i, a.k_magic)))) continue;
        const uint32_t e = __ldg(ip + i);
        if (e < (uint32_t)a.E) atomicAdd(hist + e * a.copies + copy, 1u);
        else ++bad;
      }
    }
    float acc[N];
#pragma unroll
    for (int n = 0; n < N; ++n) acc[n] = 0.f;
    float zacc = 0.f;
    for (int64_t t0 = lo + warp * L.rows; t0 < hi; t0 += kWarps * L.rows) {
      const int64_t t = t0 + L.grp;
      const bool in = t < hi;
      const bool ok = in && (!a.mask || __ldg(a.mask + t));
      Row r;
      r.load(logits + t * a.E, a.E, L.lpr, L.sub, ok, from_f32<T>(-INFINITY));
      float p[N], m, s;
      row_scores<T, VEC, NV, FULL, SIG>(r, L, a.E, ok, m, s, p);
      const float inv = ok ? 1.f / s : 0.f;
#pragma unroll
      for (int n = 0; n < N; ++n) acc[n] = fmaf(p[n], inv, acc[n]);
      if (L.sub == 0 && in) {
        a.row_stats[t] = ok ? make_float2(m, s) : make_float2(0.f, 0.f);
        if (ok) {
          ++valid;
          if (!SIG) {
            const float lse = m + logf(s);
            zacc = fmaf(lse, lse, zacc);
          }
        }
      }
    }
    // the rows of a warp, then the warps, in a fixed order
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      if (!FULL && d >= L.lpr) {
#pragma unroll
        for (int n = 0; n < N; ++n) acc[n] += __shfl_xor_sync(0xffffffffu, acc[n], d);
      }
      zacc += __shfl_xor_sync(0xffffffffu, zacc, d);
      valid += __shfl_xor_sync(0xffffffffu, valid, d);
      bad += __shfl_xor_sync(0xffffffffu, bad, d);
    }
    if (L.grp == 0) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int e = Row::elem(n / VEC, n % VEC, L.lpr, L.sub);
        if (e < a.E) red[warp * a.E + e] = acc[n];
      }
    }
    if (lane == 0) red_z[warp] = zacc, red_rows[warp] = valid, red_bad[warp] = bad;
    __syncthreads();
    const int64_t slot = (int64_t)blockIdx.x + seq;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += red[w * a.E + e];
      uint32_t c = 0;
      for (int i = 0; i < a.copies; ++i) c += hist[e * a.copies + i];
      a.part.p[slot * a.E + e] = s;
      a.part.n[slot * a.E + e] = c;
    }
    if (threadIdx.x == 0) {
      float z = 0.f;
      uint32_t v = 0, b = 0;
      for (int w = 0; w < kWarps; ++w) z += red_z[w], v += red_rows[w], b += red_bad[w];
      a.part.z[slot] = z;
      a.part.rows[slot] = v;
      a.part.bad[slot] = b;
    }
    __syncthreads();  // before the next piece writes the shared arrays
  };
  walk_sequences(a.seqs, c0, c1, piece, gap);
}

struct FinishArgs {
  Partials part;
  Seqs seqs;
  int E, k;
  int64_t chunk_rows;
  float* loss;
  float* z_loss;
  float* mean_scores;
  uint32_t* counts;
  uint32_t* tokens;
  uint32_t* status;
};

// One block per sequence: 32 experts x 8 slot lanes at a time.
__global__ void __launch_bounds__(kThreads) balance_finish_kernel(FinishArgs a) {
  __shared__ float sp[kWarps][33];
  __shared__ uint32_t sn[kWarps][33];
  __shared__ double sl[32];
  __shared__ float sz[kThreads];
  __shared__ uint32_t sv[kThreads], sb[kThreads];
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t lo = a.seqs.at(s), hi = a.seqs.at(s + 1);
  if (threadIdx.x == 0 && a.seqs.off &&
      (hi < lo || (int64_t)__ldg(a.seqs.off + s) > a.seqs.T || (int64_t)__ldg(a.seqs.off + s + 1) > a.seqs.T))
    set_status(a.status, MOE_ERR_INVALID_INDEX);
  // slots first..last hold the sequence
  int64_t first = 0, last = -1;
  if (hi > lo) {
    first = lo / a.chunk_rows + s;
    last = (hi - 1) / a.chunk_rows + s;
  }
  float z = 0.f;
  uint32_t valid = 0, bad = 0;
  for (int64_t i = first + threadIdx.x; i <= last; i += kThreads) {
    z += a.part.z[i];
    valid += a.part.rows[i];
    bad += a.part.bad[i];
  }
  sz[threadIdx.x] = z, sv[threadIdx.x] = valid, sb[threadIdx.x] = bad;
  __syncthreads();
  for (int d = kThreads / 2; d > 0; d >>= 1) {
    if (threadIdx.x < d) {
      sz[threadIdx.x] += sz[threadIdx.x + d];
      sv[threadIdx.x] += sv[threadIdx.x + d];
      sb[threadIdx.x] += sb[threadIdx.x + d];
    }
    __syncthreads();
  }
  const uint32_t rows = sv[0];
  if (threadIdx.x == 0 && sb[0]) set_status(a.status, MOE_ERR_INVALID_INDEX);
  const float inv = rows ? 1.f / (float)rows : 0.f;
  double dot = 0.0;
  for (int e0 = 0; e0 < a.E; e0 += 32) {
    const int e = e0 + lane;
    float p = 0.f;
    uint32_t n = 0;
    if (e < a.E)
      for (int64_t i = first + warp; i <= last; i += kWarps) {
        p += a.part.p[i * a.E + e];
        n += a.part.n[i * a.E + e];
      }
    sp[warp][lane] = p;
    sn[warp][lane] = n;
    __syncthreads();
    if (warp == 0 && e < a.E) {
      p = 0.f, n = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) p += sp[w][lane], n += sn[w][lane];
      a.counts[(int64_t)s * a.E + e] = n;
      if (a.mean_scores) a.mean_scores[(int64_t)s * a.E + e] = p * inv;
      dot += (double)n * (double)p;
    }
    __syncthreads();
  }
  if (warp == 0) sl[lane] = dot;
  __syncwarp();
  if (threadIdx.x == 0) {
    dot = 0.0;
    for (int i = 0; i < 32; ++i) dot += sl[i];
    const double L = (double)rows;
    a.loss[s] = rows ? (float)((double)a.E * dot / ((double)a.k * L * L)) : 0.f;
    if (a.z_loss) a.z_loss[s] = rows ? sz[0] / (float)rows : 0.f;
    a.tokens[s] = rows;
  }
}

struct BwdArgs {
  const void* logits;
  const float2* row_stats;
  const uint32_t* counts;
  const uint32_t* tokens;
  const float* dloss;
  const float* dz;
  Seqs seqs;
  int E, k, lpr;
  int64_t T, chunk_rows;
  const void* base;
  void* out;
};

template <typename T, int VEC, int NV, bool FULL, bool SIG>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(BwdArgs a) {
  constexpr int N = VEC * NV;
  using Row = RowRegs<T, VEC, NV>;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const Lanes<FULL> L(a.lpr);
  const T* logits = static_cast<const T*>(a.logits);
  const T* base = static_cast<const T*>(a.base);
  T* out = static_cast<T*>(a.out);
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk_rows;
  const int64_t c1 = min(c0 + a.chunk_rows, a.T);

  auto finish = [&](int64_t t, bool in, float (&d)[N]) {
    if (!in) return;
    if (base) {
      Row b;
      b.load(base + t * a.E, a.E, L.lpr, L.sub, true, from_f32<T>(0.f));
#pragma unroll
      for (int n = 0; n < N; ++n) d[n] += b[n];
    }
    store_row<T, VEC, NV>(out + t * a.E, a.E, L.lpr, L.sub, d);
  };
  auto gap = [&](int64_t lo, int64_t hi) {
    for (int64_t t0 = lo + warp * L.rows; t0 < hi; t0 += kWarps * L.rows) {
      float d[N];
#pragma unroll
      for (int n = 0; n < N; ++n) d[n] = 0.f;
      finish(t0 + L.grp, t0 + L.grp < hi, d);
    }
  };
  auto piece = [&](int seq, int64_t lo, int64_t hi) {
    // g about an even load, (E n - k L) / (k L^2): exact in integers, and the
    // scores sum to one, so a constant taken from g changes nothing
    const int64_t rows = (int64_t)__ldg(a.tokens + seq);
    const double kl = (double)a.k * (double)rows;
    const float up = rows ? (float)((double)__ldg(a.dloss + seq) / (kl * (double)rows)) : 0.f;
    const float zc = !SIG && a.dz && rows ? 2.f * __ldg(a.dz + seq) / (float)rows : 0.f;
    float g[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int e = Row::elem(n / VEC, n % VEC, L.lpr, L.sub);
      const int64_t c = e < a.E ? (int64_t)__ldg(a.counts + (int64_t)seq * a.E + e) : 0;
      g[n] = up * (float)(c * a.E - rows * a.k);
    }
    for (int64_t t0 = lo + warp * L.rows; t0 < hi; t0 += kWarps * L.rows) {
      const int64_t t = t0 + L.grp;
      const bool in = t < hi;
      const float2 st = in ? __ldg(a.row_stats + t) : make_float2(0.f, 0.f);
      const bool ok = st.y != 0.f;  // NaN sums count: their rows get NaN
      Row r;
      r.load(logits + t * a.E, a.E, L.lpr, L.sub, in && ok, from_f32<T>(-INFINITY));
      const float inv = ok ? 1.f / st.y : 0.f;
      float d[N], dot = 0.f;
#pragma unroll
      for (int n = 0; n < N; ++n) {
        float p, up1 = 1.f;
        if (SIG && st.x == 0.f) {
          const float ex = exp2_fast(-fabsf(r[n]) * kLog2e);  // sigmoid(|l|) = 1 / (1 + ex)
          const float hi1 = rcp_fast(1.f + ex);
          const float lo1 = ex * hi1;
          p = (r[n] > 0.f ? hi1 : lo1) * inv;
          up1 = r[n] > 0.f ? lo1 : hi1;
          if (r[n] != r[n]) p = r[n];
        } else {
          p = exp2_fast((r[n] - st.x) * kLog2e) * inv;
        }
        dot = fmaf(p, g[n], dot);
        d[n] = p * up1;
      }
      dot = L.sum(dot);
      if (!SIG) dot -= zc * (st.x + logf(st.y));
#pragma unroll
      for (int n = 0; n < N; ++n) d[n] = ok ? d[n] * (g[n] - dot) : 0.f;
      finish(t, in, d);
    }
  };
  walk_sequences(a.seqs, c0, c1, piece, gap);
}

int hist_copies(int E) {
  int c = 32;
  while (c > 1 && c * E > kHistWords) c /= 2;
  return c;
}

template <bool SIG>
struct LaunchFwd {
  FwdArgs a;
  int chunks;
  size_t smem;
  cudaStream_t s;
  template <typename T, int VEC, int NV, bool FULL>
  cudaError_t run() {
    return launch_pdl(balance_fwd_kernel<T, VEC, NV, FULL, SIG>, dim3((unsigned)chunks), dim3(kThreads), smem, s, a);
  }
};

template <bool SIG>
struct LaunchBwd {
  BwdArgs a;
  int chunks;
  cudaStream_t s;
  template <typename T, int VEC, int NV, bool FULL>
  cudaError_t run() {
    return launch_pdl(balance_bwd_kernel<T, VEC, NV, FULL, SIG>, dim3((unsigned)chunks), dim3(kThreads), 0, s, a);
  }
};

}  // namespace

size_t balance_workspace_bytes(int64_t T, int E, int64_t num_seqs) {
  const size_t slots = (size_t)(kMaxChunks < T ? kMaxChunks : T) + (size_t)num_seqs;
  return align_up(slots * (size_t)E * 8 + slots * 12, 256);
}

cudaError_t launch_balance_loss(const BalanceArgs& b, void* ws, uint32_t* status, cudaStream_t s) {
  const void* ptrs[] = {b.logits};
  const RowPlan plan = row_plan(ptrs, 1, b.dt, b.E);
  const Chunks ch = cut_rows(b.T, (int64_t)kWarps * (32 / plan.lpr), kMaxChunks);
  const size_t slots = (size_t)(kMaxChunks < b.T ? kMaxChunks : b.T) + (size_t)b.num_seqs;
  Partials part;
  part.p = static_cast<float*>(ws);
  part.n = reinterpret_cast<uint32_t*>(part.p + slots * b.E);
  part.z = reinterpret_cast<float*>(part.n + slots * b.E);
  part.rows = reinterpret_cast<uint32_t*>(part.z + slots);
  part.bad = part.rows + slots;
  FwdArgs a{};
  a.logits = b.logits;
  a.idx = b.idx;
  a.mask = b.mask;
  a.seqs = Seqs{b.seq_offsets, (int)b.num_seqs, b.T};
  a.E = b.E;
  a.k = b.k;
  a.lpr = plan.lpr;
  a.copies = hist_copies(b.E);
  a.T = b.T;
  a.chunk_rows = ch.rows;
  a.part = part;
  a.row_stats = reinterpret_cast<float2*>(b.row_stats);
  a.status = status;
  a.k_magic = b.k == 1 ? 0u : (uint32_t)((1ull << 32) / (uint32_t)b.k) + 1u;
  const size_t smem = (size_t)kWarps * b.E * 4 + (size_t)a.copies * b.E * 4;
  cudaError_t e;
  if (b.sigmoid) {
    LaunchFwd<true> f{a, ch.chunks, smem, s};
    e = with_row_variant(b.dt, plan, f);
  } else {
    LaunchFwd<false> f{a, ch.chunks, smem, s};
    e = with_row_variant(b.dt, plan, f);
  }
  if (e != cudaSuccess) return e;
  FinishArgs f{part, a.seqs, b.E, b.k, ch.rows, b.loss, b.z_loss, b.mean_scores, b.counts, b.tokens, status};
  return launch_pdl(balance_finish_kernel, dim3((unsigned)b.num_seqs), dim3(kThreads), 0, s, f);
}

cudaError_t launch_balance_loss_backward(const BalanceBwdArgs& b, cudaStream_t s) {
  const void* ptrs[] = {b.logits, b.base, b.dlogits};
  const RowPlan plan = row_plan(ptrs, 3, b.dt, b.E);
  const Chunks ch = cut_rows(b.T, (int64_t)kWarps * (32 / plan.lpr), 152 * 8);
  BwdArgs a{};
  a.logits = b.logits;
  a.row_stats = reinterpret_cast<const float2*>(b.row_stats);
  a.counts = b.counts;
  a.tokens = b.tokens;
  a.dloss = b.dloss;
  a.dz = b.dz_loss;
  a.seqs = Seqs{b.seq_offsets, (int)b.num_seqs, b.T};
  a.E = b.E;
  a.k = b.k;
  a.lpr = plan.lpr;
  a.T = b.T;
  a.chunk_rows = ch.rows;
  a.base = b.base;
  a.out = b.dlogits;
  if (b.sigmoid) {
    LaunchBwd<true> f{a, ch.chunks, s};
    return with_row_variant(b.dt, plan, f);
  }
  LaunchBwd<false> f{a, ch.chunks, s};
  return with_row_variant(b.dt, plan, f);
}

}  // namespace moe
