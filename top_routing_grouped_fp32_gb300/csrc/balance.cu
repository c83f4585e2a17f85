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
#include <cooperative_groups.h>

#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxChunks = 304;    // partials a sequence may have: two blocks per SM
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

// Sigmoid scores are normalised about 0, or about the row's maximum where all of
// them are so small that their FP32 sum would lose them (sigmoid(l) = exp(l) there).
constexpr float kFarBelow = -60.f;

// Scores of a row about `shift`, not normalised, and their sum over this lane.
template <typename Row, bool SIG>
__device__ __forceinline__ float lane_scores(const Row& r, int lpr, int E, float m, float& shift,
                                             float (&p)[Row::N]) {
  float s = 0.f;
  if (SIG && m >= kFarBelow) {
    shift = 0.f;
#pragma unroll
    for (int n = 0; n < Row::N; ++n) {
      p[n] = rcp_fast(1.f + exp2_fast(r[n] * -kLog2e));
      s += p[n];
    }
    return s;
  }
  shift = m;
  const RowExp ex(m, kLog2e);
  if (ex.wide) {
#pragma unroll
    for (int n = 0; n < Row::N; ++n) s += p[n] = ex.far(r[n]);
  } else {
#pragma unroll
    for (int n = 0; n < Row::N; ++n) s += p[n] = ex(r[n]);
  }
  return s;
}

template <typename T, int VEC, int NV, bool FULL, bool SIG>
__global__ void __launch_bounds__(kThreads, VEC * NV <= 16 ? 2 : 1) balance_fwd_kernel(FwdArgs a) {
  extern __shared__ float smem[];
  constexpr int N = VEC * NV, R = rows_at_once<VEC, NV>();
  constexpr int NI = 4;  // indices of a batch that a lane holds ahead of their use
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
  const int batch = R * L.rows;            // rows a warp takes at once, at most 128
  const int copy = lane & (a.copies - 1);  // its copy of the histogram

  auto gap = [&](int64_t lo, int64_t hi) {
    for (int64_t t = lo + threadIdx.x; t < hi; t += kThreads) a.row_stats[t] = make_float2(0.f, 0.f);
  };
  auto piece = [&](int seq, int64_t lo, int64_t hi) {
    for (int i = threadIdx.x; i < a.E * a.copies; i += kThreads) hist[i] = 0u;
    __syncthreads();
    uint32_t bad = 0, valid = 0;
    float acc[N], zacc = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) acc[n] = 0.f;

    // which rows count, as a bit per row of a batch: loaded a batch before the rows
    auto live = [&](int64_t t) {
      uint32_t bits = 0;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t tr = t + r * L.rows + L.grp;
        bits |= (uint32_t)(tr < hi && (!a.mask || __ldg(a.mask + tr))) << r;
      }
      return bits;
    };
    auto load = [&](Row& r, int64_t t, bool ok) {
      r.load(logits + t * a.E, a.E, L.lpr, L.sub, ok, from_f32<T>(-INFINITY));
    };
    int64_t t0 = lo + (int64_t)warp * batch;
    Row cur[R], nxt[R];
    uint32_t ok = live(t0), ok1 = live(t0 + (int64_t)kWarps * batch);
#pragma unroll
    for (int r = 0; r < R; ++r) load(cur[r], t0 + r * L.rows + L.grp, ok >> r & 1u);
    for (; t0 < hi; t0 += (int64_t)kWarps * batch) {
      // the next batch's rows and this batch's indices are on their way during the arithmetic
      const int64_t t1 = t0 + (int64_t)kWarps * batch;
      const int slots = (int)(min((int64_t)batch, hi - t0)) * a.k;
      const uint32_t* ip = a.idx + t0 * a.k;
      uint32_t id[NI];
#pragma unroll
      for (int i = 0; i < NI; ++i) id[i] = lane + 32 * i < slots ? __ldg(ip + lane + 32 * i) : 0u;
#pragma unroll
      for (int r = 0; r < R; ++r) load(nxt[r], t1 + r * L.rows + L.grp, ok1 >> r & 1u);
      const uint32_t ok2 = live(t1 + (int64_t)kWarps * batch);

      float p[R][N], s[R], m[R];
#pragma unroll
      for (int r = 0; r < R; ++r) m[r] = L.max(cur[r].lane_max());
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = lane_scores<Row, SIG>(cur[r], L.lpr, a.E, m[r], m[r], p[r]);
      L.sums(s);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float inv = rcp_fast(s[r]);  // p carries the factor that fix takes out, too
        if (!SIG || m[r] != 0.f) s[r] *= RowExp(m[r], kLog2e).fix;
        if (ok >> r & 1u) {
#pragma unroll
          for (int n = 0; n < N; ++n) acc[n] = fmaf(p[r][n], inv, acc[n]);
        }
      }
      // a row's statistics leave from its lane r (of few lanes: r, r + lpr, ..)
      for (int q = 0; q < R; q += L.lpr) {
        float mr = 0.f, sr = 0.f;
        bool o = false;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r == q + L.sub) mr = m[r], sr = s[r], o = ok >> r & 1u;
        const int64_t t = t0 + (q + L.sub) * L.rows + L.grp;
        if (q + L.sub < R && t < hi) {
          a.row_stats[t] = o ? make_float2(mr, sr) : make_float2(0.f, 0.f);
          if (o) {
            ++valid;
            if (!SIG) {
              const float lse = mr + logf(sr);
              zacc = fmaf(lse, lse, zacc);
            }
          }
        }
      }
      // counts of the batch's slots; a lane adds to its copy
      auto count = [&](int i, uint32_t e) {
        if (a.mask && !__ldg(a.mask + t0 + (a.k == 1 ? i : (int)__umulhi(i, a.k_magic)))) return;
        if (e < (uint32_t)a.E) atomicAdd(hist + e * a.copies + copy, 1u);
        else ++bad;
      };
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (lane + 32 * i < slots) count(lane + 32 * i, id[i]);
      for (int i = lane + 32 * NI; i < slots; i += 32) count(i, __ldg(ip + i));
#pragma unroll
      for (int r = 0; r < R; ++r) cur[r] = nxt[r];
      ok = ok1, ok1 = ok2;
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

// A cluster of blocks per sequence, each for every CL-th group of 32 experts:
// 32 experts x 32 slot lanes at a time.  Block 0 adds the blocks' shares of the
// loss in order.
constexpr int kFinishThreads = 1024;
constexpr int kFinishWarps = kFinishThreads / 32;

__global__ void __launch_bounds__(kFinishThreads) balance_finish_kernel(FinishArgs a) {
  __shared__ float sp[kFinishWarps][33];
  __shared__ uint32_t sn[kFinishWarps][33];
  __shared__ float sz[kFinishWarps];
  __shared__ uint32_t sv[kFinishWarps], sb[kFinishWarps];
  __shared__ double share;
  cg::cluster_group cl = cg::this_cluster();
  const int rank = (int)cl.block_rank(), blocks = (int)cl.num_blocks();
  const int s = blockIdx.x / blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const int64_t lo = a.seqs.at(s), hi = a.seqs.at(s + 1);
  if (rank == 0 && threadIdx.x == 0 && a.seqs.off &&
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
  for (int64_t i = first + threadIdx.x; i <= last; i += kFinishThreads) {
    z += a.part.z[i];
    valid += a.part.rows[i];
    bad += a.part.bad[i];
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    z += __shfl_xor_sync(0xffffffffu, z, d);
    valid += __shfl_xor_sync(0xffffffffu, valid, d);
    bad += __shfl_xor_sync(0xffffffffu, bad, d);
  }
  if (lane == 0) sz[warp] = z, sv[warp] = valid, sb[warp] = bad;
  double dot = 0.0;
  uint32_t rows = 0;
  for (int e0 = rank * 32; e0 < a.E; e0 += blocks * 32) {
    const int e = e0 + lane;
    float p = 0.f;
    uint32_t n = 0;
    if (e < a.E) {
#pragma unroll 4
      for (int64_t i = first + warp; i <= last; i += kFinishWarps) {
        p += a.part.p[i * a.E + e];
        n += a.part.n[i * a.E + e];
      }
    }
    sp[warp][lane] = p;
    sn[warp][lane] = n;
    __syncthreads();
    // warp w now adds the slot lanes of expert w
    p = sp[lane][warp], n = sn[lane][warp];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      p += __shfl_xor_sync(0xffffffffu, p, d);
      n += __shfl_xor_sync(0xffffffffu, n, d);
    }
    __syncthreads();
    if (lane == 0) sp[0][warp] = p, sn[0][warp] = n;
    __syncthreads();
    if (warp == 0) {
      rows = 0;
      for (int w = 0; w < kFinishWarps; ++w) rows += sv[w];
      p = sp[0][lane], n = sn[0][lane];
      if (e < a.E) {
        a.counts[(int64_t)s * a.E + e] = n;
        if (a.mean_scores) a.mean_scores[(int64_t)s * a.E + e] = rows ? p / (float)rows : 0.f;
        dot += (double)n * (double)p;
      }
    }
    __syncthreads();
  }
  if (warp == 0) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, d);
    if (lane == 0) share = dot;
  }
  cl.sync();
  if (rank == 0 && threadIdx.x == 0) {
    dot = 0.0;
    for (int b = 0; b < blocks; ++b) dot += *cl.map_shared_rank(&share, b);
    float zz = 0.f;
    uint32_t b = 0;
    rows = 0;
    for (int w = 0; w < kFinishWarps; ++w) zz += sz[w], rows += sv[w], b += sb[w];
    const double len = (double)rows;
    a.loss[s] = rows ? (float)((double)a.E * dot / ((double)a.k * len * len)) : 0.f;
    if (a.z_loss) a.z_loss[s] = rows ? zz / (float)rows : 0.f;
    a.tokens[s] = rows;
    if (b) set_status(a.status, MOE_ERR_INVALID_INDEX);
  }
  cl.sync();  // the shares are read
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
__global__ void __launch_bounds__(kThreads, VEC * NV <= 16 ? 2 : 1) balance_bwd_kernel(BwdArgs a) {
  constexpr int N = VEC * NV, R = rows_at_once<VEC, NV>();
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
  const int batch = R * L.rows;

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
    auto stats = [&](int64_t t) { return t < hi ? __ldg(a.row_stats + t) : make_float2(0.f, 0.f); };
    // rows that do not count (a sum of 0) are not read
    auto load = [&](Row& r, int64_t t, float2 st) {
      r.load(logits + t * a.E, a.E, L.lpr, L.sub, st.y != 0.f, from_f32<T>(-INFINITY));
    };
    int64_t t0 = lo + (int64_t)warp * batch;
    Row cur[R], nxt[R];
    float2 st[R], st1[R];  // a batch ahead of the rows
#pragma unroll
    for (int r = 0; r < R; ++r) {
      st[r] = stats(t0 + r * L.rows + L.grp);
      st1[r] = stats(t0 + (int64_t)kWarps * batch + r * L.rows + L.grp);
    }
#pragma unroll
    for (int r = 0; r < R; ++r) load(cur[r], t0 + r * L.rows + L.grp, st[r]);
    for (; t0 < hi; t0 += (int64_t)kWarps * batch) {
      const int64_t t1 = t0 + (int64_t)kWarps * batch;
      float2 st2[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        load(nxt[r], t1 + r * L.rows + L.grp, st1[r]);
        st2[r] = stats(t1 + (int64_t)kWarps * batch + r * L.rows + L.grp);
      }
      float d[R][N], dot[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        dot[r] = 0.f;
        if (SIG && st[r].x == 0.f) {
          const float inv = rcp_fast(st[r].y);
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const float x = cur[r][n];
            const float ex = exp2_fast(fabsf(x) * -kLog2e);  // sigmoid(|l|) = 1 / (1 + ex)
            const float up1 = rcp_fast(1.f + ex), lo1 = ex * up1;
            const float p = (x < 0.f ? lo1 : up1) * inv;
            dot[r] = fmaf(p, g[n], dot[r]);
            d[r][n] = p * (x < 0.f ? up1 : lo1);
          }
        } else {
          const RowExp ex(st[r].x, kLog2e);
          const float inv = rcp_fast(st[r].y) * ex.fix;
          if (ex.wide) {
#pragma unroll
            for (int n = 0; n < N; ++n) d[r][n] = ex.far(cur[r][n]) * inv;
          } else {
#pragma unroll
            for (int n = 0; n < N; ++n) d[r][n] = ex(cur[r][n]) * inv;
          }
#pragma unroll
          for (int n = 0; n < N; ++n) dot[r] = fmaf(d[r][n], g[n], dot[r]);
        }
      }
      L.sums(dot);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        // rows that do not count have a sum of 0; NaN sums leave NaN
        const bool ok = st[r].y != 0.f;
        if (!SIG && a.dz) dot[r] -= zc * (st[r].x + logf(st[r].y));
#pragma unroll
        for (int n = 0; n < N; ++n) d[r][n] = ok ? d[r][n] * (g[n] - dot[r]) : 0.f;
        const int64_t t = t0 + r * L.rows + L.grp;
        finish(t, t < hi, d[r]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) cur[r] = nxt[r], st[r] = st1[r], st1[r] = st2[r];
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
  // one block per group of experts while that leaves SMs without work, at most eight
  int blocks = 1;
  while (blocks < 8 && blocks * 32 < b.E && b.num_seqs * blocks < 152) blocks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(b.num_seqs * blocks));
  cfg.blockDim = dim3(kFinishThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, balance_finish_kernel, f);
}

cudaError_t launch_balance_loss_backward(const BalanceBwdArgs& b, cudaStream_t s) {
  const void* ptrs[] = {b.logits, b.base, b.dlogits};
  const RowPlan plan = row_plan(ptrs, 3, b.dt, b.E);
  const Chunks ch = cut_rows(b.T, (int64_t)kWarps * (32 / plan.lpr), 2 * kMaxChunks);
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
