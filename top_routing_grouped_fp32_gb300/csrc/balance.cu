// balance.cu -- the router's balance loss with per-expert counts and its z-loss
// (their gradient is in balance_bwd.cu).
//
// For the valid rows V_s of a sequence s (L_s of them), row scores p_te that sum
// to one over the experts and the routed slots idx [T,k]:
//   n_se   = #{(t, j) : t in V_s, idx_tj = e}
//   P_se   = 1/L_s sum_{t in V_s} p_te
//   loss_s = E sum_e n_se / (k L_s) P_se
//   z_s    = 1/L_s sum_{t in V_s} (log sum_e exp l_te)^2
//
// One pass over the logits.  A block owns a range of rows; each lane keeps the sum
// of p for its own experts in registers, the block adds its warps in a fixed order
// and writes one partial per (block, sequence) that it meets, at slot
// block + sequence (unique, since rows and sequences both ascend).  A second kernel
// adds each sequence's slots in a fixed order; a batch that one block holds needs
// none.  The counts are integers, so shared-memory atomics leave them reproducible.
//
// 524288 rows of 256 BF16 logits, top-8: 57 us, 75 % of the copy bandwidth; the main
// kernel alone takes 54 us (285 MB read, 69 instructions a row, 2.4 a cycle of a SM).
// The sums and the scores of a lane's 32 elements leave room for 16 warps a SM.  With
// sigmoid scores 70 us: two special functions a score instead of one.
#include <cooperative_groups.h>

#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHistWords = 2048;   // copies of the block's histogram share this many words

struct Partials {
  float* p;           // [slots, E] sums of the scores
  uint32_t* n;        // [slots, E] counts
  float* z;           // [slots] sums of squared log-sum-exps
  uint32_t* rows;     // [slots] valid rows
  uint32_t* bad;      // [slots] indices that are no expert
};

struct Results {
  float* loss;
  float* z_loss;       // nullable
  float* mean_scores;  // nullable
  uint32_t* counts;
  uint32_t* tokens;
  uint32_t* status;
};

// E sum n/(k L) P/L from the sum of n P_sum, without the products of large numbers
__device__ __forceinline__ float balance_of(float sum_np, int E, int k, uint32_t rows) {
  const float len = (float)rows;
  return rows ? sum_np / len * ((float)E / (float)k) / len : 0.f;
}

struct FwdArgs {
  const void* logits;
  const uint32_t* idx;
  const uint8_t* mask;
  Seqs seqs;
  int E, k, lpr, copies;
  int64_t T, chunk_rows;
  Partials part;
  float2* row_stats;
  uint32_t k_magic;  // floor(2^32 / k) + 1 (k > 1): i / k = umulhi(i, magic) while i * k < 2^32
  bool alone;        // the only block of one sequence: it writes the results
  Results res;
};

// Sigmoid scores are normalised about 0, or about the row's maximum where all of
// them are so small that sigmoid(l) = exp(l) to FP32.
constexpr float kFarBelow = -20.f;

// Scores of a row about `shift`, not normalised.
template <bool SIG, typename Row>
__device__ __forceinline__ void row_scores(const Row& r, float m, float& shift, float (&p)[Row::N]) {
  if (SIG && m >= kFarBelow) {
    shift = 0.f;
    pairwise<Row::N>(
        [&](int n) {
          // A reciprocal a score: 524288 x 256 BF16 logits take 70 us.  One for two, 1/a =
          // b / (a b), has to keep both below 2^63: it took 79 us and lost scores below 2^-63.
          const float2 x = mul2(make_float2(r[n], r[n + 1]), both(-kLog2e));
          const float2 y = add2(make_float2(exp2_fast(x.x), exp2_fast(x.y)), both(1.f));
          p[n] = rcp_fast(y.x);
          p[n + 1] = rcp_fast(y.y);
        },
        [&](int n) { p[n] = rcp_fast(1.f + exp2_fast(r[n] * -kLog2e)); });
  } else {
    shift = m;
    RowExp(m, kLog2e).row(r, p);
  }
}

template <typename T, int VEC, int NV, int LPR, bool SIG>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<T, VEC, NV>()) balance_fwd_kernel(FwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  constexpr int NI = 4;  // slots that a lane counts at once
  using Stream = RowStream<T, VEC, NV, LPR>;
  using Row = typename Stream::Row;
  constexpr int N = Row::N, S = Stream::kStages;
  float* red = reinterpret_cast<float*>(smem + kWarps * Stream::kWarpBytes);  // [kWarps][E]
  uint32_t* hist = reinterpret_cast<uint32_t*>(red + kWarps * a.E);           // [E][copies]
  __shared__ float red_z[kWarps], red_np[kWarps];
  __shared__ uint32_t red_rows[kWarps], red_bad[kWarps];

  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.res.status = 0u;
  const Lanes<LPR> L(a.lpr);
  Stream rows(L, smem, a.logits, a.E, a.T);
  const int copy = lane & (a.copies - 1), copies_log = __popc(a.copies - 1);  // its copy of the histogram
  const int batch = L.rows;                // consecutive rows that a warp takes at once
  const int step = kWarps * batch;

  auto gap = [&](int64_t lo, int64_t hi) {
    for (int64_t t = lo + threadIdx.x; t < hi; t += kThreads) a.row_stats[t] = make_float2(0.f, 0.f);
  };
  // The piece of a sequence that the block works on, and the state of this warp in it.
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk_rows, c1 = min(c0 + a.chunk_rows, a.T);
  int seq = 0;
  int64_t lo = 0, hi = a.T;
  int64_t t0;  // the batch's first row
  int left;    // rows from there on (a block has far fewer than 2^31)
  // does this group's row of a batch count: bit i for the i-th batch from here.
  // The mask's byte is fetched a batch before its bit is needed.
  uint32_t on;
  uint8_t byte;
  auto fetch = [&](int ahead) {
    const int i = ahead * step + L.grp;
    if (a.mask) byte = i < left ? __ldg(a.mask + t0 + i) : 0;
  };
  auto bit = [&](int ahead) { return (uint32_t)(ahead * step + L.grp < left && byte) << ahead; };
  // Counts of the piece's slots, 32 NI a warp at a time and behind the rows: 256
  // experts' rows with top-8 take a turn in four batches.  A turn's indices are on
  // their way since the last one; a lane adds to its copy.
  int slots, at;
  const uint32_t* ip;
  uint32_t id[NI];
  auto indices = [&]() {
    if (at + 32 * NI <= slots) {
#pragma unroll
      for (int i = 0; i < NI; ++i) id[i] = __ldg(ip + at + 32 * i);
    } else {
#pragma unroll
      for (int i = 0; i < NI; ++i) id[i] = at + lane + 32 * i < slots ? __ldg(ip + at + 32 * i) : 0u;
    }
  };
  // Asks for a piece's first rows and indices.
  auto begin = [&]() {
    t0 = lo + warp * batch;
    left = (int)(hi - t0);
    rows.start(t0, step);
    on = 0;
    byte = 1;
    uint8_t early[S];
#pragma unroll
    for (int i = 0; i < S; ++i) {
      fetch(i);
      early[i] = byte;
    }
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      byte = early[i];
      on |= bit(i);
      rows.template issue<true>(on >> i & 1u);
    }
    byte = early[S - 1];
    slots = (int)(hi - lo) * a.k;
    at = warp * 32 * NI;
    ip = a.idx + lo * a.k + lane;
    indices();
  };
  // The next piece from sequence s and row `from` on, if the block has one; rows
  // before it that lie in no sequence get their zeros.
  auto advance = [&](int s, int64_t from) {
    for (; from < c1; ++s) {
      if (s >= a.seqs.num) {
        gap(from, c1);
        return false;
      }
      lo = min(max(a.seqs.at(s), from), c1);
      hi = min(max(a.seqs.at(s + 1), lo), c1);
      if (lo > from) gap(from, lo);
      from = hi;
      seq = s;
      if (hi > lo) return true;
    }
    return false;
  };

  bool more = a.alone || advance(a.seqs.first(c0), c0);
  if (more) begin();
  while (more) {
    for (int i = threadIdx.x; i < a.E * a.copies; i += kThreads) hist[i] = 0u;
    __syncthreads();
    uint32_t bad = 0, valid = 0;
    float acc[N], zacc = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) acc[n] = 0.f;
    auto count = [&]() {
      if (!a.mask && at + 32 * NI <= slots) {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          if (id[i] < (uint32_t)a.E) atomicAdd(hist + (id[i] << copies_log) + copy, 1u);
          else ++bad;
        }
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          const int slot = at + lane + 32 * i;
          bool counts = slot < slots;
          if (a.mask && counts) counts = __ldg(a.mask + lo + (a.k == 1 ? slot : (int)__umulhi(slot, a.k_magic)));
          if (counts && id[i] < (uint32_t)a.E) atomicAdd(hist + (id[i] << copies_log) + copy, 1u);
          bad += counts && id[i] >= (uint32_t)a.E;
        }
      }
      at += kWarps * 32 * NI;
      indices();
    };
    int due = 0;  // slots of the rows that the block's warps have taken
    // A lane keeps the maximum and sum of its group's row of every lpr-th batch; then
    // the whole warp writes a row's statistics a lane.
    int turn = 0;
    float kept_m = 0.f, kept_s = 0.f;
    auto flush = [&]() {  // the batches from t0 - turn * step on
      const int64_t t = t0 + (L.sub - turn) * step + L.grp;
      const bool o = kept_s != 0.f;  // NaN sums count
      const float s = !SIG || kept_m != 0.f ? kept_s * RowExp(kept_m, kLog2e).fix() : kept_s;
      if (L.sub < turn && t < hi) {
        a.row_stats[t] = make_float2(kept_m, s);
        valid += o;
        if (!SIG && o) {
          const float lse = fmaf(log2_fast(s), kLn2, kept_m);
          zacc = fmaf(lse, lse, zacc);
        }
      }
      turn = 0;
    };
    while (left > 0) {
      Row cur;
      rows.take(cur);
      on |= bit(S - 1);
      rows.template issue<true>(on >> (S - 1) & 1u);  // (a zero row's scores times 0: no branch)
      fetch(S);
      const bool ok = on & 1u;
      if (Stream::kImage && !ok) cur.zero(rows.room, L.lpr);
      float p[N], m = L.max(cur.lane_max());
      row_scores<SIG>(cur, m, m, p);
      const float s = L.sum(lane_sum(p));
      const float inv = ok ? rcp_fast(s) : 0.f;  // p carries the factor that fix() takes out, too
      pairwise<N>([&](int n) { put(acc, n, fma2(pair(p, n), both(inv), pair(acc, n))); },
                  [&](int n) { acc[n] = fmaf(p[n], inv, acc[n]); });
      if (L.sub == turn) kept_m = ok ? m : 0.f, kept_s = ok ? s : 0.f;
      due += step * a.k;
      while (at < min(due, slots)) count();
      on >>= 1;
      t0 += step;
      left -= step;
      if (++turn == L.lpr) flush();
    }
    flush();
    while (at < slots) count();
    rows.drain();
    // the next piece's rows are on their way while this one's sums are added
    const int64_t slot = (int64_t)blockIdx.x + seq;
    more = !a.alone && advance(seq + 1, hi);
    if (more) begin();
    // the rows of a warp, then the warps, in a fixed order
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      if (d >= L.lpr) {
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
        const int e = Row::elem(n, L.lpr, L.sub);
        if (e < a.E) red[warp * a.E + e] = acc[n];
      }
    }
    if (lane == 0) red_z[warp] = zacc, red_rows[warp] = valid, red_bad[warp] = bad;
    __syncthreads();
    float z = 0.f, np = 0.f;
    uint32_t rows = 0, wrong = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) z += red_z[w], rows += red_rows[w], wrong += red_bad[w];
    const float inv = rows ? 1.f / (float)rows : 0.f;
    for (int e = threadIdx.x; e < a.E; e += kThreads) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s += red[w * a.E + e];
      uint32_t c = 0;
      for (int i = 0; i < a.copies; ++i) c += hist[e * a.copies + i];
      if (a.alone) {
        a.res.counts[e] = c;
        if (a.res.mean_scores) a.res.mean_scores[e] = rows ? s * inv : 0.f;
        np = fmaf((float)c, s, np);
      } else {
        a.part.p[slot * a.E + e] = s;
        a.part.n[slot * a.E + e] = c;
      }
    }
    if (a.alone) {
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) np += __shfl_xor_sync(0xffffffffu, np, d);
      if (lane == 0) red_np[warp] = np;
      __syncthreads();
    }
    if (threadIdx.x == 0) {
      if (a.alone) {
        np = 0.f;
        for (int w = 0; w < kWarps; ++w) np += red_np[w];
        a.res.loss[0] = balance_of(np, a.E, a.k, rows);
        if (a.res.z_loss) a.res.z_loss[0] = rows ? z * inv : 0.f;
        a.res.tokens[0] = rows;
        if (wrong) set_status(a.res.status, MOE_ERR_INVALID_INDEX);
      } else {
        a.part.z[slot] = z;
        a.part.rows[slot] = rows;
        a.part.bad[slot] = wrong;
      }
    }
    __syncthreads();  // before the next piece writes the shared arrays
  }
  rows.drain();
}

struct FinishArgs {
  Partials part;
  Seqs seqs;
  int E, k;
  int64_t chunk_rows;
  Results res;
};

// Slots first, .., first + count - 1 hold sequence s (rows fit 32 bits).
struct SlotRange {
  int64_t first;
  int count;
  __device__ __forceinline__ SlotRange(const FinishArgs& a, uint32_t s, uint32_t lo, uint32_t hi) {
    const uint32_t chunk = (uint32_t)a.chunk_rows, from = lo / chunk;
    count = hi > lo ? (int)((hi - 1) / chunk - from) + 1 : 0;
    first = (int64_t)from + s;
  }
};
__device__ __forceinline__ bool malformed(const Seqs& q, uint32_t s, uint32_t lo, uint32_t hi) {
  return q.off && (hi < lo || (int64_t)__ldg(q.off + s) > q.T || (int64_t)__ldg(q.off + s + 1) > q.T);
}
template <typename V>
__device__ __forceinline__ V warp_sum(V x) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

// Few slots a sequence: a block for each, a thread for each expert, which adds the
// slots one after another, 16 on their way at a time.  The whole loss of 65537 rows
// of 256 FP32 logits in 128 sequences (2.4 slots each) takes 24 us with it and 31 us
// with the kernel below; in 37 sequences (8.2 each, some of them long) 27 and 25 us.
__global__ void __launch_bounds__(1024) balance_finish_few_kernel(FinishArgs a) {
  __shared__ float snp[32];
  pdl_wait();
  pdl_trigger();
  const uint32_t s = blockIdx.x;
  const int e = threadIdx.x, warp = e >> 5, lane = e & 31;
  const uint32_t lo = (uint32_t)a.seqs.at(s), hi = (uint32_t)a.seqs.at(s + 1);
  const SlotRange r(a, s, lo, hi);
  constexpr int U = 16;
  float ps = 0.f, z = 0.f;
  uint32_t ns = 0, rows = 0, bad = 0;
  for (int i0 = 0; i0 < r.count; i0 += U) {
    float p[U], zz[U];
    uint32_t n[U], v[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t i = r.first + i0 + u;
      const bool in = i0 + u < r.count;
      p[u] = in && e < a.E ? __ldcg(a.part.p + i * a.E + e) : 0.f;
      n[u] = in && e < a.E ? __ldcg(a.part.n + i * a.E + e) : 0u;
      v[u] = in ? __ldcg(a.part.rows + i) : 0u;
      zz[u] = in && e == 0 ? __ldcg(a.part.z + i) : 0.f;
      b[u] = in && e == 0 ? __ldcg(a.part.bad + i) : 0u;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) ps += p[u], ns += n[u], rows += v[u], z += zz[u], bad += b[u];
  }
  if (e < a.E) {
    a.res.counts[(int64_t)s * a.E + e] = ns;
    if (a.res.mean_scores) a.res.mean_scores[(int64_t)s * a.E + e] = rows ? ps / (float)rows : 0.f;
  }
  float np = warp_sum((float)ns * ps);
  if (lane == 0) snp[warp] = np;
  __syncthreads();
  if (warp != 0) return;
  np = warp_sum(lane < (int)(blockDim.x >> 5) ? snp[lane] : 0.f);
  if (lane == 0) {
    a.res.loss[s] = balance_of(np, a.E, a.k, rows);
    if (a.res.z_loss) a.res.z_loss[s] = rows ? z / (float)rows : 0.f;
    a.res.tokens[s] = rows;
    if (bad || malformed(a.seqs, s, lo, hi)) set_status(a.res.status, MOE_ERR_INVALID_INDEX);
  }
}

// Adds a sequence's slots, 32 experts x W slot lanes at a time.  A sequence has a
// cluster of blocks, each with every blocks-th group of 32 experts; block 0 adds
// their shares of the loss in order.
template <int W>
__global__ void __launch_bounds__(32 * W) balance_finish_kernel(FinishArgs a) {
  __shared__ float sp[32][W + 1];
  __shared__ uint32_t sn[32][W + 1];
  __shared__ float sz[W], snp[W], share;
  __shared__ uint32_t sv[W], sb[W];
  cg::cluster_group cl = cg::this_cluster();
  const uint32_t part = cl.block_rank(), blocks = cl.num_blocks();
  const uint32_t s = blockIdx.x / blocks;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_trigger();
  const uint32_t lo = (uint32_t)a.seqs.at(s), hi = (uint32_t)a.seqs.at(s + 1);
  const SlotRange r(a, s, lo, hi);
  const int64_t first = r.first;
  const int count = r.count;
  // every load of a thread is on its way before the first is used: U slots a lane
  constexpr int U = 10;
  auto load = [&](uint32_t e, int i0, float (&p)[U], uint32_t (&n)[U]) {
    const float* pp = a.part.p + (first + i0) * a.E + e;
    const uint32_t* pn = a.part.n + (first + i0) * a.E + e;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = e < (uint32_t)a.E && i0 + u * W < count;
      p[u] = in ? __ldcg(pp + u * W * a.E) : 0.f;
      n[u] = in ? __ldcg(pn + u * W * a.E) : 0u;
    }
  };
  float p[U], z = 0.f, np = 0.f;
  uint32_t n[U], rows = 0, bad = 0;
  load(part * 32 + lane, warp, p, n);
  for (int i = threadIdx.x; i < count; i += 32 * W) {
    z += a.part.z[first + i];
    rows += a.part.rows[first + i];
    bad += a.part.bad[first + i];
  }
  z = warp_sum(z), rows = warp_sum(rows), bad = warp_sum(bad);
  if (lane == 0) sz[warp] = z, sv[warp] = rows, sb[warp] = bad;
  for (uint32_t e0 = part * 32; e0 < (uint32_t)a.E; e0 += blocks * 32) {
    float ps = 0.f;
    uint32_t ns = 0;
    for (int i0 = warp; i0 < count; i0 += U * W) {
      if (i0 != warp || e0 != part * 32) load(e0 + lane, i0, p, n);
#pragma unroll
      for (int u = 0; u < U; ++u) ps += p[u], ns += n[u];
    }
    sp[lane][warp] = ps;
    sn[lane][warp] = ns;
    __syncthreads();
    // a warp for each expert's slot lanes; every W experts
    rows = warp_sum(lane < W ? sv[lane] : 0u);
    const float inv = rows ? 1.f / (float)rows : 0.f;
#pragma unroll
    for (int x = warp; x < 32; x += W) {
      const float px = warp_sum(lane < W ? sp[x][lane] : 0.f);
      const uint32_t nx = warp_sum(lane < W ? sn[x][lane] : 0u);
      if (lane == 0 && e0 + x < (uint32_t)a.E) {
        a.res.counts[(int64_t)s * a.E + e0 + x] = nx;
        if (a.res.mean_scores) a.res.mean_scores[(int64_t)s * a.E + e0 + x] = rows ? px * inv : 0.f;
        np = fmaf((float)nx, px, np);
      }
    }
    __syncthreads();
  }
  if (lane == 0) snp[warp] = np;
  __syncthreads();
  if (warp == 0) {
    np = warp_sum(lane < W ? snp[lane] : 0.f);
    if (lane == 0) share = np;
  }
  if (blocks > 1) cl.sync();
  if (part == 0 && warp == 0) {
    if (blocks > 1) np = warp_sum(lane < (int)blocks ? *cl.map_shared_rank(&share, lane) : 0.f);
    z = warp_sum(lane < W ? sz[lane] : 0.f);
    bad = warp_sum(lane < W ? sb[lane] : 0u);
    rows = warp_sum(lane < W ? sv[lane] : 0u);
    if (lane == 0) {
      a.res.loss[s] = balance_of(np, a.E, a.k, rows);
      if (a.res.z_loss) a.res.z_loss[s] = rows ? z / (float)rows : 0.f;
      a.res.tokens[s] = rows;
      if (bad || malformed(a.seqs, s, lo, hi)) set_status(a.res.status, MOE_ERR_INVALID_INDEX);
    }
  }
  if (blocks > 1) cl.sync();  // the shares are read
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
  template <typename T, int VEC, int NV, int LPR>
  cudaError_t run() {
    static std::atomic<uint64_t> asked{0};
    return launch_rows(balance_fwd_kernel<T, VEC, NV, LPR, SIG>, chunks, kThreads,
                       smem + kWarps * RowStream<T, VEC, NV, LPR>::kWarpBytes, asked, s, a);
  }
};

size_t slot_count(int64_t T, int64_t num_seqs) {
  return (size_t)(kMaxBlocks < T ? kMaxBlocks : T) + (size_t)num_seqs;
}

}  // namespace

size_t balance_workspace_bytes(int64_t T, int E, int64_t num_seqs) {
  const size_t slots = slot_count(T, num_seqs);
  return align_up(slots * (size_t)E * 8 + slots * 12, 256);
}

cudaError_t launch_balance_loss(const BalanceArgs& b, void* ws, uint32_t* status, cudaStream_t s) {
  const void* ptrs[] = {b.logits};
  const RowPlan plan = row_plan(ptrs, 1, b.dt, b.E);
  // sequences are worked off one after another in a block: finer cuts where there are any
  const Chunks ch = b.seq_offsets ? cut_rows(b.T, plan_batch(plan), plan_blocks(plan), 1)
                                  : cut_rows(b.T, (int64_t)kWarps * plan_batch(plan), plan_blocks(plan));
  const size_t slots = slot_count(b.T, b.num_seqs);
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
  a.k_magic = b.k == 1 ? 0u : (uint32_t)((1ull << 32) / (uint32_t)b.k) + 1u;
  a.alone = ch.chunks == 1 && !b.seq_offsets;
  a.res = Results{b.loss, b.z_loss, b.mean_scores, b.counts, b.tokens, status};
  const size_t smem = (size_t)kWarps * b.E * 4 + (size_t)a.copies * b.E * 4;
  cudaError_t e;
  if (b.sigmoid) {
    LaunchFwd<true> f{a, ch.chunks, smem, s};
    e = with_row_variant(b.dt, plan, f);
  } else {
    LaunchFwd<false> f{a, ch.chunks, smem, s};
    e = with_row_variant(b.dt, plan, f);
  }
  if (e != cudaSuccess || a.alone) return e;
  const FinishArgs f{part, a.seqs, b.E, b.k, ch.rows, a.res};
  if (ch.chunks <= 4 * b.num_seqs)
    return launch_pdl(balance_finish_few_kernel, dim3((unsigned)b.num_seqs), dim3((unsigned)(b.E + 31) / 32 * 32), 0, s,
                      f);
  // a block for each group of experts, at most eight (a cluster)
  int blocks = 1;
  while (blocks < 8 && blocks * 32 < b.E) blocks *= 2;
  const bool many = ch.chunks / b.num_seqs >= 32;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(b.num_seqs * blocks));
  cfg.blockDim = dim3(many ? 1024 : 256);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)blocks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = blocks > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, many ? balance_finish_kernel<32> : balance_finish_kernel<8>, f);
}

}  // namespace moe
