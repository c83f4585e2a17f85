// distill_bwd.cu -- the gradient of the distillation loss (distill.cu):
//   dKL/dl_e = 1/tau (p_e - q_e)              for e in the teacher's list
//            = 1/tau p_e (1 - q_r / R)        otherwise
// from the maxima, sums and ratio q_r / R that the forward left for each row, so
// that nothing is reduced: one pass that reads the logits and writes the gradient.
// Bound by memory: 524288 rows of 256 BF16 logits with lists of 32 and a rest 107 us,
// 89 % of the copy bandwidth.
#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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

// The list's entries differ from p_e (1 - ratio): the row's gradient is laid out in
// its logits' place in shared memory, in its final type, the lanes of the list
// overwrite their entries, and the row leaves in full vectors.  A lane keeps J
// entries in registers; more are read again where they are needed.
template <typename T, int VEC, int NV, int LPR, int J>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<T, VEC, NV>(kListBlocks)) distill_bwd_kernel(BwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  using Stream = RowStream<T, VEC, NV, LPR>;
  using Row = typename Stream::Row;
  constexpr int N = Row::N, S = Stream::kStages;
  constexpr int F = 5;  // statistics of a row
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const Lanes<LPR> L(a.lpr);
  Stream rows(L, smem, a.logits, a.E, a.T);
  const int step = kWarps * L.rows;

  // rows [lo, hi) of a sequence, or (seq < 0) of none: nothing but the base
  auto piece = [&](int seq, int64_t lo, int64_t hi) {
    const uint32_t tokens = seq < 0 ? 0u : __ldg(a.tokens + seq);
    const float c = tokens ? __ldg(a.dloss + seq) * a.inv_tau / (float)tokens : 0.f;
    int64_t t0 = lo + warp * L.rows;
    int left = (int)(hi - t0);
    rows.start(t0, step);
    // A row's sum says whether it counts: the rest of it is read only then.  Bit i
    // is the i-th batch from here; sums are fetched a batch before their bit.
    auto inside = [&](int ahead) { return seq >= 0 && ahead * step + L.grp < left; };
    auto sum_at = [&](int ahead) { return inside(ahead) ? __ldg(a.row_stats + a.T + t0 + ahead * step + L.grp) : 0.f; };
    uint32_t on = 0;
    {
      float sum[S];
#pragma unroll
      for (int i = 0; i < S; ++i) sum[i] = sum_at(i);
#pragma unroll
      for (int i = 0; i < S; ++i) on |= (uint32_t)(sum[i] != 0.f) << i;
    }
#pragma unroll
    for (int i = 0; i < S - 1; ++i) rows.issue(on >> i & 1u);
    float ahead_sum = sum_at(S);
    // statistics a batch ahead: lane sub = f holds the f-th, where a row has eight
    // lanes or more; else they are loaded where they are needed
    const int mine = min(L.sub, F - 1);
    auto stat_at = [&](int ahead) {
      return L.lpr >= 8 && (on >> ahead & 1u) ? __ldg(a.row_stats + mine * a.T + t0 + ahead * step + L.grp) : 0.f;
    };
    // this lane's entries of its row's list, a batch ahead
    const ListEntries list{a.t_logits, a.t_idx, a.t_dt};
    int64_t li = (t0 + L.grp) * a.m + L.sub;
    auto entries = [&](int ahead, uint32_t (&x)[J], uint32_t (&e)[J]) {
      const bool ok = on >> ahead & 1u;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (j * L.lpr >= a.m) break;
        x[j] = list.none();
        e[j] = 0u;
        if (ok && L.sub + j * L.lpr < a.m) {
          x[j] = list.bits(li + ahead * step * a.m + j * L.lpr);
          e[j] = list.expert(li + ahead * step * a.m + j * L.lpr);
        }
      }
    };
    uint32_t x[J], e[J];
    entries(0, x, e);
    float st = stat_at(0);
    while (left > 0) {
      Row cur;
      rows.take(cur);
      __syncwarp();  // the rows lie in shared memory; the last batch has left it
      rows.issue(on >> (S - 1) & 1u);
      on |= (uint32_t)(ahead_sum != 0.f) << S;
      ahead_sum = sum_at(S + 1);
      uint32_t x1[J], e1[J];
      entries(1, x1, e1);
      const float st1 = stat_at(1);
      const int64_t t = t0 + L.grp;
      const bool in = L.grp < left, ok = on & 1u;
      auto stat = [&](int f) {
        if (L.lpr >= 8) return __shfl_sync(0xffffffffu, st, L.grp * L.lpr + f);
        return ok ? __ldg(a.row_stats + f * a.T + t) : 0.f;
      };
      const float m = stat(0), s = stat(1), mt = stat(2), sum_t = stat(3), ratio = stat(4);
      const RowExp ex(m, a.c);
      const float ps = c * rcp_fast(s) * ex.fix(), qs = c * rcp_fast(sum_t);
      // the list's gradients
      float gs[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (j * L.lpr >= a.m) break;
        gs[j] = ex.at(to_f32<T>(rows.cell((int)min(e[j], (uint32_t)a.E - 1u)))) * ps -
                exp2_fast((list.value(x[j]) - mt) * a.c) * qs;
      }
      float d[N];
      ex.row(cur, d);
      float w = ps * (1.f - ratio);
      if (isinf(w)) {  // q_r / R (1e33 at most) meets the small exponentials before a scaled dloss
        w = ps;        // (an infinity at a listed expert is overwritten)
#pragma unroll
        for (int n = 0; n < N; ++n) d[n] *= 1.f - ratio;
      }
      pairwise<N>([&](int n) { put(d, n, mul2(pair(d, n), both(w))); }, [&](int n) { d[n] *= w; });
      if (!ok) {
#pragma unroll
        for (int n = 0; n < N; ++n) d[n] = 0.f;
      }
      const int64_t at = (t0 + L.grp) * a.E;
      const T* const base = static_cast<const T*>(a.base);  // may be what this kernel writes: plain loads
      if (base) {  // into the logits' registers and their place
        cur.load(base + at + L.sub * VEC, rows.room, L.lpr, in);
#pragma unroll
        for (int n = 0; n < N; ++n) d[n] += cur[n];
        __syncwarp();
        rows.put(cur);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (j * L.lpr >= a.m) break;
          gs[j] += to_f32<T>(rows.cell((int)min(e[j], (uint32_t)a.E - 1u)));
        }
      }
      __syncwarp();
      rows.put(d);
      __syncwarp();
      const T* const row = static_cast<const T*>(a.logits) + at;
      if (ratio < 0.f) {  // -q_r: the shares of the rest about their own maximum
        auto in_list = [&](int el) {
#pragma unroll 1
          for (int j = 0; j < a.m; ++j)
            if (list.expert(t * a.m + j) == (uint32_t)el && list.bits(t * a.m + j) != list.none()) return true;
          return false;
        };
        float mo = -INFINITY, so = 0.f;
#pragma unroll 1
        for (int el = L.sub; el < a.E; el += L.lpr)
          if (!in_list(el)) mo = fmaxf(mo, to_f32<T>(__ldg(row + el)));
        for (int k = L.lpr / 2; k > 0; k >>= 1) mo = fmaxf(mo, __shfl_xor_sync(L.mask(), mo, k));
#pragma unroll 1
        for (int el = L.sub; el < a.E; el += L.lpr)
          if (!in_list(el)) so += exp2_fast((to_f32<T>(__ldg(row + el)) - mo) * a.c);
        for (int k = L.lpr / 2; k > 0; k >>= 1) so += __shfl_xor_sync(L.mask(), so, k);
#pragma unroll 1
        for (int el = L.sub; el < a.E; el += L.lpr) {
          // nothing outside but -inf: no share to give
          float g = mo == -INFINITY ? 0.f : c * ratio / so * exp2_fast((to_f32<T>(__ldg(row + el)) - mo) * a.c);
          if (base) g += to_f32<T>(base[at + el]);
          rows.cell(el) = from_f32<T>(g);  // the list's are overwritten below
        }
        __syncwarp(L.mask());
      }
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (j * L.lpr >= a.m) break;
        if (x[j] != list.none() && e[j] < (uint32_t)a.E)  // (an expert that is none: the row is NaN)
          rows.cell((int)e[j]) = from_f32<T>(gs[j]);
      }
      if (ok)
        for (int j = L.sub + J * L.lpr; j < a.m; j += L.lpr) {
          const uint32_t b = list.bits(t * a.m + j), ee = list.expert(t * a.m + j);
          if (b == list.none() || ee >= (uint32_t)a.E) continue;
          float g = ex.at(to_f32<T>(__ldg(row + ee))) * ps - exp2_fast((list.value(b) - mt) * a.c) * qs;
          if (base) g += to_f32<T>(base[at + ee]);
          rows.cell((int)ee) = from_f32<T>(g);
        }
      __syncwarp();
      rows.store(static_cast<T*>(a.out), t0, left);
      st = st1;
#pragma unroll
      for (int j = 0; j < J; ++j) x[j] = x1[j], e[j] = e1[j];
      on >>= 1;
      t0 += step;
      li += (int64_t)step * a.m;
      left -= step;
    }
    rows.drain();
    __syncwarp();
  };
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk_rows;
  walk_sequences(a.seqs, c0, min(c0 + a.chunk_rows, a.T), piece, [&](int64_t lo, int64_t hi) { piece(-1, lo, hi); });
}

struct LaunchBwd {
  BwdArgs a;
  int chunks;
  cudaStream_t s;
  template <typename T, int VEC, int NV, int LPR>
  cudaError_t run() {
    if constexpr (VEC > 1)
      if (a.m <= a.lpr) return with<T, VEC, NV, LPR, 1>();
    return with<T, VEC, NV, LPR, 4>();
  }
  template <typename T, int VEC, int NV, int LPR, int J>
  cudaError_t with() {
    static std::atomic<uint64_t> asked{0};
    return launch_rows(distill_bwd_kernel<T, VEC, NV, LPR, J>, chunks, kThreads,
                       kWarps * RowStream<T, VEC, NV, LPR>::kWarpBytes, asked, s, a);
  }
};

}  // namespace

cudaError_t launch_distill_loss_backward(const DistillBwdArgs& d, cudaStream_t s) {
  const void* ptrs[] = {d.logits, d.base, d.dlogits};
  const RowPlan plan = row_plan(ptrs, 3, d.dt, d.E);
  const Chunks ch = cut_rows(d.T, (d.seq_offsets ? 1 : kWarps) * (int64_t)plan_batch(plan), plan_blocks(plan, kListBlocks), 1);
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
  LaunchBwd f{a, ch.chunks, s};
  return with_row_variant(d.dt, plan, f);
}

}  // namespace moe
