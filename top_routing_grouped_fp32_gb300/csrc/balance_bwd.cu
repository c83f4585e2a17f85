// balance_bwd.cu -- the gradient of the balance loss and the z-loss (balance.cu).
// The counts are not differentiated.  With g_se = dloss_s E n_se / (k L_s^2),
//   softmax: dl_te = p_te (g_se - sum_i p_ti g_si) + dz_s 2 lse_t p_te / L_s
//   sigmoid: dl_te = p_te (1 - sigmoid(l_te)) (g_se - sum_i p_ti g_si)
// One pass over the logits, with the shifts and sums that the forward left; only
// sum_i p_i g_i is reduced.  Bound by memory: 524288 rows of 256 BF16 logits in 128
// padded sequences 91 us, 83 % of the copy bandwidth.
#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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

template <typename T, int VEC, int NV, int LPR, bool SIG>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<T, VEC, NV>()) balance_bwd_kernel(BwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  using Stream = RowStream<T, VEC, NV, LPR>;
  using Row = typename Stream::Row;
  constexpr int N = Row::N, S = Stream::kStages;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const Lanes<LPR> L(a.lpr);
  Stream rows(L, smem, a.logits, a.E, a.T);
  const int step = kWarps * L.rows;

  // rows [lo, hi) of a sequence, or (seq < 0) of none: nothing but the base
  auto piece = [&](int seq, int64_t lo, int64_t hi) {
    // g about an even load, (E n - k L) / (k L^2): exact in integers, and the
    // scores sum to one, so a constant taken from g changes nothing
    const uint32_t tokens = seq < 0 ? 0u : __ldg(a.tokens + seq);
    const float len = (float)tokens;
    const float up = tokens ? __ldg(a.dloss + seq) / len / (float)a.k / len : 0.f;
    const float zc = !SIG && a.dz && tokens ? 2.f * __ldg(a.dz + seq) / len : 0.f;
    float g[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int e = Row::elem(n, L.lpr, L.sub);
      const int64_t c = seq >= 0 && e < a.E ? (int64_t)__ldg(a.counts + (int64_t)seq * a.E + e) : 0;
      g[n] = up * (float)(c * a.E - (int64_t)tokens * a.k);
    }
    int64_t t0 = lo + warp * L.rows;
    int left = (int)(hi - t0);
    rows.start(t0, step);
    // Rows that do not count (a sum of 0) are not read.  A row's sum is fetched two
    // batches before its row is asked for, its statistics (again) two before their use:
    // one batch does not cover the latency.
    auto inside = [&](int ahead) { return seq >= 0 && ahead * step + L.grp < left; };
    auto sum_at = [&](int ahead) { return inside(ahead) ? __ldg(&a.row_stats[t0 + ahead * step + L.grp].y) : 0.f; };
    auto stats = [&](int ahead) {
      return inside(ahead) ? __ldg(a.row_stats + t0 + ahead * step + L.grp) : make_float2(0.f, 0.f);
    };
    float sum[S + 1];
#pragma unroll
    for (int i = 0; i <= S; ++i) sum[i] = sum_at(i);
    float2 st = stats(0), st1 = stats(1);
#pragma unroll
    for (int i = 0; i < S - 1; ++i) rows.issue(sum[i] != 0.f);
    float sum0 = sum[S - 1], sum1 = sum[S];
    while (left > 0) {
      Row cur;
      rows.take(cur);
      rows.issue(sum0 != 0.f);
      sum0 = sum1;
      sum1 = sum_at(S + 1);
      const float2 st2 = stats(2);
      const bool in = L.grp < left;
      const bool ok = st.y != 0.f;  // NaN sums leave NaN
      float d[N], dot;
      if (SIG && st.x == 0.f) {
        const float inv = rcp_fast(st.y);
        dot = 0.f;
        auto one = [&](int n, float ex, float hi1) {  // hi1 = sigmoid(|l|) = 1 / (1 + ex)
          const float x = cur[n], lo1 = ex * hi1;
          const float p = (x < 0.f ? lo1 : hi1) * inv;
          dot = fmaf(p, g[n], dot);
          d[n] = p * (x < 0.f ? hi1 : lo1);
        };
        pairwise<N>(
            [&](int n) {  // one reciprocal for two scores: 1/a = b / (a b)
              const float ex = exp2_fast(fabsf(cur[n]) * -kLog2e), ey = exp2_fast(fabsf(cur[n + 1]) * -kLog2e);
              const float b0 = 1.f + ex, b1 = 1.f + ey, q = rcp_fast(b0 * b1);
              one(n, ex, b1 * q);
              one(n + 1, ey, b0 * q);
              if (cur[n] != cur[n] || cur[n + 1] != cur[n + 1]) dot = NAN;
            },
            [&](int n) {
              const float ex = exp2_fast(fabsf(cur[n]) * -kLog2e);
              one(n, ex, rcp_fast(1.f + ex));
            });
      } else {
        const RowExp ex(st.x, kLog2e);
        const float inv = rcp_fast(st.y) * ex.fix();
        ex.row(cur, d);
        if constexpr (N > 1) {
          float2 dots[2] = {both(0.f), both(0.f)};
#pragma unroll
          for (int n = 0; n < N; n += 2) {
            put(d, n, mul2(pair(d, n), both(inv)));
            dots[n / 2 % 2] = fma2(pair(d, n), pair(g, n), dots[n / 2 % 2]);
          }
          dots[0] = add2(dots[0], dots[1]);
          dot = dots[0].x + dots[0].y;
        } else {
          d[0] *= inv;
          dot = d[0] * g[0];
        }
      }
      const int64_t at = (t0 + L.grp) * a.E + L.sub * VEC;
      if (a.base)  // into the logits' registers (vectors behind the row's end stay)
        cur.load(static_cast<const T*>(a.base) + at, rows.room, L.lpr, in);
      dot = L.sum(dot);
      if (!SIG && a.dz) dot -= zc * fmaf(log2_fast(st.y), kLn2, st.x);
      pairwise<N>([&](int n) { put(d, n, mul2(pair(d, n), add2(pair(g, n), both(-dot)))); },
                  [&](int n) { d[n] *= g[n] - dot; });
      if (!ok) {
#pragma unroll
        for (int n = 0; n < N; ++n) d[n] = 0.f;
      }
      if (a.base) {
#pragma unroll
        for (int n = 0; n < N; ++n) d[n] += cur[n];
      }
      if constexpr (Stream::kImage) {
        __syncwarp();  // every lane has read its logits
        rows.put(d);
        __syncwarp();
        rows.store(static_cast<T*>(a.out), t0, left);
      } else if (in) {
        store_row<T, VEC, NV>(static_cast<T*>(a.out) + at, rows.room, L.lpr, d);
      }
      st = st1, st1 = st2;
      t0 += step;
      left -= step;
    }
    rows.drain();
  };
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk_rows;
  walk_sequences(a.seqs, c0, min(c0 + a.chunk_rows, a.T), piece, [&](int64_t lo, int64_t hi) { piece(-1, lo, hi); });
}

template <bool SIG>
struct LaunchBwd {
  BwdArgs a;
  int chunks;
  cudaStream_t s;
  template <typename T, int VEC, int NV, int LPR>
  cudaError_t run() {
    static std::atomic<uint64_t> asked{0};
    return launch_rows(balance_bwd_kernel<T, VEC, NV, LPR, SIG>, chunks, kThreads,
                       kWarps * RowStream<T, VEC, NV, LPR>::kWarpBytes, asked, s, a);
  }
};

}  // namespace

cudaError_t launch_balance_loss_backward(const BalanceBwdArgs& b, cudaStream_t s) {
  const void* ptrs[] = {b.logits, b.base, b.dlogits};
  const RowPlan plan = row_plan(ptrs, 3, b.dt, b.E);
  const Chunks ch = cut_rows(b.T, (b.seq_offsets ? 1 : kWarps) * (int64_t)plan_batch(plan), plan_blocks(plan), 1);
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
