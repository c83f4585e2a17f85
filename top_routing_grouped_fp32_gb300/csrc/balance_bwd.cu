// balance_bwd.cu -- the gradient of the balance loss and the z-loss (balance.cu).
// The counts are not differentiated.  With g_se = dloss_s E n_se / (k L_s^2),
//   softmax: dl_te = p_te (g_se - sum_i p_ti g_si) + dz_s 2 lse_t p_te / L_s
//   sigmoid: dl_te = p_te (1 - sigmoid(l_te)) (g_se - sum_i p_ti g_si)
// One pass over the logits, with the shifts and sums that the forward left.
#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks = 304;  // two per SM

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
  constexpr int N = VEC * NV, R = rows_at_once<T, VEC, NV>();
  using Row = RowRegs<T, VEC, NV>;
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const Lanes<LPR> L(a.lpr);
  const int room = a.E - L.sub * VEC;
  const int batch = R * L.rows;

  // rows [lo, hi) of a sequence, or (seq < 0) of none: nothing but the base
  auto piece = [&](int seq, int64_t lo, int64_t hi) {
    // g about an even load, (E n - k L) / (k L^2): exact in integers, and the
    // scores sum to one, so a constant taken from g changes nothing
    const uint32_t rows = seq < 0 ? 0u : __ldg(a.tokens + seq);
    const float len = (float)rows;
    const float up = rows ? __ldg(a.dloss + seq) / len / (float)a.k / len : 0.f;
    const float zc = !SIG && a.dz && rows ? 2.f * __ldg(a.dz + seq) / len : 0.f;
    float g[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int e = Row::elem(n, L.lpr, L.sub);
      const int64_t c = seq >= 0 && e < a.E ? (int64_t)__ldg(a.counts + (int64_t)seq * a.E + e) : 0;
      g[n] = up * (float)(c * a.E - (int64_t)rows * a.k);
    }
    int64_t t0 = lo + warp * batch;
    int left = (int)(hi - t0);
    const int64_t stride = (int64_t)kWarps * batch * a.E;
    const int64_t at = (t0 + L.grp) * a.E + L.sub * VEC;
    const T* lp = static_cast<const T*>(a.logits) + at;
    const T* bp = static_cast<const T*>(a.base) + at;
    T* op = static_cast<T*>(a.out) + at;
    // rows that do not count (a sum of 0) are not read; the sums come a batch ahead
    auto stats = [&](int ahead, int r) {
      const int i = ahead * kWarps * batch + r * L.rows + L.grp;
      return seq >= 0 && i < left ? __ldg(a.row_stats + t0 + i) : make_float2(0.f, 0.f);
    };
    Row cur[R], nxt[R];
    float2 st[R], st1[R];
#pragma unroll
    for (int r = 0; r < R; ++r) st[r] = stats(0, r), st1[r] = stats(1, r);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      cur[r].fill(from_f32<T>(-INFINITY));
      nxt[r].fill(from_f32<T>(-INFINITY));
      cur[r].load(lp + r * L.rows * a.E, room, L.lpr, st[r].y != 0.f);
    }
    while (left > 0) {
      float2 st2[R];
      lp += stride;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        nxt[r].load(lp + r * L.rows * a.E, room, L.lpr, st1[r].y != 0.f);
        st2[r] = stats(2, r);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool in = r * L.rows + L.grp < left;
        const bool ok = st[r].y != 0.f;  // NaN sums leave NaN
        float d[N], dot;
        if (SIG && st[r].x == 0.f) {
          const float inv = rcp_fast(st[r].y);
          dot = 0.f;
#pragma unroll
          for (int n = 0; n < N; ++n) {
            const float x = cur[r][n];
            const float ex = exp2_fast(fabsf(x) * -kLog2e);  // sigmoid(|l|) = 1 / (1 + ex)
            const float hi1 = rcp_fast(1.f + ex), lo1 = ex * hi1;
            const float p = (x < 0.f ? lo1 : hi1) * inv;
            dot = fmaf(p, g[n], dot);
            d[n] = p * (x < 0.f ? hi1 : lo1);
          }
        } else {
          const RowExp ex(st[r].x, kLog2e);
          const float inv = rcp_fast(st[r].y) * ex.fix();
          ex.row(cur[r], d);
          if constexpr (N > 1) {
            float2 dots = both(0.f);
#pragma unroll
            for (int n = 0; n < N; n += 2) {
              put(d, n, mul2(pair(d, n), both(inv)));
              dots = fma2(pair(d, n), pair(g, n), dots);
            }
            dot = dots.x + dots.y;
          } else {
            d[0] *= inv;
            dot = d[0] * g[0];
          }
        }
        if (a.base) {  // into the logits' registers (vectors behind the row's end stay)
          cur[r].load(bp + r * L.rows * a.E, room, L.lpr, in);
        }
        dot = L.sum(dot);
        if (!SIG && a.dz) dot -= zc * fmaf(log2_fast(st[r].y), kLn2, st[r].x);
        pairwise<N>([&](int n) { put(d, n, mul2(pair(d, n), add2(pair(g, n), both(-dot)))); },
                    [&](int n) { d[n] *= g[n] - dot; });
        if (!ok) {
#pragma unroll
          for (int n = 0; n < N; ++n) d[n] = 0.f;
        }
        if (a.base) {
#pragma unroll
          for (int n = 0; n < N; ++n) d[n] += cur[r][n];
        }
        if (in) store_row<T, VEC, NV>(op + r * L.rows * a.E, room, L.lpr, d);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) cur[r] = nxt[r], st[r] = st1[r], st1[r] = st2[r];
      bp += stride;
      op += stride;
      t0 += kWarps * batch;
      left -= kWarps * batch;
    }
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
    return launch_pdl(balance_bwd_kernel<T, VEC, NV, LPR, SIG>, dim3((unsigned)chunks), dim3(kThreads), 0, s, a);
  }
};

}  // namespace

cudaError_t launch_balance_loss_backward(const BalanceBwdArgs& b, cudaStream_t s) {
  const void* ptrs[] = {b.logits, b.base, b.dlogits};
  const RowPlan plan = row_plan(ptrs, 3, b.dt, b.E);
  const Chunks ch = cut_rows(b.T, plan_batch(plan), kMaxBlocks);
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
