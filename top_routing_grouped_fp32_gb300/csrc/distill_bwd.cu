// distill_bwd.cu -- the gradient of the distillation loss (distill.cu):
//   dKL/dl_e = 1/tau (p_e - q_e)              for e in the teacher's list
//            = 1/tau p_e (1 - q_r / R)        otherwise
// from the maxima, sums and ratio q_r / R that the forward left for each row, so
// that nothing is reduced: one pass that reads the logits and writes the gradient.
#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxBlocks = 304;  // two per SM

// Entries of a row's list that a lane keeps in registers; more are read again
// where they are needed.
template <typename T, int VEC, int NV>
constexpr int list_regs() {
  return 4 / rows_at_once<T, VEC, NV>();
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
template <typename T, int VEC, int NV, int LPR>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<T, VEC, NV>()) distill_bwd_kernel(BwdArgs a) {
  using Row = RowRegs<T, VEC, NV>;
  constexpr int N = Row::N, R = rows_at_once<T, VEC, NV>(), J = list_regs<T, VEC, NV>();
  constexpr int F = 5;  // statistics of a row
  extern __shared__ __align__(16) unsigned char row_smem[];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5;
  const Lanes<LPR> L(a.lpr);
  const int room = a.E - L.sub * VEC;
  const int batch = R * L.rows;
  const int pitch = (int)align_up((size_t)a.E * sizeof(T), 16) / (int)sizeof(T);
  T* buf = reinterpret_cast<T*>(row_smem) + (warp * batch + L.grp) * pitch;  // r-th row: + r * rows * pitch

  // rows [lo, hi) of a sequence, or (seq < 0) of none: nothing but the base
  auto piece = [&](int seq, int64_t lo, int64_t hi) {
    const uint32_t tokens = seq < 0 ? 0u : __ldg(a.tokens + seq);
    const float c = tokens ? __ldg(a.dloss + seq) * a.inv_tau / (float)tokens : 0.f;
    int64_t t0 = lo + warp * batch;
    int left = (int)(hi - t0);
    const int64_t stride = (int64_t)kWarps * batch * a.E;
    int64_t at = (t0 + L.grp) * a.E;  // this group's first row of the batch, in elements
    const T* const logits = static_cast<const T*>(a.logits);
    const T* const base = static_cast<const T*>(a.base);
    Row cur[R], nxt[R];
    // statistics: lane sub = f holds the f-th (rows of eight lanes or more), or
    // the sum alone, which says whether the row counts
    const int mine = L.lpr >= 8 ? min(L.sub, F - 1) : 1;
    auto stats = [&](int ahead, int r) {
      const int i = ahead * kWarps * batch + r * L.rows + L.grp;
      return seq >= 0 && i < left ? __ldg(a.row_stats + mine * a.T + t0 + i) : 0.f;
    };
    auto stat = [&](float own, int64_t t, bool ok, int f) {
      if (L.lpr >= 8) return __shfl_sync(0xffffffffu, own, L.grp * L.lpr + f);
      return ok ? __ldg(a.row_stats + f * a.T + t) : 0.f;
    };
    auto sum_of = [&](float own) { return L.lpr >= 8 ? __shfl_sync(0xffffffffu, own, L.grp * L.lpr + 1) : own; };
    const ListEntries list{a.t_logits, a.t_idx, a.t_dt};
    int64_t li = (t0 + L.grp) * a.m + L.sub;
    float st[R], st1[R], s[R], s1[R];
    uint32_t x[R][J], x1[R][J], e[R][J], e1[R][J];
    auto lists = [&](int ahead, const float (&s)[R], uint32_t (&x)[R][J], uint32_t (&e)[R][J]) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t i = li + (int64_t)(ahead * kWarps * batch + r * L.rows) * a.m;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (j * L.lpr >= a.m) break;
          x[r][j] = list.none();
          e[r][j] = 0u;
          if (s[r] != 0.f && L.sub + j * L.lpr < a.m) {
            x[r][j] = list.bits(i + j * L.lpr);
            e[r][j] = list.expert(i + j * L.lpr);
          }
        }
      }
    };
#pragma unroll
    for (int r = 0; r < R; ++r) st[r] = stats(0, r), st1[r] = stats(1, r);
#pragma unroll
    for (int r = 0; r < R; ++r) {
      s[r] = sum_of(st[r]);
      cur[r].fill(from_f32<T>(-INFINITY));
      nxt[r].fill(from_f32<T>(-INFINITY));
      cur[r].load(logits + at + (L.sub * VEC + r * L.rows * a.E), room, L.lpr, s[r] != 0.f);
    }
    lists(0, s, x, e);
    while (left > 0) {
      float st2[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s1[r] = sum_of(st1[r]);
        nxt[r].load(logits + at + stride + (L.sub * VEC + r * L.rows * a.E), room, L.lpr, s1[r] != 0.f);
        st2[r] = stats(2, r);
      }
      lists(1, s1, x1, e1);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t t = t0 + r * L.rows + L.grp;
        const bool in = r * L.rows + L.grp < left;
        const bool ok = s[r] != 0.f;  // the row counted; NaN sums leave NaN
        const float m = stat(st[r], t, ok, 0), mt = stat(st[r], t, ok, 2), sum_t = stat(st[r], t, ok, 3),
                    ratio = stat(st[r], t, ok, 4);
        const RowExp ex(m, a.c);
        const float ps = c * rcp_fast(s[r]) * ex.fix(), qs = c * rcp_fast(sum_t);
        T* out = buf + r * L.rows * pitch;
        // the list's gradients, from the row's logits (and then the base's elements)
        // laid out in shared memory
        cur[r].keep(out + L.sub * VEC, room, L.lpr);
        __syncwarp();
        float gs[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (j * L.lpr >= a.m) break;
          gs[j] = ex.at(to_f32<T>(out[min(e[r][j], (uint32_t)a.E - 1u)])) * ps -
                  exp2_fast((list.value(x[r][j]) - mt) * a.c) * qs;
        }
        float d[N];
        ex.row(cur[r], d);
        const float w = ps * (1.f - ratio);
        pairwise<N>([&](int n) { put(d, n, mul2(pair(d, n), both(w))); }, [&](int n) { d[n] *= w; });
        if (!ok) {
#pragma unroll
          for (int n = 0; n < N; ++n) d[n] = 0.f;
        }
        if (a.base) {  // into the logits' registers (vectors behind the row's end stay)
          cur[r].load(base + at + (L.sub * VEC + r * L.rows * a.E), room, L.lpr, in);
#pragma unroll
          for (int n = 0; n < N; ++n) d[n] += cur[r][n];
          __syncwarp();
          cur[r].keep(out + L.sub * VEC, room, L.lpr);
          __syncwarp();
#pragma unroll
          for (int j = 0; j < J; ++j) {
            if (j * L.lpr >= a.m) break;
            gs[j] += to_f32<T>(out[min(e[r][j], (uint32_t)a.E - 1u)]);
          }
        }
        __syncwarp();
        store_row<T, VEC, NV>(out + L.sub * VEC, room, L.lpr, d);
        __syncwarp();
        if (ratio < 0.f) {  // -q_r: the shares of the rest about their own maximum
          auto listed = [&](int el) {
#pragma unroll 1
            for (int j = 0; j < a.m; ++j)
              if (list.expert(t * a.m + j) == (uint32_t)el && list.bits(t * a.m + j) != list.none()) return true;
            return false;
          };
          const T* row = logits + at + r * L.rows * a.E;
          float mo = -INFINITY, so = 0.f;
#pragma unroll 1
          for (int el = L.sub; el < a.E; el += L.lpr)
            if (!listed(el)) mo = fmaxf(mo, to_f32<T>(__ldg(row + el)));
          for (int k = L.lpr / 2; k > 0; k >>= 1) mo = fmaxf(mo, __shfl_xor_sync(L.mask(), mo, k));
#pragma unroll 1
          for (int el = L.sub; el < a.E; el += L.lpr)
            if (!listed(el)) so += exp2_fast((to_f32<T>(__ldg(row + el)) - mo) * a.c);
          for (int k = L.lpr / 2; k > 0; k >>= 1) so += __shfl_xor_sync(L.mask(), so, k);
#pragma unroll 1
          for (int el = L.sub; el < a.E; el += L.lpr) {
            // nothing outside but -inf: no share to give
            float g = mo == -INFINITY ? 0.f : c * ratio / so * exp2_fast((to_f32<T>(__ldg(row + el)) - mo) * a.c);
            if (a.base) g += to_f32<T>(__ldg(base + at + r * L.rows * a.E + el));
            out[el] = from_f32<T>(g);  // the list's are overwritten below
          }
          __syncwarp(L.mask());
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
          if (j * L.lpr >= a.m) break;
          if (x[r][j] != list.none() && e[r][j] < (uint32_t)a.E)  // (an expert that is none: the row is NaN)
            out[e[r][j]] = from_f32<T>(gs[j]);
        }
        if (ok)
          for (int j = L.sub + J * L.lpr; j < a.m; j += L.lpr) {
            const uint32_t b = list.bits(t * a.m + j), ee = list.expert(t * a.m + j);
            if (b == list.none() || ee >= (uint32_t)a.E) continue;
            float g = ex.at(to_f32<T>(__ldg(logits + at + r * L.rows * a.E + ee))) * ps -
                      exp2_fast((list.value(b) - mt) * a.c) * qs;
            if (a.base) g += to_f32<T>(__ldg(base + at + r * L.rows * a.E + ee));
            out[ee] = from_f32<T>(g);
          }
      }
      __syncwarp();
#pragma unroll
      for (int r = 0; r < R; ++r) {
        if (r * L.rows + L.grp < left) {
          const T* from = buf + r * L.rows * pitch + L.sub * VEC;
          T* to = static_cast<T*>(a.out) + at + (L.sub * VEC + r * L.rows * a.E);
#pragma unroll
          for (int v = 0; v < NV; ++v) {
            if (v * L.lpr * VEC >= room) continue;
            if constexpr (VEC > 1)
              *reinterpret_cast<uint4*>(to + v * L.lpr * VEC) = *reinterpret_cast<const uint4*>(from + v * L.lpr * VEC);
            else
              to[v * L.lpr] = from[v * L.lpr];
          }
        }
        cur[r] = nxt[r];
        st[r] = st1[r], st1[r] = st2[r], s[r] = s1[r];
#pragma unroll
        for (int j = 0; j < J; ++j) x[r][j] = x1[r][j], e[r][j] = e1[r][j];
      }
      __syncwarp();  // before the next batch is laid out
      at += stride;
      t0 += kWarps * batch;
      li += (int64_t)kWarps * batch * a.m;
      left -= kWarps * batch;
    }
  };
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk_rows;
  walk_sequences(a.seqs, c0, min(c0 + a.chunk_rows, a.T), piece, [&](int64_t lo, int64_t hi) { piece(-1, lo, hi); });
}

struct LaunchBwd {
  BwdArgs a;
  int chunks;
  size_t smem;
  cudaStream_t s;
  template <typename T, int VEC, int NV, int LPR>
  cudaError_t run() {
    return launch_pdl(distill_bwd_kernel<T, VEC, NV, LPR>, dim3((unsigned)chunks), dim3(kThreads), smem, s, a);
  }
};

}  // namespace

cudaError_t launch_distill_loss_backward(const DistillBwdArgs& d, cudaStream_t s) {
  const void* ptrs[] = {d.logits, d.base, d.dlogits};
  const RowPlan plan = row_plan(ptrs, 3, d.dt, d.E);
  const int batch = plan_batch(plan);
  const Chunks ch = cut_rows(d.T, batch, kMaxBlocks);
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
  LaunchBwd f{a, ch.chunks, (size_t)kWarps * batch * align_up((size_t)d.E * dtype_size(d.dt), 16), s};
  return with_row_variant(d.dt, plan, f);
}

}  // namespace moe
