// distill.cu -- distillation of a router from a teacher's top logits (its gradient
// is in distill_bwd.cu, the teacher's side in distill_targets.cu).
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
//
// 524288 rows of 256 BF16 logits with lists of 8 and a rest: 84 us, 54 % of the copy
// bandwidth.  Bound by issue: 130 instructions a row, 2.7 a cycle of a SM.
#include "internal.h"
#include "rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// Below this, beside the exponential of the row's maximum, the student's mass outside
// the list is taken about its own maximum, and -q_r stands in the place of q_r / R.
constexpr float kFarBelow = 1e-30f;

// q log(q/p) - q + p from d = log(q/p); its series where the terms nearly cancel
// (|d| < 1/2: the first term left out is below 2^-24 of the sum).
// Without branches: both forms cost less than the divergence between them.
__device__ __forceinline__ float kl_term(float q, float p, float d) {
  float h = fmaf(d, -1.f / 362880.f, 1.f / 40320.f);
  h = fmaf(-d, h, 1.f / 5040.f);
  h = fmaf(-d, h, 1.f / 720.f);
  h = fmaf(-d, h, 1.f / 120.f);
  h = fmaf(-d, h, 1.f / 24.f);
  h = fmaf(-d, h, 1.f / 6.f);
  h = fmaf(-d, h, 1.f / 2.f);
  const float t = fabsf(d) < 0.5f ? q * d * d * h : fmaf(q, d, p - q);
  return q == 0.f ? p : t;  // no mass: its limit
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
  float* part_loss;     // [slots]
  uint32_t* part_rows;  // [slots]
  uint32_t* part_bad;   // [slots] lists with an index that is no expert or is there twice
  bool alone;           // the only block of one sequence: it writes the results
  float* loss;
  uint32_t* tokens;
  float* row_loss;
  float* row_stats;
  uint32_t* status;
};

// A row's lanes hold its logits and, entry sub, sub + lpr, .., its list.  Which of
// its elements are listed is a word of bits for each lane, set by the list's
// lanes in shared memory, so that the mass outside the list is summed as it is and
// not as a difference.  A lane keeps J entries in registers (1 where that holds the
// list: for lists of 8 of 256 and 524288 rows it took 98 us where 4 took 106); more are read again
// where they are needed.  What a row needs once, and no other lane waits for, is
// left until a warp can do it for a row a lane.
template <typename T, int VEC, int NV, int LPR, int J>
__global__ void __launch_bounds__(kThreads, blocks_per_sm<T, VEC, NV>(kListBlocks)) distill_fwd_kernel(FwdArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  using Stream = RowStream<T, VEC, NV, LPR>;
  using Row = typename Stream::Row;
  constexpr int N = Row::N, S = Stream::kStages;
  __shared__ uint32_t listed[kWarps][32];
  __shared__ float red_l[kWarps];
  __shared__ uint32_t red_n[kWarps], red_b[kWarps];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0u;
  const Lanes<LPR> L(a.lpr);
  Stream rows(L, smem, a.logits, a.E, a.T);
  const int step = kWarps * L.rows;
  uint32_t* const words = &listed[warp][L.grp * L.lpr];
  auto owner = [&](uint32_t e) { return (e / VEC) & (L.lpr - 1); };  // the lane that holds element e
  auto bit_of = [&](uint32_t e) { return 1u << ((e / VEC >> rows.lpr_log) * VEC + e % VEC); };

  auto gap = [&](int64_t lo, int64_t hi) {
    for (int64_t t = lo + threadIdx.x; t < hi; t += kThreads) {
      a.row_loss[t] = 0.f;
#pragma unroll
      for (int f = 0; f < 5; ++f) a.row_stats[f * a.T + t] = 0.f;
    }
  };
  auto piece = [&](int seq, int64_t lo, int64_t hi) {
    float loss = 0.f;
    uint32_t counted = 0, broken = 0;
    int64_t t0 = lo + warp * L.rows;
    int left = (int)(hi - t0);
    rows.start(t0, step);
    // does this group's row of a batch count: bit i for the i-th batch from here.
    // The mask's byte is fetched a batch before its bit is needed.
    uint32_t on = 0;
    uint8_t byte = 1, early[S];
    auto fetch = [&](int ahead) {
      const int i = ahead * step + L.grp;
      if (a.mask) byte = i < left ? __ldg(a.mask + t0 + i) : 0;
    };
    auto bit = [&](int ahead) { return (uint32_t)(ahead * step + L.grp < left && byte) << ahead; };
#pragma unroll
    for (int i = 0; i < S; ++i) {
      fetch(i);
      early[i] = byte;
    }
#pragma unroll
    for (int i = 0; i < S - 1; ++i) {
      byte = early[i];
      on |= bit(i);
      rows.issue(on >> i & 1u);
    }
    byte = early[S - 1];
    // this lane's entries of its row's list, a batch ahead
    const ListEntries list{a.t_logits, a.t_idx, a.t_dt};
    int64_t li = (t0 + L.grp) * a.m + L.sub;
    auto entries = [&](int ahead, uint32_t (&x)[J], uint32_t (&e)[J], float& rest) {
      const bool ok = on >> ahead & 1u;
      rest = ok && a.t_rest ? __ldg(a.t_rest + t0 + ahead * step + L.grp) : -INFINITY;
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
    float rest;
    entries(0, x, e, rest);
    // A lane keeps its group's row of every lpr-th batch: the list's part of KL, the
    // maxima and sums of both sides (student's sum 0: the row does not count), the mass
    // outside the list (or, far below the row, its log, which is negative) and the rest.
    struct Kept {
      float kl, m, s, mt, st, out, rest;
    } kept = {};
    int turn = 0;
    auto flush = [&]() {  // the batches from t0 - turn * step on
      const int64_t t = t0 + (L.sub - turn) * step + L.grp;
      if (L.sub < turn && t < hi) {
        const float fix = RowExp(kept.m, a.c).fix();
        const float s = kept.s * fix;
        float kl = kept.kl, ratio = 0.f;
        const bool far = kept.out < 0.f;
        const float p = far ? 0.f : kept.out * rcp_fast(kept.s);
        if (a.t_rest) {
          const float ln_out = far ? kept.out : logf(kept.out * fix);
          const float inv_st = rcp_fast(kept.st);
          const float q = exp2_fast((kept.rest - kept.mt) * a.c) * inv_st;
          kl += kl_term(q, p, (kept.rest - kept.mt) * a.inv_tau - ln_out + log2_fast(s * inv_st) * kLn2);
          ratio = far ? -q : q * rcp_fast(p);
        } else {
          kl += p;
        }
        if (s != s || kept.st != kept.st) kl = ratio = NAN;  // (a far rest would leave -q_r)
        const bool ok = kept.s != 0.f;
        a.row_loss[t] = ok ? kl : 0.f;
        a.row_stats[t] = kept.m;
        a.row_stats[a.T + t] = ok ? s : 0.f;
        a.row_stats[2 * a.T + t] = kept.mt;
        a.row_stats[3 * a.T + t] = kept.st;
        a.row_stats[4 * a.T + t] = ok ? ratio : 0.f;
        if (ok) loss += kl;
        counted += ok;
      }
      turn = 0;
    };
    while (left > 0) {
      Row cur;
      rows.take(cur);
      listed[warp][lane] = 0u;
      __syncwarp();  // the rows and the words lie in shared memory
      on |= bit(S - 1);
      rows.issue(on >> (S - 1) & 1u);
      fetch(S);
      uint32_t x1[J], e1[J];
      float rest1;
      entries(1, x1, e1, rest1);
      const int64_t t = t0 + L.grp;
      bool ok = on & 1u;
      // calls f(x, e) for this lane's entries behind those in registers
      auto others = [&](auto f) {
        if (ok)
          for (int j = L.sub + J * L.lpr; j < a.m; j += L.lpr) {
            const uint32_t b = list.bits(t * a.m + j);
            if (b != list.none()) f(list.value(b), list.expert(t * a.m + j));
          }
      };
      // the teacher's maximum, and the bits of the list's experts
      float mt = rest;
      bool nan = rest != rest || rest == INFINITY, bad = false;
      auto note = [&](float xx, uint32_t ee) {
        mt = fmaxf(mt, xx);  // passes over NaN
        nan |= xx != xx || xx == INFINITY;
        if (ee >= (uint32_t)a.E || (atomicOr(words + owner(ee), bit_of(ee)) & bit_of(ee))) bad = true;
      };
      float xs[J], ys[J];  // an entry that is not there has xs = -inf
#pragma unroll
      for (int j = 0; j < J; ++j) {
        xs[j] = -INFINITY;
        if (j * L.lpr >= a.m) break;
        xs[j] = list.value(x[j]);
        ys[j] = to_f32<T>(rows.cell((int)min(e[j], (uint32_t)a.E - 1u)));
        if (xs[j] != -INFINITY) note(xs[j], e[j]);
      }
      others(note);
      mt = L.max(mt);
      nan = L.any(nan);
      bad = L.any(bad);
      ok = ok && (mt != -INFINITY || nan);  // else no target
      const float m = L.max(cur.lane_max());
      __syncwarp();
      const uint32_t mine = listed[warp][lane];
      // the student's mass outside the list, and both sides' masses in it
      const RowExp ex(m, a.c);
      float out = 0.f;
      {
        float p[N], part[4] = {0.f, 0.f, 0.f, 0.f};
        ex.row(cur, p);
#pragma unroll
        for (int n = 0; n < N; ++n)
          if (!(mine & (1u << n))) part[n % 4] += p[n];
        out = (part[0] + part[1]) + (part[2] + part[3]);
      }
      const float eq_rest = exp2_fast((rest - mt) * a.c);
      float st = L.sub == 0 ? eq_rest : 0.f, sp = 0.f;
      float eq[J], ep[J];
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (j * L.lpr >= a.m) break;
        eq[j] = exp2_fast((xs[j] - mt) * a.c);
        ep[j] = xs[j] != -INFINITY ? ex.at(ys[j]) : 0.f;
        st += eq[j];
        sp += ep[j];
      }
      others([&](float xx, uint32_t ee) {
        st += exp2_fast((xx - mt) * a.c);
        if (ee < (uint32_t)a.E) sp += ex.at(to_f32<T>(rows.cell((int)ee)));
      });
      out = L.sum(out);
      st = L.sum(st);
      const float s0 = out + L.sum(sp);  // with the factor that fix() takes out
      // log of the mass outside the list about its own maximum where it is far below the row's
      float kept_out = out;
      if (ok && a.t_rest && out < kFarBelow) {
        float mo = -INFINITY, so = 0.f;
#pragma unroll 1
        for (int el = L.sub; el < a.E; el += L.lpr)
          if (!(words[owner(el)] & bit_of(el))) mo = fmaxf(mo, to_f32<T>(rows.cell(el)));
        for (int d = L.lpr / 2; d > 0; d >>= 1) mo = fmaxf(mo, __shfl_xor_sync(L.mask(), mo, d));
#pragma unroll 1
        for (int el = L.sub; el < a.E; el += L.lpr)
          if (!(words[owner(el)] & bit_of(el))) so += exp2_fast((to_f32<T>(rows.cell(el)) - mo) * a.c);
        for (int d = L.lpr / 2; d > 0; d >>= 1) so += __shfl_xor_sync(L.mask(), so, d);
        kept_out = mo == -INFINITY ? -INFINITY : (mo - m) * a.inv_tau + logf(so);
      }
      const float inv_s = rcp_fast(s0), inv_st = rcp_fast(st);
      const float dz = log2_fast(s0 * ex.fix() * inv_st) * kLn2;  // as in flush()
      float kl = 0.f;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        if (j * L.lpr >= a.m) break;
        const float term = kl_term(eq[j] * inv_st, ep[j] * inv_s, ((xs[j] - mt) - (ys[j] - m)) * a.inv_tau + dz);
        kl += xs[j] != -INFINITY ? term : 0.f;
      }
      others([&](float xx, uint32_t ee) {
        if (ee >= (uint32_t)a.E) return;
        const float y = to_f32<T>(rows.cell((int)ee));
        kl += kl_term(exp2_fast((xx - mt) * a.c) * inv_st, ex.at(y) * inv_s,
                      ((xx - mt) - (y - m)) * a.inv_tau + dz);
      });
      kl = L.sum(kl);
      if (L.sub == turn) {
        kept = ok ? Kept{kl, m, bad || nan ? NAN : s0, mt, st, kept_out, rest} : Kept{};
        broken += ok && bad;
      }
      __syncwarp();  // before the next batch takes this one's place
#pragma unroll
      for (int j = 0; j < J; ++j) x[j] = x1[j], e[j] = e1[j];
      rest = rest1;
      on >>= 1;
      t0 += step;
      li += (int64_t)step * a.m;
      left -= step;
      if (++turn == L.lpr) flush();
    }
    flush();
    rows.drain();
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
      if (a.alone) {
        a.loss[0] = n ? l / (float)n : 0.f;
        a.tokens[0] = n;
        if (b) set_status(a.status, MOE_ERR_INVALID_INDEX);
      } else {
        const int64_t slot = (int64_t)blockIdx.x + seq;
        a.part_loss[slot] = l;
        a.part_rows[slot] = n;
        a.part_bad[slot] = b;
      }
    }
    __syncthreads();
  };
  if (a.alone) {
    piece(0, 0, a.T);
    return;
  }
  const int64_t c0 = (int64_t)blockIdx.x * a.chunk_rows;
  walk_sequences(a.seqs, c0, min(c0 + a.chunk_rows, a.T), piece, gap);
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

struct LaunchFwd {
  FwdArgs a;
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
    return launch_rows(distill_fwd_kernel<T, VEC, NV, LPR, J>, chunks, kThreads,
                       kWarps * RowStream<T, VEC, NV, LPR>::kWarpBytes, asked, s, a);
  }
};

size_t slot_count(int64_t T, int64_t num_seqs) { return (size_t)(kMaxBlocks < T ? kMaxBlocks : T) + (size_t)num_seqs; }

}  // namespace

size_t distill_workspace_bytes(int64_t T, int64_t num_seqs) { return align_up(slot_count(T, num_seqs) * 12, 256); }

cudaError_t launch_distill_loss(const DistillArgs& d, void* ws, uint32_t* status, cudaStream_t s) {
  const void* ptrs[] = {d.logits};
  const RowPlan plan = row_plan(ptrs, 1, d.dt, d.E);
  // sequences are worked off one after another in a block: finer cuts where there are any
  const Chunks ch = d.seq_offsets ? cut_rows(d.T, plan_batch(plan), plan_blocks(plan, kListBlocks), 1)
                                  : cut_rows(d.T, (int64_t)kWarps * plan_batch(plan), plan_blocks(plan, kListBlocks));
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
  a.alone = ch.chunks == 1 && !d.seq_offsets;
  a.loss = d.loss;
  a.tokens = d.tokens;
  a.row_loss = d.row_loss;
  a.row_stats = d.row_stats;
  a.status = status;
  LaunchFwd f{a, ch.chunks, s};
  const cudaError_t e = with_row_variant(d.dt, plan, f);
  if (e != cudaSuccess || a.alone) return e;
  FinishArgs fin{a.part_loss, a.part_rows, a.part_bad, a.seqs, ch.rows, d.loss, d.tokens, status};
  return launch_pdl(distill_finish_kernel, dim3((unsigned)((d.num_seqs + kWarps - 1) / kWarps)), dim3(kThreads), 0,
                    s, fin);
}

}  // namespace moe
