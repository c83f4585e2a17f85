// internal.h -- launchers shared between the translation units of the library.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/moe.h"

namespace moe {

// ---- routing (route.cu) ----------------------------------------------------
cudaError_t launch_route(const void* logits, moe_dtype ldt, int64_t T, int E, int k, int renorm,
                         uint32_t* idx, void* weights, float* w32, uint32_t* status_reset,
                         cudaStream_t s);

// selected router weights (FP32) and, when dw != nullptr, their logit gradient
cudaError_t launch_router_backward(const void* logits, moe_dtype ldt, int64_t T, int E,
                                   const uint32_t* idx, int k, const float* dw, int scoring,
                                   int renorm, float scale, void* dlogits, float* w_out,
                                   cudaStream_t s);
cudaError_t launch_route_sigmoid_grouped(const void* logits, moe_dtype ldt, int64_t T, int E,
                                         const float* bias, int k, int groups, int sel_groups,
                                         int top_two, int renorm, float scale, uint32_t* idx,
                                         void* weights, float* w32, cudaStream_t s);

// ---- dispatch (dispatch.cu) ------------------------------------------------
constexpr int kDispatchChunk = 256;  // tokens per block of the dispatch kernels
inline int64_t dispatch_chunks(int64_t T) { return (T + kDispatchChunk - 1) / kDispatchChunk; }
// bytes of scratch the dispatch kernels need (chunk counts and chunk bases)
size_t dispatch_scratch_bytes(int64_t T, int E);
cudaError_t launch_dispatch(const uint32_t* idx, int64_t T, int E, int k, uint32_t* offsets,
                            uint32_t* row_experts, uint32_t* perm, void* scratch,
                            uint32_t* status, cudaStream_t s, uint32_t* slot_row = nullptr);
// x_disp in token order from the slot -> row map the scatter wrote (16-byte
// rows and pointers, top_k <= 64; cudaErrorInvalidValue otherwise)
cudaError_t launch_gather_tokens(const void* x, moe_dtype dt, int64_t H, int k, const uint32_t* slot_row,
                                 int64_t T, void* x_disp, cudaStream_t s);
// fixed device scratch for moe_dispatch_noalloc (size limit and address)
size_t dispatch_noalloc_scratch_limit();
cudaError_t dispatch_noalloc_scratch(void** out);
cudaError_t launch_gather(const void* x, moe_dtype dt, int64_t H, int k, const uint32_t* perm,
                          const uint32_t* offsets, int E, int64_t N, void* x_disp, cudaStream_t s);

// ---- training losses of the router (balance*.cu, distill*.cu) -----------------
struct BalanceArgs {
  const void* logits;
  moe_dtype dt;
  const uint32_t* idx;
  const uint8_t* mask;          // nullable
  const uint32_t* seq_offsets;  // nullable
  int64_t T;
  int E, k;
  int64_t num_seqs;
  bool sigmoid;
  float* loss;
  float* z_loss;       // nullable
  float* mean_scores;  // nullable
  uint32_t* counts;
  uint32_t* tokens;
  float* row_stats;    // [T, 2], 8-byte aligned
};
struct BalanceBwdArgs {
  const void* logits;
  moe_dtype dt;
  const float* row_stats;
  const uint32_t* counts;
  const uint32_t* tokens;
  const uint32_t* seq_offsets;
  int64_t T;
  int E, k;
  int64_t num_seqs;
  bool sigmoid;
  const float* dloss;
  const float* dz_loss;  // nullable
  const void* base;      // nullable
  void* dlogits;
};
// partial sums of the forward (behind the workspace's header)
size_t balance_workspace_bytes(int64_t T, int E, int64_t num_seqs);
cudaError_t launch_balance_loss(const BalanceArgs& b, void* ws, uint32_t* status, cudaStream_t s);
cudaError_t launch_balance_loss_backward(const BalanceBwdArgs& b, cudaStream_t s);

struct DistillArgs {
  const void* logits;
  moe_dtype dt;
  const uint32_t* t_idx;
  const void* t_logits;
  moe_dtype t_dt;
  const float* t_rest;          // nullable
  const uint8_t* mask;          // nullable
  const uint32_t* seq_offsets;  // nullable
  int64_t T;
  int E, m;
  int64_t num_seqs;
  float temperature;
  float* loss;
  uint32_t* tokens;
  float* row_loss;
  float* row_stats;  // [5, T]
};
struct DistillBwdArgs {
  const void* logits;
  moe_dtype dt;
  const uint32_t* t_idx;
  const void* t_logits;
  moe_dtype t_dt;
  const float* row_stats;
  const uint32_t* tokens;
  const uint32_t* seq_offsets;
  int64_t T;
  int E, m;
  int64_t num_seqs;
  float temperature;
  const float* dloss;
  const void* base;  // nullable
  void* dlogits;
};
size_t distill_workspace_bytes(int64_t T, int64_t num_seqs);
cudaError_t launch_distill_loss(const DistillArgs& d, void* ws, uint32_t* status, cudaStream_t s);
cudaError_t launch_distill_loss_backward(const DistillBwdArgs& d, cudaStream_t s);
cudaError_t launch_distill_targets(const void* logits, moe_dtype dt, int64_t T, int E, int m, float temperature,
                                   uint32_t* idx, void* top, float* rest, cudaStream_t s);

// ---- microscaled rows (mx.cu) ------------------------------------------------
cudaError_t launch_mx_quantize(const void* x, moe_dtype dt, int64_t R, int64_t C, moe_mx_format fmt,
                               uint8_t* values, uint8_t* scales, cudaStream_t s);
// n output rows: row r of the R held ones, or row perm[r] / k (zero past R)
cudaError_t launch_mx_dequantize(const uint8_t* values, const uint8_t* scales, moe_mx_format fmt, int64_t R,
                                 int64_t C, const uint32_t* perm, int k, int64_t n, void* out, moe_dtype dt,
                                 cudaStream_t s);
// 16-bit rows to e2m1 in dispatch order, scales in the order of the products.
// With slot_row, source row t goes to rows slot_row[t k + j].  Without, rows are
// in order and the offsets are a caller's: they are checked (clamp_offsets),
// written to off_ok, and *status is set.
cudaError_t launch_mx4_rows(const void* x, moe_dtype dt, int64_t rows, int64_t C, const uint32_t* slot_row, int k,
                            const uint32_t* offsets, int E, uint32_t* off_ok, uint32_t* status, uint8_t* values,
                            uint8_t* scales, int num_sms, cudaStream_t s);
// the same with the dispatch, for T k <= mx4_small_slots(): sorts idx [T, k],
// writes offsets [E+1], perm [T k] and zeroes *status
int64_t mx4_small_slots();
cudaError_t launch_mx4_dispatch_rows(const void* x, moe_dtype dt, int64_t T, int64_t C, const uint32_t* idx, int k,
                                     int E, uint32_t* offsets, uint32_t* perm, uint32_t* status, uint8_t* values,
                                     uint8_t* scales, int num_sms, cudaStream_t s);
// weight scales [E, rows, C/32] in the order of the products
cudaError_t launch_mx4_weight_scales(const uint8_t* scales, int64_t E, int64_t rows, int64_t C, uint8_t* out,
                                     cudaStream_t s);
cudaError_t launch_slot_sum_f32(const float* slots, int64_t T, int k, int64_t H, void* y, moe_dtype dt,
                                cudaStream_t s);

// ---- 4-bit experts (gemm_mx4.cu) ----------------------------------------------
struct Mx4Weights;  // prebuilt tensor maps of one 4-bit expert-weight set
// gate, up [E,I,H/2] and down [E,H,I/2] packed; sg, su, sd: scales in product order
Mx4Weights* mx4_weights_create(const void* gate, const void* up, const void* down, const uint8_t* sg,
                               const uint8_t* su, const uint8_t* sd, int64_t E, int64_t I, int64_t H,
                               const char** err);
void mx4_weights_destroy(Mx4Weights* w);
// bytes of the re-ordered scales of rows of C values
size_t mx4_weight_scale_bytes(int64_t rows, int64_t C);
// bytes of the scales of N activation rows of C values in product order
size_t mx4_row_scale_bytes(int64_t N, int64_t E, int64_t C);
struct Mx4Args {
  bool gate_up;             // h = silu(g) u, in 4 bits (hq, hs); else out = A . W_down^T
  int E;
  int64_t N, I, H;
  const void* a;            // packed rows [N, K/2]
  const void* a_scales;
  const uint32_t* offsets;
  void* hq;
  void* hs;
  void* out;                // [N, H] in dt, or FP32 slots [T*k, H] (perm given)
  moe_dtype dt;
  const uint32_t* perm;     // with weights: row r goes to slot perm[r], times its weight
  const void* weights;
  moe_dtype wdt;
  uint32_t* status;
};
cudaError_t launch_gemm_mx4(const Mx4Args& a, const Mx4Weights* w, int num_sms, cudaStream_t s);

// ---- combine (combine.cu) --------------------------------------------------
cudaError_t launch_invert_perm(const uint32_t* perm, int64_t N, uint32_t* slot_row, cudaStream_t s);
cudaError_t launch_combine(const void* expert_out, moe_dtype dt, const uint32_t* slot_row,
                           const void* weights, moe_dtype wdt, int64_t T, int k, int64_t H,
                           void* y, cudaStream_t s);
// dexpert[r] = w[perm[r]] * dy[t], dweights[perm[r]] = <expert_out[r], dy[t]>
cudaError_t launch_combine_backward(const void* expert_out, moe_dtype dt, const uint32_t* perm,
                                    const void* weights, moe_dtype wdt, const void* dy, int64_t T,
                                    int k, int64_t H, void* dexpert, float* dweights, cudaStream_t s);
// y[t] = sum_j slots[t*k+j] (weights already applied), ascending j
cudaError_t launch_slot_sum(const void* slots, moe_dtype dt, int64_t T, int k, int64_t H, void* y,
                            cudaStream_t s);

// ---- grouped GEMMs ---------------------------------------------------------
enum GemmMode {
  kGateUpSwiglu = 0,
  kDownPlain = 1,
  kDownWeighted = 2,
  // backward products (tcgen05 path only; da = dout W_down and dinput use kDownPlain)
  kSwigluBwd = 4,   // g, u recomputed, then [dg | du] (out) and a (out2), 16-bit
  kWgrad = 5,       // per-expert FP32 weight-gradient tiles over the padded rows
  kPartial = 6,     // one part of K, FP32 rows
};

struct GemmArgs {
  int mode;
  moe_dtype dt;
  int E;
  int64_t N;          // rows of the A operand (dispatched rows)
  int64_t K;          // reduction length
  int64_t n_out;      // output columns (I for gate/up, H for down)
  const void* A;      // [N, K]
  const void* B0;     // gate (gate/up) or down weights
  const void* B1;     // up (gate/up) or nullptr
  const uint32_t* offsets;
  void* out;          // [N, n_out] (or [T*k, n_out] slots for weighted mode)
  const uint32_t* perm;
  const void* weights;
  moe_dtype wdt;
  uint32_t* status;
  // gate/up of the tcgen05 path: also hold g and u in 8 bits (mx.cuh), or null
  uint8_t* ck_g;
  uint8_t* ck_u;
  uint8_t* ck_gs;
  uint8_t* ck_us;
};

// Backward of the SwiGLU experts (gemm_bwd.cu): FP32 accumulate, any dtype.
struct ExpertsBwdArgs {
  moe_dtype dt;
  int E;
  int64_t N, H, I;
  const void* x_disp;   // [N, H]
  const void* dout;     // [N, H] gradient of the expert outputs
  const void* gate;     // [E, I, H]
  const void* up;       // [E, I, H]
  const void* down;     // [E, H, I]
  const uint32_t* offsets;
  float* g;             // [N, I] scratch: recomputed gate product
  float* u;             // [N, I] scratch: recomputed up product
  float* act;           // [N, I] scratch: silu(g) * u
  float* dg;            // [N, I] scratch
  float* du;            // [N, I] scratch
  void* dinput;         // [N, H] in dt
  float* dgate;         // [E, I, H]
  float* dup;           // [E, I, H]
  float* ddown;         // [E, H, I]
  uint32_t* status;     // device status word (bounded waits of the tensor-core path)
};
cudaError_t launch_experts_backward(const ExpertsBwdArgs& a, cudaStream_t s);

// offsets of a staged expert call, clamped to [previous, N] (rowpad.cu); a
// clamped entry sets MOE_ERR_INVALID_INDEX in *status
cudaError_t launch_sanitize_offsets(const uint32_t* offsets, int E, int64_t N, uint32_t* out,
                                   uint32_t* status, cudaStream_t s);
// the same, also the status word's first value and, unless null, pad (below)
cudaError_t launch_check_offsets(const uint32_t* offsets, int E, int64_t N, uint32_t* out, uint32_t* status,
                                 uint32_t* pad, cudaStream_t s);
// The 64-padded row space of the tensor-core backward (rowpad.cu)
cudaError_t launch_pad_offsets(const uint32_t* offsets, int E, uint32_t* pad, cudaStream_t s);
cudaError_t launch_pad_rows(const void* src, int64_t C, const uint32_t* offsets, const uint32_t* pad,
                            int E, int64_t npad_max, void* dst, cudaStream_t s);

// the last (rows of e) % 64 rows of each expert's segment, at row 64 e, zeros behind
cudaError_t launch_tail_rows(const void* src, int64_t C, const uint32_t* offsets, int E, void* dst, cudaStream_t s);
// out [E, n] in dt = sum over the k parts of parts [E, k, n], in order
cudaError_t launch_join_parts(const float* parts, int E, int k, int64_t n, void* out, moe_dtype dt, cudaStream_t s);
// rows of the segments of out [N, H] in dt = sum over the k parts [k, N, H], in order
cudaError_t launch_join_rows(const float* parts, int k, int64_t N, int64_t H, const uint32_t* offsets, int E, void* out,
                             moe_dtype dt, cudaStream_t s);
// pad_rows from 8-bit tokens: dispatched row r is token perm[r] / k (zeros past T)
cudaError_t launch_pad_rows_mx8(const uint8_t* x, const uint8_t* scales, int64_t T, int64_t C, const uint32_t* perm,
                                int k, const uint32_t* offsets, const uint32_t* pad, int E, int64_t npad_max,
                                void* dst, moe_dtype dt, cudaStream_t s);

// SIMT FP32-accumulate path (gemm_simt.cu): any dtype and shape
cudaError_t launch_gemm_simt(const GemmArgs& a, cudaStream_t s);

// tcgen05 path (gemm_tc.cu): F16/BF16, K and n_out multiples of 8, 16-byte aligned
struct TcWeights;  // prebuilt tensor maps of one expert-weight set
TcWeights* tc_weights_create(const void* gate, const void* up, const void* down, moe_dtype dt,
                             int64_t E, int64_t I, int64_t H, const char** err);
void tc_weights_destroy(TcWeights* w);
cudaError_t launch_gemm_tc(const GemmArgs& a, const TcWeights* w, int num_sms, cudaStream_t s);
bool tc_supported(moe_dtype dt, int64_t I, int64_t H);
// Expert backward on the tcgen05 engine (F16/BF16): scratch of
// experts_backward_tc_workspace(...) bytes at `ws` (1024-byte aligned);
// a.g/u/act/dg/du are not used.
size_t experts_backward_tc_workspace(int64_t N, int E, int64_t H, int64_t I);
cudaError_t launch_experts_backward_tc(const ExpertsBwdArgs& a, const TcWeights* w, void* ws,
                                       int num_sms, cudaStream_t s);
// Expert backward from 8-bit checkpoints (F16/BF16, tcgen05); weight gradients
// in dt; scratch of experts_backward_ck_workspace(...) bytes, 1024-byte aligned
struct ExpertsCkBwdArgs {
  moe_dtype dt;
  int E, k;
  int64_t T, N, H, I;
  const uint8_t* x;         // e4m3 tokens [T, H]
  const uint8_t* x_scales;  // [T, ceil(H/32)]
  const uint32_t* perm;
  const uint32_t* offsets_in;  // the caller's
  uint32_t* offsets;           // checked copy, written first
  const uint8_t* g;         // e4m3 [N, I]
  const uint8_t* g_scales;  // [N, ceil(I/32)]
  const uint8_t* u;
  const uint8_t* u_scales;
  const void* dout;
  const void* gate;
  const void* up;
  const void* down;
  void* dinput;
  void* dgate;
  void* dup;
  void* ddown;
  uint32_t* status;
};
size_t experts_backward_ck_workspace(int64_t N, int E, int64_t H, int64_t I, int num_sms);
cudaError_t launch_experts_backward_ck(const ExpertsCkBwdArgs& a, void* ws, int num_sms, cudaStream_t s);
// a kernel whose bounded wait is made to expire (failure-path self-test)
cudaError_t launch_bounded_wait_selftest(uint32_t* status, uint64_t limit_ns, cudaStream_t s);

}  // namespace moe
