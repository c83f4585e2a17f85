// api_mx.cu -- the microscaled calls of include/moe.h: rows to 4 and 8 bits and
// back, experts on 4-bit operands, and the expert training step that keeps its
// activations in 8 bits.  Checks, workspaces and the order of the launches.
#include <algorithm>
#include <climits>
#include <new>

#include "api.h"

struct moe_mx4_experts {
  moe_dtype dt;
  int64_t E, I, H;
  int device;
  int num_sms;
  moe::Mx4Weights* w;
};

namespace {

using namespace moe::api;

bool valid_format(moe_mx_format f) { return f == MOE_MXFP4 || f == MOE_MXFP8; }

uint64_t value_bytes(int64_t R, int64_t C, moe_mx_format f) {
  return (uint64_t)R * (f == MOE_MXFP4 ? (C + 1) / 2 : C);
}
uint64_t scale_bytes(int64_t R, int64_t C) { return (uint64_t)R * ((C + 31) / 32); }

moe_status check_rows(int64_t n, const char* name) {
  if (n < 0) return fail(MOE_ERR_SHAPE, "%s must be >= 0 (got %lld)", name, (long long)n);
  if (n > kMaxRows) return fail(MOE_ERR_UNSUPPORTED, "%s=%lld exceeds 2^31-1", name, (long long)n);
  return MOE_OK;
}

moe_status check_mx4(const moe_mx4_experts* x) {
  if (!x) return fail(MOE_ERR_INVALID_ARG, "experts handle is NULL");
  int dev = -1;
  MOE_TRY_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  if (dev != x->device)
    return fail(MOE_ERR_INVALID_ARG, "experts live on device %d but device %d is current", x->device, dev);
  return MOE_OK;
}

struct Mx4Layout {
  size_t offsets, xq, xs, hq, hs;              // every call
  size_t idx, weights, perm, scratch, slot_row, slots;  // the fused forward
  size_t total;
};

void rows_layout(Cursor& c, Mx4Layout& L, const moe_mx4_experts* x, int64_t N) {
  L.offsets = c.take((size_t)(x->E + 1) * 4);
  L.xq = c.take((size_t)N * x->H / 2);
  L.xs = c.take(moe::mx4_row_scale_bytes(N, x->E, x->H));
  L.hq = c.take((size_t)N * x->I / 2);
  L.hs = c.take(moe::mx4_row_scale_bytes(N, x->E, x->I));
}

Mx4Layout staged_layout(const moe_mx4_experts* x, int64_t N) {
  Cursor c;
  Mx4Layout L{};
  rows_layout(c, L, x, N);
  L.total = c.off;
  return L;
}

Mx4Layout fused_layout(const moe_mx4_experts* x, int64_t T, int32_t k, moe_dtype ldt) {
  const size_t N = (size_t)T * k;
  Cursor c;
  Mx4Layout L{};
  rows_layout(c, L, x, (int64_t)N);
  L.idx = c.take(N * 4);
  L.weights = c.take(N * dtype_size(ldt));
  L.perm = c.take(N * 4);
  L.scratch = c.take(moe::dispatch_scratch_bytes(T, (int)x->E));
  L.slot_row = c.take(N * 4);
  L.slots = c.take(N * (size_t)x->H * 4);
  L.total = c.off;
  return L;
}

// The two products over rows that are in 4 bits already.
moe_status run_mx4(const moe_mx4_experts* x, int64_t N, const uint32_t* offsets, void* ws, const Mx4Layout& L,
                   void* out, const uint32_t* perm, const void* weights, moe_dtype wdt, cudaStream_t s) {
  moe::Mx4Args a{};
  a.gate_up = true;
  a.E = (int)x->E;
  a.N = N;
  a.I = x->I;
  a.H = x->H;
  a.a = at<void>(ws, L.xq);
  a.a_scales = at<void>(ws, L.xs);
  a.offsets = offsets;
  a.hq = at<void>(ws, L.hq);
  a.hs = at<void>(ws, L.hs);
  a.dt = x->dt;
  a.wdt = MOE_F32;
  a.status = status_word(ws);
  MOE_TRY_CUDA(moe::launch_gemm_mx4(a, x->w, x->num_sms, s), "4-bit gate/up product launch");
  a.gate_up = false;
  a.a = at<void>(ws, L.hq);
  a.a_scales = at<void>(ws, L.hs);
  a.out = out;
  a.perm = perm;
  a.weights = weights;
  a.wdt = wdt;
  MOE_TRY_CUDA(moe::launch_gemm_mx4(a, x->w, x->num_sms, s), "4-bit down product launch");
  return MOE_OK;
}

// Route: cudaError_t(uint32_t* idx, void* weights, cudaStream_t)
template <typename Route>
moe_status mx4_forward(moe_mx4_experts_t x, const void* xin, const void* logits, moe_dtype ldt, int64_t T, int32_t k,
                       const Route& route, void* y, void* ws, size_t ws_bytes, cudaStream_t s) {
  if (T == 0) return ok();
  if (!xin || !logits || !y) return fail(MOE_ERR_INVALID_ARG, "x, logits and y must be non-NULL");
  if (!aligned16(xin) || !aligned16(y)) return fail(MOE_ERR_INVALID_ARG, "x and y must be 16-byte aligned");
  const Mx4Layout L = fused_layout(x, T, k, ldt);
  moe_status st = check_ws(ws, ws_bytes, L.total);
  if (st != MOE_OK) return st;
  const int E = (int)x->E;
  uint32_t* idx = at<uint32_t>(ws, L.idx);
  uint32_t* offsets = at<uint32_t>(ws, L.offsets);
  uint32_t* perm = at<uint32_t>(ws, L.perm);
  uint32_t* slot_row = at<uint32_t>(ws, L.slot_row);
  void* w = at<void>(ws, L.weights);
  float* slots = at<float>(ws, L.slots);
  MOE_TRY_CUDA(route(idx, w, s), "routing kernel launch");
  if (T * k <= moe::mx4_small_slots()) {
    MOE_TRY_CUDA(moe::launch_mx4_dispatch_rows(xin, x->dt, T, x->H, idx, k, E, offsets, perm, status_word(ws),
                                               at<uint8_t>(ws, L.xq), at<uint8_t>(ws, L.xs), x->num_sms, s),
                 "4-bit dispatch launch");
  } else {
    MOE_TRY_CUDA(moe::launch_dispatch(idx, T, E, k, offsets, nullptr, perm, at<void>(ws, L.scratch), status_word(ws),
                                      s, slot_row),
                 "dispatch kernel launch");
    MOE_TRY_CUDA(moe::launch_mx4_rows(xin, x->dt, T, x->H, slot_row, k, offsets, E, nullptr, nullptr,
                                      at<uint8_t>(ws, L.xq), at<uint8_t>(ws, L.xs), x->num_sms, s),
                 "4-bit row launch");
  }
  if ((st = run_mx4(x, T * k, offsets, ws, L, slots, perm, w, ldt, s)) != MOE_OK) return st;
  MOE_TRY_CUDA(moe::launch_slot_sum_f32(slots, T, k, x->H, y, x->dt, s), "combine kernel launch");
  return ok();
}

}  // namespace

extern "C" {

// ---- microscaled rows ------------------------------------------------------
moe_status moe_mx_quantize(const void* x, moe_dtype dt, int64_t R, int64_t C, moe_mx_format fmt, uint8_t* values,
                           uint8_t* scales, cudaStream_t stream) {
  if (!valid_dtype(dt)) return fail(MOE_ERR_DTYPE, "x dtype %d is not F32/F16/BF16", (int)dt);
  if (!valid_format(fmt)) return fail(MOE_ERR_DTYPE, "format %d is not MXFP4/MXFP8", (int)fmt);
  moe_status st;
  if ((st = check_rows(R, "R")) != MOE_OK || (st = check_dim(C, "C")) != MOE_OK) return st;
  if (R == 0) return ok();
  if (!x || !values || !scales) return fail(MOE_ERR_INVALID_ARG, "x, values and scales must be non-NULL");
  if (reinterpret_cast<uintptr_t>(x) % dtype_size(dt) != 0) return fail(MOE_ERR_INVALID_ARG, "x is misaligned for its dtype");
  const uint64_t xb = (uint64_t)R * C * dtype_size(dt), vb = value_bytes(R, C, fmt), sb = scale_bytes(R, C);
  if (overlap(values, vb, x, xb) || overlap(scales, sb, x, xb) || overlap(values, vb, scales, sb))
    return fail(MOE_ERR_INVALID_ARG, "x, values and scales must not overlap");
  MOE_TRY_CUDA(moe::launch_mx_quantize(x, dt, R, C, fmt, values, scales, stream), "quantise launch");
  return ok();
}

moe_status moe_mx_dequantize(const uint8_t* values, const uint8_t* scales, moe_mx_format fmt, int64_t R, int64_t C,
                             const uint32_t* perm, int32_t top_k, int64_t n, void* out, moe_dtype dt,
                             cudaStream_t stream) {
  if (!valid_dtype(dt)) return fail(MOE_ERR_DTYPE, "out dtype %d is not F32/F16/BF16", (int)dt);
  if (!valid_format(fmt)) return fail(MOE_ERR_DTYPE, "format %d is not MXFP4/MXFP8", (int)fmt);
  moe_status st;
  if ((st = check_rows(R, "R")) != MOE_OK || (st = check_rows(n, "n")) != MOE_OK ||
      (st = check_dim(C, "C")) != MOE_OK)
    return st;
  if (top_k < 1) return fail(MOE_ERR_INVALID_ARG, "top_k must be >= 1 (got %d)", top_k);
  if (n == 0) return ok();  // (an empty map has no address)
  if (!perm && n != R)
    return fail(MOE_ERR_SHAPE, "n=%lld must be R=%lld without perm", (long long)n, (long long)R);
  if (!perm && top_k != 1) return fail(MOE_ERR_INVALID_ARG, "top_k=%d needs perm", top_k);
  if (!out || (R > 0 && (!values || !scales)))
    return fail(MOE_ERR_INVALID_ARG, "values, scales and out must be non-NULL");
  if (reinterpret_cast<uintptr_t>(out) % dtype_size(dt) != 0 || reinterpret_cast<uintptr_t>(perm) % 4 != 0)
    return fail(MOE_ERR_INVALID_ARG, "out or perm is misaligned");
  const uint64_t ob = (uint64_t)n * C * dtype_size(dt);
  if (overlap(out, ob, values, value_bytes(R, C, fmt)) || overlap(out, ob, scales, scale_bytes(R, C)) ||
      (perm && overlap(out, ob, perm, (uint64_t)n * 4)))
    return fail(MOE_ERR_INVALID_ARG, "out must not overlap values, scales or perm");
  MOE_TRY_CUDA(moe::launch_mx_dequantize(values, scales, fmt, R, C, perm, top_k, n, out, dt, stream),
               "dequantise launch");
  return ok();
}

// ---- 4-bit experts -----------------------------------------------------------
size_t moe_mx4_experts_scale_bytes(int64_t E, int64_t I, int64_t H) {
  if (E < 1 || E > kMaxE || I < 1 || I > kMaxDim || H < 1 || H > kMaxDim) return 0;
  return 2 * moe::mx4_weight_scale_bytes(E * I, H) + moe::mx4_weight_scale_bytes(E * H, I);
}

moe_status moe_mx4_experts_create(const uint8_t* gate, const uint8_t* gate_scales, const uint8_t* up,
                                  const uint8_t* up_scales, const uint8_t* down, const uint8_t* down_scales,
                                  moe_dtype dt, int64_t E, int64_t I, int64_t H, void* buffer, size_t buffer_bytes,
                                  cudaStream_t stream, moe_mx4_experts_t* out) {
  if (!out) return fail(MOE_ERR_INVALID_ARG, "out handle pointer is NULL");
  *out = nullptr;
  if (dt != MOE_F16 && dt != MOE_BF16) return fail(MOE_ERR_DTYPE, "4-bit experts take F16 or BF16 rows (dtype %d)", (int)dt);
  if (E < 1) return fail(MOE_ERR_SHAPE, "E must be >= 1 (got %lld)", (long long)E);
  if (E > kMaxE) return fail(MOE_ERR_UNSUPPORTED, "E=%lld exceeds the supported 1024", (long long)E);
  moe_status st;
  if ((st = check_dim(I, "I")) != MOE_OK || (st = check_dim(H, "H")) != MOE_OK) return st;
  if (I % 32 != 0 || H % 32 != 0)
    return fail(MOE_ERR_UNSUPPORTED, "4-bit experts need H and I in whole blocks of 32 (I=%lld H=%lld)", (long long)I,
                (long long)H);
  if (!gate || !up || !down || !gate_scales || !up_scales || !down_scales)
    return fail(MOE_ERR_INVALID_ARG, "gate, up, down and their scales must be non-NULL");
  if (!aligned16(gate) || !aligned16(up) || !aligned16(down))
    return fail(MOE_ERR_INVALID_ARG, "expert weight values must be 16-byte aligned");
  if (!buffer || !aligned256(buffer)) return fail(MOE_ERR_INVALID_ARG, "scale_buffer must be non-NULL and 256-byte aligned");
  if (buffer_bytes < moe_mx4_experts_scale_bytes(E, I, H))
    return fail(MOE_ERR_INVALID_ARG, "scale_buffer too small: %zu bytes given, %zu needed", buffer_bytes,
                moe_mx4_experts_scale_bytes(E, I, H));
  // (each tensor's scales are re-ordered while the others' wait, and the values are used as they are)
  const uint64_t vb = value_bytes(E * I, H, MOE_MXFP4), sb = scale_bytes(E * I, H), db = scale_bytes(E * H, I);
  const Range scratch[1] = {{buffer, moe_mx4_experts_scale_bytes(E, I, H)}};
  const Range held[6] = {{gate, vb}, {up, vb}, {down, vb}, {gate_scales, sb}, {up_scales, sb}, {down_scales, db}};
  if (!apart(scratch, held))
    return fail(MOE_ERR_INVALID_ARG, "scale_buffer must not overlap the weights or their scales");
  int dev = -1;
  MOE_TRY_CUDA(cudaGetDevice(&dev), "cudaGetDevice");
  const void* ptrs[7] = {gate, up, down, gate_scales, up_scales, down_scales, buffer};
  for (const void* p : ptrs) {
    cudaPointerAttributes a{};
    MOE_TRY_CUDA(cudaPointerGetAttributes(&a, p), "cudaPointerGetAttributes");
    if (a.type != cudaMemoryTypeDevice && a.type != cudaMemoryTypeManaged)
      return fail(MOE_ERR_INVALID_ARG, "expert weights must be device memory");
    if (a.device != dev) return fail(MOE_ERR_INVALID_ARG, "expert weights must live on the current device %d", dev);
  }
  int sms = 0;
  MOE_TRY_CUDA(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "cudaDeviceGetAttribute");
  uint8_t* sg = static_cast<uint8_t*>(buffer);
  uint8_t* su = sg + moe::mx4_weight_scale_bytes(E * I, H);
  uint8_t* sd = su + moe::mx4_weight_scale_bytes(E * I, H);
  const char* err = "";
  moe::Mx4Weights* w = moe::mx4_weights_create(gate, up, down, sg, su, sd, E, I, H, &err);
  if (!w) return fail(MOE_ERR_CUDA, "%s", err);
  moe_mx4_experts* x = new (std::nothrow) moe_mx4_experts{dt, E, I, H, dev, sms, w};
  cudaError_t e = x ? moe::launch_mx4_weight_scales(gate_scales, E, I, H, sg, stream) : cudaErrorMemoryAllocation;
  if (e == cudaSuccess) e = moe::launch_mx4_weight_scales(up_scales, E, I, H, su, stream);
  if (e == cudaSuccess) e = moe::launch_mx4_weight_scales(down_scales, E, H, I, sd, stream);
  if (e != cudaSuccess) {
    moe::mx4_weights_destroy(w);
    delete x;
    return cuda_fail(e, "4-bit expert scales");
  }
  *out = x;
  return ok();
}

void moe_mx4_experts_destroy(moe_mx4_experts_t x) {
  if (!x) return;
  moe::mx4_weights_destroy(x->w);
  delete x;
}

size_t moe_mx4_experts_workspace_size(moe_mx4_experts_t x, int64_t N) {
  if (!x || N < 0 || N > kMaxRows) return 0;
  return staged_layout(x, N).total;
}

moe_status moe_mx4_experts_forward(moe_mx4_experts_t x, const void* x_disp, int64_t N, const uint32_t* offsets,
                                   void* expert_out, void* ws, size_t ws_bytes, cudaStream_t stream) {
  moe_status st = check_mx4(x);
  if (st != MOE_OK) return st;
  if (N < 0 || N > kMaxRows) return fail(MOE_ERR_SHAPE, "N=%lld out of range", (long long)N);
  if (N == 0) return ok();
  if (!x_disp || !offsets || !expert_out)
    return fail(MOE_ERR_INVALID_ARG, "x_disp, offsets and expert_out must be non-NULL");
  if (!aligned16(x_disp) || !aligned16(expert_out))
    return fail(MOE_ERR_INVALID_ARG, "x_disp and expert_out must be 16-byte aligned");
  const Mx4Layout L = staged_layout(x, N);
  if ((st = check_ws(ws, ws_bytes, L.total)) != MOE_OK) return st;
  uint32_t* off_ok = at<uint32_t>(ws, L.offsets);
  MOE_TRY_CUDA(moe::launch_mx4_rows(x_disp, x->dt, N, x->H, nullptr, 1, offsets, (int)x->E, off_ok, status_word(ws),
                                    at<uint8_t>(ws, L.xq), at<uint8_t>(ws, L.xs), x->num_sms, stream),
               "4-bit row launch");
  st = run_mx4(x, N, off_ok, ws, L, expert_out, nullptr, nullptr, MOE_F32, stream);
  return st == MOE_OK ? ok() : st;
}

size_t moe_mx4_forward_workspace_size(moe_mx4_experts_t x, int64_t T, int32_t top_k, moe_dtype ldt) {
  if (!x || T < 0 || top_k < 1 || T > kMaxRows / top_k || !valid_dtype(ldt)) return 0;
  return fused_layout(x, T, top_k, ldt).total;
}

moe_status moe_mx4_forward(moe_mx4_experts_t x, const void* xin, const void* logits, moe_dtype ldt, int64_t T,
                           int32_t top_k, int renormalize, void* y, void* ws, size_t ws_bytes, cudaStream_t stream) {
  moe_status st = check_mx4(x);
  if (st != MOE_OK) return st;
  if (!valid_dtype(ldt)) return fail(MOE_ERR_DTYPE, "logits dtype %d is not F32/F16/BF16", (int)ldt);
  if ((st = check_tek(T, x->E, top_k)) != MOE_OK) return st;
  const int E = (int)x->E;
  auto route = [=](uint32_t* idx, void* w, cudaStream_t s) {
    return moe::launch_route(logits, ldt, T, E, top_k, renormalize, idx, w, nullptr, nullptr, s);
  };
  return mx4_forward(x, xin, logits, ldt, T, top_k, route, y, ws, ws_bytes, stream);
}

moe_status moe_mx4_forward_sigmoid_grouped(moe_mx4_experts_t x, const void* xin, const void* logits, moe_dtype ldt,
                                           int64_t T, const float* bias, const moe_group_routing_options* opt,
                                           void* y, void* ws, size_t ws_bytes, cudaStream_t stream) {
  moe_status st = check_mx4(x);
  if (st != MOE_OK) return st;
  if (!valid_dtype(ldt)) return fail(MOE_ERR_DTYPE, "logits dtype %d is not F32/F16/BF16", (int)ldt);
  if ((st = check_group_options(T, x->E, opt)) != MOE_OK) return st;
  const int E = (int)x->E;
  const moe_group_routing_options o = *opt;
  auto route = [=](uint32_t* idx, void* w, cudaStream_t s) {
    return moe::launch_route_sigmoid_grouped(logits, ldt, T, E, bias, o.top_k, o.groups, o.selected_groups,
                                             o.group_top_two, o.renormalize, o.scale, idx, w, nullptr, s);
  };
  return mx4_forward(x, xin, logits, ldt, T, o.top_k, route, y, ws, ws_bytes, stream);
}

}  // extern "C"
