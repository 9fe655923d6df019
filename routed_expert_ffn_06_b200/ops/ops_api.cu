// ops_api.cu -- the C ABI declared in include/moe_ops.h: argument validation
// and the launches of each entry point.
#include <cuda_runtime.h>
#include <math.h>

#include "ops.h"

namespace moe {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Two ranges of bytes have one in common.
bool overlap(const void* p, size_t np, const void* q, size_t nq) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return a < b + nq && b < a + np && np && nq;
}

moe_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return MOE_OK;
  cudaGetLastError();
  return MOE_ERR_CUDA;
}

// A row pitch in elements: 0 stands for d; false when it is not usable.
bool pitch(int64_t ld, int d, long long* out) {
  *out = ld == 0 ? d : ld;
  return *out >= d && *out % 8 == 0;
}

moe_status validate_mat(const moe_fp8_mat* w) {
  if (!w || !w->codes || !w->scales) return MOE_ERR_INVALID_ARG;
  if (w->n < 1 || w->n > 65536 || w->k < 16 || w->k > 65536 || w->k % 16 || w->groups < 1 ||
      w->groups > 1024 || (long long)w->n * w->groups >= (1ll << 31))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(w->codes, 16) || !aligned(w->scales, 4)) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

moe_status gemm(const moe_fp8_mat* w, const uint8_t* a, const float* a_scales, int32_t M,
                const int32_t* offsets, void* c, void* ws, void* stream) {
  moe_status s = validate_mat(w);
  if (s != MOE_OK) return s;
  if (M < 0 || !a || !a_scales || !c) return MOE_ERR_INVALID_ARG;
  if (M > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!offsets && w->groups != 1) return MOE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(a_scales, 4) || !aligned(c, 2) || !aligned(offsets, 4) ||
      !aligned(ws, 256))
    return MOE_ERR_MISALIGNED;
  const size_t cb = (size_t)M * w->n * 2;
  if (overlap(c, cb, a, (size_t)M * w->k) ||
      overlap(c, cb, a_scales, (size_t)M * blocks128(w->k) * 4))
    return MOE_ERR_INVALID_ARG;
  if ((s = check_device()) != MOE_OK) return s;
  if (M == 0) return MOE_OK;
  GemmArgs g;
  g.M = M;
  g.N = w->n;
  g.K = w->k;
  g.G = w->groups;
  g.a = a;
  g.a_scales = a_scales;
  g.w = w->codes;
  g.w_scales = w->scales;
  g.offsets = offsets;
  g.c = static_cast<uint16_t*>(c);
  g.ctl = static_cast<Control*>(ws);
  return from_cuda(launch_fp8_gemm(g, static_cast<cudaStream_t>(stream)));
}

bool bad_width(int v) { return v < 32 || v > 4096 || v % 32; }

moe_status validate_fp8_layer(const moe_fp8_layer* l) {
  if (!l) return MOE_ERR_INVALID_ARG;
  if (bad_width(l->d_model) || bad_width(l->ffn) || (l->shared_ffn != 0 && bad_width(l->shared_ffn)))
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (l->top_k < 1 || l->top_k > 16 || l->n_experts < l->top_k || l->n_experts > 1024)
    return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!l->router_w || !l->gate_up || !l->gate_up_scales || !l->down || !l->down_scales)
    return MOE_ERR_INVALID_ARG;
  if (l->shared_ffn && (!l->shared_gate_up || !l->shared_gate_up_scales || !l->shared_down ||
                        !l->shared_down_scales))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(l->router_w, 16) || !aligned(l->gate_up, 16) || !aligned(l->down, 16) ||
      !aligned(l->gate_up_scales, 4) || !aligned(l->down_scales, 4) || !aligned(l->router_bias, 4))
    return MOE_ERR_MISALIGNED;
  if (l->shared_ffn && (!aligned(l->shared_gate_up, 16) || !aligned(l->shared_down, 16) ||
                        !aligned(l->shared_gate_up_scales, 4) || !aligned(l->shared_down_scales, 4)))
    return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

Fp8LayerDev to_dev(const moe_fp8_layer* l) {
  Fp8LayerDev L;
  L.d = l->d_model;
  L.E = l->n_experts;
  L.F = l->ffn;
  L.k = l->top_k;
  L.Fs = l->shared_ffn;
  L.Wr = l->router_w;
  L.bias = l->router_bias;
  L.gu = l->gate_up;
  L.gus = l->gate_up_scales;
  L.dn = l->down;
  L.dns = l->down_scales;
  L.sgu = l->shared_gate_up;
  L.sgus = l->shared_gate_up_scales;
  L.sdn = l->shared_down;
  L.sdns = l->shared_down_scales;
  return L;
}

}  // namespace

cudaError_t allow_smem(const void* kernel, size_t most) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_norm_block(const moe_norm* n, const void* x, const void* y_or_null,
                          const void* gate_or_null, int32_t T, void* x_out_or_null,
                          void* h_or_null, uint8_t* codes_or_null, float* scales_or_null,
                          void* stream) {
  if (!n || !x || T < 0) return MOE_ERR_INVALID_ARG;
  if (n->flags & ~(MOE_NORM_F_POST | MOE_NORM_F_ZERO_CENTRED | MOE_NORM_F_STREAM_F32 |
                   MOE_NORM_F_SIGMOID))
    return MOE_ERR_INVALID_ARG;
  if (n->gate_kind < MOE_GATE_NONE || n->gate_kind > MOE_GATE_FULL) return MOE_ERR_INVALID_ARG;
  if (!(n->eps > 0.f) || !isfinite(n->eps) || !isfinite(n->stream_scale) ||
      !isfinite(n->branch_scale))
    return MOE_ERR_INVALID_ARG;
  if (n->d < 8 || n->d > 8192 || n->d % 8 || T > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!codes_or_null != !scales_or_null) return MOE_ERR_INVALID_ARG;
  if (!x_out_or_null && !h_or_null && !codes_or_null) return MOE_ERR_INVALID_ARG;
  const bool gated = y_or_null && n->gate_kind != MOE_GATE_NONE;
  if (gated && !gate_or_null) return MOE_ERR_INVALID_ARG;
  NormArgs a = {};
  if (!pitch(n->x_ld, n->d, &a.x_ld) || !pitch(n->y_ld, n->d, &a.y_ld) ||
      !pitch(n->gate_ld, n->d, &a.gate_ld) || !pitch(n->x_out_ld, n->d, &a.x_out_ld) ||
      !pitch(n->h_ld, n->d, &a.h_ld))
    return MOE_ERR_INVALID_ARG;
  // in-place rows are read whole before they are written only where they coincide
  if ((x_out_or_null == x && a.x_out_ld != a.x_ld) ||
      (h_or_null && h_or_null == y_or_null && a.h_ld != a.y_ld) || h_or_null == x ||
      (x_out_or_null && (x_out_or_null == y_or_null || x_out_or_null == h_or_null)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(y_or_null, 16) || !aligned(x_out_or_null, 16) ||
      !aligned(h_or_null, 16) || !aligned(n->pre_w, 16) || !aligned(n->post_w, 16) ||
      !aligned(codes_or_null, 8) || !aligned(scales_or_null, 4) ||
      (gated && !aligned(gate_or_null, n->gate_kind == MOE_GATE_TOKEN ? 2 : 16)))
    return MOE_ERR_MISALIGNED;
  moe_status s = check_device();
  if (s != MOE_OK) return s;
  if (T == 0) return MOE_OK;
  a.d = n->d;
  a.T = T;
  a.gate_kind = gated ? n->gate_kind : MOE_GATE_NONE;
  a.post = (n->flags & MOE_NORM_F_POST) && y_or_null;
  a.sigmoid = n->flags & MOE_NORM_F_SIGMOID;
  a.eps = n->eps;
  a.inv_d = (float)(1.0 / n->d);
  a.a = n->stream_scale;
  a.b = n->branch_scale;
  a.w_off = (n->flags & MOE_NORM_F_ZERO_CENTRED) ? 1.f : 0.f;
  a.pre_w = n->pre_w;
  a.post_w = n->post_w;
  a.x = x;
  a.y = static_cast<const uint16_t*>(y_or_null);
  a.gate = static_cast<const uint16_t*>(gate_or_null);
  a.x_out = x_out_or_null;
  a.h = static_cast<uint16_t*>(h_or_null);
  a.codes = codes_or_null;
  a.scales = scales_or_null;
  return from_cuda(launch_norm_block(a, n->flags & MOE_NORM_F_STREAM_F32,
                                     static_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_quant(const void* x, int64_t ld, int32_t T, int32_t d, uint8_t* codes,
                         float* scales, void* stream) {
  if (!x || !codes || !scales || T < 0) return MOE_ERR_INVALID_ARG;
  if (d < 8 || d > 65536 || d % 8 || T > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  long long p;
  if (!pitch(ld, d, &p)) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(codes, 8) || !aligned(scales, 4)) return MOE_ERR_MISALIGNED;
  moe_status s = check_device();
  if (s != MOE_OK) return s;
  if (T == 0) return MOE_OK;
  return from_cuda(launch_fp8_quant(static_cast<const uint16_t*>(x), p, T, d, codes, scales,
                                    static_cast<cudaStream_t>(stream)));
}

moe_status moe_fp8_gemm(const moe_fp8_mat* w, const uint8_t* a, const float* a_scales, int32_t M,
                        void* c_bf16, void* ws_or_null, void* stream) {
  return gemm(w, a, a_scales, M, nullptr, c_bf16, ws_or_null, stream);
}

moe_status moe_fp8_gemm_grouped(const moe_fp8_mat* w, const uint8_t* a, const float* a_scales,
                                int32_t M, const int32_t* offsets, void* c_bf16, void* ws_or_null,
                                void* stream) {
  if (!offsets) return MOE_ERR_INVALID_ARG;
  return gemm(w, a, a_scales, M, offsets, c_bf16, ws_or_null, stream);
}

moe_status moe_fp8_gemm_plan(const moe_fp8_mat* w, int32_t M, int32_t grouped, int32_t plan[3]) {
  moe_status s = validate_mat(w);
  if (s != MOE_OK) return s;
  if (M < 1 || !plan || (!grouped && w->groups != 1)) return MOE_ERR_INVALID_ARG;
  if (M > kMaxRows) return MOE_ERR_UNSUPPORTED_SHAPE;
  const GemmPlan p = plan_fp8_gemm(M, w->n, w->groups, grouped != 0, sm_count());
  plan[0] = p.bn;
  plan[1] = p.a_rows;
  plan[2] = p.stages;
  return MOE_OK;
}

size_t moe_fp8_layer_workspace_bytes(const moe_fp8_layer* layer, int32_t max_tokens) {
  if (validate_fp8_layer(layer) != MOE_OK || max_tokens < 0 || max_tokens > MOE_FP8_LAYER_MAX_T)
    return 0;
  return fp8_layer_ws_bytes(to_dev(layer));
}

moe_status moe_fp8_layer_forward(const moe_fp8_layer* layer, const void* x_bf16, int32_t T,
                                 void* y_bf16, int32_t* ids_or_null, float* w_or_null, void* ws,
                                 size_t ws_bytes, void* stream) {
  moe_status s = validate_fp8_layer(layer);
  if (s != MOE_OK) return s;
  if (T < 0 || !x_bf16 || !y_bf16 || !ws || x_bf16 == y_bf16) return MOE_ERR_INVALID_ARG;
  if (T > MOE_FP8_LAYER_MAX_T) return MOE_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(x_bf16, 16) || !aligned(y_bf16, 16) || !aligned(ws, 256) ||
      !aligned(ids_or_null, 4) || !aligned(w_or_null, 4))
    return MOE_ERR_MISALIGNED;
  const Fp8LayerDev L = to_dev(layer);
  if (overlap(x_bf16, (size_t)T * L.d * 2, y_bf16, (size_t)T * L.d * 2)) return MOE_ERR_INVALID_ARG;
  if (ws_bytes < fp8_layer_ws_bytes(L)) return MOE_ERR_WORKSPACE_TOO_SMALL;
  if ((s = check_device()) != MOE_OK) return s;
  for (int t0 = 0; t0 < T; t0 += kFp8Window) {
    const int n = T - t0 < kFp8Window ? T - t0 : kFp8Window;
    s = from_cuda(launch_fp8_layer(L, static_cast<const uint16_t*>(x_bf16) + (size_t)t0 * L.d, n,
                                   static_cast<uint16_t*>(y_bf16) + (size_t)t0 * L.d,
                                   ids_or_null ? ids_or_null + (size_t)t0 * L.k : nullptr,
                                   w_or_null ? w_or_null + (size_t)t0 * L.k : nullptr,
                                   static_cast<char*>(ws), static_cast<cudaStream_t>(stream)));
    if (s != MOE_OK) return s;
  }
  return MOE_OK;
}

}  // extern "C"
