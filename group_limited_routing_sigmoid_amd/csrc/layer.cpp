// C ABI of the operators around the expert block: host-side checks, then one
// launch.  See include/beam_moe.h for the contract of every entry point.
#include <math.h>

#include "layer.h"

using namespace beam;

namespace {

// Shape and scalar checks shared by the two directions.
int check_norm(int64_t T, int64_t H, int32_t dtype, float eps, float alpha, float beta) {
  if (T < 0 || H < 1 || (dtype != BEAM_F32 && dtype != BEAM_BF16)) return BEAM_ERR_INVALID_ARG;
  if (!(eps > 0.0f) || !isfinite(eps) || !isfinite(alpha) || !isfinite(beta))
    return BEAM_ERR_INVALID_ARG;
  if (H > kNormMaxH || T > norm_max_tokens(static_cast<int>(H))) return BEAM_ERR_UNSUPPORTED;
  return BEAM_OK;
}

// gate and gate_cols belong together, and a gate needs a block output (the
// tensors of an empty batch have no address).
bool gate_ok(int64_t T, const void* o, const void* gate, int64_t gate_cols, int64_t H) {
  if (gate_cols != 0 && gate_cols != 1 && gate_cols != H) return false;
  return T == 0 || (gate ? o && gate_cols > 0 : gate_cols == 0);
}

}  // namespace

extern "C" {

int beam_moe_norm_residual(int64_t T, int64_t H, int32_t dtype, const void* o,
                           const float* post_weight, const void* gate, int64_t gate_cols,
                           const float* pre_weight, float eps, float alpha, float beta,
                           const float* residual, float* residual_out, void* x,
                           uint8_t* x_codes, float* x_scales, void* stream) {
  const int st = check_norm(T, H, dtype, eps, alpha, beta);
  if (st != BEAM_OK) return st;
  if (!gate_ok(T, o, gate, gate_cols, H)) return BEAM_ERR_INVALID_ARG;
  if (x_codes && H % 128) return BEAM_ERR_UNSUPPORTED;
  if (T == 0) return BEAM_OK;
  if (!residual || (o && (!post_weight || !residual_out))) return BEAM_ERR_INVALID_ARG;
  if (!o && !pre_weight) return BEAM_ERR_INVALID_ARG;  // nothing to compute
  if (pre_weight ? (!x && !x_codes) : (x || x_codes)) return BEAM_ERR_INVALID_ARG;
  if ((x_codes == nullptr) != (x_scales == nullptr)) return BEAM_ERR_INVALID_ARG;
  const void* ptrs[] = {o, post_weight, gate, pre_weight, residual, residual_out, x, x_codes,
                        x_scales};
  for (const void* q : ptrs)
    if (!aligned16(q)) return BEAM_ERR_INVALID_ARG;
  NormArgs a;
  a.o = o;
  a.post = post_weight;
  a.gate = gate;
  a.pre = pre_weight;
  a.residual = residual;
  a.residual_out = residual_out;
  a.x = x;
  a.xq = x_codes;
  a.xs = x_scales;
  a.H = static_cast<int>(H);
  a.gate_cols = static_cast<int>(gate_cols);
  a.eps = eps;
  a.alpha = alpha;
  a.beta = beta;
  return hip_status(launch_norm_residual(a, T, dtype, static_cast<hipStream_t>(stream)));
}

int beam_moe_norm_residual_workspace_bytes(int64_t T, int64_t H, size_t* bytes) {
  if (!bytes || T < 0 || H < 1) return BEAM_ERR_INVALID_ARG;
  if (H > kNormMaxH || T > norm_max_tokens(static_cast<int>(H))) return BEAM_ERR_UNSUPPORTED;
  *bytes = static_cast<size_t>(norm_grad_groups(T, static_cast<int>(H))) * 2 * static_cast<size_t>(H) * sizeof(float);
  return BEAM_OK;
}

int beam_moe_norm_residual_backward(int64_t T, int64_t H, int32_t dtype, const void* o,
                                    const float* post_weight, const void* gate,
                                    int64_t gate_cols, const float* pre_weight, float eps,
                                    float alpha, float beta, const float* residual_out,
                                    const float* d_residual_out, const void* d_x,
                                    float* d_residual, void* d_o, void* d_gate,
                                    float* d_pre_weight, float* d_post_weight,
                                    void* workspace, size_t ws_bytes, void* stream) {
  int st = check_norm(T, H, dtype, eps, alpha, beta);
  if (st != BEAM_OK) return st;
  if (!gate_ok(T, o, gate, gate_cols, H)) return BEAM_ERR_INVALID_ARG;
  if (T > 0) {
    // without a block output only x has a gradient of its own
    if (!d_x && (!d_residual_out || !o)) return BEAM_ERR_INVALID_ARG;
    if (!residual_out || !d_residual) return BEAM_ERR_INVALID_ARG;
    if (d_x && (!pre_weight || !d_pre_weight)) return BEAM_ERR_INVALID_ARG;
    if (o && (!post_weight || !d_o || !d_post_weight)) return BEAM_ERR_INVALID_ARG;
    if (gate && !d_gate) return BEAM_ERR_INVALID_ARG;
  }
  const void* ptrs[] = {o,      post_weight, gate,   pre_weight,   residual_out, d_residual_out,
                        d_x,    d_residual,  d_o,    d_gate,       d_pre_weight, d_post_weight};
  for (const void* q : ptrs)
    if (!aligned16(q)) return BEAM_ERR_INVALID_ARG;
  size_t need = 0;
  st = beam_moe_norm_residual_workspace_bytes(T, H, &need);
  if (st != BEAM_OK) return st;
  if (need && (!workspace || ws_bytes < need)) return BEAM_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return BEAM_ERR_INVALID_ARG;
  NormGradArgs a;
  a.o = o;
  a.post = post_weight;
  a.gate = gate;
  a.pre = pre_weight;
  a.r = residual_out;
  a.d_res = d_residual_out;
  a.dx = d_x;
  a.d_residual = d_residual;
  a.d_o = d_o;
  a.d_gate = d_gate;
  a.part = static_cast<float*>(workspace);
  a.T = T;
  a.H = static_cast<int>(H);
  a.gate_cols = static_cast<int>(gate_cols);
  a.eps = eps;
  a.alpha = o ? alpha : 1.0f;  // without o the stream passes unscaled
  a.beta = beta;
  // gradients of weights that took no part are not written
  float* dp = (d_x || T == 0) ? d_pre_weight : nullptr;
  float* dq = (o || T == 0) ? d_post_weight : nullptr;
  return hip_status(
      launch_norm_residual_backward(a, dtype, dp, dq, static_cast<hipStream_t>(stream)));
}

int beam_moe_quant_e4m3_2d(int64_t rows, int64_t cols, int32_t dtype, int32_t block,
                           const void* v, uint8_t* q, float* s, uint8_t* qt, float* st,
                           void* stream) {
  if (rows < 0 || cols < 0 || (dtype != BEAM_F32 && dtype != BEAM_BF16) ||
      (block != 0 && block != 1))
    return BEAM_ERR_INVALID_ARG;
  if (rows > 0x7FFFFFFF || cols > 0x7FFFFFFF ||
      ceil_div(rows, 128) * ceil_div(cols, 128) > kQuantMaxTiles)
    return BEAM_ERR_UNSUPPORTED;
  if (rows == 0 || cols == 0) return BEAM_OK;
  if (!v || (!q && !qt) || !q != !s || !qt != !st) return BEAM_ERR_INVALID_ARG;
  if (!aligned16(v) || !aligned16(q) || !aligned16(s) || !aligned16(qt) || !aligned16(st))
    return BEAM_ERR_INVALID_ARG;
  return hip_status(launch_quant_2d(rows, cols, dtype, block != 0, v, q, s, qt, st,
                                    static_cast<hipStream_t>(stream)));
}

int beam_moe_matmul_e4m3(int64_t M, int64_t N, int64_t K, const uint8_t* a, const float* sa,
                         int64_t sa_row, int64_t sa_block, const uint8_t* b, const float* sb,
                         int64_t sb_row, int64_t sb_block, int32_t b_rows, int32_t dtype, void* y,
                         void* stream) {
  if (M < 0 || N < 0 || K < 0 || (dtype != BEAM_F32 && dtype != BEAM_BF16) ||
      (b_rows != 0 && b_rows != 1))
    return BEAM_ERR_INVALID_ARG;
  if (K % 128 || K > kMatmulMaxK || M > kMatmulMaxRows || N > kMatmulMaxRows ||
      M * N > kMatmulMaxOut)
    return BEAM_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return BEAM_OK;
  if (!y || (K > 0 && (!a || !sa || !b || !sb))) return BEAM_ERR_INVALID_ARG;
  if (sa_row < 0 || sa_block < 0 || sb_row < 0 || sb_block < 0) return BEAM_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(sa) || !aligned16(b) || !aligned16(sb) || !aligned16(y))
    return BEAM_ERR_INVALID_ARG;
  const int64_t za[2] = {sa_row, sa_block}, zb[2] = {sb_row, sb_block};
  return hip_status(launch_matmul_e4m3(M, N, K, a, sa, za, b, sb, zb, b_rows != 0, dtype, y,
                                       static_cast<hipStream_t>(stream)));
}

}  // extern "C"
