// Declarations shared by the operators around the expert block (layer.cpp,
// norm.hip, matmul_fp8.hip).
#pragma once

#include "common.h"
#include "internal.h"

namespace beam {

// norm.hip: the norms around a block, its gate and the residual stream
struct NormArgs {
  const void* o;          // [T, H] block output, or null: r' = residual
  const float* post;      // [H]
  const void* gate;       // [T, H] or [T, 1], or null
  const float* pre;       // [H], or null: no x
  const float* residual;  // [T, H]
  float* residual_out;    // [T, H] (with o)
  void* x;                // [T, H], or null
  uint8_t* xq;            // [T, H] e4m3 codes, or null
  float* xs;              // [T, H/128]
  int H, gate_cols;       // gate_cols: 0 (none), 1 or H
  float eps, alpha, beta;
};
struct NormGradArgs {
  const void* o;
  const float* post;
  const void* gate;
  const float* pre;
  const float* r;      // [T, H] the forward's residual stream r'
  const float* d_res;  // [T, H] gradient of r' from later, or null
  const void* dx;      // [T, H] gradient of x, or null
  float* d_residual;   // [T, H]
  void* d_o;
  void* d_gate;
  float* part;         // workspace [groups][2][H]
  int64_t T;
  int H, gate_cols;
  float eps, alpha, beta;
};
// Workgroups of the backward pass, each with its share of the weights' gradients.
int norm_grad_groups(int64_t T, int H);
int64_t norm_max_tokens(int H);  // a launch holds fewer than 2^32 threads
constexpr int kNormMaxH = 16384;  // 1024 threads of 16 columns
hipError_t launch_norm_residual(const NormArgs& a, int64_t T, int32_t dtype, hipStream_t s);
hipError_t launch_norm_residual_backward(const NormGradArgs& a, int32_t dtype, float* d_pre,
                                         float* d_post, hipStream_t s);
// matmul_fp8.hip: dense e4m3 products and their operands' quantisation
hipError_t launch_quant_2d(int64_t rows, int64_t cols, int32_t dtype, bool block, const void* v,
                           uint8_t* q, float* s, uint8_t* qt, float* st, hipStream_t stream);
// Byte offsets inside a tile of 256 rows are 32-bit; tiles are counted in 31.
constexpr int64_t kMatmulMaxK = 1 << 22, kMatmulMaxRows = (1 << 23) - 128;
constexpr int64_t kQuantMaxTiles = (int64_t{1} << 23) - 1;  // of 512 threads, under 2^32 in all
constexpr int64_t kMatmulMaxOut = int64_t{1} << 38;
hipError_t launch_matmul_e4m3(int64_t M, int64_t N, int64_t K, const uint8_t* a, const float* sa,
                              const int64_t* sa_stride, const uint8_t* b, const float* sb,
                              const int64_t* sb_stride, bool rows, int32_t dtype, void* y,
                              hipStream_t s);

// A block's scale s = e4m3_scale(amax) and the quotients v / s of its values,
// bit for bit the binary32 divisions of the recipe, in three instructions a
// quotient instead of about eleven.  With y = RN(1/b), q = RN(v y), the
// remainder v - q b is exact in one fused multiply-add and RN(q + remainder y)
// is the correctly rounded quotient; and y itself is RN(y0 + (1 - b y0) y0)
// from an approximation y0 within an ulp (P. Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", 1990, which
// excepts divisors whose significand is all ones), as long as nothing under-
// or overflows: with amax from 2^-80 to 2^90 only a quotient below 2^-25 can,
// which any rounding turns into the code 0.  Other blocks divide.  (Tested
// for every significand of amax: the scale's bits, and the codes of values on
// and beside the midpoints of neighbouring codes.)
struct BlockDivisor {
  float s, y;
  bool fast;
  __device__ __forceinline__ explicit BlockDivisor(float amax) {
    constexpr float kBy448 = 1.0f / 448.0f;
    const float q = amax * kBy448;
    s = __builtin_fmaf(__builtin_fmaf(q, 448.0f, -amax), -kBy448, q);
    fast = amax >= 0x1p-80f && amax <= 0x1p90f && (__float_as_uint(s) & 0x7FFFFFu) != 0x7FFFFFu;
    if (!fast) s = e4m3_scale(amax);
    const float y0 = __builtin_amdgcn_rcpf(s);
    y = __builtin_fmaf(__builtin_fmaf(-s, y0, 1.0f), y0, y0);
  }
  // With the remainder's and the reciprocal's signs turned, a quotient of -0
  // keeps its sign.
  __device__ __forceinline__ float quotient(float v) const {
    const float q = v * y;
    return __builtin_fmaf(__builtin_fmaf(q, s, -v), -y, q);
  }
  // The codes of four values no larger than the block's amax: quotients of at
  // most 448 (1 + 2^-23), which need no clamp, where the scale is not
  // subnormal.
  __device__ __forceinline__ uint32_t codes(const float (&v)[4]) const {
    if (fast) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[0]), quotient(v[1]), 0, false);
      return static_cast<uint32_t>(
          __builtin_amdgcn_cvt_pk_fp8_f32(quotient(v[2]), quotient(v[3]), lo, true));
    }
    // a NaN (also an infinity over the scale it makes) stays one
    auto code = [&](float x) { return x == x ? sat448(x) : x; };
    const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(code(v[0] / s), code(v[1] / s), 0, false);
    return static_cast<uint32_t>(
        __builtin_amdgcn_cvt_pk_fp8_f32(code(v[2] / s), code(v[3] / s), lo, true));
  }
  __device__ __forceinline__ uint2 codes(const float (&v)[8]) const {
    const float lo[4] = {v[0], v[1], v[2], v[3]}, hi[4] = {v[4], v[5], v[6], v[7]};
    return make_uint2(codes(lo), codes(hi));
  }
};

}  // namespace beam
