// The step between two blocks of a layer stack, in one pass over the token:
// the norm after a block, its gate, the scaled fp32 residual stream and the
// norm before the next block,
//   y  = o / sqrt(mean(o^2) + eps) * w_post
//   r' = alpha r + beta sigmoid(gate) y
//   x  = r' / sqrt(mean(r'^2) + eps) * w_pre
// (SandwichNorm with a depth-scaled residual stream: "Reflection Beam",
// section "Hybrid Attention and Unusual Residuals"; pretraining paragraph of
// "Reflection AI Introduces Beam ...").  x leaves in bf16 or fp32, or as e4m3
// codes with a scale for each 128 columns (the recipe of beam_moe_quant_e4m3
// on the unrounded x) for a product that takes those.
//
// One workgroup holds one token's row in registers, so every input is read
// and every output written once: both directions are bound by those bytes.
// Sums of squares and dot products are binary32, reduced lane by lane, then
// wave by wave in a fixed order.
#include "common.h"
#include "internal.h"

namespace beam {
namespace {

constexpr int kMaxWaves = 16;

template <typename IO, int VEC>
__device__ __forceinline__ void load_vec(const IO* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    if constexpr (sizeof(IO) == 2) v[0] = bf16_bits_to_f32(*p);
    else v[0] = *p;
  } else if constexpr (sizeof(IO) == 2) {
    const u32x4 q = ld16(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(q[i] << 16);
      v[2 * i + 1] = __uint_as_float(q[i] & 0xFFFF0000u);
    }
  } else {
    const u32x4 a = ld16(p), b = ld16(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = __uint_as_float(a[i]);
      v[4 + i] = __uint_as_float(b[i]);
    }
  }
}

template <typename IO, int VEC>
__device__ __forceinline__ void store_vec(IO* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    if constexpr (sizeof(IO) == 2) *p = f32_to_bf16_bits(v[0]);
    else *p = v[0];
  } else if constexpr (sizeof(IO) == 2) {
    u32x4 q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i])) |
             (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i + 1])) << 16);
    st16(p, q);
  } else {
    st16(p, u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                  __float_as_uint(v[3])});
    st16(p + 4, u32x4{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                      __float_as_uint(v[7])});
  }
}

// Sums over the workgroup of N values a thread, the same bits in every
// thread; sh [N][kMaxWaves] must not be in use by an earlier sum that a wave
// may still be reading.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*sh)[kMaxWaves]) {
  const int wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
#pragma unroll
  for (int off = kWave / 2; off >= 1; off >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor(v[i], off);
  if (threadIdx.x % kWave == 0)
#pragma unroll
    for (int i = 0; i < N; ++i) sh[i][wave] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = 0.0f;
    for (int w = 0; w < waves; ++w) v[i] += sh[i][w];
  }
}

// sigmoid from t = e^-|g| with the hardware exponential and reciprocal (each
// within about 1 ulp of binary32, the exponent's rounding adding |g| 2^-24):
// far inside what the gate's own type resolves, and a third of the
// instructions of the exact forms.  d is its derivative.
__device__ __forceinline__ float sigmoid_fast(float g, float& d) {
  const float t = __expf(-fabsf(g));
  const float r = __builtin_amdgcn_rcpf(1.0f + t);
  d = t * r * r;
  return g >= 0.0f ? r : t * r;
}

template <typename IO, int VEC, int NC>
__global__ __launch_bounds__(1024) void norm_residual(NormArgs a) {
  __shared__ float sh[2][1][kMaxWaves];
  const int64_t t = blockIdx.x, base = t * a.H;
  const int H = a.H;
  const IO* o = a.o ? static_cast<const IO*>(a.o) + base : nullptr;
  const IO* gate = static_cast<const IO*>(a.gate);
  float r[NC][VEC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * VEC;
    if (c < H) load_vec<float, VEC>(a.residual + base + c, r[i]);
    else
#pragma unroll
      for (int j = 0; j < VEC; ++j) r[i][j] = 0.0f;
  }
  if (o) {
    float ov[NC][VEC], gv[NC][VEC];
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * VEC;
      if (c < H) {
        load_vec<IO, VEC>(o + c, ov[i]);
        if (a.gate_cols > 1) load_vec<IO, VEC>(gate + base + c, gv[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) ov[i][j] = 0.0f;
      }
    }
    float scale = a.beta, dummy;
    if (a.gate_cols == 1) {
      float g[1];
      load_vec<IO, 1>(gate + t, g);
      scale *= sigmoid_fast(g[0], dummy);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss[0] = __builtin_fmaf(ov[i][j], ov[i][j], ss[0]);
    block_sum<1>(ss, sh[0]);
    const float inv = 1.0f / sqrtf(ss[0] / static_cast<float>(H) + a.eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * VEC;
      if (c >= H) continue;
      float w[VEC];
      load_vec<float, VEC>(a.post + c, w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float y = ov[i][j] * inv * w[j];
        if (a.gate_cols > 1) y *= sigmoid_fast(gv[i][j], dummy);
        r[i][j] = __builtin_fmaf(a.alpha, r[i][j], scale * y);
      }
      store_vec<float, VEC>(a.residual_out + base + c, r[i]);
    }
  }
  if (!a.pre) return;
  float ss[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NC; ++i)
#pragma unroll
    for (int j = 0; j < VEC; ++j) ss[0] = __builtin_fmaf(r[i][j], r[i][j], ss[0]);
  block_sum<1>(ss, sh[1]);
  const float inv = 1.0f / sqrtf(ss[0] / static_cast<float>(H) + a.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * VEC;
    if (c >= H) continue;
    float w[VEC], x[VEC];
    load_vec<float, VEC>(a.pre + c, w);
#pragma unroll
    for (int j = 0; j < VEC; ++j) x[j] = r[i][j] * inv * w[j];
    if (a.x) store_vec<IO, VEC>(static_cast<IO*>(a.x) + base + c, x);
    if constexpr (VEC == 8) {
      if (a.xq) {
        // a block's 128 columns are 16 aligned lanes of one wave (H % 128 ==
        // 0 here, so all of them or none are inside the row)
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
        const float sc = e4m3_scale(m);
        const uint32_t lo = e4m3x4(x[0] / sc, x[1] / sc, x[2] / sc, x[3] / sc);
        const uint32_t hi = e4m3x4(x[4] / sc, x[5] / sc, x[6] / sc, x[7] / sc);
        *reinterpret_cast<uint2*>(a.xq + base + c) = make_uint2(lo, hi);
        if (c % 128 == 0) a.xs[(base + c) / 128] = sc;
      }
    }
  }
}

// Gradients.  With rhat = r' inv_r, ohat = o inv_o, g the gate's sigmoid,
//   dr'    = d_r' + inv_r (w_pre dx - rhat mean(w_pre dx rhat))
//   dr     = alpha dr'
//   dn     = beta g dr'          (gradient of y)
//   d_gate = beta dr' y g (1 - g)  (summed over the row for a token gate)
//   d_o    = inv_o (w_post dn - ohat mean(w_post dn ohat))
//   d_pre  = sum_t dx rhat,  d_post = sum_t dn ohat
// r' is the forward's output, so nothing else is kept from it.  A workgroup
// walks over tokens blockIdx.x, blockIdx.x + gridDim.x, ... and holds its
// share of the weights' gradients in registers; the shares of all
// workgroups go to the workspace and are added in a fixed order by
// norm_weight_grad (no atomics).
template <typename IO, int VEC, int NC>
__global__ __launch_bounds__(1024) void norm_residual_backward(NormGradArgs a) {
  __shared__ float sh[2][3][kMaxWaves], sh2[1][kMaxWaves];
  const int H = a.H;
  const float rh = 1.0f / static_cast<float>(H);
  float w_pre[NC][VEC], w_post[NC][VEC], g_pre[NC][VEC], g_post[NC][VEC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) w_pre[i][j] = w_post[i][j] = g_pre[i][j] = g_post[i][j] = 0.0f;
    if (c < H) {
      if (a.dx) load_vec<float, VEC>(a.pre + c, w_pre[i]);
      if (a.o) load_vec<float, VEC>(a.post + c, w_post[i]);
    }
  }
  int par = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
    const int64_t base = t * H;
    float r[NC][VEC], dx[NC][VEC], dr[NC][VEC], o[NC][VEC], gv[NC][VEC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) r[i][j] = dx[i][j] = dr[i][j] = o[i][j] = gv[i][j] = 0.0f;
      if (c < H) {
        if (a.dx) {
          load_vec<float, VEC>(a.r + base + c, r[i]);
          load_vec<IO, VEC>(static_cast<const IO*>(a.dx) + base + c, dx[i]);
        }
        if (a.d_res) load_vec<float, VEC>(a.d_res + base + c, dr[i]);
        if (a.o) load_vec<IO, VEC>(static_cast<const IO*>(a.o) + base + c, o[i]);
        if (a.gate_cols > 1)
          load_vec<IO, VEC>(static_cast<const IO*>(a.gate) + base + c, gv[i]);
      }
    }
    float tg = 1.0f, tdg = 0.0f;  // a token gate's sigmoid and derivative
    if (a.gate_cols == 1) {
      float g[1];
      load_vec<IO, 1>(static_cast<const IO*>(a.gate) + t, g);
      tg = sigmoid_fast(g[0], tdg);
    }
    float s[3] = {0.0f, 0.0f, 0.0f};  // sum r'^2, sum w_pre dx r', sum o^2
#pragma unroll
    for (int i = 0; i < NC; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        s[0] = __builtin_fmaf(r[i][j], r[i][j], s[0]);
        s[1] = __builtin_fmaf(w_pre[i][j] * dx[i][j], r[i][j], s[1]);
        s[2] = __builtin_fmaf(o[i][j], o[i][j], s[2]);
      }
    block_sum<3>(s, sh[par]);
    const float inv_r = 1.0f / sqrtf(s[0] * rh + a.eps);
    const float inv_o = 1.0f / sqrtf(s[2] * rh + a.eps);
    const float k_r = a.dx ? (s[1] * inv_r * rh) * inv_r * inv_r : 0.0f;
    float u[1] = {0.0f};  // sum w_post dn o (without a token gate's sigmoid)
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = (threadIdx.x + i * blockDim.x) * VEC;
      float out[VEC], dgate[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        g_pre[i][j] = __builtin_fmaf(dx[i][j], r[i][j] * inv_r, g_pre[i][j]);
        float d = dr[i][j] + inv_r * (w_pre[i][j] * dx[i][j]) - r[i][j] * k_r;
        out[j] = a.alpha * d;
        d *= a.beta;
        if (a.gate_cols > 1) {
          float dg;
          const float g = sigmoid_fast(gv[i][j], dg);
          dgate[j] = d * (o[i][j] * inv_o * w_post[i][j]) * dg;
          d *= g;
        }
        dr[i][j] = d;  // gradient of y but for a token gate's sigmoid
        u[0] = __builtin_fmaf(w_post[i][j] * d, o[i][j], u[0]);
      }
      if (c < H) {
        store_vec<float, VEC>(a.d_residual + base + c, out);
        if (a.gate_cols > 1) store_vec<IO, VEC>(static_cast<IO*>(a.d_gate) + base + c, dgate);
      }
    }
    if (a.o) {
      block_sum<1>(u, sh2);
      const float k_o = (u[0] * tg * inv_o * rh) * inv_o * inv_o;
      if (a.gate_cols == 1 && threadIdx.x == 0) {
        const float dg[1] = {u[0] * inv_o * tdg};
        store_vec<IO, 1>(static_cast<IO*>(a.d_gate) + t, dg);
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const int c = (threadIdx.x + i * blockDim.x) * VEC;
        float out[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          const float dn = tg * dr[i][j];
          g_post[i][j] = __builtin_fmaf(dn, o[i][j] * inv_o, g_post[i][j]);
          out[j] = inv_o * (w_post[i][j] * dn) - o[i][j] * k_o;
        }
        if (c < H) store_vec<IO, VEC>(static_cast<IO*>(a.d_o) + base + c, out);
      }
    }
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * H;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = (threadIdx.x + i * blockDim.x) * VEC;
    if (c >= H) continue;
    if (a.dx) store_vec<float, VEC>(part + c, g_pre[i]);
    if (a.o) store_vec<float, VEC>(part + H + c, g_post[i]);
  }
}

// d_w[c] = sum over the n workgroups' shares, 64 columns a workgroup: four
// waves each add every fourth share, then meet in LDS in wave order.
__global__ __launch_bounds__(256) void norm_weight_grad(const float* __restrict__ part, int n,
                                                        int H, float* __restrict__ d_pre,
                                                        float* __restrict__ d_post) {
  __shared__ float sh[4][kWave];
  float* out = blockIdx.y == 0 ? d_pre : d_post;
  if (!out) return;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int c = blockIdx.x * kWave + lane;
  float s = 0.0f;
  if (c < H)
    for (int i = wave; i < n; i += 4)
      s += part[(static_cast<int64_t>(i) * 2 + blockIdx.y) * H + c];
  sh[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < H) out[c] = ((sh[0][lane] + sh[1][lane]) + sh[2][lane]) + sh[3][lane];
}

// Threads of a row: rows of a multiple of 8 columns take 8 consecutive
// columns a thread (16-byte accesses; every such row starts 16-byte aligned),
// others single ones.
struct RowShape {
  int vec, nc, threads;
};
RowShape row_shape(int H) {
  RowShape s;
  s.vec = H % 8 == 0 ? 8 : 1;
  const int chunks = H / s.vec;
  s.nc = s.vec == 8 ? (chunks <= 1024 ? 1 : 2) : (chunks <= 4096 ? 4 : 16);
  s.threads = static_cast<int>(ceil_div(ceil_div(chunks, s.nc), kWave)) * kWave;
  return s;
}

}  // namespace

int norm_grad_groups(int64_t T) { return static_cast<int>(T < 512 ? T : 512); }

#define BEAM_NORM_SHAPES(RUN)                            \
  if (rs.vec == 8 && rs.nc == 1) RUN(8, 1);              \
  else if (rs.vec == 8) RUN(8, 2);                       \
  else if (rs.nc == 4) RUN(1, 4);                        \
  else RUN(1, 16)

hipError_t launch_norm_residual(const NormArgs& a, int64_t T, int32_t dtype, hipStream_t s) {
  const RowShape rs = row_shape(a.H);
  const dim3 grid(static_cast<unsigned>(T)), block(rs.threads);
#define BEAM_NORM(V, N)                                                                       \
  do {                                                                                        \
    if (dtype == BEAM_BF16)                                                                   \
      hipLaunchKernelGGL((norm_residual<uint16_t, V, N>), grid, block, 0, s, a);              \
    else                                                                                      \
      hipLaunchKernelGGL((norm_residual<float, V, N>), grid, block, 0, s, a);                 \
  } while (0)
  BEAM_NORM_SHAPES(BEAM_NORM);
#undef BEAM_NORM
  return hipGetLastError();
}

hipError_t launch_norm_residual_backward(const NormGradArgs& a, int32_t dtype, float* d_pre,
                                         float* d_post, hipStream_t s) {
  const RowShape rs = row_shape(a.H);
  const int n = norm_grad_groups(a.T);
  const dim3 grid(n), block(rs.threads);
  if (n > 0) {
#define BEAM_NORM(V, N)                                                                       \
  do {                                                                                        \
    if (dtype == BEAM_BF16)                                                                   \
      hipLaunchKernelGGL((norm_residual_backward<uint16_t, V, N>), grid, block, 0, s, a);     \
    else                                                                                      \
      hipLaunchKernelGGL((norm_residual_backward<float, V, N>), grid, block, 0, s, a);        \
  } while (0)
    BEAM_NORM_SHAPES(BEAM_NORM);
#undef BEAM_NORM
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (d_pre || d_post)
    hipLaunchKernelGGL(norm_weight_grad, dim3(static_cast<unsigned>(ceil_div(a.H, kWave)), 2),
                       dim3(256), 0, s, a.part, n, a.H, d_pre, d_post);
  return hipGetLastError();
}

}  // namespace beam
