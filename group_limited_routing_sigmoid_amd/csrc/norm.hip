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
#include <algorithm>
#include <type_traits>

#include "layer.h"

namespace beam {
namespace {

constexpr int kMaxWaves = 16;
constexpr int kVec = 8;  // columns of a thread's chunk

// Rows of a multiple of 8 columns start 16-byte aligned and end with a chunk
// (TAIL 0).  Others (TAIL 1) start anywhere, and their last chunk is the
// row's last 8 columns: it shares some with the chunk before, of which both
// threads write the same values and only the other one's count in sums.  The
// card reads and writes 16 bytes at any address that the type allows, so every
// row goes in whole chunks, but for rows of fewer than 8 columns (TAIL 2).
// (8,192 rows of 5,119, bf16, forward with a gate for each channel: 124 us, with
// gradients 276, against 115 and 258 for 5,120; value by value 296 and 1,489.)
struct Place {
  int slot, col;  // first column by the thread's number and of its chunk
  int skip;       // columns of the chunk that another thread's sums count
  bool live;
};
template <int TAIL>
__device__ __forceinline__ Place place(int i, int H) {
  Place p;
  p.slot = (threadIdx.x + i * blockDim.x) * kVec;
  p.col = TAIL ? min(p.slot, max(H - kVec, 0)) : p.slot;
  p.skip = TAIL ? p.slot - p.col : 0;
  p.live = p.slot < H;
  return p;
}

typedef u32x4 u32x4_2 __attribute__((aligned(2)));
typedef u32x4 u32x4_4 __attribute__((aligned(4)));
template <typename IO, int TAIL>
struct Chunk {
  static constexpr int kWords = kVec * static_cast<int>(sizeof(IO)) / 16;
  using Word = std::conditional_t<!TAIL, u32x4, std::conditional_t<sizeof(IO) == 2, u32x4_2, u32x4_4>>;
  u32x4 w[kWords];  // as they lie in memory (bf16 ones two to a register)
  // n: columns of the row; of fewer than 8 the others count as zeros.
  __device__ __forceinline__ void load(const IO* p, int n) {
    if (TAIL != 2) {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = *reinterpret_cast<const Word*>(p + i * (kVec / kWords));
    } else {
      zero();
#pragma unroll
      for (int j = 0; j < kVec - 1; ++j)
        if (j < n) {
          if constexpr (sizeof(IO) == 2) w[0][j / 2] |= static_cast<uint32_t>(p[j]) << (16 * (j % 2));
          else w[j / 4][j % 4] = __float_as_uint(p[j]);
        }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = u32x4{0, 0, 0, 0};
  }
  // Makes the compiler forget values it has unpacked (it would rather keep
  // them, in twice the registers, than unpack again).
  __device__ __forceinline__ void repack() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(IO) == 2) {
      const uint32_t v = w[0][j / 2];
      return __uint_as_float(j % 2 ? v & 0xFFFF0000u : v << 16);
    } else {
      return __uint_as_float(w[j / 4][j % 4]);
    }
  }
};

template <typename IO, int TAIL>
__device__ __forceinline__ void load_vec(const IO* p, int n, float (&v)[kVec]) {
  Chunk<IO, TAIL> c;
  c.load(p, n);
#pragma unroll
  for (int j = 0; j < kVec; ++j) v[j] = c.get(j);
}

template <typename IO, int TAIL>
__device__ __forceinline__ void store_vec(IO* p, int n, const float (&v)[kVec]) {
  Chunk<IO, TAIL> c;
  if constexpr (sizeof(IO) == 2) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c.w[0][i] = static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i])) |
                  (static_cast<uint32_t>(f32_to_bf16_bits(v[2 * i + 1])) << 16);
  } else {
#pragma unroll
    for (int j = 0; j < kVec; ++j) c.w[j / 4][j % 4] = __float_as_uint(v[j]);
  }
  if (TAIL != 2) {
#pragma unroll
    for (int i = 0; i < Chunk<IO, TAIL>::kWords; ++i)
      *reinterpret_cast<typename Chunk<IO, TAIL>::Word*>(p + i * (kVec / Chunk<IO, TAIL>::kWords)) = c.w[i];
  } else {
#pragma unroll
    for (int j = 0; j < kVec - 1; ++j)
      if (j < n) {
        if constexpr (sizeof(IO) == 2) p[j] = static_cast<uint16_t>(c.w[0][j / 2] >> (16 * (j % 2)));
        else p[j] = v[j];
      }
  }
}

template <typename IO>
__device__ __forceinline__ float load_one(const IO* p) {
  if constexpr (sizeof(IO) == 2) return bf16_bits_to_f32(*p);
  else return *p;
}
template <typename IO>
__device__ __forceinline__ void store_one(IO* p, float v) {
  if constexpr (sizeof(IO) == 2) *p = f32_to_bf16_bits(v);
  else *p = v;
}

// Adds another lane's value in one data-parallel move: CTRL swaps neighbours
// or pairs, mirrors half rows or rows of 16, or hands a row's last lane to
// the next rows (which then hold the sum so far; the last lane ends with all).
template <int CTRL>
__device__ __forceinline__ float dpp_add(float v) {
  return v + __uint_as_float(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
                 0, static_cast<int>(__float_as_uint(v)), CTRL, 0xF, 0xF, false)));
}

// Sums over the workgroup of N values a thread, the same bits in every
// thread; sh [N][kMaxWaves] must not be in use by an earlier sum that a wave
// may still be reading.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*sh)[kMaxWaves]) {
  const int wave = threadIdx.x / kWave, waves = blockDim.x / kWave;
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_add<0xB1>(v[i]);   // quad_perm(1, 0, 3, 2)
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_add<0x4E>(v[i]);   // quad_perm(2, 3, 0, 1)
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_add<0x141>(v[i]);  // row_half_mirror
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_add<0x140>(v[i]);  // row_mirror
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_add<0x142>(v[i]);  // row_bcast:15
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = dpp_add<0x143>(v[i]);  // row_bcast:31
  if (threadIdx.x % kWave == kWave - 1)
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

template <typename IO, int TAIL, int NC>
__global__ __launch_bounds__(1024) void norm_residual(NormArgs a) {
  __shared__ float sh[2][1][kMaxWaves];
  const int64_t t = blockIdx.x, base = t * a.H;
  const int H = a.H;
  const IO* o = a.o ? static_cast<const IO*>(a.o) + base : nullptr;
  const IO* gate = static_cast<const IO*>(a.gate);
  float r[NC][kVec];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const Place at = place<TAIL>(i, H);
    const int c = at.col;
    if (at.live) load_vec<float, TAIL>(a.residual + base + c, H, r[i]);
    else
#pragma unroll
      for (int j = 0; j < kVec; ++j) r[i][j] = 0.0f;
  }
  if (o) {
    float ov[NC][kVec], gv[NC][kVec];
    float ss[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const Place at = place<TAIL>(i, H);
      const int c = at.col;
      if (at.live) {
        load_vec<IO, TAIL>(o + c, H, ov[i]);
        if (a.gate_cols > 1) load_vec<IO, TAIL>(gate + base + c, H, gv[i]);
      } else {
#pragma unroll
        for (int j = 0; j < kVec; ++j) ov[i][j] = 0.0f;
      }
    }
    float scale = a.beta, dummy;
    if (a.gate_cols == 1) {
      scale *= sigmoid_fast(load_one(gate + t), dummy);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int skip = place<TAIL>(i, H).skip;
#pragma unroll
      for (int j = 0; j < kVec; ++j)
        if (j >= skip) ss[0] = __builtin_fmaf(ov[i][j], ov[i][j], ss[0]);
    }
    if (TAIL) {
      // residual_out may be the residual: this thread has its columns before
      // another one, past the sum's barrier, writes those that they share
#pragma unroll
      for (int i = 0; i < NC; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) asm volatile("" : "+v"(r[i][j]));
    }
    block_sum<1>(ss, sh[0]);
    const float inv = 1.0f / sqrtf(ss[0] / static_cast<float>(H) + a.eps);
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const Place at = place<TAIL>(i, H);
      const int c = at.col;
      if (!at.live) continue;
      float w[kVec];
      load_vec<float, TAIL>(a.post + c, H, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        float y = ov[i][j] * inv * w[j];
        if (a.gate_cols > 1) y *= sigmoid_fast(gv[i][j], dummy);
        r[i][j] = __builtin_fmaf(a.alpha, r[i][j], scale * y);
      }
      store_vec<float, TAIL>(a.residual_out + base + c, H, r[i]);
    }
  }
  if (!a.pre) return;
  float ss[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int skip = place<TAIL>(i, H).skip;
#pragma unroll
    for (int j = 0; j < kVec; ++j)
      if (j >= skip) ss[0] = __builtin_fmaf(r[i][j], r[i][j], ss[0]);
  }
  block_sum<1>(ss, sh[1]);
  const float inv = 1.0f / sqrtf(ss[0] / static_cast<float>(H) + a.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const Place at = place<TAIL>(i, H);
    const int c = at.col;
    if (!at.live) continue;
    float w[kVec], x[kVec];
    load_vec<float, TAIL>(a.pre + c, H, w);
#pragma unroll
    for (int j = 0; j < kVec; ++j) x[j] = r[i][j] * inv * w[j];
    if (a.x) store_vec<IO, TAIL>(static_cast<IO*>(a.x) + base + c, H, x);
    if constexpr (!TAIL) {
      if (a.xq) {
        // a block's 128 columns are 16 aligned lanes of one wave (H % 128 ==
        // 0 here, so all of them or none are inside the row)
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[j]));
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
        const BlockDivisor d(m);
        *reinterpret_cast<uint2*>(a.xq + base + c) = d.codes(x);
        if (c % 128 == 0) a.xs[(base + c) / 128] = d.s;
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
// norm_weight_grad (no atomics).  The weights lie in LDS and the inputs stay
// packed as they lie in memory, so that two workgroups of a 5,120-column row
// share a compute unit and one's loads run beside the other's sums: 8,191
// tokens, bf16, one gate a token, 160 us, 4.7 TB/s (everything unpacked in
// registers, one workgroup a unit: 181 us; the next token's loads issued
// ahead instead: 165 us; half the threads with twice the columns: 186 us).
// With a gate for each channel 197 us, the same 4.7 TB/s.  Rows of more than
// 8,192 columns take two chunks a thread, whose sums, weights' shares and packed
// inputs exceed the 128 registers that 1,024 threads leave: up to 35 of them
// spill without a gate a channel (8,192 x 16,384, one gate a token: 507 us, 4.8
// TB/s all the same), 64 to 99 with one (1,114 us, 2.7 TB/s).
// O: there is a block output; DX: there is a gradient of x; CG: a gate for
// each channel (or none, or one a token, in the other form).
template <typename IO, int TAIL, int NC, bool O, bool DX, bool CG>
__global__ __launch_bounds__(1024, NC == 1 && !CG ? 5 : 4) void norm_residual_backward(NormGradArgs a) {
  __shared__ float sh[2][3][kMaxWaves], sh2[1][kMaxWaves];
  extern __shared__ __attribute__((aligned(16))) float wts[];  // w_pre, then w_post
  const int H = a.H, post = blockDim.x * NC * kVec;
  const float rh = 1.0f / static_cast<float>(H);
  float g_pre[NC][kVec], g_post[NC][kVec];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    // a thread reads only what it wrote
    const Place pl = place<TAIL>(i, H);
    const int c = pl.col;
    float w[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) g_pre[i][j] = g_post[i][j] = w[j] = 0.0f;
    if (DX) {
      if (pl.live) load_vec<float, TAIL>(a.pre + c, H, w);
      store_vec<float, 0>(wts + pl.slot, kVec, w);
    }
    if (O) {
      if (pl.live) load_vec<float, TAIL>(a.post + c, H, w);
      store_vec<float, 0>(wts + post + pl.slot, kVec, w);
    }
  }
  struct Row {
    Chunk<float, TAIL> r[NC], dr[NC];
    Chunk<IO, TAIL> dx[NC], o[NC], gv[NC];
  };
  auto load = [&](Row& x, int64_t t) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const Place pl = place<TAIL>(i, H);
      const int c = pl.col;
      const int64_t at = t * H + c;
      if (pl.live) {
        if (DX) x.r[i].load(a.r + at, H), x.dx[i].load(static_cast<const IO*>(a.dx) + at, H);
        if (O) x.o[i].load(static_cast<const IO*>(a.o) + at, H);
        if (a.d_res) x.dr[i].load(a.d_res + at, H);
        if (CG) x.gv[i].load(static_cast<const IO*>(a.gate) + at, H);
      }
    }
  };
  Row x;
#pragma unroll
  for (int i = 0; i < NC; ++i) x.r[i].zero(), x.dr[i].zero(), x.dx[i].zero(), x.o[i].zero(), x.gv[i].zero();
  int par = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, par ^= 1) {
    const int64_t base = t * H;
    load(x, t);
    float tg = 1.0f, tdg = 0.0f;  // a token gate's sigmoid and derivative
    if (O && !CG && a.gate_cols == 1)
      tg = sigmoid_fast(load_one(static_cast<const IO*>(a.gate) + t), tdg);
    float s[3] = {0.0f, 0.0f, 0.0f};  // sum r'^2, sum w_pre dx r', sum o^2
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const Place pl = place<TAIL>(i, H);
      const int c = pl.col;
      float w[kVec];
      if (DX) load_vec<float, 0>(wts + pl.slot, kVec, w);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if (j < pl.skip) continue;
        const float rv = x.r[i].get(j), ov = x.o[i].get(j);
        if (DX) {
          s[0] = __builtin_fmaf(rv, rv, s[0]);
          s[1] = __builtin_fmaf(w[j] * x.dx[i].get(j), rv, s[1]);
        }
        if (O) s[2] = __builtin_fmaf(ov, ov, s[2]);
      }
    }
    if (TAIL)  // as in the forward: d_residual may be d_residual_out
#pragma unroll
      for (int i = 0; i < NC; ++i) x.dr[i].repack();
    block_sum<3>(s, sh[par]);
#pragma unroll
    for (int i = 0; i < NC; ++i) x.r[i].repack(), x.dx[i].repack(), x.o[i].repack();
    const float inv_r = 1.0f / sqrtf(s[0] * rh + a.eps);
    const float inv_o = 1.0f / sqrtf(s[2] * rh + a.eps);
    const float k_r = (s[1] * inv_r * rh) * inv_r * inv_r;
    float u[1] = {0.0f};  // sum w_post dn o (without a token gate's sigmoid)
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const Place pl = place<TAIL>(i, H);
      const int c = pl.col;
      float out[kVec], dgate[kVec], wp[kVec], wq[kVec];
      if (DX) load_vec<float, 0>(wts + pl.slot, kVec, wp);
      if (O) load_vec<float, 0>(wts + post + pl.slot, kVec, wq);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        float d = x.dr[i].get(j);
        if (DX) {
          const float rv = x.r[i].get(j), xv = x.dx[i].get(j);
          g_pre[i][j] = __builtin_fmaf(xv, rv * inv_r, g_pre[i][j]);
          d = d + inv_r * (wp[j] * xv) - rv * k_r;
        }
        out[j] = a.alpha * d;
        if (O) {
          const float ov = x.o[i].get(j);
          d *= a.beta;
          if (CG) {
            float dg;
            const float g = sigmoid_fast(x.gv[i].get(j), dg);
            dgate[j] = d * (ov * inv_o * wq[j]) * dg;
            d *= g;
          }
          // gradient of y but for a token gate's sigmoid, in dr's place
          x.dr[i].w[j / 4][j % 4] = __float_as_uint(d);
          if (j >= pl.skip) u[0] = __builtin_fmaf(wq[j] * d, ov, u[0]);
        }
      }
      if (pl.live) {
        store_vec<float, TAIL>(a.d_residual + base + c, H, out);
        if (CG) store_vec<IO, TAIL>(static_cast<IO*>(a.d_gate) + base + c, H, dgate);
      }
    }
    if (O) {
      block_sum<1>(u, sh2);
#pragma unroll
      for (int i = 0; i < NC; ++i) x.o[i].repack();
      const float k_o = (u[0] * tg * inv_o * rh) * inv_o * inv_o;
      if (!CG && a.gate_cols == 1 && threadIdx.x == 0)
        store_one(static_cast<IO*>(a.d_gate) + t, u[0] * inv_o * tdg);
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const Place pl = place<TAIL>(i, H);
        const int c = pl.col;
        float out[kVec], wq[kVec];
        load_vec<float, 0>(wts + post + pl.slot, kVec, wq);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float dn = tg * x.dr[i].get(j), ov = x.o[i].get(j);
          g_post[i][j] = __builtin_fmaf(dn, ov * inv_o, g_post[i][j]);
          out[j] = inv_o * (wq[j] * dn) - ov * k_o;
        }
        if (pl.live) store_vec<IO, TAIL>(static_cast<IO*>(a.d_o) + base + c, H, out);
      }
    }
    // Chunks that the next token's loads do not replace: without d_res, and
    // those past the row's end, where a token whose sums are not finite leaves
    // NaN that would reach the next ones' sums.
#pragma unroll
    for (int i = 0; i < NC; ++i)
      if (!a.d_res || !place<TAIL>(i, H).live) x.dr[i].zero();
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * 2 * H;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const Place pl = place<TAIL>(i, H);
    const int c = pl.col;
    if (!pl.live) continue;
    if (DX) store_vec<float, TAIL>(part + c, H, g_pre[i]);
    if (O) store_vec<float, TAIL>(part + H + c, H, g_post[i]);
  }
}

// d_w[c] = sum over the n workgroups' shares, 64 columns a workgroup: sixteen
// waves each add every sixteenth share, then meet in LDS in wave order.
__global__ __launch_bounds__(1024) void norm_weight_grad(const float* __restrict__ part, int n,
                                                         int H, float* __restrict__ d_pre,
                                                         float* __restrict__ d_post) {
  __shared__ float sh[16][kWave];
  float* out = blockIdx.y == 0 ? d_pre : d_post;
  if (!out) return;
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int c = blockIdx.x * kWave + lane;
  float s = 0.0f;
  if (c < H)
#pragma unroll 8
    for (int i = wave; i < n; i += 16)
      s += part[(static_cast<int64_t>(i) * 2 + blockIdx.y) * H + c];
  sh[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < H) {
#pragma unroll
    for (int w = 1; w < 16; ++w) s += sh[w][lane];
    out[c] = s;
  }
}

// Threads of a row: one chunk of 8 columns each or two.  `pairs`: two also
// where one would do (rows of more than 2,048 columns; the forward of many
// tokens: 16,384 gated tokens of 5,120 211 against 215 us, while one token is
// faster spread over more threads).
struct RowShape {
  int nc, threads;
};
RowShape row_shape(int H, bool pairs) {
  RowShape s;
  const int chunks = static_cast<int>(ceil_div(H, kVec));
  s.nc = chunks <= (pairs ? 256 : 1024) ? 1 : 2;
  s.threads = static_cast<int>(ceil_div(ceil_div(chunks, s.nc), kWave)) * kWave;
  return s;
}

}  // namespace

int64_t norm_max_tokens(int H) { return 0xFFFFFFFF / row_shape(H, false).threads; }

// Workgroups of the gradients: two a compute unit of rows of four waves and
// more, up to six of narrower ones, whose tokens would otherwise queue for a
// few waves (16,384 tokens of 70, 300 and 1,000 with gradients: 46, 50 and 99
// us; with two 78, 80 and 125; 2,000 columns: 190 us with two, 207 with five).
int norm_grad_groups(int64_t T, int H) {
  const int waves = row_shape(H, false).threads / kWave;
  const int64_t n = 256 * std::clamp(8 / waves, 2, 6);
  return static_cast<int>(T < n ? T : n);
}

#define BEAM_NORM_SHAPES(RUN, H)                                          \
  if ((H) % kVec == 0 && rs.nc == 1) RUN(0, 1);                           \
  else if ((H) % kVec == 0) RUN(0, 2);                                    \
  else if ((H) < kVec) RUN(2, 1);                                         \
  else if (rs.nc == 1) RUN(1, 1);                                         \
  else RUN(1, 2)

hipError_t launch_norm_residual(const NormArgs& a, int64_t T, int32_t dtype, hipStream_t s) {
  const RowShape rs = row_shape(a.H, T >= 1024);
  const dim3 grid(static_cast<unsigned>(T)), block(rs.threads);
#define BEAM_NORM(V, N)                                                                       \
  do {                                                                                        \
    if (dtype == BEAM_BF16)                                                                   \
      hipLaunchKernelGGL((norm_residual<uint16_t, V, N>), grid, block, 0, s, a);              \
    else                                                                                      \
      hipLaunchKernelGGL((norm_residual<float, V, N>), grid, block, 0, s, a);                 \
  } while (0)
  BEAM_NORM_SHAPES(BEAM_NORM, a.H);
#undef BEAM_NORM
  return hipGetLastError();
}

hipError_t launch_norm_residual_backward(const NormGradArgs& a, int32_t dtype, float* d_pre,
                                         float* d_post, hipStream_t s) {
  const RowShape rs = row_shape(a.H, false);
  const int n = norm_grad_groups(a.T, a.H);
  const dim3 grid(n), block(rs.threads);
  const size_t lds = 2 * static_cast<size_t>(rs.threads) * rs.nc * kVec * sizeof(float);
  if (n > 0) {
#define BEAM_NORM(V, N)                                                                       \
  do {                                                                                        \
    if (dtype == BEAM_BF16) BEAM_NORM2(uint16_t, V, N);                                       \
    else BEAM_NORM2(float, V, N);                                                             \
  } while (0)
#define BEAM_NORM2(IO, V, N)                                                                  \
  do {                                                                                        \
    if (!a.o) BEAM_NORM3(IO, V, N, false, true, false);                                       \
    else if (a.gate_cols > 1 && a.dx) BEAM_NORM3(IO, V, N, true, true, true);                 \
    else if (a.gate_cols > 1) BEAM_NORM3(IO, V, N, true, false, true);                        \
    else if (a.dx) BEAM_NORM3(IO, V, N, true, true, false);                                   \
    else BEAM_NORM3(IO, V, N, true, false, false);                                            \
  } while (0)
#define BEAM_NORM3(IO, V, N, O, DX, CG)                                                       \
  hipLaunchKernelGGL((norm_residual_backward<IO, V, N, O, DX, CG>), grid, block, lds, s, a)
    BEAM_NORM_SHAPES(BEAM_NORM, a.H);
#undef BEAM_NORM3
#undef BEAM_NORM2
#undef BEAM_NORM
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (d_pre || d_post)
    hipLaunchKernelGGL(norm_weight_grad, dim3(static_cast<unsigned>(ceil_div(a.H, kWave)), 2),
                       dim3(1024), 0, s, a.part, n, a.H, d_pre, d_post);
  return hipGetLastError();
}

}  // namespace beam
