// Router of the Beam MoE block on gfx950.
//
// The router computes sigmoid scores over the experts, adds a per-expert bias
// used only to choose experts, keeps the best groups, picks the top-K experts
// inside them and normalises their unbiased scores to sum to the routed scale
// ("Reflection Releases Beam: An Open 501B-Parameter MoE Model Under Apache
// 2.0", section "Where Beam Saves and Where the Memory Bill Comes In";
// "Hugging Face releases Beam ..." MoE paragraph; bias from the
// load-balancing paragraph of "Reflection AI Introduces Beam ...").  The
// group score is the sum of a group's best two biased scores, DeepSeek-V3's
// rule (arXiv 2412.19437, section 2.1.2), which the pages invoke.
//
// Kernels:
//   router_logits_*  logits = x W_r^T in fp32 (for many tokens the same
//                    three-term split feeds the dense tile GEMM of the
//                    grouped expert path, split over H).  With bf16 activations the
//                    fp32 router weights are split exactly into three bf16
//                    terms (hi + mid + lo), so every product is exact and the
//                    matrix cores accumulate in fp32.  The reduction over H
//                    may be split into `ks` partial sums for parallelism.
//   router_select    one wavefront per token: sums the partials in a fixed
//                    order, then routes in binary32 exactly as specified
//                    (sigmoid from a fixed binary64 evaluation, ties to the
//                    lower index), so indices and weights are bitwise
//                    reproducible from the fp32 logits.  Scores may instead be
//                    the softmax over all experts, the weights unnormalised.
//   route_backward   one wavefront per token: the gradient of the weights in
//                    the logits, scores recomputed in binary32.
//
// This translation unit is compiled with -ffp-contract=off.
#include <type_traits>

#include "common.h"
#include "internal.h"

namespace beam {
namespace {

// ---- logits: bf16 activations, bf16x3 split of fp32 weights, MFMA -------

__device__ __forceinline__ void split3(const float* w, bf16x8& hi, bf16x8& mid,
                                       bf16x8& lo) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float v = w[j];
    const bf16 h = static_cast<bf16>(v);
    const float r1 = v - static_cast<float>(h);
    const bf16 m = static_cast<bf16>(r1);
    const float r2 = r1 - static_cast<float>(m);
    hi[j] = h;
    mid[j] = m;
    lo[j] = static_cast<bf16>(r2);
  }
}

// grid (ceil(T/32), ceil(E/64), ks), four waves: 32 tokens x 64 experts (32
// in the last block when E % 64 == 32) over columns [z*kchunk, (z+1)*kchunk)
// of H.  Wave w takes the w-th quarter of those columns; the four partial
// tiles meet in LDS and are added in wave order.  With few tokens the
// kernel is bound by how much of W_r is in flight, so each wave issues the
// loads of four 16-column steps before their products.
constexpr int kLgWaves = 4;

__global__ __launch_bounds__(kLgWaves * kWave) void router_logits_mfma(
    const uint16_t* __restrict__ x, const float* __restrict__ wr,
    float* __restrict__ part, int64_t T, int H, int E, int kchunk) {
  __shared__ float red[kLgWaves - 1][2][16][kWave];
  const int wave = threadIdx.x / kWave, lane = threadIdx.x % kWave;
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 32;
  const int e0 = blockIdx.y * 64;
  const int z = blockIdx.z;
  const int kq = kchunk / kLgWaves;
  const int kb = z * kchunk + wave * kq + 8 * (lane / 32);
  int64_t tr = t0 + (lane % 32);
  if (tr > T - 1) tr = T - 1;
  const uint16_t* xp = x + tr * H + kb;
  // without a second 32-expert half the wave reads the first half twice and
  // stores one (keeps the loop free of branches)
  const bool has1 = e0 + 32 < E;  // wave-uniform
  const float* wp0 = wr + static_cast<int64_t>(e0 + lane % 32) * H + kb;
  const float* wp1 = wr + static_cast<int64_t>(has1 ? e0 + 32 + lane % 32 : e0 + lane % 32) * H + kb;
  f32x16 acc0 = {}, acc1 = {};
#pragma unroll 4
  for (int k = 0; k < kq; k += 16) {
    const bf16x8 a = as_bf16x8(ld16(xp + k));
    float w0[8], w1[8];
    *reinterpret_cast<u32x4*>(w0) = ld16(wp0 + k);
    *reinterpret_cast<u32x4*>(w0 + 4) = ld16(wp0 + k + 4);
    *reinterpret_cast<u32x4*>(w1) = ld16(wp1 + k);
    *reinterpret_cast<u32x4*>(w1 + 4) = ld16(wp1 + k + 4);
    bf16x8 h0, m0, l0, h1, m1, l1;
    split3(w0, h0, m0, l0);
    split3(w1, h1, m1, l1);
    acc0 = mfma32x32x16(a, l0, acc0);
    acc1 = mfma32x32x16(a, l1, acc1);
    acc0 = mfma32x32x16(a, m0, acc0);
    acc1 = mfma32x32x16(a, m1, acc1);
    acc0 = mfma32x32x16(a, h0, acc0);
    acc1 = mfma32x32x16(a, h1, acc1);
  }
  if (wave > 0) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      red[wave - 1][0][r][lane] = acc0[r];
      red[wave - 1][1][r][lane] = acc1[r];
    }
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int w = 0; w < kLgWaves - 1; ++w) {
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      acc0[r] = acc0[r] + red[w][0][r][lane];
      acc1[r] = acc1[r] + red[w][1][r][lane];
    }
  }
  float* out = part + static_cast<int64_t>(z) * T * E;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int64_t t = t0 + 8 * (r / 4) + 4 * (lane / 32) + (r % 4);
    if (t < T) {
      out[t * E + e0 + lane % 32] = acc0[r];
      if (has1) out[t * E + e0 + 32 + lane % 32] = acc1[r];
    }
  }
}

// ---- exact three-term bf16 split of the fp32 router matrix ---------------
// w3 [E, 3H]: row e = [smallest term | middle term | bf16 rounding of W_r[e]];
// the three add up to W_r[e] exactly.
__global__ __launch_bounds__(256) void router_split(const float* __restrict__ wr,
                                                    uint16_t* __restrict__ w3, int E, int H) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= static_cast<int64_t>(E) * H) return;
  const int64_t e = i / H, k = i % H;
  const float v = wr[i];
  const bf16 h = static_cast<bf16>(v);
  const float r1 = v - static_cast<float>(h);
  const bf16 m = static_cast<bf16>(r1);
  const float r2 = r1 - static_cast<float>(m);
  uint16_t* row = w3 + e * 3 * H;
  row[k] = __builtin_bit_cast(uint16_t, static_cast<bf16>(r2));
  row[H + k] = __builtin_bit_cast(uint16_t, m);
  row[2 * H + k] = __builtin_bit_cast(uint16_t, h);
}

// ---- logits: generic fp32 dot products (fp32 activations, small layers) --

__global__ __launch_bounds__(256) void router_logits_valu(
    const void* __restrict__ x, int x_bf16, const float* __restrict__ wr,
    float* __restrict__ part, int64_t T, int H, int E, int kchunk) {
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  const int z = blockIdx.y;
  if (i >= T * E) return;
  const int64_t t = i / E;
  const int e = static_cast<int>(i % E);
  const int k0 = z * kchunk;
  float acc = 0.0f;
  for (int k = k0; k < k0 + kchunk; ++k) {
    const float xv = x_bf16
        ? bf16_bits_to_f32(static_cast<const uint16_t*>(x)[t * H + k])
        : static_cast<const float*>(x)[t * H + k];
    acc = __builtin_fmaf(xv, wr[static_cast<int64_t>(e) * H + k], acc);
  }
  part[static_cast<int64_t>(z) * T * E + i] = acc;
}

// ---- routing --------------------------------------------------------------

// sigmoid32(l) = 1/(1+e^-l) evaluated in binary64 and rounded once to
// binary32.  e^z: Cody & Waite reduction z = n ln2 + r (ln2 as a 32-bit head
// plus a tail), then the degree-13 Taylor polynomial of e^r in Horner form
// with fused multiply-adds; coefficients are the binary64 roundings of 1/j!.
// Every step is an IEEE-exact binary64 operation, so any conforming
// evaluation of this sequence returns the same bits.
__device__ __forceinline__ double exp64(double z) {
  const double n = __builtin_rint(z * 0x1.71547652b82fep+0);
  double r = __builtin_fma(-n, 0x1.62e42feep-1, z);
  r = __builtin_fma(-n, 0x1.a39ef35793c76p-33, r);
  double p = 0x1.6124613a86d09p-33;          // 1/13!
  p = __builtin_fma(p, r, 0x1.1eed8eff8d898p-29);  // 1/12!
  p = __builtin_fma(p, r, 0x1.ae64567f544e4p-26);  // 1/11!
  p = __builtin_fma(p, r, 0x1.27e4fb7789f5cp-22);  // 1/10!
  p = __builtin_fma(p, r, 0x1.71de3a556c734p-19);  // 1/9!
  p = __builtin_fma(p, r, 0x1.a01a01a01a01ap-16);  // 1/8!
  p = __builtin_fma(p, r, 0x1.a01a01a01a01ap-13);  // 1/7!
  p = __builtin_fma(p, r, 0x1.6c16c16c16c17p-10);  // 1/6!
  p = __builtin_fma(p, r, 0x1.1111111111111p-7);   // 1/5!
  p = __builtin_fma(p, r, 0x1.5555555555555p-5);   // 1/4!
  p = __builtin_fma(p, r, 0x1.5555555555555p-3);   // 1/3!
  p = __builtin_fma(p, r, 0x1.0p-1);               // 1/2!
  p = __builtin_fma(p, r, 1.0);                    // 1/1!
  p = __builtin_fma(p, r, 1.0);                    // 1/0!
  return __builtin_ldexp(p, static_cast<int>(n));
}

__device__ __forceinline__ float sigmoid32(float l) {
  if (l <= -104.0f) return 0.0f;
  if (l >= 40.0f) return 1.0f;
  const double q = 1.0 / (1.0 + exp64(-static_cast<double>(l)));
  return static_cast<float>(q);
}

// Order-preserving map of a finite binary32 to uint32 (larger float, larger
// key); +0 and -0 map to the same key after canonicalisation.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}

constexpr int kSelWaves = 4;
constexpr int kMaxE = 1024;
constexpr int kMaxKs = 16;   // the plan splits the router's reduction at most 16 ways
constexpr int kMaxK = 16;

// ---- wave-wide helpers --------------------------------------------------
// Reductions over the wave in data-parallel moves: swap neighbours, swap
// pairs (quad permutations), mirror the half rows, mirror the row; every lane
// then holds its row of 16's result, and the rows meet in the last lane.  All
// need every lane active.

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return static_cast<uint32_t>(
      __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, 0xF, 0xF, true));
}

// Maximum over the wave, returned uniform.
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, dpp<0xB1>(v));   // quad_perm(1, 0, 3, 2)
  v = max(v, dpp<0x4E>(v));   // quad_perm(2, 3, 0, 1)
  v = max(v, dpp<0x141>(v));  // row_half_mirror
  v = max(v, dpp<0x140>(v));  // row_mirror
  v = max(v, dpp<0x142>(v));  // row_bcast:15, the row before's
  v = max(v, dpp<0x143>(v));  // row_bcast:31, the first two rows'
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

__device__ __forceinline__ float readlane_f(float v, int l) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), l));
}

__device__ __forceinline__ float wave_max_f32(float v) {
  auto step = [&](uint32_t o) { v = fmaxf(v, __uint_as_float(o)); };
  step(dpp<0xB1>(__float_as_uint(v)));
  step(dpp<0x4E>(__float_as_uint(v)));
  step(dpp<0x141>(__float_as_uint(v)));
  step(dpp<0x140>(__float_as_uint(v)));
  step(dpp<0x142>(__float_as_uint(v)));
  step(dpp<0x143>(__float_as_uint(v)));
  return readlane_f(v, 63);
}

__device__ __forceinline__ double wave_sum_f64(double v) {
  auto move = [&](auto ctrl) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = dpp<decltype(ctrl)::value>(static_cast<uint32_t>(b));
    const uint64_t hi = dpp<decltype(ctrl)::value>(static_cast<uint32_t>(b >> 32));
    v += __builtin_bit_cast(double, lo | (hi << 32));
  };
  move(std::integral_constant<int, 0xB1>{});
  move(std::integral_constant<int, 0x4E>{});
  move(std::integral_constant<int, 0x141>{});
  move(std::integral_constant<int, 0x140>{});
  move(std::integral_constant<int, 0x142>{});
  move(std::integral_constant<int, 0x143>{});
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), 63);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), 63);
  return __builtin_bit_cast(double, static_cast<uint64_t>(lo) | (static_cast<uint64_t>(hi) << 32));
}

// Softmax scores of a token, one wave: s_e = e^(l_e - m) / sum_j e^(l_j - m)
// with m the largest logit, the exponentials, their sum and its reciprocal
// (one a token) in binary64, rounded once to binary32 (the selection compares
// these values, so they are held to the rounding of the exact softmax, as the
// sigmoids are).  Exponents below -105 give 0: such a score is below half the
// smallest binary32 value, and 1024 of them are below the sum's last bit.  A
// row whose logits are all -infinity has m = -infinity, every comparison false
// and the scores 0; a NaN or +infinity makes every score of its row NaN.
// Needs every lane active; l of places past the last expert is -infinity.
template <int EPL>
__device__ __forceinline__ void softmax32(const float (&l)[EPL], float (&s)[EPL]) {
  float m = l[0];
#pragma unroll
  for (int j = 1; j < EPL; ++j) m = fmaxf(m, l[j]);
  m = wave_max_f32(m);
  bool bad = false;
#pragma unroll
  for (int j = 0; j < EPL; ++j) bad |= !(l[j] <= 3.402823466e38f);
  double ez[EPL], sum = 0.0;
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    // no branch, so that the exponentials of a lane overlap
    const double z = static_cast<double>(l[j]) - static_cast<double>(m);
    const double v = exp64(__builtin_fmax(z, -105.0));
    ez[j] = z > -105.0 ? v : 0.0;
    sum += ez[j];
  }
  sum = wave_sum_f64(sum);
  // 1 / sum within 2^-52 by two steps from the hardware's approximation (sum
  // lies between 1 and 1024)
  double inv = __builtin_amdgcn_rcp(sum);
  inv = __builtin_fma(__builtin_fma(-sum, inv, 1.0), inv, inv);
  inv = __builtin_fma(__builtin_fma(-sum, inv, 1.0), inv, inv);
  if (sum == 0.0) inv = 0.0;
  if (__ballot(bad)) inv = __builtin_nan("");
#pragma unroll
  for (int j = 0; j < EPL; ++j) s[j] = static_cast<float>(ez[j] * inv);
}

// grid ceil(T/4), block 256: wave w routes token 4*blockIdx.x + w, holding
// EPL experts per lane in registers (lane l: experts l*EPL .. l*EPL+EPL-1).
// KS is 1 (one partial per logit) or kMaxKs (ks <= kMaxKs partials).  SEG:
// a group's experts are the 2^lg = gs/EPL lanes of one aligned segment, so
// group maxima are butterflies within the segment; otherwise
// lane g scans group g's biased scores from LDS (one pad word per 32 keeps
// the scan's lanes on distinct banks).  SM: softmax scores.
__device__ __forceinline__ int upad(int e) { return e + (e >> 5); }

template <int EPL, int KS, bool SEG, bool SM>
__global__ __launch_bounds__(256) void router_select(
    const float* __restrict__ part, int ks, int vec4, int64_t T, int E, int G,
    int TG, int K, int topn, int lg, int normed, float scale, const float* __restrict__ bias,
    float* __restrict__ logits_out, int32_t* __restrict__ idx_out,
    float* __restrict__ w_out) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kSelWaves + wave;
  const bool valid = t < T;   // wave-uniform
  const int64_t tc = valid ? t : T - 1;
  const int gs = E / G;
  const float ninf = -__builtin_huge_valf();

  // 1. logits (fixed-order sum of the partials), scores, biased scores.
  // Every load is issued before the first add: indices are clamped into
  // range instead of branched on, and the clamped values are not used.
  // With vec4 (E % 4 == 0: 16-byte aligned rows) a lane's experts come four
  // to a 16-byte load.
  float pz[EPL][KS], bz[EPL], lv[EPL], sv[EPL], u[EPL];
  if (EPL % 4 == 0 && vec4) {
#pragma unroll
    for (int j = 0; j < EPL; j += 4) {
      const int e = min(lane * EPL + j, E - 4);
#pragma unroll
      for (int z = 0; z < KS; ++z) {
        const u32x4 v = ld16(part + (static_cast<int64_t>(min(z, ks - 1)) * T + tc) * E + e);
#pragma unroll
        for (int q = 0; q < 4 && j + q < EPL; ++q) pz[j + q][z] = __uint_as_float(v[q]);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = min(lane * EPL + j, E - 1);
#pragma unroll
      for (int z = 0; z < KS; ++z)
        pz[j][z] = part[(static_cast<int64_t>(min(z, ks - 1)) * T + tc) * E + e];
    }
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) bz[j] = 0.0f;
  if (bias) {
    if (EPL % 4 == 0 && vec4) {
#pragma unroll
      for (int j = 0; j < EPL; j += 4) {
        const u32x4 v = ld16(bias + min(lane * EPL + j, E - 4));
#pragma unroll
        for (int q = 0; q < 4 && j + q < EPL; ++q) bz[j + q] = __uint_as_float(v[q]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) bz[j] = bias[min(lane * EPL + j, E - 1)];
    }
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane * EPL + j;
    float l = pz[j][0];
#pragma unroll
    for (int z = 1; z < KS; ++z)
      if (z < ks) l = l + pz[j][z];
    if (SM) lv[j] = l;
    else sv[j] = sigmoid32(l);
    if (valid && e < E && logits_out) logits_out[t * E + e] = l;
  }
  if constexpr (SM) {
    if (E < kWave * EPL)
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (lane * EPL + j >= E) lv[j] = ninf;
    softmax32<EPL>(lv, sv);
  }
#pragma unroll
  for (int j = 0; j < EPL; ++j) u[j] = sv[j] + bz[j];  // past E: no group, no key

  // 2. group scores: sum of the topn (1 or 2) largest biased scores (a
  // repeated value counts twice).  gsc ends in lane g for group g.  Not
  // needed where every group is kept.
  float gsc = ninf;
  uint64_t keep = ~uint64_t{0} >> (64 - G);
  const bool limited = TG < G;
  if (SEG && limited) {
    float t1 = ninf, t2 = ninf;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if (u[j] > t1) {
        t2 = t1;
        t1 = u[j];
      } else if (u[j] > t2) {
        t2 = u[j];
      }
    }
    auto meet = [&](float o1, float o2) {
      const float n2 = fmaxf(fminf(t1, o1), fmaxf(t2, o2));
      t1 = fmaxf(t1, o1);
      t2 = n2;
    };
    auto move = [&](auto ctrl) {
      constexpr int c = decltype(ctrl)::value;
      meet(__uint_as_float(dpp<c>(__float_as_uint(t1))), __uint_as_float(dpp<c>(__float_as_uint(t2))));
    };
    if (lg > 0) move(std::integral_constant<int, 0xB1>{});
    if (lg > 1) move(std::integral_constant<int, 0x4E>{});
    if (lg > 2) move(std::integral_constant<int, 0x141>{});
    if (lg > 3) move(std::integral_constant<int, 0x140>{});
    for (int off = 16; off < (1 << lg); off <<= 1) meet(__shfl_xor(t1, off), __shfl_xor(t2, off));
    const float mine = (topn == 1) ? t1 : t1 + t2;
    gsc = __shfl(mine, min(lane, G - 1) << lg);
  } else if (limited) {
    __shared__ float u_sh[kSelWaves][kMaxE + kMaxE / 32];
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      const int e = lane * EPL + j;
      if (e < E) u_sh[wave][upad(e)] = u[j];
    }
    __syncthreads();
    if (lane < G) {
      float t1 = ninf, t2 = ninf;
      for (int j = 0; j < gs; ++j) {
        const float v = u_sh[wave][upad(lane * gs + j)];
        if (v > t1) {
          t2 = t1;
          t1 = v;
        } else if (v > t2) {
          t2 = v;
        }
      }
      gsc = (topn == 1) ? t1 : t1 + t2;
    }
  }
  if (!valid) return;

  // 3. keep the TG best groups (ties: lower group id): bit g of `keep`
  if (limited) {
    int rank = 0;
    for (int g = 0; g < G; ++g) {
      const float o = readlane_f(gsc, g);
      rank += (o > gsc) || (o == gsc && g < lane);
    }
    keep = __ballot(lane < G && rank < TG);
  }

  // 4. top-K of the eligible experts by biased score.  key: ordered scores (0:
  // not a candidate; 1 at least, also for a NaN of all ones).  The K-th key is
  // found by halving an interval of keys: lo with at least K keys above it,
  // hi with fewer, until exactly K are above lo or, where the K-th key is held
  // more than once, hi is that key.  A count is one comparison a key and
  // scalar work beside the other waves' vector work; from four powers of two
  // below the largest key it takes about seven.  (52,001 tokens of 256
  // experts, softmax, top 8: 40 us, bound by its 345 vector instructions a token; K rounds
  // of the wave's largest key over sorted lanes: 48.)
  uint32_t key[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) {
    const int e = lane * EPL + j;
    // a segment past the last group has no bit in keep
    key[j] = (SEG ? (keep >> (lane >> lg)) & 1 : e < E && ((keep >> (e / gs)) & 1)) ? max(ordered(u[j]), 1u) : 0;
  }
  auto above = [&](uint32_t x) {
    int n = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) n += __builtin_popcountll(__ballot(key[j] > x));
    return n;
  };
  uint32_t best = key[0];
#pragma unroll
  for (int j = 1; j < EPL; ++j) best = max(best, key[j]);
  uint32_t hi = wave_max_u32(best);
  uint32_t lo = hi - min(hi, 4u << 23);
  int n = above(lo);
  if (n < K) {
    hi = lo;
    lo = 0;  // K <= TG*E/G keys at least are above 0
    n = above(0);
  }
  while (n != K && hi - lo > 1) {
    const uint32_t mid = lo + (hi - lo) / 2;
    const int m = above(mid);
    if (m >= K) {
      lo = mid;
      n = m;
    } else {
      hi = mid;
    }
  }
  uint64_t chosen[EPL];  // bit l: expert j of lane l
#pragma unroll
  for (int j = 0; j < EPL; ++j) chosen[j] = __ballot(key[j] > lo);
  // number of experts before the lane's first, of those marked in c
  auto before = [&](const uint64_t (&c)[EPL]) {
    uint32_t p = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      p = __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(c[j] >> 32),
                                    __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(c[j]), p));
    return static_cast<int>(p);
  };
  if (n != K) {  // of the keys equal to hi only the first ones
    uint64_t same[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) same[j] = __ballot(key[j] == hi);
    int left = K - above(hi) - before(same);
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      chosen[j] = __ballot(key[j] > hi || (key[j] == hi && left > 0));
      left -= key[j] == hi ? 1 : 0;
    }
  }
  // the chosen, exactly K, in the experts' order to lanes 0 .. K - 1
  __shared__ __attribute__((aligned(16))) u32x4 pick[kSelWaves][kMaxK];
  {
    int p = before(chosen);
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (__builtin_amdgcn_inverse_ballot_w64(chosen[j])) {
        pick[wave][p] =
            u32x4{key[j], static_cast<uint32_t>(lane * EPL + j), __float_as_uint(sv[j]), 0};
        ++p;
      }
  }
  wave_order();
  const u32x4 mine = pick[wave][min(lane, K - 1)];
  // rank order: larger key first, then lower index.  Lane l compares choice
  // l % 16 with choices l / 16, 4 + l / 16, ..: bit l of a round's ballot is
  // set where the other one comes first.
  int rank = lane;
  {
    const int r = lane % kMaxK, own = pick[wave][min(r, K - 1)][0];
    int n = 0;
    for (int i0 = 0; i0 < K; i0 += kWave / kMaxK) {
      const int i = i0 + lane / kMaxK;
      const uint32_t o = pick[wave][min(i, K - 1)][0], k = own;
      const uint64_t b = __ballot(i < K && (o > k || (o == k && i < r)));
      const uint32_t of_r = 0x00010001u << r;  // r's column
      n += __builtin_popcount(static_cast<uint32_t>(b) & of_r) +
           __builtin_popcount(static_cast<uint32_t>(b >> 32) & of_r);
    }
    if (lane < K) rank = n;
  }
  const float my_s = __builtin_bit_cast(
      float, __builtin_amdgcn_ds_permute(4 * rank, static_cast<int>(mine[2])));  // ranked scores
  // their sum in rank order: with each step a lane adds its score to the lane
  // before's sum, so that after K - 1 lane K - 1 holds ((s_0 + s_1) + s_2) ..
  float D = my_s;
  for (int k = 1; k < K; ++k) D = __uint_as_float(dpp<0x111>(__float_as_uint(D))) + my_s;  // row_shr:1
  D = readlane_f(D, K - 1);
  // 5. weights: (s / D) * scale, two binary32 roundings (0 where every chosen
  // score is 0), or s * scale
  if (lane < K) {
    const float q = !normed ? my_s : D == 0.0f ? 0.0f : my_s / D;
    idx_out[t * K + rank] = static_cast<int32_t>(mine[1]);
    w_out[t * K + lane] = q * scale;
  }
}

// ---- gradient ---------------------------------------------------------------

// 1 / (1 + e^-l) and its derivative, from t = e^-|l| so that neither loses
// the small side: s = 1/(1+t) or t/(1+t), s (1 - s) = t / (1+t)^2.
__device__ __forceinline__ void sigmoid_grad(float l, float& s, float& ds) {
  const float t = expf(-fabsf(l));
  const float r = 1.0f / (1.0f + t);
  s = l >= 0.0f ? r : t * r;
  ds = t * r * r;
}

// Sum over lanes 0..15, in every one of them (a wave's choices, K <= 16).
__device__ __forceinline__ float sum16(float v) {
  auto step = [&](uint32_t o) { v += __uint_as_float(o); };
  step(dpp<0xB1>(__float_as_uint(v)));
  step(dpp<0x4E>(__float_as_uint(v)));
  step(dpp<0x141>(__float_as_uint(v)));
  step(dpp<0x140>(__float_as_uint(v)));
  return v;
}

// One wave per token; lane l holds experts l*EPL .. l*EPL + EPL - 1 of the
// row, lanes 0..K-1 also a choice each.  The choices' gradients meet the row
// in LDS; where an expert is named twice every lane instead adds the choices
// that name its experts in rank order, so no sum depends on timing.  Bound by
// reading and writing the logits' rows: a sigmoid row is only written, its K
// chosen logits being gathered (16,384 rows of 256, softmax: 9.2 us; every
// lane adding every choice: 12.4).
template <int EPL, bool SM>
__global__ __launch_bounds__(256) void route_backward(
    const float* __restrict__ logits, const int32_t* __restrict__ idx,
    const float* __restrict__ dw, int vec4, int64_t T, int E, int K, int normed, float scale,
    float* __restrict__ dl) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), lane = threadIdx.x % kWave;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kSelWaves + wave;
  if (t >= T) return;  // wave-uniform
  __shared__ __attribute__((aligned(16))) float sh[kSelWaves][kWave * EPL];
  const float* row = logits + t * E;
  float p[EPL];
  float m = 0.0f, rs = 0.0f;
  if constexpr (SM) {  // p = e^(l - m), rs = 1 / their sum
    if (EPL % 4 == 0 && vec4) {
#pragma unroll
      for (int j = 0; j < EPL; j += 4) {
        const u32x4 v = ld16(row + min(lane * EPL + j, E - 4));
#pragma unroll
        for (int q = 0; q < 4 && j + q < EPL; ++q) p[j + q] = __uint_as_float(v[q]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < EPL; ++j) p[j] = row[min(lane * EPL + j, E - 1)];
    }
  }
  int e_k = -1;
  float d_k = 0.0f, l_k = 0.0f;
  if (lane < K) {
    e_k = idx[t * K + lane];
    if (e_k < 0 || e_k >= E) e_k = -1;
    if (e_k >= 0) {
      d_k = dw[t * K + lane];
      l_k = row[e_k];
    }
  }
  if constexpr (SM) {
    m = -__builtin_huge_valf();
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      if (lane * EPL + j >= E) p[j] = -__builtin_huge_valf();
      m = fmaxf(m, p[j]);
    }
    m = wave_max_f32(m);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) {
      p[j] = p[j] == -__builtin_huge_valf() ? 0.0f : expf(p[j] - m);
      sum += p[j];
    }
    sum = sum16(sum);
    sum += __uint_as_float(dpp<0x142>(__float_as_uint(sum)));  // rows 0 and 1, 2 and 3
    sum += __uint_as_float(dpp<0x143>(__float_as_uint(sum)));  // all, in the last lane
    sum = readlane_f(sum, kWave - 1);
    rs = sum == 0.0f ? 0.0f : 1.0f / sum;
  }
  // the choices: scores, then the gradient g of each choice's own logit
  float s_k = 0.0f, ds_k = 0.0f;
  if (e_k >= 0) {
    if (SM) s_k = l_k == -__builtin_huge_valf() ? 0.0f : expf(l_k - m) * rs;
    else sigmoid_grad(l_k, s_k, ds_k);
  }
  float D = 1.0f;
  if (normed) {
    D = sum16(s_k);
    D = D == 0.0f ? __builtin_huge_valf() : D;  // all scores 0: every quotient below is 0
  }
  // lanes 0..15 hold the sum; the dense form needs it in every lane
  const float c = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(
                                                __builtin_bit_cast(int, sum16(d_k * (s_k / D)))));
  float g;
  if (SM) g = scale * (s_k / D) * (normed ? d_k - c : d_k);
  else g = scale * (ds_k / D) * (normed ? d_k - c : d_k);
  const float back = (SM && !normed) ? scale * c * rs : 0.0f;
  float out[EPL];
#pragma unroll
  for (int j = 0; j < EPL; ++j) out[j] = SM ? -back * p[j] : 0.0f;
  // an expert named twice: lane l compares choice l % 16 with l / 16, ..
  uint64_t twice = 0;
  for (int i0 = 0; i0 < K; i0 += kWave / 16) {
    const int i = i0 + lane / 16;
    const int ei = __shfl(e_k, i % 16), er = __shfl(e_k, lane % 16);
    twice |= __ballot(i < lane % 16 && ei >= 0 && ei == er);
  }
  if (!twice) {
    // through LDS: zeros, the choices' gradients where they belong, the row
    float* row_g = sh[wave];
#pragma unroll
    for (int j = 0; j < EPL; ++j) row_g[lane * EPL + j] = 0.0f;
    wave_order();
    if (e_k >= 0) row_g[e_k] = g;
    wave_order();
#pragma unroll
    for (int j = 0; j < EPL; ++j) out[j] += row_g[lane * EPL + j];
  } else {
    for (int k = 0; k < K; ++k) {
      const int e = __builtin_amdgcn_readlane(e_k, k);
      const float gk = readlane_f(g, k);
#pragma unroll
      for (int j = 0; j < EPL; ++j)
        if (lane * EPL + j == e) out[j] += gk;
    }
  }
  float* o = dl + t * E;
  if (EPL % 4 == 0 && vec4) {
#pragma unroll
    for (int j = 0; j < EPL; j += 4)
      if (lane * EPL + j < E) {
        u32x4 v;
#pragma unroll
        for (int q = 0; q < 4 && j + q < EPL; ++q) v[q] = __float_as_uint(out[j + q]);
        st16(o + lane * EPL + j, v);
      }
  } else {
#pragma unroll
    for (int j = 0; j < EPL; ++j)
      if (lane * EPL + j < E) o[lane * EPL + j] = out[j];
  }
}

}  // namespace

hipError_t launch_route_backward(const Plan& p, const float* logits, const int32_t* idx,
                                 const float* d_w, float* d_logits, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(p.T, kSelWaves)));
  const int epl = static_cast<int>(ceil_div(p.E, kWave));
  const int vec4 = p.E % 4 == 0;
#define BEAM_RB(EPL)                                                                         \
  do {                                                                                       \
    if (p.softmax)                                                                           \
      hipLaunchKernelGGL((route_backward<EPL, true>), grid, dim3(256), 0, s, logits, idx,    \
                         d_w, vec4, p.T, p.E, p.K, p.normed ? 1 : 0, p.scale, d_logits);     \
    else                                                                                     \
      hipLaunchKernelGGL((route_backward<EPL, false>), grid, dim3(256), 0, s, logits, idx,   \
                         d_w, vec4, p.T, p.E, p.K, p.normed ? 1 : 0, p.scale, d_logits);     \
  } while (0)
  if (epl <= 1) BEAM_RB(1);
  else if (epl <= 2) BEAM_RB(2);
  else if (epl <= 4) BEAM_RB(4);
  else if (epl <= 8) BEAM_RB(8);
  else BEAM_RB(16);
#undef BEAM_RB
  return hipGetLastError();
}

hipError_t launch_router(const Plan& p, const void* x, const float* w_router,
                         const float* bias, float* logits_out,
                         const float* logits_in, int32_t* idx, float* w,
                         void* ws, hipStream_t s, Timer* tm) {
  const float* part = logits_in;
  int ks = 1;
  if (!logits_in) {
    ks = p.ks;
    float* buf = ws_at<float>(ws, p.off_part);
    const int kchunk = p.H / ks;
    if (p.router_gemm) {
      uint16_t* w3 = ws_at<uint16_t>(ws, p.off_w3);
      const int64_t n = static_cast<int64_t>(p.E) * p.H;
      BEAM_LAUNCH(tm, "router_split", router_split, dim3(static_cast<unsigned>(ceil_div(n, 256))),
                  dim3(256), 0, s, w_router, w3, p.E, p.H);
      const hipError_t e = launch_router_gemm(p, x, w3, buf, s, tm);
      if (e != hipSuccess) return e;
    } else if (p.act == BEAM_BF16 && p.E % 32 == 0) {
      dim3 grid(static_cast<unsigned>(ceil_div(p.T, 32)), static_cast<unsigned>(ceil_div(p.E, 64)), ks);
      BEAM_LAUNCH(tm, "router_logits_mfma", router_logits_mfma, grid, dim3(kLgWaves * kWave), 0, s,
                         static_cast<const uint16_t*>(x), w_router, buf, p.T,
                         p.H, p.E, kchunk);
    } else {
      dim3 grid(static_cast<unsigned>(ceil_div(p.T * p.E, 256)), ks);
      BEAM_LAUNCH(tm, "router_logits_valu", router_logits_valu, grid, dim3(256), 0, s, x,
                         p.act == BEAM_BF16 ? 1 : 0, w_router, buf, p.T, p.H,
                         p.E, kchunk);
    }
    part = buf;
  }
  const float* lo = logits_in ? nullptr : logits_out;
  dim3 grid(static_cast<unsigned>(ceil_div(p.T, kSelWaves)));
  const int epl = static_cast<int>(ceil_div(p.E, kWave));
  const int eplp = epl <= 1 ? 1 : epl <= 2 ? 2 : epl <= 4 ? 4 : epl <= 8 ? 8 : 16;
  const int gs = p.E / p.G, seg_l = gs / eplp;
  const bool seg = gs % eplp == 0 && (seg_l & (seg_l - 1)) == 0;
  const int lg = seg ? __builtin_ctz(static_cast<unsigned>(seg_l)) : 0;
  // partials live in the workspace and given logits are 16-byte aligned
  // (checked at the boundary), so rows of E % 4 == 0 floats are too
  const int vec4 = p.E % 4 == 0;
#define BEAM_SEL4(EPL, KS, SEG, SM)                                            \
  BEAM_LAUNCH(tm, "router_select", (router_select<EPL, KS, SEG, SM>), grid, dim3(256), 0, s, part, \
              ks, vec4, p.T, p.E, p.G, p.TG, p.K, p.topn, lg, p.normed ? 1 : 0, p.scale, bias, \
              const_cast<float*>(lo), idx, w)
#define BEAM_SEL3(EPL, KS, SEG)                                                \
  do {                                                                         \
    if (p.softmax) BEAM_SEL4(EPL, KS, SEG, true);                              \
    else BEAM_SEL4(EPL, KS, SEG, false);                                       \
  } while (0)
#define BEAM_SEL(EPL)                                                          \
  do {                                                                         \
    if (ks == 1) {                                                             \
      if (seg) BEAM_SEL3(EPL, 1, true); else BEAM_SEL3(EPL, 1, false);         \
    } else {                                                                   \
      if (seg) BEAM_SEL3(EPL, kMaxKs, true); else BEAM_SEL3(EPL, kMaxKs, false); \
    }                                                                          \
  } while (0)
  if (ks > kMaxKs) return hipErrorInvalidValue;
  if (eplp == 1) BEAM_SEL(1);
  else if (eplp == 2) BEAM_SEL(2);
  else if (eplp == 4) BEAM_SEL(4);
  else if (eplp == 8) BEAM_SEL(8);
  else BEAM_SEL(16);
#undef BEAM_SEL4
#undef BEAM_SEL3
#undef BEAM_SEL
  return hipGetLastError();
}

}  // namespace beam
