// Norms of query and key heads, their rotation by position and the keys' and
// values' way into a paged cache, in one pass, and the gradients:
//   n = x / sqrt(mean(x^2) + eps) * w     per head of D values
//   (n_a, n_b) turned by pos * f_i        pairs (i, i + rot/2) or (2i, 2i+1)
//   q times (1 + (pos + 1) / L)^e
// (RMSNorm on queries and keys, rotation in the sliding-window layers and the
// query's temperature in the global ones: "Reflection Releases Beam ...",
// section "Hybrid Attention and Unusual Residuals".)
//
// A head is held by a group of lanes, 8 values a lane, so every input is read
// and every output written once: both directions are bound by those bytes.  A
// wave stays with one token: each lane takes the sine and cosine of one pair
// (two at D > 128) and all heads of the token take theirs from LDS.  An angle
// is reduced in binary64, in quarter turns: what is left is off by 2^-26 of a quarter
// turn and by 2^-52 of the turns taken off (two roundings of them, 2^-22 near position
// 2^30 at a radian each).  One token a wave and the next step's loads ahead of the
// work: 16,381 tokens of 48 + 8 heads of 128 into a cache take 101 us (5.3 TB/s; fp32
// 231, 4.6); waves that stay for several tokens, with loads ahead across them, took
// 139, and two to eight waves a token 119 to 173.
#include <algorithm>

#include "serve.h"

namespace beam {
namespace {

constexpr int kRopeWaves = 4;
constexpr double kQuartersPerRadian = 0.63661977236758134308;  // 2 / pi

// (cos, sin) of pos * f quarter turns
__device__ __forceinline__ float2 turn(int pos, double f) {
  const double u = static_cast<double>(pos) * f;
  const double n = rint(u);
  float s, c;
  sincospif(0.5f * static_cast<float>(u - n), &s, &c);
  const int quarter = static_cast<int>(n - 4.0 * floor(0.25 * n));
  if (quarter & 1) {
    const float t = c;
    c = -s;
    s = t;
  }
  return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

// Sum over the LPH lanes of a head, by data-parallel moves: neighbours, pairs,
// then each half of 8 and of 16 lanes mirrored.
template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#define BEAM_ADD(ctrl) \
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), ctrl, 0xF, 0xF, true))
  if (LPH >= 2) BEAM_ADD(0xB1);
  if (LPH >= 4) BEAM_ADD(0x4E);
  if (LPH >= 8) BEAM_ADD(0x141);
  if (LPH >= 16) BEAM_ADD(0x140);
#undef BEAM_ADD
  if (LPH >= 32) v += __shfl_xor(v, 16);
  return v;
}

// A lane's 8 values of a turn: with o a value's partner, y = c v + s o.
struct Turn {
  float c[8], s[8];
  int partner;  // lane of the partners (pairs half a rotation apart; else itself)
};
template <int LPH>
__device__ __forceinline__ void make_turn(const RopeArgs& a, int pos, const double* freq,
                                          float2* cs, int lane, Turn& t) {
  const int pairs = a.rot / 2, col = lane % LPH * 8;
  t.partner = lane;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    t.c[j] = 1.0f;
    t.s[j] = 0.0f;
  }
  if (a.rot == 0) return;
  for (int i = lane; i < pairs; i += kWave) cs[i] = turn(pos, freq[i]);
  wave_order();
  if (col < a.rot) {
    const bool second = !a.interleaved && col >= pairs;
    if (!a.interleaved) t.partner = second ? lane - pairs / 8 : lane + pairs / 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = cs[a.interleaved ? (col + j) / 2 : second ? col - pairs + j : col + j];
      t.c[j] = v.x;
      t.s[j] = (a.interleaved ? j % 2 == 0 : !second) ? -v.y : v.y;
    }
  }
  wave_order();  // the next token's pairs
}

// The partners of a lane's values (every lane of the wave calls it).
template <typename IO>
__device__ __forceinline__ void partners(const RopeArgs& a, const Turn& t, const Eight<IO>& e,
                                         float (&o)[8]) {
  if (a.interleaved || a.rot == 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = e.get(j ^ 1);
    return;
  }
  Eight<IO> x;
#pragma unroll
  for (int i = 0; i < Eight<IO>::kWords; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) x.w[i][j] = __shfl(static_cast<int>(e.w[i][j]), t.partner);
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = x.get(j);
}

__device__ __forceinline__ float temperature(const RopeArgs& a, int pos) {
  if (a.temp_length == 0.0f) return 1.0f;
  return powf(1.0f + (static_cast<float>(pos) + 1.0f) / a.temp_length, a.temp_exponent);
}

// Where token t's key and value go: an element offset, or -1.
__device__ __forceinline__ int64_t place(const RopeArgs& a, int64_t t, int pos) {
  const Cache& c = a.cache;
  const int64_t row = a.rows ? a.rows[t] : t;
  if (row < 0 || row >= c.seqs || pos < 0) return -1;
  const int slot = pos >> c.shift;
  if (slot >= c.cols) return -1;
  const int page = c.tables[row * c.cols + slot];
  if (page < 0 || page >= c.pages) return -1;
  return page * c.page_stride + (pos & ((1 << c.shift) - 1)) * c.token_stride;
}

// What the workgroup's waves share: both weights, the frequencies in quarter
// turns a position, and each wave's sines and cosines.
struct Shared {
  float w[2][kMaxHeadDim];
  double freq[kMaxHeadDim / 2];
  float2 pairs[kRopeWaves][kMaxHeadDim / 2];
  __device__ __forceinline__ void stage(const RopeArgs& a) {
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
      w[0][c] = a.wq[c];
      w[1][c] = a.wk[c];
    }
    for (int i = threadIdx.x; i < a.rot / 2; i += blockDim.x)
      freq[i] = a.inv_freq[i] * kQuartersPerRadian;
    __syncthreads();
  }
};

// Lane groups of LPH lanes hold a head; a wave takes 64 / LPH heads at a step:
// first the queries', then the keys', then the values' (which are copied).
// `parts` waves share a token.  Loads are never masked (a lane without a head
// reads its step's last one, one past D the head's first values, which stay out of
// the head's sums), so that the next step's are on their way while one is worked
// on; stores are.
template <typename IO, int LPH>
__global__ __launch_bounds__(kRopeWaves* kWave) void rope_forward(RopeArgs a, int parts) {
  constexpr int kHeads = kWave / LPH;
  __shared__ Shared sh;
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRopeWaves + wave;
  const int64_t t = min<int64_t>(id / parts, a.T - 1);
  int i = static_cast<int>(id % parts);
  const bool in = lane % LPH * 8 < a.D;
  const int col = in ? lane % LPH * 8 : 0, sub = lane / LPH;
  const int nq = (a.Hq + kHeads - 1) / kHeads, nk = (a.Hkv + kHeads - 1) / kHeads;
  const IO* q = static_cast<const IO*>(a.q) + t * a.q_stride + col;
  const IO* k = static_cast<const IO*>(a.k) + t * a.k_stride + col;
  const IO* v = static_cast<const IO*>(a.v) + t * a.v_stride + col;
  auto read = [&](const IO* p, int step, int H) {
    Eight<IO> e;
    e.load(p + min(step * kHeads + sub, H - 1) * a.D);
    return e;
  };
  // what the wave starts with
  Eight<IO> e = i < nq ? read(q, i, a.Hq) : i < nq + nk ? read(k, i - nq, a.Hkv)
                : a.cache.k ? read(v, i - nq - nk, a.Hkv) : read(k, 0, a.Hkv);
  const int pos = a.pos ? a.pos[t] : 0;
  sh.stage(a);
  if (id / parts >= a.T) return;
  const int64_t at = a.cache.k ? place(a, t, pos) : -1;
  Turn tn;
  make_turn<LPH>(a, pos, sh.freq, sh.pairs[wave], lane, tn);
  const float per = 1.0f / static_cast<float>(a.D);
  // y = inv (c v + s o) with the weights and the scale in c and s
  float c[8], s[8];
  auto factors = [&](const float* w, float scale) {
    const int other = tn.partner % LPH * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] = tn.c[j] * w[col + j] * scale;
      s[j] = tn.s[j] * w[a.interleaved ? col + (j ^ 1) : other + j] * scale;
    }
  };
  auto normed = [&](Eight<IO>& e) {
    float x[8], o[8], ss = 0.0f;
    partners(a, tn, e, o);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      x[j] = e.get(j);
      ss += x[j] * x[j];
    }
    const float inv = __builtin_amdgcn_rsqf(head_sum<LPH>(in ? ss * per : 0.0f) + a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = (x[j] * c[j] + o[j] * s[j]) * inv;
    e.set(x);
  };
  if (i < nq) {
    factors(sh.w[0], temperature(a, pos));
    IO* out = static_cast<IO*>(a.q_out) + t * a.Hq * a.D + col;
    do {
      const Eight<IO> next = i + parts < nq ? read(q, i + parts, a.Hq)
                                            : read(k, min(i + parts - nq, nk - 1), a.Hkv);
      normed(e);
      const int h = i * kHeads + sub;
      if (in && h < a.Hq) e.store(out + h * a.D);
      e = next;
      i += parts;
    } while (i < nq);
    // (where its next step is a value's, the wave has read a key's in vain)
    if (a.cache.k && i >= nq + nk) e = read(v, min(i - nq - nk, nk - 1), a.Hkv);
  }
  i -= nq;
  if (i < nk) {
    factors(sh.w[1], 1.0f);
    do {
      Eight<IO> next = e;
      if (i + parts < nk) next = read(k, i + parts, a.Hkv);
      else if (at >= 0) next = read(v, min(i + parts - nk, nk - 1), a.Hkv);
      normed(e);
      const int h = i * kHeads + sub;
      if (in && h < a.Hkv) {
        if (a.k_out) e.store(static_cast<IO*>(a.k_out) + (t * a.Hkv + h) * a.D + col);
        if (at >= 0) e.store(static_cast<IO*>(a.cache.k) + at + h * a.cache.head_stride + col);
      }
      e = next;
      i += parts;
    } while (i < nk);
  }
  if (at < 0) return;
  for (i -= nk; i < nk; i += parts) {
    const Eight<IO> next = read(v, min(i + parts, nk - 1), a.Hkv);
    const int h = i * kHeads + sub;
    if (in && h < a.Hkv) e.store(static_cast<IO*>(a.cache.v) + at + h * a.cache.head_stride + col);
    e = next;
  }
}

// Gradients: with d the gradient turned back (and scaled), xhat = x inv,
//   dw += d xhat,  dx = inv (d w - xhat mean(d w xhat)).
// A wave takes every gridDim-th token, keeps the weights' sums of its lanes'
// columns, and the workgroup leaves one sum for each column and weight.
template <typename IO, int LPH>
__global__ __launch_bounds__(kRopeWaves* kWave) void rope_backward(RopeGradArgs g) {
  constexpr int kHeads = kWave / LPH;
  const RopeArgs& a = g.f;
  __shared__ Shared sh;
  __shared__ float sums[kRopeWaves][kHeads][LPH * 8];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const bool in = lane % LPH * 8 < a.D;
  const int col = in ? lane % LPH * 8 : 0, sub = lane / LPH;
  const float per = 1.0f / static_cast<float>(a.D);
  sh.stage(a);
  float acc[2][8] = {};
  const int64_t every = static_cast<int64_t>(gridDim.x) * kRopeWaves;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRopeWaves + wave; t < a.T; t += every) {
    const IO* x[2] = {static_cast<const IO*>(a.q) + t * a.q_stride + col,
                      static_cast<const IO*>(a.k) + t * a.k_stride + col};
    const IO* dy[2] = {static_cast<const IO*>(g.dq_out) + t * a.Hq * a.D + col,
                       static_cast<const IO*>(g.dk_out) + t * a.Hkv * a.D + col};
    Eight<IO> ex, ed;
    auto read = [&](int kind, int i, int H) {
      const int off = min(i * kHeads + sub, H - 1) * a.D;
      ex.load(x[kind] + off);
      ed.load(dy[kind] + off);
    };
    read(0, 0, a.Hq);
    const int pos = a.pos ? a.pos[t] : 0;
    Turn tn;
    make_turn<LPH>(a, pos, sh.freq, sh.pairs[wave], lane, tn);
    const float temp = temperature(a, pos);
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int H = kind ? a.Hkv : a.Hq, n = (H + kHeads - 1) / kHeads;
      IO* dx = static_cast<IO*>(kind ? g.dk : g.dq) + t * H * a.D + col;
      const float scale = kind ? 1.0f : temp;
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = sh.w[kind][col + j];
      for (int i = 0; i < n; ++i) {
        const Eight<IO> nx = ex, nd = ed;
        if (i + 1 < n) read(kind, i + 1, H);
        else if (kind == 0) read(1, 0, a.Hkv);
        float v[8], d[8], o[8], ss = 0.0f;
        partners(a, tn, nd, o);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = nx.get(j);
          ss += v[j] * v[j];
          d[j] = (nd.get(j) * tn.c[j] - o[j] * tn.s[j]) * scale;
        }
        const float inv = __builtin_amdgcn_rsqf(head_sum<LPH>(in ? ss * per : 0.0f) + a.eps);
        const bool live = in && i * kHeads + sub < H;
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] *= inv;
          acc[kind][j] += live ? d[j] * v[j] : 0.0f;
          d[j] *= w[j];
          dot += d[j] * v[j];
        }
        const float mean = head_sum<LPH>(in ? dot * per : 0.0f);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = inv * (d[j] - v[j] * mean);
        if (live) {
          Eight<IO> out;
          out.set(d);
          out.store(dx + (i * kHeads + sub) * a.D);
        }
      }
    }
  }
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[wave][sub][lane % LPH * 8 + j] = acc[kind][j];
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
      float s = 0.0f;
      for (int i = 0; i < kRopeWaves; ++i)
#pragma unroll 4
        for (int j = 0; j < kHeads; ++j) s += sums[i][j][c];
      g.part[(static_cast<int64_t>(blockIdx.x) * 2 + kind) * a.D + c] = s;
    }
  }
}

// The workgroups' shares added: 8 columns a workgroup, 32 threads a column.
constexpr int kSumCols = 8, kSumRows = 32;
__global__ __launch_bounds__(kSumCols* kSumRows) void rope_weight_sums(const float* part, int groups,
                                                                        int D, float* d_wq,
                                                                        float* d_wk) {
  __shared__ float sums[kSumRows][kSumCols + 1];
  const int in = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols;
  const int c = blockIdx.x * kSumCols + in;  // D is a multiple of 8
  float s = 0.0f;
#pragma unroll 8
  for (int g = row; g < groups; g += kSumRows) s += part[static_cast<int64_t>(g) * 2 * D + c];
  sums[row][in] = s;
  __syncthreads();
  if (row) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < kSumRows; ++i) s += sums[i][in];
  (c < D ? d_wq : d_wk)[c < D ? c : c - D] = s;
}

int lanes_per_head(int D) {
  int n = 1;
  while (n * 8 < D) n *= 2;
  return n;
}

template <typename IO, typename F>
hipError_t by_lanes(int D, F f) {
  switch (lanes_per_head(D)) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    case 8: return f(std::integral_constant<int, 8>());
    case 16: return f(std::integral_constant<int, 16>());
    default: return f(std::integral_constant<int, 32>());
  }
}

template <typename IO>
hipError_t forward(const RopeArgs& a, hipStream_t s) {
  return by_lanes<IO>(a.D, [&](auto lanes) {
    constexpr int kLanes = decltype(lanes)::value, kHeads = kWave / kLanes;
    // few tokens: a token's heads over several waves, down to one step each
    const int64_t steps = ceil_div(a.Hq, kHeads) + (a.cache.k ? 2 : 1) * ceil_div(a.Hkv, kHeads);
    const int64_t parts = std::max<int64_t>(1, std::min(steps, 4096 / std::max<int64_t>(1, a.T)));
    const int64_t blocks = ceil_div(a.T * parts, kRopeWaves);
    hipLaunchKernelGGL((rope_forward<IO, kLanes>), dim3(blocks), dim3(kRopeWaves * kWave), 0, s, a,
                       static_cast<int>(parts));
    return hipGetLastError();
  });
}

template <typename IO>
hipError_t backward(const RopeGradArgs& a, float* d_wq, float* d_wk, hipStream_t s) {
  const int groups = rope_grad_groups(a.f.T);
  if (groups) {
    const hipError_t e = by_lanes<IO>(a.f.D, [&](auto lanes) {
      hipLaunchKernelGGL((rope_backward<IO, decltype(lanes)::value>), dim3(groups),
                         dim3(kRopeWaves * kWave), 0, s, a);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(rope_weight_sums, dim3(2 * a.f.D / kSumCols), dim3(kSumCols * kSumRows), 0, s, a.part,
                     groups, a.f.D, d_wq, d_wk);
  return hipGetLastError();
}

}  // namespace

// Three workgroups a compute unit, as their registers allow (8,191 tokens with the
// forward: 128 us; two 133, four 141).
int rope_grad_groups(int64_t T) {
  return static_cast<int>(std::min<int64_t>(ceil_div(T, kRopeWaves), 768));
}

hipError_t launch_qk_norm_rope(const RopeArgs& a, int32_t dtype, hipStream_t s) {
  return dtype == BEAM_BF16 ? forward<uint16_t>(a, s) : forward<float>(a, s);
}

hipError_t launch_qk_norm_rope_backward(const RopeGradArgs& a, int32_t dtype, float* d_wq,
                                        float* d_wk, hipStream_t s) {
  return dtype == BEAM_BF16 ? backward<uint16_t>(a, d_wq, d_wk, s)
                            : backward<float>(a, d_wq, d_wk, s);
}

}  // namespace beam
