// Norms of query and key heads, their rotation by position and the keys' and
// values' way into a paged cache, in one pass, and the gradients:
//   n = x / sqrt(mean(x^2) + eps) * w     per head of D values
//   (n_a, n_b) turned by pos * f_i        pairs (i, i + rot/2) or (2i, 2i+1)
//   q times (1 + (pos + 1) / L)^e
// (RMSNorm on queries and keys, rotation in the sliding-window layers and the
// query's temperature in the global ones: "Reflection Beam", section "Hybrid
// Attention and Unusual Residuals".)
//
// A head is held by a group of lanes, 8 values a lane, so every input is read
// and every output written once: both directions are bound by those bytes.  A
// wave stays with one token: each lane takes the sine and cosine of one pair
// (two at D > 128) and all heads of the token take theirs from LDS.  An angle
// is reduced in binary64, in quarter turns, so that what is left is exact to
// 2^-26 of a quarter turn at any position.
#include <algorithm>

#include "serve.h"

namespace beam {
namespace {

constexpr int kRopeWaves = 4;
constexpr double kQuartersPerRadian = 0.63661977236758134308;  // 2 / pi

// (cos, sin) of pos * f
__device__ __forceinline__ float2 turn(int pos, double f) {
  const double u = static_cast<double>(pos) * (f * kQuartersPerRadian);
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

template <int LPH>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int m = 1; m < LPH; m *= 2) v += __shfl_xor(v, m);
  return v;
}

// What a lane needs to turn its 8 values: for each the cosine and the sine with
// the sign that meets its partner's value.
struct Turn {
  float c[8], s[8];
  int partner;  // lane of the partner's values (pairs half a rotation apart)
  bool turns;
};
template <int LPH>
__device__ __forceinline__ Turn make_turn(const RopeArgs& a, int pos, float2* cs, int lane) {
  const int pairs = a.rot / 2, chunk = lane % LPH, col = chunk * 8;
  Turn t;
  t.turns = col < a.rot;
  t.partner = lane;
  if (a.rot == 0) return t;
  for (int i = lane; i < pairs; i += kWave) cs[i] = turn(pos, a.inv_freq[i]);
  wave_order();
  if (!t.turns) return t;
  const bool second = !a.interleaved && col >= pairs;
  if (!a.interleaved) t.partner = second ? lane - pairs / 8 : lane + pairs / 8;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 v = cs[a.interleaved ? (col + j) / 2 : second ? col - pairs + j : col + j];
    t.c[j] = v.x;
    t.s[j] = (a.interleaved ? j % 2 == 0 : !second) ? -v.y : v.y;
  }
  wave_order();  // the next token's pairs
  return t;
}

// y = the turned v, where `back` turns the other way.  Every lane of the wave
// calls it.
template <int LPH, bool back>
__device__ __forceinline__ void rotate(const RopeArgs& a, const Turn& t, float (&v)[8]) {
  if (a.rot == 0) return;
  float other[8];
  if (a.interleaved) {
#pragma unroll
    for (int j = 0; j < 8; ++j) other[j] = v[j ^ 1];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) other[j] = __shfl(v[j], t.partner);
  }
  if (!t.turns) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float s = back ? -t.s[j] : t.s[j];
    v[j] = v[j] * t.c[j] + other[j] * s;
  }
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

// Lane groups of LPH lanes hold a head; a wave takes 64 / LPH heads at a time:
// first the queries', then the keys', then the values' (which are copied).
// `parts` waves share a token.
template <typename IO, int LPH>
__global__ __launch_bounds__(kRopeWaves* kWave) void rope_forward(RopeArgs a, int parts) {
  constexpr int kHeads = kWave / LPH;
  __shared__ float2 pairs[kRopeWaves][kMaxHeadDim / 2];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRopeWaves + wave;
  const int64_t t = id / parts;
  const int part = static_cast<int>(id % parts);
  if (t >= a.T) return;
  const int pos = a.pos ? a.pos[t] : 0;
  const int col = lane % LPH * 8, sub = lane / LPH;
  const bool in = col < a.D;
  const Turn tn = make_turn<LPH>(a, pos, pairs[wave], lane);
  const float temp = temperature(a, pos);
  const int64_t at = a.cache.k ? place(a, t, pos) : -1;
  const int nq = (a.Hq + kHeads - 1) / kHeads, nk = (a.Hkv + kHeads - 1) / kHeads;
  float w[8];
  auto weights = [&](const float* p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = in ? p[col + j] : 0.0f;
  };
  auto normed = [&](const IO* x, bool live, float scale, Eight<IO>& e) {
    if (live) e.load(x);
    else e.zero();
    float v[8], ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = e.get(j);
      ss += v[j] * v[j];
    }
    const float inv = 1.0f / sqrtf(head_sum<LPH>(ss) / static_cast<float>(a.D) + a.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = v[j] * inv * w[j];
    rotate<LPH, false>(a, tn, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= scale;
    e.set(v);
  };
  weights(a.wq);
  const IO* q = static_cast<const IO*>(a.q) + t * a.q_stride + col;
  IO* qo = static_cast<IO*>(a.q_out) + t * a.Hq * a.D + col;
  int i = part;
  for (; i < nq; i += parts) {
    const int h = i * kHeads + sub;
    const bool live = in && h < a.Hq;
    Eight<IO> e;
    normed(q + h * a.D, live, temp, e);
    if (live) e.store(qo + h * a.D);
  }
  weights(a.wk);
  for (i -= nq; i < nk; i += parts) {
    const int h = i * kHeads + sub;
    const bool live = in && h < a.Hkv;
    Eight<IO> e;
    normed(static_cast<const IO*>(a.k) + t * a.k_stride + h * a.D + col, live, 1.0f, e);
    if (live && a.k_out)
      e.store(static_cast<IO*>(a.k_out) + (t * a.Hkv + h) * a.D + col);
    if (live && at >= 0)
      e.store(static_cast<IO*>(a.cache.k) + at + h * a.cache.head_stride + col);
  }
  if (at < 0) return;
  for (i -= nk; i < nk; i += parts) {
    const int h = i * kHeads + sub;
    if (!in || h >= a.Hkv) continue;
    Eight<IO> e;
    e.load(static_cast<const IO*>(a.v) + t * a.v_stride + h * a.D + col);
    e.store(static_cast<IO*>(a.cache.v) + at + h * a.cache.head_stride + col);
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
  __shared__ float2 pairs[kRopeWaves][kMaxHeadDim / 2];
  __shared__ float sums[kRopeWaves][kHeads][LPH * 8];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const int col = lane % LPH * 8, sub = lane / LPH;
  const bool in = col < a.D;
  float acc[2][8] = {};
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRopeWaves;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRopeWaves + wave; t < a.T; t += step) {
    const int pos = a.pos ? a.pos[t] : 0;
    const Turn tn = make_turn<LPH>(a, pos, pairs[wave], lane);
    const float temp = temperature(a, pos);
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const int H = kind ? a.Hkv : a.Hq;
      const IO* x = static_cast<const IO*>(kind ? a.k : a.q) +
                    t * (kind ? a.k_stride : a.q_stride) + col;
      const IO* dy = static_cast<const IO*>(kind ? g.dk_out : g.dq_out) + t * H * a.D + col;
      IO* dx = static_cast<IO*>(kind ? g.dk : g.dq) + t * H * a.D + col;
      float w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = in ? (kind ? a.wk : a.wq)[col + j] : 0.0f;
      const float scale = kind ? 1.0f : temp;
      for (int h0 = 0; h0 < H; h0 += kHeads) {
        const int h = h0 + sub;
        const bool live = in && h < H;
        Eight<IO> ex, ed;
        if (live) {
          ex.load(x + h * a.D);
          ed.load(dy + h * a.D);
        } else {
          ex.zero();
          ed.zero();
        }
        float v[8], d[8], ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] = ex.get(j);
          d[j] = ed.get(j) * scale;
          ss += v[j] * v[j];
        }
        const float inv = 1.0f / sqrtf(head_sum<LPH>(ss) / static_cast<float>(a.D) + a.eps);
        rotate<LPH, true>(a, tn, d);
        float dot = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[j] *= inv;
          acc[kind][j] += d[j] * v[j];
          d[j] *= w[j];
          dot += d[j] * v[j];
        }
        const float mean = head_sum<LPH>(dot) / static_cast<float>(a.D);
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = inv * (d[j] - v[j] * mean);
        if (live) {
          ed.set(d);
          ed.store(dx + h * a.D);
        }
      }
    }
  }
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) sums[wave][sub][col + j] = acc[kind][j];
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
      float s = 0.0f;
      for (int i = 0; i < kRopeWaves; ++i)
        for (int j = 0; j < kHeads; ++j) s += sums[i][j][c];
      g.part[(static_cast<int64_t>(blockIdx.x) * 2 + kind) * a.D + c] = s;
    }
  }
}

// The workgroups' shares added: 16 columns a workgroup, 16 threads a column.
__global__ __launch_bounds__(256) void rope_weight_sums(const float* part, int groups, int D,
                                                         float* d_wq, float* d_wk) {
  __shared__ float sums[16][17];
  const int c = blockIdx.x * 16 + threadIdx.x % 16, row = threadIdx.x / 16;
  float s = 0.0f;
  if (c < 2 * D)
    for (int g = row; g < groups; g += 16) s += part[static_cast<int64_t>(g) * 2 * D + c];
  sums[row][threadIdx.x % 16] = s;
  __syncthreads();
  if (row || c >= 2 * D) return;
  s = 0.0f;
  for (int i = 0; i < 16; ++i) s += sums[i][threadIdx.x];
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
  const int groups = rope_grad_groups(a.f.T, a.f.Hq, a.f.Hkv, a.f.D);
  if (groups) {
    const hipError_t e = by_lanes<IO>(a.f.D, [&](auto lanes) {
      hipLaunchKernelGGL((rope_backward<IO, decltype(lanes)::value>), dim3(groups),
                         dim3(kRopeWaves * kWave), 0, s, a);
      return hipGetLastError();
    });
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(rope_weight_sums, dim3(ceil_div(2 * a.f.D, 16)), dim3(256), 0, s, a.part,
                     groups, a.f.D, d_wq, d_wk);
  return hipGetLastError();
}

}  // namespace

int rope_grad_groups(int64_t T, int, int, int) {
  return static_cast<int>(std::min<int64_t>(ceil_div(T, kRopeWaves), 1024));
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
