// Log probabilities of given tokens with the entropy of the distribution and
// its best alternatives, in one reading of the logits, and their gradient:
//   z = scale cap tanh(l / cap)      (no cap: scale l)
//   logp = z - ln S,  S = sum exp(z),  entropy = ln S - sum z exp(z) / S
//   dl_j = z'(l_j) (g ([j = target] - p_j) - h p_j (logp_j + entropy))
// (logits capped by tanh at 30: "Reflection Beam", section "Hybrid Attention
// and Unusual Residuals".)
//
// A row is cut into pieces of at most 16,384 logits, which a workgroup holds in
// registers: the largest first (the cap keeps the order, so the raw logits are
// compared), then the sums relative to each thread's own largest, in base 2:
// S and sum (z - m) exp(z - m), which meet by rescaling.  Few rows get smaller
// pieces, so that they fill the card.  The alternatives are taken in turn: a
// wave's best by the largest value and the lowest index, after which the lane
// that held it looks for its next.  A second kernel joins a row's pieces.
// Bound by reading the logits (with the cap: by two exponentials and a
// reciprocal an element).
#include <algorithm>
#include <climits>

#include "serve.h"

namespace beam {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kChunk = kThreads * 8;   // logits of a workgroup's step
constexpr int kMaxSteps = 8;
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.0e38f;

typedef u32x4 u32x4_2 __attribute__((aligned(2)));
typedef u32x4 u32x4_4 __attribute__((aligned(4)));

// Eight logits of a row that starts anywhere; those past n are `none`.
template <typename IO>
__device__ __forceinline__ void load8(Eight<IO>& e, const IO* p, int64_t n) {
  using Word = std::conditional_t<sizeof(IO) == 2, u32x4_2, u32x4_4>;
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < e.kWords; ++i)
      e.w[i] = *reinterpret_cast<const Word*>(p + i * (8 / e.kWords));
    return;
  }
  constexpr uint32_t kNone = sizeof(IO) == 2 ? 0xFF80FF80u : 0xFF800000u;  // -infinity
#pragma unroll
  for (int i = 0; i < e.kWords; ++i) e.w[i] = u32x4{kNone, kNone, kNone, kNone};
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < n) {
      if constexpr (sizeof(IO) == 2) {
        const int sh = 16 * (j % 2);
        e.w[0][j / 2] = (e.w[0][j / 2] & ~(0xFFFFu << sh)) | static_cast<uint32_t>(p[j]) << sh;
      } else {
        e.w[j / 4][j % 4] = __float_as_uint(p[j]);
      }
    }
}
template <typename IO>
__device__ __forceinline__ void store8(const Eight<IO>& e, IO* p, int64_t n) {
  using Word = std::conditional_t<sizeof(IO) == 2, u32x4_2, u32x4_4>;
  if (n >= 8) {
#pragma unroll
    for (int i = 0; i < e.kWords; ++i)
      *reinterpret_cast<Word*>(p + i * (8 / e.kWords)) = e.w[i];
    return;
  }
#pragma unroll
  for (int j = 0; j < 7; ++j)
    if (j < n) {
      if constexpr (sizeof(IO) == 2) p[j] = static_cast<uint16_t>(e.w[0][j / 2] >> (16 * (j % 2)));
      else p[j] = __uint_as_float(e.w[j / 4][j % 4]);
    }
}
template <typename IO>
__device__ __forceinline__ float value(IO v) {
  if constexpr (sizeof(IO) == 2) return bf16_bits_to_f32(v);
  else return v;
}

// z in base 2, and with the cap r = 1 / (1 + e^(2 l / cap)): z = a (1 - 2 r),
// dz/dl = 4 r (1 - r) scale.
struct Cap {
  float a, b;  // no cap: z = b l;  cap: z = a - 2 a r, r of exp2(b l)
  bool on;
};
__host__ __device__ __forceinline__ Cap make_cap(float softcap, float scale) {
  Cap c;
  c.on = softcap > 0.0f;
  c.a = scale * softcap * kLog2E;
  c.b = c.on ? 2.0f * kLog2E / softcap : scale * kLog2E;
  return c;
}
template <bool CAP>
__device__ __forceinline__ float z_of(const Cap& c, float l, float& r) {
  if constexpr (!CAP) return c.b * l;
  r = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(c.b * l));
  return c.a - 2.0f * c.a * r;
}
__device__ __forceinline__ float z_of(const Cap& c, float l) {
  if (l == -INFINITY) return l;
  float r;
  return c.on ? z_of<true>(c, l, r) : z_of<false>(c, l, r);
}

// Sums relative to 2^m: s of 2^(z - m), w of (z - m) 2^(z - m).
struct Sums {
  float m, s, w;
};
__device__ __forceinline__ Sums meet(const Sums& x, const Sums& y) {
  Sums o;
  o.m = fmaxf(x.m, y.m);
  // (a side without logits has s and w 0 and any m)
  const float dx = fmaxf(x.m - o.m, -1e30f), dy = fmaxf(y.m - o.m, -1e30f);
  const float fx = __builtin_amdgcn_exp2f(dx), fy = __builtin_amdgcn_exp2f(dy);
  o.s = x.s * fx + y.s * fy;
  o.w = (x.w + dx * x.s) * fx + (y.w + dy * y.s) * fy;
  return o;
}
__device__ __forceinline__ Sums wave_meet(Sums v) {
#pragma unroll
  for (int i = 1; i < kWave; i *= 2) {
    const Sums o = {__shfl_xor(v.m, i), __shfl_xor(v.s, i), __shfl_xor(v.w, i)};
    v = meet(v, o);
  }
  return v;
}

// A candidate: the highest value, then the lowest index.  index INT_MAX: none.
struct Best {
  float v;
  int i;
};
__device__ __forceinline__ bool before(float v, int i, const Best& b) {
  return v > b.v || (v == b.v && i < b.i);
}
// The wave's best, in every lane.
__device__ __forceinline__ Best wave_best(const Best& mine) {
  Best b = mine;
#pragma unroll
  for (int i = 1; i < kWave; i *= 2) {
    const float v = __shfl_xor(b.v, i);
    const int x = __shfl_xor(b.i, i);
    if (before(v, x, b)) b = Best{v, x};
  }
  return b;
}
constexpr Best kNobody = {-INFINITY, INT_MAX};
// A NaN ranks first, so that a row's alternatives are always different tokens.
__device__ __forceinline__ float ranked(float v) { return v == v ? v : INFINITY; }

// The best `top` of the wave's lanes' candidates, one after another; next(last)
// gives the calling lane's best behind `last`.  Lane i keeps the i-th.
template <typename F>
__device__ __forceinline__ Best take_best(int top, Best mine, F next) {
  const int lane = threadIdx.x % kWave;
  Best kept = kNobody;
  for (int k = 0; k < top; ++k) {
    const Best b = wave_best(mine);
    if (lane == k) kept = b;
    if (b.i != INT_MAX && mine.i == b.i) mine = next(b);
  }
  return kept;
}

struct Shared {
  Sums sums[kWaves];
  Best best[kWaves][kMaxTop];
};
// The waves' sums and best meet in wave 0 (whose lanes i < top get the i-th best).
__device__ __forceinline__ void join(Shared& sh, int top, Sums& sums, Best& kept) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  sums = wave_meet(sums);
  if (lane == 0) sh.sums[wave] = sums;
  if (lane < top) sh.best[wave][lane] = kept;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int i = 1; i < kWaves; ++i) sums = meet(sums, sh.sums[i]);
  if (top == 0) return;
  Best mine = kNobody;
  if (lane % kMaxTop < top) mine = sh.best[lane / kMaxTop][lane % kMaxTop];
  kept = take_best(top, mine, [](const Best&) { return kNobody; });
}
static_assert(kWaves * kMaxTop == kWave, "one lane for each wave's candidate");

// A row's results, by wave 0.
template <typename IO>
__device__ __forceinline__ void finish(const ScoreArgs& a, const Cap& c, int64_t t,
                                       const Sums& u, const Best& kept) {
  const int lane = threadIdx.x % kWave;
  const bool none = u.s == 0.0f;  // every logit masked
  const float log2s = __log2f(u.s);
  const float lse2 = none ? -INFINITY : u.m + log2s;
  const IO* row = static_cast<const IO*>(a.logits) + t * a.stride;
  if (lane == 0) {
    a.lse[t] = lse2 * kLn2;
    a.entropy[t] = none ? 0.0f : (log2s - u.w / u.s) * kLn2;
    if (a.logprobs) {
      const int64_t x = a.targets[t];
      float lp = 0.0f;
      if (x >= 0 && x < a.V) {
        const float z = z_of(c, value(row[x]));
        lp = z == -INFINITY ? z : (z - lse2) * kLn2;
        if (u.s != u.s) lp = u.s;
      }
      a.logprobs[t] = lp;
    }
  }
  if (lane < a.top) {
    const float z = z_of(c, value(row[kept.i]));
    a.top_ids[t * a.top + lane] = kept.i;
    float lp = z == -INFINITY ? z : (z - lse2) * kLn2;
    if (u.s != u.s) lp = u.s;
    a.top_logprobs[t * a.top + lane] = lp;
  }
}

// A piece of a row: `len` logits, STEPS steps of the workgroup at most.
template <typename IO, int STEPS, bool CAP, bool TOP>
__global__ __launch_bounds__(kThreads) void score_pieces(ScoreArgs a, Cap c, int pieces, int len,
                                                          float* part) {
  __shared__ Shared sh;
  const int64_t t = blockIdx.x / pieces;
  const int piece = blockIdx.x % pieces;
  const int first = piece * len, end = min(first + len, a.V);
  const IO* row = static_cast<const IO*>(a.logits) + t * a.stride;
  const int base = first + static_cast<int>(threadIdx.x) * 8;
  Eight<IO> e[STEPS];
#pragma unroll
  for (int k = 0; k < STEPS; ++k) load8(e[k], row + base + k * kChunk, end - (base + k * kChunk));
  float top = -INFINITY;
#pragma unroll
  for (int k = 0; k < STEPS; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) top = fmaxf(top, e[k].get(j));
  Sums u;
  float r;
  top = fmaxf(top, kLowest);
  u.m = fmaxf(z_of<CAP>(c, top, r), kLowest);
  u.s = u.w = 0.0f;
#pragma unroll
  for (int k = 0; k < STEPS; ++k)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float l = e[k].get(j);
      if constexpr (CAP) {
        const float d = z_of<CAP>(c, l, r) - u.m;
        float p = __builtin_amdgcn_exp2f(d);
        p = l == -INFINITY ? 0.0f : p;
        u.w += p * d;
        u.s += p;
      } else {  // the difference first: exact for logits alike, however large
        const float d = c.b * (l - top), p = __builtin_amdgcn_exp2f(d);
        u.w += p * fmaxf(d, -160.0f);  // 0, not NaN, where p is 0
        u.s += p;
      }
    }
  Best kept = kNobody;
  if constexpr (TOP) {
    auto next = [&](const Best& last) {
      Best b = kNobody;
#pragma unroll
      for (int k = 0; k < STEPS; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = ranked(e[k].get(j));
          const int i = base + k * kChunk + j;
          if (i < end && before(v, i, b) && (v < last.v || (v == last.v && i > last.i)))
            b = Best{v, i};
        }
      return b;
    };
    kept = take_best(a.top, next(Best{INFINITY, -1}), next);
  }
  join(sh, TOP ? a.top : 0, u, kept);
  if (threadIdx.x >= kWave) return;
  if (pieces == 1) {
    finish<IO>(a, c, t, u, kept);
    return;
  }
  float* to = part + static_cast<int64_t>(blockIdx.x) * (4 + 2 * a.top);
  if (threadIdx.x == 0) {
    to[0] = u.m;
    to[1] = u.s;
    to[2] = u.w;
  }
  if (TOP && static_cast<int>(threadIdx.x) < a.top) {
    to[4 + threadIdx.x] = kept.v;
    to[4 + a.top + threadIdx.x] = __int_as_float(kept.i);
  }
}

// Joins a row's pieces.
template <typename IO>
__global__ __launch_bounds__(kThreads) void score_join(ScoreArgs a, Cap c, int pieces,
                                                        const float* part) {
  __shared__ Shared sh;
  const int64_t t = blockIdx.x;
  const int size = 4 + 2 * a.top;
  const float* row = part + t * pieces * size;
  Sums u = {kLowest, 0.0f, 0.0f};
  for (int i = threadIdx.x; i < pieces; i += kThreads) {
    const float* p = row + static_cast<int64_t>(i) * size;
    u = meet(u, Sums{p[0], p[1], p[2]});
  }
  Best kept = kNobody;
  if (a.top) {
    auto next = [&](const Best& last) {
      Best b = kNobody;
      for (int x = threadIdx.x; x < pieces * a.top; x += kThreads) {
        const float* p = row + static_cast<int64_t>(x / a.top) * size + 4 + x % a.top;
        const float v = p[0];
        const int i = __float_as_int(p[a.top]);
        if (i != INT_MAX && before(v, i, b) && (v < last.v || (v == last.v && i > last.i)))
          b = Best{v, i};
      }
      return b;
    };
    kept = take_best(a.top, next(Best{INFINITY, -1}), next);
  }
  join(sh, a.top, u, kept);
  if (threadIdx.x < kWave) finish<IO>(a, c, t, u, kept);
}

template <typename IO, bool CAP>
__global__ __launch_bounds__(kThreads) void score_backward(ScoreGradArgs a, Cap c, int pieces,
                                                            int len) {
  const int64_t t = blockIdx.x / pieces;
  const int first = blockIdx.x % pieces * len, end = min(first + len, a.V);
  const IO* row = static_cast<const IO*>(a.logits) + t * a.stride;
  IO* out = static_cast<IO*>(a.d_logits) + t * a.d_stride;
  const int64_t target = a.targets ? a.targets[t] : -1;
  const bool counts = target >= 0 && target < a.V;
  const float g = counts && a.d_logprobs ? a.d_logprobs[t] * a.scale : 0.0f;
  const float h = a.d_entropy ? a.d_entropy[t] * a.scale : 0.0f;
  const float lse2 = a.lse[t] * kLog2E;
  const float both = g + h * a.entropy[t], h2 = h * kLn2;
  const int at = counts ? static_cast<int>(target) : -1;
  for (int i = first + static_cast<int>(threadIdx.x) * 8; i < end; i += kChunk) {
    Eight<IO> e;
    load8(e, row + i, end - i);
    float d[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float l = e.get(j);
      float r;
      const float logp = fminf(fmaxf(z_of<CAP>(c, l, r) - lse2, -200.0f), 0.0f);
      const float p = __builtin_amdgcn_exp2f(logp);
      d[j] = -p * (both + h2 * logp);
    }
    if (at >= i && at < i + 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] += at == i + j ? g : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float l = e.get(j);
      if constexpr (CAP) {
        float r;
        z_of<CAP>(c, l, r);
        d[j] *= 4.0f * r * (1.0f - r);
      }
      d[j] = l == -INFINITY ? 0.0f : d[j];
    }
    e.set(d);
    store8(e, out + i, end - i);
  }
}

// Steps of a piece: 8, or fewer where that leaves the card empty.
int steps_for(int64_t T, int64_t V) {
  int steps = kMaxSteps;
  while (steps > 1 && T * ceil_div(V, int64_t{kChunk} * steps) < 1024) steps /= 2;
  return steps;
}
struct Cut {
  int pieces, len;
};
// Pieces of like length, a multiple of 8.
Cut cut(int64_t V, int steps) {
  Cut c;
  c.pieces = static_cast<int>(ceil_div(V, int64_t{kChunk} * steps));
  c.len = static_cast<int>(ceil_div(ceil_div(V, c.pieces), 8) * 8);
  return c;
}

template <typename IO, int STEPS, bool CAP>
void pieces_top(const ScoreArgs& a, const Cap& c, const Cut& k, float* part, hipStream_t s) {
  const dim3 grid(a.T * k.pieces), block(kThreads);
  if (a.top)
    hipLaunchKernelGGL((score_pieces<IO, STEPS, CAP, true>), grid, block, 0, s, a, c, k.pieces,
                       k.len, part);
  else
    hipLaunchKernelGGL((score_pieces<IO, STEPS, CAP, false>), grid, block, 0, s, a, c, k.pieces,
                       k.len, part);
}
template <typename IO, bool CAP>
void pieces_steps(const ScoreArgs& a, const Cap& c, int steps, const Cut& k, float* part,
                  hipStream_t s) {
  switch (steps) {
    case 1: return pieces_top<IO, 1, CAP>(a, c, k, part, s);
    case 2: return pieces_top<IO, 2, CAP>(a, c, k, part, s);
    case 4: return pieces_top<IO, 4, CAP>(a, c, k, part, s);
    default: return pieces_top<IO, 8, CAP>(a, c, k, part, s);
  }
}

template <typename IO>
hipError_t forward(const ScoreArgs& a, float* part, hipStream_t s) {
  const Cap c = make_cap(a.softcap, a.scale);
  const int steps = steps_for(a.T, a.V);
  const Cut k = cut(a.V, steps);
  if (c.on) pieces_steps<IO, true>(a, c, steps, k, part, s);
  else pieces_steps<IO, false>(a, c, steps, k, part, s);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || k.pieces == 1) return e;
  hipLaunchKernelGGL((score_join<IO>), dim3(a.T), dim3(kThreads), 0, s, a, c, k.pieces, part);
  return hipGetLastError();
}

template <typename IO>
hipError_t backward(const ScoreGradArgs& a, hipStream_t s) {
  const Cap c = make_cap(a.softcap, a.scale);
  const Cut k = cut(a.V, steps_for(a.T, a.V));
  const dim3 grid(a.T * k.pieces), block(kThreads);
  if (c.on)
    hipLaunchKernelGGL((score_backward<IO, true>), grid, block, 0, s, a, c, k.pieces, k.len);
  else
    hipLaunchKernelGGL((score_backward<IO, false>), grid, block, 0, s, a, c, k.pieces, k.len);
  return hipGetLastError();
}

}  // namespace

int64_t score_pieces_count(int64_t T, int64_t V) { return T * cut(V, steps_for(T, V)).pieces; }

size_t score_workspace(int64_t T, int64_t V, int top) {
  const int64_t n = score_pieces_count(T, V);
  return n == T ? 0 : static_cast<size_t>(n) * (4 + 2 * top) * sizeof(float);
}

hipError_t launch_token_logprobs(const ScoreArgs& a, int32_t dtype, void* ws, hipStream_t s) {
  float* part = static_cast<float*>(ws);
  return dtype == BEAM_BF16 ? forward<uint16_t>(a, part, s) : forward<float>(a, part, s);
}

hipError_t launch_token_logprobs_backward(const ScoreGradArgs& a, int32_t dtype, hipStream_t s) {
  return dtype == BEAM_BF16 ? backward<uint16_t>(a, s) : backward<float>(a, s);
}

}  // namespace beam
