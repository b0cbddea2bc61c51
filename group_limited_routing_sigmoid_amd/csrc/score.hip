// Log probabilities of given tokens with the entropy of the distribution and
// its best alternatives, in one reading of the logits (ordinary ones), and their
// gradient:
//   z = scale cap tanh(l / cap)      (no cap: scale l)
//   logp = z - ln S,  S = sum exp(z),  entropy = ln S - sum z exp(z) / S
//   dl_j = z'(l_j) (g ([j = target] - p_j) - h p_j (logp_j + entropy))
// (logits capped by tanh at 30: "Reflection Releases Beam ...", section "Hybrid
// Attention and Unusual Residuals".)
//
// A row is cut into pieces, more of them for few rows, so that they fill the
// card.  Without alternatives a workgroup runs through its piece with the sums
// relative to each thread's largest logit so far, in base 2: S and sum (z - m)
// exp(z - m), which meet by rescaling; under a cap of ordinary size, whose z
// binary32's exponentials hold as they are, m is 0.  With alternatives the piece,
// of at most 16,384 logits, is held in registers (the cap keeps the order, so the
// raw logits are compared): the n-th largest of a wave's lanes' largest is a bar
// that at least n logits reach and few more, those meet in LDS, and each finds its
// rank by counting (2,048 x 131,072 bf16 with 16: 201 us, 5: 142, none: 100; one
// after another by the wave's largest 562 and 240).  A wave whose lanes with any
// unmasked logit are fewer than the alternatives has no bar, and one with more than
// 64 equal logits at it no room: those read their logits again for each alternative
// (50 scattered words a row of the same shape, 16 alternatives: 3.6 ms).  A second
// kernel joins a row's pieces.  Bound by reading the logits; with the cap by two
// exponentials and a reciprocal an element as much (4,096 x 100,003 bf16: 165 us among
// many calls, 5.0 TB/s, 195 to 238 among the first few, as the clock holds; without a
// cap 148; the gradient 311, 5.3 TB/s).
#include <algorithm>
#include <cfloat>

#include "serve.h"

namespace beam {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kChunk = kThreads * 8;   // logits of a workgroup's step
constexpr int kMaxSteps = 8;
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

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
// Rows start anywhere.  What runs through them steps in whole 16 bytes of memory
// (4,096 x 100,003 bf16, capped: 166 us, 100,000 164), so that its first and last
// eight may lie over the row's ends: `skew` is how many values the row starts behind
// such a place.
template <typename IO>
__device__ __forceinline__ int skew_of(const IO* row) {
  return static_cast<int>(reinterpret_cast<uintptr_t>(row) % 16 / sizeof(IO));
}
// Eight logits from i on, of which those outside [0, V) are masked ones.
template <typename IO>
__device__ __forceinline__ void load_over(Eight<IO>& e, const IO* row, int i, int V) {
  if (i >= 0) return load8(e, row + i, V - i);
  load8(e, row, 0);
#pragma unroll
  for (int j = 1; j < 8; ++j)
    if (i + j >= 0 && i + j < V) {
      if constexpr (sizeof(IO) == 2) {
        const int sh = 16 * (j % 2);
        e.w[0][j / 2] = (e.w[0][j / 2] & ~(0xFFFFu << sh)) | static_cast<uint32_t>(row[i + j]) << sh;
      } else {
        e.w[j / 4][j % 4] = __float_as_uint(row[i + j]);
      }
    }
}
template <typename IO>
__device__ __forceinline__ void store_over(const Eight<IO>& e, IO* row, int i, int V) {
  if (i >= 0) return store8(e, row + i, V - i);
#pragma unroll
  for (int j = 1; j < 8; ++j)
    if (i + j >= 0 && i + j < V) {
      if constexpr (sizeof(IO) == 2) row[i + j] = static_cast<uint16_t>(e.w[0][j / 2] >> (16 * (j % 2)));
      else row[i + j] = __uint_as_float(e.w[j / 4][j % 4]);
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
  float a, b;  // no cap: z = b l;  cap: r of exp2(b l)
  float scale;
  float unit;  // of Sums::m in base 2
  float near;  // logits below it have a series (tanh_series)
  bool on;
};
__host__ __device__ __forceinline__ Cap make_cap(float softcap, float scale) {
  Cap c;
  c.on = softcap > 0.0f;
  c.scale = scale;
  c.a = scale * softcap * kLog2E;
  c.b = c.on ? 2.0f * kLog2E / softcap : scale * kLog2E;
  c.unit = c.on ? 1.0f : c.b;
  c.near = 1.0f / c.b;
  return c;
}
// How z is made: without a cap, with one, and with one small enough that 2^z and
// its sums need no maximum (a z of 2^24 logits, 96 2^96 2^24 at most) and that 1 - 2 r
// has bits enough.
enum Form { kPlain, kCapped, kSmall };
constexpr float kSmallCap = 96.0f;
Form form_of(const Cap& c) { return !c.on ? kPlain : c.a <= kSmallCap ? kSmall : kCapped; }

__device__ __forceinline__ float r_of(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x));
}
// tanh(u) by its series to u^11 where |u| <= 0.35 (2^-26 of itself is left out), u = x
// ln 2 / 2 of an exponent |x| < 1 in base 2.
__device__ __forceinline__ float tanh_series(float x) {
  const float u = x * (0.5f * kLn2), q = u * u;
  float p = __builtin_fmaf(q, -1382.0f / 155925.0f, 62.0f / 2835.0f);
  p = __builtin_fmaf(q, p, -17.0f / 315.0f);
  p = __builtin_fmaf(q, p, 2.0f / 15.0f);
  p = __builtin_fmaf(q, p, -1.0f / 3.0f);
  return __builtin_fmaf(q * u, p, u);
}
// A capped z in base 2.  1 - 2 r cancels where r is near a half, which leaves 16 2^-24
// of the cap: under a small one less than the sums' own errors.  Past it logits below
// 0.35 caps take the series, the others r of |l|: 20 2^-24 of z itself.  Where a wave
// has only the former, as under a cap far above its logits, the latter is not
// worked out (NEAR).  4,096 x 100,003 bf16 of deviation 4: caps of 30 and 50 178 and
// 161 us, of 80 and 1,000 238 and 233 (a small one's way 196), a z of 2.5 times a cap
// of 30, in whose every wave some need r, 361; gradients 311, 310, 325, 329 and 435.
template <Form F, bool NEAR = false>
__device__ __forceinline__ float capped(const Cap& c, float l) {
  const float x = c.b * l;
  if constexpr (F == kSmall) return c.a - 2.0f * c.a * r_of(x);
  const float near = c.a * tanh_series(x);
  if constexpr (NEAR) return near;
  const float far = __builtin_copysignf(c.a - 2.0f * c.a * r_of(fabsf(x)), x);
  return fabsf(l) < c.near ? near : far;
}
// Whether none of the wave's logits needs more than the series (masked ones, infinite
// ones and NaNs need no z).
template <typename IO>
__device__ __forceinline__ bool all_near(const Cap& c, const Eight<IO>& e) {
  const uint32_t from = __float_as_uint(c.near);
  uint32_t least = 0xFFFFFFFFu;
#pragma unroll
  for (int j = 0; j < 8; ++j) least = min(least, (__float_as_uint(e.get(j)) & 0x7FFFFFFFu) - from);
  return !__any(least < 0x7F800000u - from);
}
// z - m in nats, of a logit and what sums are relative to.  Without a cap the
// difference of the logits comes first: it has a scaled value where the lowest
// logit itself has none.
__device__ __forceinline__ float z_from(const Cap& c, float l, float m) {
  if (l == -INFINITY) return l;  // masked
  if (!c.on) return c.scale * (l - m);
  return ((c.a <= kSmallCap ? capped<kSmall>(c, l) : capped<kCapped>(c, l)) - m) * kLn2;
}
// Times a logit: at most 5e-7 of a finite one, an infinite one all the same.
constexpr float kTrace = 0x1p-149f;

// Sums relative to m, a logit without a cap, else a z in base 2: with d = z - z(m)
// in base 2, s of 2^d, w of d 2^d.
struct Sums {
  float m, s, w;
};
// In base 2, and finite, so that it times 0 is 0.
__device__ __forceinline__ float apart(const Cap& c, float m, float to) {
  return fmaxf((m - to) * c.unit, -1e30f);
}
__device__ __forceinline__ Sums meet(const Cap& c, const Sums& x, const Sums& y) {
  Sums o;
  o.m = fmaxf(x.m, y.m);
  // (a side without logits has s and w 0 and any m)
  const float dx = apart(c, x.m, o.m), dy = apart(c, y.m, o.m);
  const float fx = __builtin_amdgcn_exp2f(dx), fy = __builtin_amdgcn_exp2f(dy);
  o.s = x.s * fx + y.s * fy;
  o.w = (x.w + dx * x.s) * fx + (y.w + dy * y.s) * fy;
  return o;
}

// ln sum exp(z) of sums whose s has the logarithm ln_s, held to binary32's range.
__device__ __forceinline__ float lse_of(const Cap& c, float m, float ln_s) {
  return (c.on ? m * kLn2 : fminf(fmaxf(c.scale * m, -FLT_MAX), FLT_MAX)) + ln_s;
}

// Reductions over the wave by data-parallel moves; the result in every lane.
template <typename F>
__device__ __forceinline__ float wave_reduce(float v, F f) {
#define BEAM_STEP(ctrl, rows)                                                                \
  v = f(v, __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(v), __float_as_int(v), \
                                                      ctrl, rows, 0xF, false)))
  BEAM_STEP(0xB1, 0xF);   // neighbours, pairs, halves of 8, of 16
  BEAM_STEP(0x4E, 0xF);
  BEAM_STEP(0x141, 0xF);
  BEAM_STEP(0x140, 0xF);
#undef BEAM_STEP
  const float a = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0)),
              b = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16)),
              c = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32)),
              d = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
  return f(f(a, b), f(c, d));
}
__device__ __forceinline__ float wave_max(float v) {
  return wave_reduce(v, [](float x, float y) { return fmaxf(x, y); });
}
__device__ __forceinline__ float wave_sum(float v) {
  return wave_reduce(v, [](float x, float y) { return x + y; });
}
// Indexes below 2^24 as binary32 are exact, and so is their order.
__device__ __forceinline__ int wave_min(int v) {
  return static_cast<int>(-wave_max(-static_cast<float>(v)));
}
__device__ __forceinline__ Sums wave_meet(const Cap& c, const Sums& v) {
  Sums o;
  o.m = wave_max(v.m);
  const float d = apart(c, v.m, o.m), f = __builtin_amdgcn_exp2f(d);
  o.s = wave_sum(v.s * f);
  o.w = wave_sum((v.w + d * v.s) * f);
  return o;
}

// A candidate: the highest value, then the lowest index.
constexpr int kNoIndex = 1 << 24;
struct Best {
  float v;
  int i;  // kNoIndex: none
};
constexpr Best kNobody = {-INFINITY, kNoIndex};
// The wave's best, in every lane.
__device__ __forceinline__ Best wave_best(const Best& mine) {
  Best b;
  b.v = wave_max(mine.v);
  b.i = wave_min(mine.v == b.v ? mine.i : kNoIndex);
  return b;
}
// Whether (v, i) ranks behind `last`.
__device__ __forceinline__ bool behind(float v, int i, const Best& last) {
  return v < last.v || (v == last.v && i > last.i);
}

// The best `top` of c candidates in LDS, one a lane, by counting those before each;
// lane i gets the i-th.  One wave's.
__device__ __forceinline__ Best by_rank(Best* list, int c, int top) {
  const int lane = threadIdx.x % kWave;
  const Best mine = lane < c ? list[lane] : kNobody;
  int rank = 0;
  for (int j = 0; j < c; ++j) {
    const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mine.v), j));
    const int i = __builtin_amdgcn_readlane(mine.i, j);
    rank += v > mine.v || (v == mine.v && i < mine.i);
  }
  wave_order();
  if (lane < c && rank < top) list[rank] = mine;
  wave_order();
  return lane < min(top, c) ? list[lane] : kNobody;
}

struct Shared {
  Sums sums[kWaves];
  Best best[kWaves * kMaxTop];
  Best found[kWaves][kWave];  // a wave's candidates
  int many[kWaves];
};
// The waves' sums and best meet in wave 0, whose lanes i < top get the i-th best.
__device__ __forceinline__ void join(Shared& sh, const Cap& c, int top, Sums& sums, Best& kept) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  sums = wave_meet(c, sums);
  if (lane == 0) sh.sums[wave] = sums;
  if (lane < top) sh.best[wave * top + lane] = kept;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int i = 1; i < kWaves; ++i) sums = meet(c, sums, sh.sums[i]);
  if (top == 0) return;
  // (a wave's nobodies are no candidates)
  Best mine = lane < kWaves * top ? sh.best[lane] : kNobody;
  const uint64_t some = __ballot(mine.i != kNoIndex);
  const int at = __popcll(some & ((uint64_t{1} << lane) - 1));
  wave_order();
  if (mine.i != kNoIndex) sh.best[at] = mine;
  wave_order();
  kept = by_rank(sh.best, __popcll(some), top);
}
static_assert(kWaves * kMaxTop == kWave, "one lane for each wave's candidate");

// A row's target and its logit, read ahead of what they meet.
struct Target {
  float l;
  bool counts;
};
template <typename IO>
__device__ __forceinline__ Target target_of(const ScoreArgs& a, int64_t t) {
  Target g = {0.0f, false};
  if (!a.logprobs) return g;
  const int64_t x = a.targets[t];
  g.counts = x >= 0 && x < a.V;
  if (g.counts) g.l = value(static_cast<const IO*>(a.logits)[t * a.stride + x]);
  return g;
}
// A row's results, by wave 0.
template <typename IO>
__device__ __forceinline__ void finish(const ScoreArgs& a, const Cap& c, int64_t t,
                                       const Sums& u, const Best& kept, const Target& g) {
  const int lane = threadIdx.x % kWave;
  const bool none = u.s == 0.0f;      // every logit masked
  const bool bad = !(u.s <= FLT_MAX);  // a NaN or +infinity among them
  const float log2s = bad ? NAN : __log2f(u.s), lns = log2s * kLn2;
  auto logp = [&](float l) {
    const float d = z_from(c, l, u.m);
    return d == -INFINITY && !bad ? d : d - lns;
  };
  if (lane == 0) {
    a.lse[t] = none ? -INFINITY : lse_of(c, u.m, lns);
    a.entropy[t] = none ? 0.0f : (log2s - u.w / u.s) * kLn2;
    if (a.logprobs) a.logprobs[t] = g.counts ? logp(g.l) : 0.0f;
  }
  if (a.top == 0) return;
  // where NaNs leave too few, the first tokens stand in, so that they differ
  const bool few = __any(lane < a.top && kept.i == kNoIndex);
  if (lane < a.top) {
    a.top_ids[t * a.top + lane] = few ? lane : kept.i;
    a.top_logprobs[t * a.top + lane] = few ? NAN : logp(kept.v);
  }
}

// What a thread's sums are relative to: a logit, and under a large cap its z (base
// 2).  kSmall: to 0, and w is a sum of r.
struct Ref {
  float l, z;
};
template <Form F>
__device__ __forceinline__ Ref ref_of(const Cap& c, float l) {
  Ref r = {fmaxf(l, -FLT_MAX), 0.0f};
  if constexpr (F == kCapped) r.z = capped<kCapped>(c, r.l);
  return r;
}
template <Form F, bool NEAR>
__device__ __forceinline__ void add(const Cap& c, float l, const Ref& ref, float& s, float& w) {
  if constexpr (F == kPlain) {
    // the difference first: exact for logits alike, however large
    const float d = c.b * (l - ref.l), p = __builtin_amdgcn_exp2f(d);
    s += p;
    w += p * fmaxf(d, -160.0f);  // 0, not NaN, where p is 0
  } else if constexpr (F == kCapped) {
    // (not past the largest logit's by its rounding, which 2^d would not hold under a
    // very large cap; 0 for the NaN of an infinity's series)
    const float d = fminf(capped<F, NEAR>(c, l) - ref.z, 0.0f);
    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(l, kTrace, d));
    s += p;
    w += p * d;
  } else {
    const float r = r_of(c.b * l);
    const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(-2.0f * c.a, r, __builtin_fmaf(l, kTrace, c.a)));
    s += p;
    w += p * r;
  }
}
template <Form F, typename IO>
__device__ __forceinline__ void add8(const Cap& c, const Eight<IO>& e, const Ref& ref, float& s, float& w) {
  if (F == kCapped && all_near(c, e)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) add<F, true>(c, e.get(j), ref, s, w);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) add<F, false>(c, e.get(j), ref, s, w);
  }
}
template <Form F>
__device__ __forceinline__ Sums sums_of(const Cap& c, const Ref& ref, float s, float w) {
  if constexpr (F == kPlain) return Sums{ref.l, s, w};
  else if constexpr (F == kCapped) return Sums{ref.z, s, w};
  else return Sums{0.0f, s, c.a * s - 2.0f * c.a * w};
}

// Workspace: four floats of sums for each piece of each row, then the pieces'
// best, `top` each.
__device__ __forceinline__ void put_sums(float* part, int64_t i, const Sums& u) {
  *reinterpret_cast<f32x4*>(part + 4 * i) = f32x4{u.m, u.s, u.w, 0.0f};
}
__device__ __forceinline__ Best* best_of(float* part, int64_t T, int pieces, int64_t i, int top) {
  return reinterpret_cast<Best*>(part + 4 * T * pieces) + i * top;
}

// The thread's sums of a row's logits [first, end), read as it goes, the next ones
// ahead; first is a place of whole 16 bytes.
template <Form F, typename IO>
__device__ __forceinline__ Sums run_through(const Cap& c, const IO* row, int first, int end) {
  Ref ref = ref_of<F>(c, -FLT_MAX);
  float s = 0.0f, w = 0.0f;
  auto use = [&](const Eight<IO>& e) {
    if constexpr (F != kSmall) {
      float top = e.get(0);
#pragma unroll
      for (int j = 1; j < 8; ++j) top = fmaxf(top, e.get(j));
      if (top > ref.l) {  // raise the maximum
        const Ref to = ref_of<F>(c, top);
        const float d = fmaxf(F == kPlain ? c.b * (ref.l - to.l) : ref.z - to.z, -1e30f);
        const float f = __builtin_amdgcn_exp2f(d);
        w = (w + d * s) * f;
        s *= f;
        ref = to;
      }
    }
    add8<F>(c, e, ref, s, w);
  };
  // the step over the row's start; whole ones, four at a time; what is left
  const int in = static_cast<int>(threadIdx.x) * 8;
  int i = first;
  auto step = [&] {
    Eight<IO> e;
    load_over(e, row, i + in, end);
    use(e);
    i += kChunk;
  };
  if (i < 0) step();
  constexpr int kAhead = 4;
  for (; i + kAhead * kChunk <= end; i += kAhead * kChunk) {
    Eight<IO> e[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) e[u].load(row + i + in + u * kChunk);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) use(e[u]);
  }
  while (i < end) step();
  return sums_of<F>(c, ref, s, w);
}

// Sums of a piece of a row.
template <typename IO, Form F>
__global__ __launch_bounds__(kThreads) void score_sums(ScoreArgs a, Cap c, int pieces, int len,
                                                        float* part) {
  __shared__ Shared sh;
  const int64_t t = blockIdx.x / pieces;
  const IO* row = static_cast<const IO*>(a.logits) + t * a.stride;
  const int first = static_cast<int>(blockIdx.x % pieces) * len - skew_of(row);
  Sums u = run_through<F>(c, row, first, min(first + len, a.V));
  Best kept = kNobody;
  join(sh, c, 0, u, kept);
  if (threadIdx.x >= kWave) return;
  if (pieces == 1) finish<IO>(a, c, t, u, kept, target_of<IO>(a, t));
  else if (threadIdx.x == 0) put_sums(part, blockIdx.x, u);
}

// Sums and the best `top` of a piece of a row of `len` logits, STEPS steps of the
// workgroup at most, held in registers.
template <typename IO, int STEPS, Form F>
__global__ __launch_bounds__(kThreads) void score_top(ScoreArgs a, Cap c, int pieces, int len,
                                                       float* part) {
  __shared__ Shared sh;
  const int64_t t = blockIdx.x / pieces;
  const int first = blockIdx.x % pieces * len, end = min(first + len, a.V);
  const IO* row = static_cast<const IO*>(a.logits) + t * a.stride;
  const int base = first + static_cast<int>(threadIdx.x) * 8, lane = threadIdx.x % kWave;
  Eight<IO> e[STEPS];
#pragma unroll
  for (int k = 0; k < STEPS; ++k) load8(e[k], row + base + k * kChunk, end - (base + k * kChunk));
  float most[STEPS], all = -INFINITY;  // of each eight, of the lane
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    most[k] = e[k].get(0);
#pragma unroll
    for (int j = 1; j < 8; ++j) most[k] = fmaxf(most[k], e[k].get(j));
    all = fmaxf(all, most[k]);
  }
  const Ref ref = ref_of<F>(c, all);
  float s = 0.0f, w = 0.0f;
#pragma unroll
  for (int k = 0; k < STEPS; ++k) {
    e[k].repack();
    add8<F>(c, e[k], ref, s, w);
    e[k].repack();
  }
  // The top-th largest of the lanes' largest: at least `top` logits reach it, and
  // seldom many more.  Those meet in LDS.
  const int wave = threadIdx.x / kWave;
  const float highest = wave_max(all);
  float bar = highest, rest = all;
  for (int x = 0, reach = 0; x < a.top && reach < a.top; ++x) {
    if (x) bar = wave_max(rest);
    reach += __popcll(__ballot(rest == bar));
    if (rest == bar) rest = -INFINITY;
  }
  int found = kWave + 1;
  if (first + wave * kWave * 8 >= end) {
    found = 0;  // no logit is the wave's
  } else if (bar > -INFINITY) {
    if (lane == 0) sh.many[wave] = 0;
    wave_order();
#pragma unroll
    for (int k = 0; k < STEPS; ++k)
      if (most[k] >= bar)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = e[k].get(j);
          if (v >= bar) {
            const int at = atomicAdd(&sh.many[wave], 1);
            if (at < kWave) sh.found[wave][at] = Best{v, base + k * kChunk + j};
          }
        }
    wave_order();
    found = __builtin_amdgcn_readfirstlane(sh.many[wave]);
  }
  Best kept = kNobody;
  if (found <= kWave) {
    kept = by_rank(sh.found[wave], found, a.top);
  } else if (highest == -INFINITY) {
    // all masked: the first ones
    const int i = first + wave * kWave * 8 + lane;
    if (lane < a.top && i < end) kept = Best{-INFINITY, i};
  } else {
    // logits alike in their hundreds, or masked ones among the best: one after
    // another, each lane's next by reading its logits again
    Best last = {INFINITY, -1};
    for (int x = 0; x < a.top; ++x) {
      Best mine = kNobody;
      for (int k = 0; k < STEPS; ++k) {
        const int i0 = base + k * kChunk;
        for (int i = i0; i < min(i0 + 8, end); ++i) {
          const float v = value(row[i]);
          if (behind(v, i, last) && (v > mine.v || mine.i == kNoIndex)) mine = Best{v, i};
        }
      }
      last = wave_best(mine);
      if (lane == x) kept = last;
    }
  }
  Sums u = sums_of<F>(c, ref, s, w);
  join(sh, c, a.top, u, kept);
  if (threadIdx.x >= kWave) return;
  if (pieces == 1) {
    finish<IO>(a, c, t, u, kept, target_of<IO>(a, t));
    return;
  }
  if (lane == 0) put_sums(part, blockIdx.x, u);
  if (lane < a.top) best_of(part, a.T, pieces, blockIdx.x, a.top)[lane] = kept;
}

// Joins a row's pieces.  Each piece's best are in order: a thread stands at the
// first one of its piece that is not taken yet, all of them in LDS (`staged` of
// them; 0: there are more pieces than threads, and each looks through its own).
template <typename IO>
__global__ __launch_bounds__(kThreads) void score_join(ScoreArgs a, Cap c, int pieces,
                                                        float* part, int staged) {
  __shared__ Shared sh;
  extern __shared__ Best all[];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x % kWave;
  const Best* best = best_of(part, a.T, pieces, t * pieces, a.top);
#pragma unroll 4
  for (int x = threadIdx.x; x < staged; x += kThreads) all[x] = best[x];
  Sums u = {-FLT_MAX, 0.0f, 0.0f};
  for (int i = threadIdx.x; i < pieces; i += kThreads) {
    const f32x4 p = *reinterpret_cast<const f32x4*>(part + 4 * (t * pieces + i));
    u = meet(c, u, Sums{p[0], p[1], p[2]});
  }
  const Target g = target_of<IO>(a, t);
  Best kept = kNobody;
  if (a.top) {
    __syncthreads();
    int at = threadIdx.x * a.top;
    const int stop = min(at + a.top, staged);
    auto first = [&](const Best& last) {
      Best b = kNobody;
      if (staged) return at < stop ? all[at] : b;
      for (int i = threadIdx.x; i < pieces; i += kThreads)
        for (int x = 0; x < a.top; ++x) {
          const Best y = best[i * a.top + x];
          if (!behind(y.v, y.i, last)) continue;
          if (y.v > b.v || (y.v == b.v && y.i < b.i)) b = y;
          break;
        }
      return b;
    };
    Best mine = first(Best{INFINITY, -1});
    // (a wave without a piece has nobody)
    const int rounds = threadIdx.x - lane < pieces ? a.top : 0;
    for (int k = 0; k < rounds; ++k) {
      const Best b = wave_best(mine);
      if (lane == k) kept = b;
      if (mine.i == b.i && b.i != kNoIndex) {
        ++at;
        mine = first(b);
      }
    }
  }
  // with pieces in one wave alone, its best are the row's
  join(sh, c, pieces > kWave ? a.top : 0, u, kept);
  if (threadIdx.x < kWave) finish<IO>(a, c, t, u, kept, g);
}

// p comes from z and lse, which is the logits' sum and their size in one binary32
// number: past kFar its rounding alone moves every p of the row by 2^-17 and more, and
// a row of the type's lowest value has no ln S left.  Such a row is its first
// piece's workgroup's alone, which forms its largest logit and the sum beside it once
// more before anything is written (in the logits' place, too), and takes them if they
// make the given lse up to two steps: one of more words than the row's, as a shard of
// a vocabulary has, stays as it is.  4,096 x 100,003 bf16:
// 315 us, all rows far 534; 1 x 100,003 12.4 and 26.5.
constexpr float kFar = 128.0f;
template <typename IO, Form F>
__global__ __launch_bounds__(kThreads) void score_backward(ScoreGradArgs a, Cap c, int pieces,
                                                            int len) {
  const int64_t t = blockIdx.x / pieces;
  const IO* row = static_cast<const IO*>(a.logits) + t * a.stride;
  const int skew = skew_of(row), from = blockIdx.x % pieces * len;
  int first = from - skew, end = min(first + len, a.V);
  IO* out = static_cast<IO*>(a.d_logits) + t * a.d_stride;
  const int64_t target = a.targets ? a.targets[t] : -1;
  const bool counts = target >= 0 && target < a.V;
  const float g = counts && a.d_logprobs ? a.d_logprobs[t] * a.scale : 0.0f;
  const float h = a.d_entropy ? a.d_entropy[t] * a.scale : 0.0f;
  const float given = a.lse[t], lse = given == -INFINITY ? 0.0f : given;  // (all masked: p is 0)
  // ln p is z less two numbers: 0 and lse, or the largest z and ln S (kCapped in base 2,
  // kPlain with the largest logit)
  float most = 0.0f, log_sum = F == kPlain ? lse : lse * kLog2E;
  if constexpr (F != kSmall) {
    if (fabsf(lse) >= kFar) {
      if (from) return;
      __shared__ Sums waves[kWaves];
      first = -skew;
      end = a.V;
      const Sums mine = wave_meet(c, run_through<F>(c, row, first, end));
      if (threadIdx.x % kWave == 0) waves[threadIdx.x / kWave] = mine;
      __syncthreads();
      Sums u = waves[0];
#pragma unroll
      for (int i = 1; i < kWaves; ++i) u = meet(c, u, waves[i]);
      const float log2s = __log2f(u.s);
      if (fabsf(lse_of(c, u.m, log2s * kLn2) - lse) <= fabsf(lse) * 0x1p-22f) {
        most = u.m;
        log_sum = F == kPlain ? log2s * kLn2 : log2s;
      }
    }
  }
  const float both = -(g + h * a.entropy[t]), h2 = -h * kLn2;
  const int at = counts ? static_cast<int>(target) : -1;
  // a logit's gradient, in which the target's own g is missing; q: z'
  auto gradient = [&](auto near, float l, float& q) {
    if constexpr (F == kSmall) {
      const float r = r_of(c.b * l), r4 = 4.0f * r;
      const float logp = __builtin_fmaf(-2.0f * c.a, r, c.a - log_sum);
      const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(l, kTrace, logp));
      q = __builtin_fmaf(-r4, r, r4);
      return p * __builtin_fmaf(h2, logp, both) * q;
    } else if constexpr (F == kCapped) {
      // as capped, with z' of the same terms
      const float x = c.b * l, t = tanh_series(x);
      float z = c.a * t;
      q = __builtin_fmaf(-t, t, 1.0f);
      if constexpr (!decltype(near)::value) {
        const float r = r_of(fabsf(x)), r4 = 4.0f * r;
        const float far = __builtin_copysignf(c.a - 2.0f * c.a * r, x), far_q = __builtin_fmaf(-r4, r, r4);
        const bool low = fabsf(l) < c.near;
        z = low ? z : far;
        q = low ? q : far_q;
      }
      const float logp = fminf(z - most - log_sum, 0.0f);
      const float p = __builtin_amdgcn_exp2f(__builtin_fmaf(l, kTrace, logp));
      q = l == -INFINITY ? 0.0f : q;
      return p * __builtin_fmaf(h2, logp, both) * q;
    } else {
      q = 1.0f;
      const float d = __builtin_fmaf(c.scale, l - most, -log_sum);
      const float logp = fminf(fmaxf(d * kLog2E, -200.0f), 0.0f);
      return __builtin_amdgcn_exp2f(logp) * __builtin_fmaf(h2, logp, both);
    }
  };
  auto use = [&](Eight<IO>& e, int i) {
    float d[8], q;
    if (F == kCapped && all_near(c, e)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = gradient(std::true_type(), e.get(j), q);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = gradient(std::false_type(), e.get(j), q);
    }
    if (at >= i && at < i + 8) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at == i + j && e.get(j) != -INFINITY) {
          gradient(std::false_type(), e.get(j), q);
          d[j] += g * q;
        }
    }
    e.set(d);
  };
  const int in = static_cast<int>(threadIdx.x) * 8;
  int i = first;
  auto step = [&] {
    Eight<IO> e;
    load_over(e, row, i + in, end);
    use(e, i + in);
    store_over(e, out, i + in, end);
    i += kChunk;
  };
  if (i < 0) step();
  constexpr int kAhead = 2;
  for (; i + kAhead * kChunk <= end; i += kAhead * kChunk) {
    Eight<IO> e[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) e[u].load(row + i + in + u * kChunk);
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      use(e[u], i + in + u * kChunk);
      store8(e[u], out + i + in + u * kChunk, 8);
    }
  }
  while (i < end) step();
}

// Steps of a piece: `most`, or fewer where that leaves the card empty.
int steps_for(int64_t T, int64_t V, int most) {
  int steps = most;
  while (steps > 1 && T * ceil_div(V, int64_t{kChunk} * steps) < 1024) steps /= 2;
  return steps;
}
// Without alternatives a piece is as long as fills the card.
constexpr int kLongSteps = 1 << 13;
int most_steps(int top) { return top ? kMaxSteps : kLongSteps; }
struct Cut {
  int pieces, len;
};
// Pieces of like length, a multiple of 8; `over`: values that a row's first eight
// may start before it.
Cut cut(int64_t V, int steps, int over) {
  Cut c;
  c.pieces = static_cast<int>(ceil_div(V, int64_t{kChunk} * steps));
  c.len = static_cast<int>(ceil_div(ceil_div(V + over, c.pieces), 8) * 8);
  return c;
}

template <typename IO, Form F>
void pieces(const ScoreArgs& a, const Cap& c, int steps, const Cut& k, float* part, hipStream_t s) {
  const dim3 grid(a.T * k.pieces), block(kThreads);
#define BEAM_TOP(n) \
  hipLaunchKernelGGL((score_top<IO, n, F>), grid, block, 0, s, a, c, k.pieces, k.len, part)
  if (!a.top)
    hipLaunchKernelGGL((score_sums<IO, F>), grid, block, 0, s, a, c, k.pieces, k.len, part);
  else if (steps == 1) BEAM_TOP(1);
  else if (steps == 2) BEAM_TOP(2);
  else if (steps == 4) BEAM_TOP(4);
  else BEAM_TOP(8);
#undef BEAM_TOP
}

template <typename IO>
hipError_t forward(const ScoreArgs& a, float* part, hipStream_t s) {
  const Cap c = make_cap(a.softcap, a.scale);
  const int steps = steps_for(a.T, a.V, most_steps(a.top));
  const Cut k = cut(a.V, steps, a.top ? 0 : 7);
  switch (form_of(c)) {
    case kPlain: pieces<IO, kPlain>(a, c, steps, k, part, s); break;
    case kCapped: pieces<IO, kCapped>(a, c, steps, k, part, s); break;
    default: pieces<IO, kSmall>(a, c, steps, k, part, s);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || k.pieces == 1) return e;
  const int staged = k.pieces <= kThreads ? k.pieces * a.top : 0;
  hipLaunchKernelGGL((score_join<IO>), dim3(a.T), dim3(kThreads), staged * sizeof(Best), s, a, c,
                     k.pieces, part, staged);
  return hipGetLastError();
}

template <typename IO>
hipError_t backward(const ScoreGradArgs& a, hipStream_t s) {
  const Cap c = make_cap(a.softcap, a.scale);
  const Cut k = cut(a.V, steps_for(a.T, a.V, kMaxSteps), 7);
  const dim3 grid(a.T * k.pieces), block(kThreads);
  switch (form_of(c)) {
    case kPlain:
      hipLaunchKernelGGL((score_backward<IO, kPlain>), grid, block, 0, s, a, c, k.pieces, k.len);
      break;
    case kCapped:
      hipLaunchKernelGGL((score_backward<IO, kCapped>), grid, block, 0, s, a, c, k.pieces, k.len);
      break;
    default:
      hipLaunchKernelGGL((score_backward<IO, kSmall>), grid, block, 0, s, a, c, k.pieces, k.len);
  }
  return hipGetLastError();
}

}  // namespace

int64_t score_pieces_count(int64_t T, int64_t V) {
  return T * cut(V, steps_for(T, V, kMaxSteps), 0).pieces;
}

size_t score_workspace(int64_t T, int64_t V, int top) {
  const int n = cut(V, steps_for(T, V, most_steps(top)), 0).pieces;
  return n == 1 ? 0 : static_cast<size_t>(T) * n * (4 + 2 * top) * sizeof(float);
}

hipError_t launch_token_logprobs(const ScoreArgs& a, int32_t dtype, void* ws, hipStream_t s) {
  float* part = static_cast<float*>(ws);
  return dtype == BEAM_BF16 ? forward<uint16_t>(a, part, s) : forward<float>(a, part, s);
}

hipError_t launch_token_logprobs_backward(const ScoreGradArgs& a, int32_t dtype, hipStream_t s) {
  return dtype == BEAM_BF16 ? backward<uint16_t>(a, s) : backward<float>(a, s);
}

}  // namespace beam
