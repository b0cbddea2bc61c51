// Attention of one new token of every sequence over its cached tokens:
//   out_h = softmax(scale q_h K^T) V [* sigmoid(gate_h)]
// for the query heads of a key-value head together, over the last `window`
// tokens or all ("Reflection Beam", section "Hybrid Attention and Unusual
// Residuals").
//
// Bound by reading the keys and values once.  The query heads of one key-value
// head (up to 16; more go in blocks of 16) are the 16 columns of the matrix
// instructions, and a wave takes 16 tokens at a time:
//   S^T[token][head] = K Q^T     bf16 16x16x32 (fp32 cache: fp32 16x16x4), K's
//                                rows straight from memory
//   O^T[value][head] += V^T P^T  fp32 16x16x4
// Lane l of the first product's result holds tokens 4 (l/16) + r of head l % 16,
// r < 4; the r-th fp32 instruction takes of P^T exactly that element from each
// lane, and of V^T the row of token 4 (l/16) + r: 16 lanes read one token's
// values in whole lines, which become the values' columns 8 (l % 16) + j of
// eight products.  So neither keys, values nor probabilities ever change lanes or
// pass through LDS, and probabilities stay binary32.  The running maximum is
// raised only when a score passes it by 2^8 (any of the wave's), so the usual
// step has no exchange between lanes and no rescaling; the sums of one lane's
// tokens meet the other lanes' at the end.
//
// The work is counted in units of 64 tokens (16 for each of a workgroup's four
// waves) over all sequences and key-value heads.  Where a sequence can hold only
// few units (a window) a workgroup takes one key-value head of one sequence.
// Else the units are dealt evenly to as many workgroups as run at once, whatever
// the sequences' lengths: each finds its first one from the lengths, and leaves
// sums for the heads that it did not see whole, which a second kernel joins.
#include <algorithm>

#include "serve.h"

namespace beam {
namespace {

constexpr int kUnit = 64;    // tokens of a unit
constexpr int kStep = 16;    // tokens of a wave's step
constexpr int kWaves = 4;
constexpr int kRows = 16;    // query heads of a block
constexpr int kMaxSplit = 1024;
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.0e38f;  // a maximum that any score passes
constexpr float kLazy = 8.0f;        // binary orders that a score may pass the maximum by

// What a workgroup knows of one sequence.
struct Seq {
  int first, end;  // tokens that take part
  int unit0, units;
};
__device__ __forceinline__ Seq seq_of(int len, int window, int most) {
  Seq q;
  q.end = min(max(len, 0), most);
  q.first = window ? max(q.end - window, 0) : 0;
  q.unit0 = q.first / kUnit;
  q.units = max((q.end + kUnit - 1) / kUnit - q.unit0, 1);
  return q;
}

struct Segment {  // of one sequence's one block of heads
  int64_t id;     // sequence * blocks of heads + block
  int seq, block;
  int from, to;   // units, from the sequence's first
};

__device__ __forceinline__ float wave_max16(float v) {
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float wave_sum16(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

template <typename IO>
__device__ __forceinline__ float to_f32(IO v) {
  if constexpr (sizeof(IO) == 2) return bf16_bits_to_f32(v);
  else return v;
}
template <typename IO>
__device__ __forceinline__ IO from_f32(float v) {
  if constexpr (sizeof(IO) == 2) return f32_to_bf16_bits(v);
  else return v;
}

__device__ __forceinline__ f32x4 mfma16x16x4(float a, float b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x4f32(a, b, c, 0, 0, 0);
}

// A lane's share of 16 tokens' keys or values.
//   keys    token l % 16, values of the l/16-th quarter of each 32 (fp32: 16)
//   values  tokens 4 (l/16) + r; of each, kCols neighbouring values at
//           kCols (l % 16) + 16 kCols i
template <typename IO, int DK>
struct Tile {
  static constexpr bool kHalf = sizeof(IO) == 2;
  static constexpr int kPart = 16 / static_cast<int>(sizeof(IO));  // values of 16 bytes
  static constexpr int kK = DK / 4 / kPart;                        // loads of a key
  static constexpr int kCols = std::min(kPart, DK / 16);
  static constexpr int kV = DK / 16 / kCols;                       // loads of a token's values
  u32x4 k[kK];
  u32x4 v[4][kV];  // kCols 4 of bf16: the first two words
};

// out[x] for a head's element: the gate and the rounding
template <typename IO>
__device__ __forceinline__ void put(const AttendArgs& a, int64_t x, float v) {
  if (a.gate) v /= 1.0f + __expf(-to_f32(static_cast<const IO*>(a.gate)[x]));
  static_cast<IO*>(a.out)[x] = from_f32<IO>(v);
}

// WHOLE: a workgroup takes whole segments.  PAGED16: pages of 16 tokens or
// more, so that a wave's step lies in one page.
template <typename IO, int DK, bool PAGED16>
struct Attend {
  using T = Tile<IO, DK>;
  static constexpr int kAcc = DK / 16;
  static constexpr int kPad = 4;

  struct Shared {
    float o[kWaves][kRows][DK + kPad];
    float m[kWaves][kRows], l[kWaves][kRows];
  };

  const AttendArgs& a;
  const int lane, wave, group, rows_blocks;
  u32x4 q[T::kK];
  f32x4 acc[kAcc];
  float m, l;
  Seq s;
  const int32_t* table;
  const IO* kb;
  const IO* vb;
  int table_base, pages;  // this wave's pages, one a lane, from step table_base on

  __device__ Attend(const AttendArgs& args)
      : a(args), lane(threadIdx.x % kWave),
        wave(__builtin_amdgcn_readfirstlane(threadIdx.x / kWave)), group(args.Hq / args.Hkv),
        rows_blocks((group + kRows - 1) / kRows) {}

  // The page of the wave's i-th step of a segment, from the 64 that it holds.
  __device__ __forceinline__ int page_of(int unit, int i) {
    if (i - table_base >= kWave || table_base < 0) {
      table_base = i;
      const int token = (unit + lane) * kUnit + wave * kStep;  // step i + lane is unit + lane
      const int slot = min(token, s.end - 1) >> a.cache.shift;
      pages = table[max(slot, 0)];
    }
    return __builtin_amdgcn_readlane(pages, i - table_base);
  }

  __device__ __forceinline__ void load(T& t, bool& none, int& bad, int unit, int i) {
    const int token0 = unit * kUnit + wave * kStep;
    const Cache& c = a.cache;
    const int mask = (1 << c.shift) - 1;
    const int sub = lane / 16, row = lane % 16;
    none = token0 >= s.end || token0 + kStep <= s.first;
    bad = 0;
    if (none) return;
    int kcol[T::kK], vcol[T::kV];
    (void)kcol;
    (void)vcol;
    auto read = [&](const IO* kp, const IO* const (&vp)[4]) {
#pragma unroll
      for (int j = 0; j < T::kK; ++j) {
        const int col = (4 * j + sub) * T::kPart;
        t.k[j] = ld16(kp + (col < a.D ? col : 0));
      }
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int j = 0; j < T::kV; ++j) {
          const int col = (16 * j + row) * T::kCols;
          const IO* p = vp[r] + (col < a.D ? col : 0);
          if constexpr (sizeof(IO) * T::kCols == 16) t.v[r][j] = ld16(p);
          else {
            const uint2 x = *reinterpret_cast<const uint2*>(p);
            t.v[r][j] = u32x4{x.x, x.y, 0, 0};
          }
        }
    };
    const int lo = s.first, hi = s.end - 1;
    if constexpr (PAGED16) {
      const int page = page_of(unit, i);
      if (page < 0 || page >= c.pages) {
        none = true;
        return;
      }
      // places before the first token and behind the last are read as those
      const int64_t base = page * c.page_stride;
      const int in0 = token0 & mask, l0 = max(lo - token0, 0), h0 = min(hi - token0, kStep - 1);
      const IO* kp = kb + base;
      const IO* vp = vb + base;
      const IO* vr[4];
#pragma unroll
      for (int r = 0; r < 4; ++r)
        vr[r] = vp + (in0 + min(max(4 * sub + r, l0), h0)) * c.token_stride;
      read(kp + (in0 + min(max(row, l0), h0)) * c.token_stride, vr);
    } else {
      // a page for every token: the key's lane looks it up
      const int token = min(max(token0 + row, lo), hi);
      int page = table[token >> c.shift];
      const bool wrong = page < 0 || page >= c.pages;
      if (wrong) page = 0;
      const int64_t off = page * c.page_stride + (token & mask) * c.token_stride;
      bad = wrong ? 1 : 0;
      const IO* vr[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int from = 4 * sub + r;
        const uint32_t lo32 = __shfl(static_cast<int>(off), from);
        const uint32_t hi32 = __shfl(static_cast<int>(off >> 32), from);
        vr[r] = vb + static_cast<int64_t>(static_cast<uint64_t>(hi32) << 32 | lo32);
      }
      read(kb + off, vr);
    }
  }

  __device__ __forceinline__ void use(T& t, bool none, int bad, int unit) {
    if (none) return;
    const int token0 = unit * kUnit + wave * kStep, sub = lane / 16;
    f32x4 sc = {0, 0, 0, 0};
    if constexpr (T::kHalf) {
#pragma unroll
      for (int j = 0; j < T::kK; ++j)
        sc = mfma16x16x32(as_bf16x8(t.k[j]), as_bf16x8(q[j]), sc);
    } else {
#pragma unroll
      for (int j = 0; j < T::kK; ++j)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          sc = mfma16x16x4(__uint_as_float(t.k[j][x]), __uint_as_float(q[j][x]), sc);
    }
    const float f = a.scale * kLog2E;
    float p[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) p[r] = sc[r] * f;
    if (token0 < s.first || token0 + kStep > s.end) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int token = token0 + 4 * sub + r;
        if (token < s.first || token >= s.end) p[r] = -INFINITY;
      }
    }
    if constexpr (!PAGED16) {
      if (__any(bad)) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (__shfl(bad, 4 * sub + r)) {
            p[r] = -INFINITY;
#pragma unroll
            for (int j = 0; j < T::kV; ++j) t.v[r][j] = u32x4{0, 0, 0, 0};
          }
      }
    }
    const float top = fmaxf(fmaxf(p[0], p[1]), fmaxf(p[2], p[3]));
    if (__any(top > m + kLazy)) {
      const float to = fmaxf(m, wave_max16(top));
      const float by = __builtin_amdgcn_exp2f(m - to);
      m = to;
      l *= by;
#pragma unroll
      for (int j = 0; j < kAcc; ++j) acc[j] *= by;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      p[r] = __builtin_amdgcn_exp2f(p[r] - m);
      l += p[r];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < T::kV; ++j)
#pragma unroll
        for (int x = 0; x < T::kCols; ++x) {
          float v;
          if constexpr (T::kHalf)
            v = __uint_as_float(x % 2 ? t.v[r][j][x / 2] & 0xFFFF0000u : t.v[r][j][x / 2] << 16);
          else
            v = __uint_as_float(t.v[r][j][x]);
          acc[j * T::kCols + x] = mfma16x16x4(v, p[r], acc[j * T::kCols + x]);
        }
  }

  // One segment: its units, the waves' sums joined, and the result or its part.
  __device__ void run(const Segment& g, bool whole, int64_t piece, Shared& sh) {
    const int kvh = g.block / rows_blocks, r0 = g.block % rows_blocks * kRows;
    const int rows = min(kRows, group - r0);
    const int sub = lane / 16, row = lane % 16;
    const int64_t head0 = static_cast<int64_t>(g.seq) * a.Hq + kvh * group + r0;
    table = a.cache.tables + static_cast<int64_t>(g.seq) * a.cache.cols;
    kb = static_cast<const IO*>(a.cache.k) + kvh * a.cache.head_stride;
    vb = static_cast<const IO*>(a.cache.v) + kvh * a.cache.head_stride;
    table_base = -1;
#pragma unroll
    for (int j = 0; j < T::kK; ++j) {
      const int col = (4 * j + sub) * T::kPart;
      q[j] = row < rows && col < a.D
                 ? ld16(static_cast<const IO*>(a.q) + (head0 + row) * a.D + col)
                 : u32x4{0, 0, 0, 0};
    }
#pragma unroll
    for (int j = 0; j < kAcc; ++j) acc[j] = f32x4{0, 0, 0, 0};
    m = kLowest;
    l = 0.0f;
    // two tiles: one is read while the other is used
    T t0, t1;
    bool n0 = true, n1 = true;
    int b0 = 0, b1 = 0;
    const int unit = s.unit0 + g.from, n = g.to - g.from;
    load(t0, n0, b0, unit, 0);
    for (int i = 0; i < n; i += 2) {
      n1 = true;
      if (i + 1 < n) load(t1, n1, b1, unit + i + 1, i + 1);
      use(t0, n0, b0, unit + i);
      n0 = true;
      if (i + 2 < n) load(t0, n0, b0, unit + i + 2, i + 2);
      use(t1, n1, b1, unit + i + 1);
    }
    l = wave_sum16(l);
    // the waves' parts meet
    __syncthreads();
    if (sub == 0) {
      sh.m[wave][row] = m;
      sh.l[wave][row] = l;
    }
    if (row < rows) {
      // lane's values: those of rows 4 sub + r of the instructions' results
#pragma unroll
      for (int j = 0; j < T::kV; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int x = 0; x < T::kCols; ++x)
            sh.o[wave][row][(16 * j + 4 * sub + r) * T::kCols + x] = acc[j * T::kCols + x][r];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < rows * DK; e += kWaves * kWave) {
      const int rr = e / DK, d = e % DK;
      if (d >= a.D) continue;
      float mm = sh.m[0][rr];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, sh.m[w][rr]);
      float ll = 0.0f, oo = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float by = __builtin_amdgcn_exp2f(sh.m[w][rr] - mm);
        ll += sh.l[w][rr] * by;
        oo += sh.o[w][rr][d] * by;
      }
      if (whole) {
        put<IO>(a, (head0 + rr) * a.D + d, ll > 0.0f || ll != ll ? oo / ll : 0.0f);
        if (d == 0 && a.lse)
          a.lse[head0 + rr] = ll > 0.0f || ll != ll ? (mm + __log2f(ll)) * kLn2 : -INFINITY;
      } else {
        float* part = a.part + piece * kRows * (a.D + 2);
        part[rr * a.D + d] = oo;
        if (d == 0) {
          part[kRows * a.D + 2 * rr] = mm;
          part[kRows * a.D + 2 * rr + 1] = ll;
        }
      }
    }
  }
};

// A workgroup for each block of heads of each sequence.
template <typename IO, int DK, bool PAGED16>
__global__ __launch_bounds__(kWaves* kWave) void attend_whole(AttendArgs a) {
  using A = Attend<IO, DK, PAGED16>;
  __shared__ typename A::Shared sh;
  A at(a);
  const int blocks = a.Hkv * at.rows_blocks;
  Segment g;
  g.id = blockIdx.x;
  g.seq = blockIdx.x / blocks;
  g.block = blockIdx.x % blocks;
  at.s = seq_of(a.lengths[g.seq], a.window, a.cache.cols << a.cache.shift);
  g.from = 0;
  g.to = at.s.units;
  at.run(g, true, 0, sh);
}

// Units dealt evenly.  `marks` [segments][2]: the workgroups that hold a
// segment's first and last unit.
template <typename IO, int DK, bool PAGED16>
__global__ __launch_bounds__(kWaves* kWave) void attend_split(AttendArgs a, int32_t* marks,
                                                               int least) {
  using A = Attend<IO, DK, PAGED16>;
  __shared__ typename A::Shared sh;
  A at(a);
  const int blocks = a.Hkv * at.rows_blocks, most = a.cache.cols << a.cache.shift;
  const int seqs = static_cast<int>(a.cache.seqs), lane = at.lane;
  // every wave counts the units for itself
  int64_t total = 0;
  for (int b = lane; b < seqs; b += kWave) total += seq_of(a.lengths[b], a.window, most).units;
#pragma unroll
  for (int i = 1; i < kWave; i *= 2) total += __shfl_xor(total, i);
  total *= blocks;
  const int64_t each = max<int64_t>(ceil_div(total, gridDim.x), least);
  int64_t unit = each * blockIdx.x;
  const int64_t stop = min<int64_t>(unit + each, total);
  if (unit >= stop) return;
  // the sequence of the first unit
  int b = 0;
  int64_t before = 0;
  for (int b0 = 0; b0 < seqs; b0 += kWave) {
    const int64_t mine = b0 + lane < seqs
                             ? static_cast<int64_t>(blocks) *
                                   seq_of(a.lengths[b0 + lane], a.window, most).units
                             : 0;
    int64_t sum = mine;
#pragma unroll
    for (int i = 1; i < kWave; i *= 2) {
      const int64_t x = __shfl_up(sum, i);
      if (lane >= i) sum += x;
    }
    const uint64_t past = __ballot(before + sum > unit);
    if (past) {
      const int at_lane = __ffsll(static_cast<long long>(past)) - 1;
      b = b0 + at_lane;
      before += __shfl(sum - mine, at_lane);
      break;
    }
    before += __shfl(sum, kWave - 1);
  }
  b = __builtin_amdgcn_readfirstlane(b);
  at.s = seq_of(a.lengths[b], a.window, most);
  const int64_t in = unit - before;
  Segment g;
  g.seq = b;
  g.block = __builtin_amdgcn_readfirstlane(static_cast<int>(in / at.s.units));
  g.from = __builtin_amdgcn_readfirstlane(static_cast<int>(in % at.s.units));
  while (unit < stop) {
    g.id = static_cast<int64_t>(g.seq) * blocks + g.block;
    g.to = static_cast<int>(min<int64_t>(at.s.units, g.from + (stop - unit)));
    const bool begins = g.from == 0, ends = g.to == at.s.units;
    if (threadIdx.x == 0) {
      if (begins) marks[2 * g.id] = blockIdx.x;
      if (ends) marks[2 * g.id + 1] = blockIdx.x;
    }
    at.run(g, begins && ends, blockIdx.x + g.id, sh);
    unit += g.to - g.from;
    g.from = 0;
    if (++g.block == blocks) {
      g.block = 0;
      if (++g.seq < seqs) at.s = seq_of(a.lengths[g.seq], a.window, most);
    }
  }
}

// Joins the parts of one query head: a workgroup's threads take its values, in
// as many shares of the parts as fit.
template <typename IO>
__global__ __launch_bounds__(256) void attend_join(AttendArgs a, const int32_t* marks) {
  __shared__ float o[256], sm[256], sl[256];
  const int group = a.Hq / a.Hkv, rows_blocks = (group + kRows - 1) / kRows;
  const int head = blockIdx.x % a.Hq, seq = blockIdx.x / a.Hq;
  const int r = head % group;
  const int64_t id = (static_cast<int64_t>(seq) * a.Hkv + head / group) * rows_blocks + r / kRows;
  const int from = marks[2 * id], to = marks[2 * id + 1];
  if (from == to) return;
  const int rr = r % kRows;
  const int64_t size = kRows * (a.D + 2);
  const float* part = a.part + (from + id) * size;
  const int n = to - from + 1;
  // statistics: a thread for each part
  float m = kLowest;
  for (int i = threadIdx.x; i < n; i += 256) m = fmaxf(m, part[i * size + kRows * a.D + 2 * rr]);
  sm[threadIdx.x] = m;
  __syncthreads();
  for (int i = 128; i; i /= 2) {
    if (threadIdx.x < i) sm[threadIdx.x] = fmaxf(sm[threadIdx.x], sm[threadIdx.x + i]);
    __syncthreads();
  }
  m = sm[0];
  const int shares = 256 / a.D, d = threadIdx.x % a.D, share = threadIdx.x / a.D;
  float ll = 0.0f, oo = 0.0f;
  if (share < shares)
    for (int i = share; i < n; i += shares) {
      const float* p = part + i * size;
      const float by = __builtin_amdgcn_exp2f(p[kRows * a.D + 2 * rr] - m);
      ll += p[kRows * a.D + 2 * rr + 1] * by;
      oo += p[rr * a.D + d] * by;
    }
  o[threadIdx.x] = oo;
  sl[threadIdx.x] = ll;
  __syncthreads();
  if (share) return;
  for (int i = 1; i < shares; ++i) {
    ll += sl[i * a.D + d];
    oo += o[i * a.D + d];
  }
  const bool some = ll > 0.0f || ll != ll;
  const int64_t at = static_cast<int64_t>(seq) * a.Hq + head;
  put<IO>(a, at * a.D + d, some ? oo / ll : 0.0f);
  if (d == 0 && a.lse) a.lse[at] = some ? (m + __log2f(ll)) * kLn2 : -INFINITY;
}

int64_t segments(int64_t seqs, int Hq, int Hkv) {
  return seqs * Hkv * ceil_div(Hq / Hkv, kRows);
}

template <typename IO, int DK, bool PAGED16>
hipError_t launch(const AttendArgs& a, hipStream_t s) {
  const int64_t segs = segments(a.cache.seqs, a.Hq, a.Hkv);
  const int64_t most = static_cast<int64_t>(a.cache.cols) << a.cache.shift;
  // units that a segment can have
  const int64_t units = a.window && a.window < most ? ceil_div(a.window - 1, kUnit) + 1
                                                    : ceil_div(most, kUnit);
  const dim3 block(kWaves * kWave);
  if (units <= 2 || (segs >= 512 && units <= 16)) {
    hipLaunchKernelGGL((attend_whole<IO, DK, PAGED16>), dim3(segs), block, 0, s, a);
    return hipGetLastError();
  }
  int32_t* marks = reinterpret_cast<int32_t*>(
      a.part + (kMaxSplit + segs) * kRows * (a.D + 2));
  const int64_t grid = std::min<int64_t>(DK == 256 ? 512 : 768, segs * units);
  hipLaunchKernelGGL((attend_split<IO, DK, PAGED16>), dim3(grid), block, 0, s, a, marks, 2);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attend_join<IO>), dim3(a.cache.seqs * a.Hq), dim3(256), 0, s, a, marks);
  return hipGetLastError();
}

template <typename IO, int DK>
hipError_t by_page(const AttendArgs& a, hipStream_t s) {
  return a.cache.shift >= 4 ? launch<IO, DK, true>(a, s) : launch<IO, DK, false>(a, s);
}

template <typename IO>
hipError_t by_head(const AttendArgs& a, hipStream_t s) {
  return a.D <= 64 ? by_page<IO, 64>(a, s) : a.D <= 128 ? by_page<IO, 128>(a, s)
                                                        : by_page<IO, 256>(a, s);
}

}  // namespace

size_t attend_workspace(int64_t seqs, int Hq, int Hkv, int D) {
  if (seqs == 0) return 0;
  const int64_t segs = segments(seqs, Hq, Hkv);
  return static_cast<size_t>(kMaxSplit + segs) * kRows * (D + 2) * sizeof(float) +
         static_cast<size_t>(segs) * 2 * sizeof(int32_t);
}

hipError_t launch_paged_attention(const AttendArgs& a, int32_t dtype, hipStream_t s) {
  return dtype == BEAM_BF16 ? by_head<uint16_t>(a, s) : by_head<float>(a, s);
}

}  // namespace beam
