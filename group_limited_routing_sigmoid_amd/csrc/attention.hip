// Attention of one new token of every sequence over its cached tokens:
//   out_h = softmax(scale q_h K^T) V [* sigmoid(gate_h)]
// for the query heads of a key-value head together, over the last `window`
// tokens or all ("Reflection Releases Beam ...", section "Hybrid Attention and
// Unusual Residuals").
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
// waves; 256 where sixteen waves share a sequence).  Where a sequence can hold
// only few units (a window) a workgroup takes one block of heads of one sequence.
// Else the units of all sequences are cut into slices of one size, whatever the
// sequences' lengths, a workgroup for each slice and block of heads (neighbouring
// workgroups read the heads of the same tokens at the same time): each finds its
// first unit from the lengths, and leaves sums for the sequences that it did not
// see whole, which a second kernel joins.
// 1,000,003 tokens of 8 heads of 128: 690 us, 5.9 TB/s (6.35 is what reading alone
// reaches); 64 sequences of 100 to 32,000: 257 us, 5.7; 256 windows of 512: 96 to 98.
#include <algorithm>

#include "serve.h"

namespace beam {
namespace {

constexpr int kStep = 16;    // tokens of a wave's step
constexpr int kRows = 16;    // query heads of a block
constexpr int kSplitWaves = 4;
constexpr int kSlots = 512;  // workgroups that the split form fills
constexpr float kLog2E = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLowest = -3.0e38f;  // a maximum that any score passes
constexpr float kLazy = 8.0f;        // binary orders that a score may pass the maximum by

// What a workgroup knows of one sequence.
struct Seq {
  int first, end;  // tokens that take part
  int unit0, units;
};
template <int kUnit>
__device__ __forceinline__ Seq seq_of(int len, int window, int most) {
  Seq q;
  q.end = min(max(len, 0), most);
  q.first = window ? max(q.end - window, 0) : 0;
  q.unit0 = q.first / kUnit;
  q.units = max((q.end + kUnit - 1) / kUnit - q.unit0, 1);
  return q;
}

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

// 16 bytes that are read once (700 us instead of 708 for 1,000,003 tokens, 267
// instead of 280 for 64 sequences, 102 instead of 105 for 256 windows of 512).
__device__ __forceinline__ u32x4 once(const char* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
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

// A sequence's units [from, to), counted from its first, for one block of heads.
struct Segment {
  int seq, block, from, to;
};

// FAST: pages of 16 tokens or more, so that a wave's step lies in one page, and D
// = DK; else a lane looks up its token's page and masks the values past D.
template <typename IO, int DK, bool FAST, int W>
struct Attend {
  using T = Tile<IO, DK>;
  static constexpr int kWaves = W, kUnit = W * kStep;
  static constexpr int kAcc = DK / 16;
  static constexpr int kPad = 4;

  // LDS where the waves' sums meet: maxima and sums of probabilities, then the
  // sums of values of each wave's heads.
  static int shared_bytes(int group) {
    return kWaves * (2 * kRows + std::min(group, kRows) * (DK + kPad)) * static_cast<int>(sizeof(float));
  }

  const AttendArgs& a;
  const int lane, wave, sub, row, group, rows_blocks;
  u32x4 q[T::kK];
  f32x4 acc[kAcc];
  float m, l;
  Seq s;
  const int32_t* table;
  const char* kb;  // the cache's first key and value of the block's head
  const char* vb;
  int table_base, pages;  // FAST: this wave's pages, one a lane, from step table_base on
  T t;

  __device__ Attend(const AttendArgs& args)
      : a(args), lane(threadIdx.x % kWave),
        wave(__builtin_amdgcn_readfirstlane(threadIdx.x / kWave)), sub(lane / 16), row(lane % 16),
        group(args.Hq / args.Hkv), rows_blocks((group + kRows - 1) / kRows) {}

  // Where a step's keys and values lie.
  struct Place {
    bool bad;  // FAST: the step's page is none; else that of the lane's token `row`
    const char* key;    // FAST: of the page's place, the same for the wave; else of the lane's rows
    const char* value[4];
    uint32_t off_k, off_v[4];  // FAST: the lane's bytes from there
  };

  // The page of the wave's i-th step, of the 64 steps that it holds.
  __device__ __forceinline__ int page_of(int unit, int i) {
    if (table_base < 0 || i - table_base >= kWave) {
      table_base = i;
      const int token = (unit + lane) * kUnit + wave * kStep;  // step i + lane
      pages = table[min(token, s.end - 1) >> a.cache.shift];
    }
    return __builtin_amdgcn_readlane(pages, i - table_base);
  }

  // Places before the first token that takes part and behind the last are read
  // as those, and count as nothing.
  __device__ __forceinline__ Place place(int unit, int i) {
    const Cache& c = a.cache;
    const int token0 = unit * kUnit + wave * kStep, mask = (1 << c.shift) - 1;
    constexpr int kSize = sizeof(IO);
    Place p;
    if constexpr (FAST) {
      int page = page_of(unit, i);
      p.bad = page < 0 || page >= c.pages;
      if (p.bad) page = 0;
      const uint32_t step = static_cast<uint32_t>(c.token_stride) * kSize;
      const int64_t base = (page * c.page_stride + (token0 & mask) * c.token_stride) * kSize;
      p.key = kb + base;
      p.value[0] = vb + base;
      uint32_t k = row, v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = 4 * sub + r;
      if (token0 < s.first || token0 + kStep > s.end) {
        const uint32_t lo = max(s.first - token0, 0), hi = min(s.end - 1 - token0, kStep - 1);
        k = min(max(k, lo), hi);
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = min(max(v[r], lo), hi);
      }
      p.off_k = k * step + sub * 16;
#pragma unroll
      for (int r = 0; r < 4; ++r) p.off_v[r] = v[r] * step + row * (T::kCols * kSize);
    } else {
      // a page for every token: the key's lane looks it up
      const int token = min(max(token0 + row, s.first), s.end - 1);
      int page = table[token >> c.shift];
      p.bad = page < 0 || page >= c.pages;
      if (p.bad) page = 0;
      const int64_t off = (page * c.page_stride + (token & mask) * c.token_stride) * kSize;
      p.key = kb + off;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t lo = __shfl(static_cast<int>(off), 4 * sub + r);
        const uint32_t hi = __shfl(static_cast<int>(off >> 32), 4 * sub + r);
        p.value[r] = vb + static_cast<int64_t>(static_cast<uint64_t>(hi) << 32 | lo);
      }
    }
    return p;
  }

  // Not FAST: values past D are the row's first ones, which meet zeros.
  __device__ __forceinline__ int in_row(int col) const {
    return (col < a.D ? col : 0) * static_cast<int>(sizeof(IO));
  }
  __device__ __forceinline__ void load_keys(const Place& p) {
#pragma unroll
    for (int j = 0; j < T::kK; ++j)
      t.k[j] = once(p.key + (FAST ? p.off_k + 64 * j : in_row((4 * j + sub) * T::kPart)));
  }
  __device__ __forceinline__ void load_values(const Place& p) {
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < T::kV; ++j) {
        const char* x = FAST ? p.value[0] + p.off_v[r] + 16 * T::kCols * sizeof(IO) * j
                             : p.value[r] + in_row((16 * j + row) * T::kCols);
        if constexpr (sizeof(IO) * T::kCols == 16) t.v[r][j] = once(x);
        else {
          const uint2 w = *reinterpret_cast<const uint2*>(x);
          t.v[r][j] = u32x4{w.x, w.y, 0, 0};
        }
      }
  }

  __device__ __forceinline__ f32x4 products() const {
    f32x4 sc = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < T::kK; ++j) {
      if constexpr (T::kHalf) sc = mfma16x16x32(as_bf16x8(t.k[j]), as_bf16x8(q[j]), sc);
      else
#pragma unroll
        for (int x = 0; x < 4; ++x)
          sc = mfma16x16x4(__uint_as_float(t.k[j][x]), __uint_as_float(q[j][x]), sc);
    }
    return sc;
  }

  // Probabilities relative to the running maximum.
  __device__ __forceinline__ void soften(const f32x4& sc, int unit, const Place& at, float (&p)[4]) {
    const int token0 = unit * kUnit + wave * kStep;
    const float f = a.scale * kLog2E;
#pragma unroll
    for (int r = 0; r < 4; ++r) p[r] = sc[r] * f;
    if (token0 < s.first || token0 + kStep > s.end) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int token = token0 + 4 * sub + r;
        if (token < s.first || token >= s.end) p[r] = -INFINITY;
      }
    }
    if (__any(at.bad)) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (FAST || __shfl(static_cast<int>(at.bad), 4 * sub + r)) {
          p[r] = -INFINITY;
#pragma unroll
          for (int j = 0; j < T::kV; ++j) t.v[r][j] = u32x4{0, 0, 0, 0};
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
  }

  __device__ __forceinline__ void weigh(const float (&p)[4]) {
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

  // One segment: its units, the waves' sums joined, and the result, or where
  // `part` is given its sums.
  __device__ void run(const Segment& g, float* part, float* shared) {
    const int kvh = g.block / rows_blocks, r0 = g.block % rows_blocks * kRows;
    const int rows = min(kRows, group - r0);
    const int64_t head0 = static_cast<int64_t>(g.seq) * a.Hq + kvh * group + r0;
    table = a.cache.tables + static_cast<int64_t>(g.seq) * a.cache.cols;
    const int64_t head = kvh * a.cache.head_stride * static_cast<int64_t>(sizeof(IO));
    kb = static_cast<const char*>(a.cache.k) + head;
    vb = static_cast<const char*>(a.cache.v) + head;
    table_base = -1;
    // the wave's steps with tokens that take part
    const int unit = s.unit0 + g.from, n = g.to - g.from, begin = unit * kUnit + wave * kStep;
    int i = begin + kStep <= s.first ? 1 : 0;  // the first unit alone holds earlier ones
    const int stop = min(n, (s.end - begin + kUnit - 1) / kUnit);
#pragma unroll
    for (int j = 0; j < kAcc; ++j) acc[j] = f32x4{0, 0, 0, 0};
    m = kLowest;
    l = 0.0f;
    if (i < stop) {
#pragma unroll
      for (int j = 0; j < T::kK; ++j) {
        const int col = (4 * j + sub) * T::kPart;
        q[j] = row < rows && col < a.D
                   ? ld16(static_cast<const IO*>(a.q) + (head0 + row) * a.D + col)
                   : u32x4{0, 0, 0, 0};
      }
      Place now = place(unit + i, i);
      load_keys(now);
      load_values(now);
      // the next step's keys are read from when this one's are used up, and its
      // values likewise
      float p[4];
      for (; i + 1 < stop; ++i) {
        const Place next = place(unit + i + 1, i + 1);
        const f32x4 sc = products();
        load_keys(next);
        soften(sc, unit + i, now, p);
        weigh(p);
        load_values(next);
        now = next;
      }
      soften(products(), unit + i, now, p);
      weigh(p);
    }
    l = wave_sum16(l);
    // the waves' parts meet
    float* const sm = shared;
    float* const sl = sm + kWaves * kRows;
    float* const so = sl + kWaves * kRows;
    __syncthreads();
    if (sub == 0) {
      sm[wave * kRows + row] = m;
      sl[wave * kRows + row] = l;
    }
    if (row < rows) {
      // lane's values: those of rows 4 sub + r of the instructions' results
#pragma unroll
      for (int j = 0; j < T::kV; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int x = 0; x < T::kCols; ++x)
            so[(wave * rows + row) * (DK + kPad) + (16 * j + 4 * sub + r) * T::kCols + x] =
                acc[j * T::kCols + x][r];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < rows * DK; e += kWaves * kWave) {
      const int rr = e / DK, d = e % DK;
      if (d >= a.D) continue;
      float mm = sm[rr];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) mm = fmaxf(mm, sm[w * kRows + rr]);
      float ll = 0.0f, oo = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float by = __builtin_amdgcn_exp2f(sm[w * kRows + rr] - mm);
        ll += sl[w * kRows + rr] * by;
        oo += so[(w * rows + rr) * (DK + kPad) + d] * by;
      }
      if (!part) {
        put<IO>(a, (head0 + rr) * a.D + d, ll > 0.0f || ll != ll ? oo / ll : 0.0f);
        if (d == 0 && a.lse)
          a.lse[head0 + rr] = ll > 0.0f || ll != ll ? (mm + __log2f(ll)) * kLn2 : -INFINITY;
      } else {
        part[rr * a.D + d] = oo;
        if (d == 0) {
          part[kRows * a.D + 2 * rr] = mm;
          part[kRows * a.D + 2 * rr + 1] = ll;
        }
      }
    }
  }
};

// A workgroup for each block of heads of each sequence.  Bound to 128 registers, so
// that 1,024 workgroups share the card (256 windows of 512: 99 us, with three a
// compute unit 102; two sequences a workgroup, the second one's first loads before
// the first one's join, 103).
template <typename IO, int DK, bool FAST, int W>
__global__ __launch_bounds__(W* kWave, W == 4 && DK <= 128 && FAST && sizeof(IO) == 2 ? 4 : 1)
void attend_whole(AttendArgs a) {
  using A = Attend<IO, DK, FAST, W>;
  extern __shared__ float sh[];
  A at(a);
  const int blocks = a.Hkv * at.rows_blocks;
  Segment g;
  g.seq = blockIdx.x / blocks;
  g.block = blockIdx.x % blocks;
  at.s = seq_of<A::kUnit>(a.lengths[g.seq], a.window, a.cache.cols << a.cache.shift);
  g.from = 0;
  g.to = at.s.units;
  at.run(g, nullptr, sh);
}

// Sum of v over the wave's lanes up to this one, by data-parallel moves.
__device__ __forceinline__ uint32_t wave_scan(uint32_t v) {
#define BEAM_SCAN(ctrl, rows) \
  v += static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), ctrl, rows, 0xF, false))
  BEAM_SCAN(0x111, 0xF);  // from 1, 2, 4, 8 lanes below in the row of 16
  BEAM_SCAN(0x112, 0xF);
  BEAM_SCAN(0x114, 0xF);
  BEAM_SCAN(0x118, 0xF);
  BEAM_SCAN(0x142, 0xA);  // the first and third row's sums to the next row
  BEAM_SCAN(0x143, 0xC);  // the first half's to the second
#undef BEAM_SCAN
  return v;
}

// What a slice leaves for the second kernel: a sequence that begins in it and
// ends in another one.
struct Open {
  int32_t seq;   // -1: none
  int32_t last;  // the slice that it ends in
};
// A slice's sums for a block of heads: of the sequence that came from the slice
// before (which 0), and of the one that goes on to the next (1).
__host__ __device__ constexpr int64_t part_size(int D) { return kRows * (D + 2); }
__device__ __forceinline__ float* part_of(const AttendArgs& a, int blocks, int slice, int block,
                                          int which) {
  return a.part + ((static_cast<int64_t>(slice) * blocks + block) * 2 + which) * part_size(a.D);
}

// The units of all sequences in slices of one size.
template <typename IO, int DK, bool FAST>
__global__ __launch_bounds__(kSplitWaves* kWave) void attend_split(AttendArgs a, Open* open, int slices) {
  using A = Attend<IO, DK, FAST, kSplitWaves>;
  extern __shared__ float sh[];
  A at(a);
  const int blocks = a.Hkv * at.rows_blocks, most = a.cache.cols << a.cache.shift;
  const int seqs = static_cast<int>(a.cache.seqs), lane = at.lane;
  const int slice = blockIdx.x / blocks;
  // every wave counts the units for itself
  auto units = [&](int b) -> uint32_t {
    return b < seqs ? seq_of<A::kUnit>(a.lengths[b], a.window, most).units : 0;
  };
  uint32_t total = 0;
  for (int b = lane; b < seqs; b += kWave) total += units(b);
  total = __builtin_amdgcn_readlane(wave_scan(total), kWave - 1);
  const uint32_t each = (total + slices - 1) / slices;  // a sequence has at least one
  uint32_t unit = each * slice;
  const uint32_t stop = min(unit + each, total);
  if (unit >= total) {
    if (threadIdx.x == 0) open[slice] = Open{-1, 0};
    return;
  }
  // the sequence of the first unit
  int b = 0;
  uint32_t before = 0;
  for (int b0 = 0; b0 < seqs; b0 += kWave) {
    const uint32_t mine = units(b0 + lane), sum = before + wave_scan(mine);
    const uint64_t past = __ballot(sum > unit);
    if (past) {
      const int x = __ffsll(static_cast<long long>(past)) - 1;
      b = b0 + x;
      before = __builtin_amdgcn_readlane(sum - mine, x);
      break;
    }
    before = __builtin_amdgcn_readlane(sum, kWave - 1);
  }
  Segment g;
  g.seq = __builtin_amdgcn_readfirstlane(b);
  g.block = blockIdx.x % blocks;
  at.s = seq_of<A::kUnit>(a.lengths[g.seq], a.window, most);
  g.from = static_cast<int>(unit - before);
  Open left = {-1, 0};
  while (unit < stop) {
    g.to = static_cast<int>(min<uint32_t>(at.s.units, g.from + (stop - unit)));
    const bool begins = g.from == 0, ends = g.to == at.s.units;
    // (the next sequence's length on its way)
    const int length = a.lengths[min(g.seq + 1, seqs - 1)];
    if (begins && !ends)
      left = Open{g.seq, static_cast<int32_t>((unit + at.s.units - 1) / each)};
    at.run(g, begins && ends ? nullptr : part_of(a, blocks, slice, g.block, begins), sh);
    unit += g.to - g.from;
    g.from = 0;
    if (++g.seq < seqs) at.s = seq_of<A::kUnit>(length, a.window, most);
  }
  if (threadIdx.x == 0) open[slice] = left;
}

// Joins the parts of the sequence that begins in a slice and ends in a later
// one, for one query head: 32 lanes take four values each (of up to 128; D 256
// in two turns), eight of such groups the parts in turn.
template <typename IO>
__global__ __launch_bounds__(256) void attend_join(AttendArgs a, const Open* open) {
  __shared__ float by[kSlots];
  __shared__ float red[4][2];
  __shared__ f32x4 sums[8][32];
  const Open w = open[blockIdx.x / a.Hq];
  if (w.seq < 0) return;
  const int first = blockIdx.x / a.Hq, head = blockIdx.x % a.Hq;
  const int group = a.Hq / a.Hkv, rows_blocks = (group + kRows - 1) / kRows;
  const int blocks = a.Hkv * rows_blocks, in = head % group;
  const int block = head / group * rows_blocks + in / kRows, rr = in % kRows;
  const int n = w.last - first + 1;
  auto part = [&](int i) -> const float* {  // the beginning, then what came over
    return part_of(a, blocks, first + i, block, i == 0);
  };
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  float m = kLowest;
  for (int i = threadIdx.x; i < n; i += 256) m = fmaxf(m, part(i)[kRows * a.D + 2 * rr]);
#pragma unroll
  for (int i = 1; i < kWave; i *= 2) m = fmaxf(m, __shfl_xor(m, i));
  if (lane == 0) red[wave][0] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
  float l = 0.0f;
  for (int i = threadIdx.x; i < n; i += 256) {
    const float* p = part(i) + kRows * a.D + 2 * rr;
    const float f = __builtin_amdgcn_exp2f(p[0] - m);
    by[i] = f;
    l += p[1] * f;
  }
#pragma unroll
  for (int i = 1; i < kWave; i *= 2) l += __shfl_xor(l, i);
  if (lane == 0) red[wave][1] = l;
  __syncthreads();
  l = (red[0][1] + red[1][1]) + (red[2][1] + red[3][1]);
  const bool some = l > 0.0f || l != l;
  const int64_t at = static_cast<int64_t>(w.seq) * a.Hq + head;
  const int col = threadIdx.x % 32, share = threadIdx.x / 32;
  for (int d0 = 0; d0 < a.D; d0 += 128) {
    const int d = d0 + 4 * col;
    f32x4 o = {0, 0, 0, 0};
    if (d < a.D) {
#pragma unroll 4
      for (int i = share; i < n; i += 8) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(part(i) + rr * a.D + d);
        o += v * by[i];
      }
    }
    __syncthreads();
    sums[share][col] = o;
    __syncthreads();
    if (share == 0 && d < a.D) {
      for (int i = 1; i < 8; ++i) o += sums[i][col];
#pragma unroll
      for (int j = 0; j < 4; ++j) put<IO>(a, at * a.D + d + j, some ? o[j] / l : 0.0f);
    }
  }
  if (threadIdx.x == 0 && a.lse) a.lse[at] = some ? (m + __log2f(l)) * kLn2 : -INFINITY;
}

int head_blocks(int Hq, int Hkv) { return Hkv * static_cast<int>(ceil_div(Hq / Hkv, kRows)); }
// Slices of the split form: two workgroups a compute unit in all.  (1,000,003
// tokens and 64 sequences of 100 to 32,000, 8 heads of 128: 700 and 267 us; one a
// unit 729 and 301, three 705 and 271.)
int slices_of(int blocks) {
  return std::max(1, kSlots / blocks);
}

template <typename IO, int DK, bool FAST, int W>
hipError_t whole(const AttendArgs& a, int64_t segs, hipStream_t s) {
  const int shared = Attend<IO, DK, FAST, W>::shared_bytes(a.Hq / a.Hkv);
  hipLaunchKernelGGL((attend_whole<IO, DK, FAST, W>), dim3(segs), dim3(W * kWave), shared, s, a);
  return hipGetLastError();
}

template <typename IO, int DK, bool FAST>
hipError_t launch(const AttendArgs& a, hipStream_t s) {
  constexpr int W = kSplitWaves;
  const int blocks = head_blocks(a.Hq, a.Hkv);
  const int64_t segs = a.cache.seqs * blocks;
  const int64_t most = static_cast<int64_t>(a.cache.cols) << a.cache.shift;
  // tokens and units that a sequence can have
  const int64_t tokens = a.window && a.window < most ? a.window + W * kStep : most;
  const int64_t units = ceil_div(tokens, W * kStep);
  const int slices = static_cast<int>(std::min<int64_t>(slices_of(blocks), a.cache.seqs * units));
  // Two units or fewer: nothing to split.  Up to 17 (a window of 1,024): whole
  // sequences fill the card from 512 on, and with sixteen waves for each from 128
  // on (32 sequences of 900 or 500 tokens, 8 heads: 24 and 16 us, in slices 34 and
  // 22; 8 of 900 20, in slices 17).  Up to six units sixteen waves take a step or two
  // each, in one launch (250 tokens 8.7 us, 300 9.4, in slices 11; 500 tokens 11.6 and
  // in slices 10).  A slice may be one unit, a step for each wave (2,000 tokens 11.4
  // us, with two at least 12.7).
  if (slices <= 1 || units <= 2 || (segs >= 512 && units <= 17)) return whole<IO, DK, FAST, W>(a, segs, s);
  if constexpr (FAST && sizeof(IO) == 2 && DK <= 128)
    if ((segs >= 128 && units <= 17) || units <= 6) return whole<IO, DK, FAST, 16>(a, segs, s);
  const dim3 block(W * kWave);
  const int shared = Attend<IO, DK, FAST, W>::shared_bytes(a.Hq / a.Hkv);
  Open* open = reinterpret_cast<Open*>(a.part + static_cast<int64_t>(slices_of(blocks)) * blocks *
                                                    2 * part_size(a.D));
  hipLaunchKernelGGL((attend_split<IO, DK, FAST>), dim3(slices * blocks), block, shared, s, a, open,
                     slices);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((attend_join<IO>), dim3(slices * a.Hq), dim3(256), 0, s, a, open);
  return hipGetLastError();
}

template <typename IO, int DK>
hipError_t by_page(const AttendArgs& a, hipStream_t s) {
  return a.cache.shift >= 4 && a.D == DK ? launch<IO, DK, true>(a, s) : launch<IO, DK, false>(a, s);
}

template <typename IO>
hipError_t by_head(const AttendArgs& a, hipStream_t s) {
  return a.D <= 64 ? by_page<IO, 64>(a, s) : a.D <= 128 ? by_page<IO, 128>(a, s)
                                                        : by_page<IO, 256>(a, s);
}

}  // namespace

size_t attend_workspace(int64_t seqs, int Hq, int Hkv, int D) {
  if (seqs == 0) return 0;
  const int blocks = head_blocks(Hq, Hkv), slices = slices_of(blocks);
  return static_cast<size_t>(slices) * (blocks * 2 * part_size(D) * sizeof(float) + sizeof(Open));
}

hipError_t launch_paged_attention(const AttendArgs& a, int32_t dtype, hipStream_t s) {
  return dtype == BEAM_BF16 ? by_head<uint16_t>(a, s) : by_head<float>(a, s);
}

}  // namespace beam
