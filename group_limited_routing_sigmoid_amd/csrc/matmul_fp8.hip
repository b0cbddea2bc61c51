// The product of two e4m3 matrices with a scale for each block of 128 along
// the reduction, y[m,n] = sum_kb sa[m,kb] sb[n,kb] sum_{k in kb} a[m,k] b[n,k],
// dense (the expert path's grouped products are its own kernels), and the
// quantiser that makes its operands in both orientations.
//
// Each 128-deep block's products are summed by the matrix cores into fresh
// registers and added to the result's with one fused multiply-add by the
// block's scale: no ratio of scales is formed, so blocks of any size mix.  That
// scale is the two operands' product in binary32, which so has to be a normal
// number (or 0): of quantised blocks that meet, the largest values multiply to
// between 2^-108 and 2^145.  Scales applied one after the other would not need
// that, at a second multiplication for every sum of every block.
//
// How the sums round.  The e4m3 matrix instructions (every form of them,
// measured) add eight consecutive products aligned to the largest one's
// exponent and cut each at 2^-13 of it, and add those sums in binary32: on
// normal data 1.5e-5 of the result, an eightieth of what rounding to bf16
// then loses, so bf16 results are made with them.  A binary32 result would
// show it, so those are made with the bf16 instructions at half the rate
// (2.07 against 4.04 PFLOP/s measured), which hold every product and sum
// binary32: an e4m3 value is a bf16 value, and one conversion instruction
// expands two codes.
#include <algorithm>
#include <type_traits>

#include "grouped_tile.h"
#include "layer.h"

namespace beam {
namespace {

constexpr int kRow = 128;  // bytes of a tile row: one block of 128 codes

// D = A(16x128) * B(128x16) + C on e4m3 codes (format 0, unit E8M0 scales).
// Lane l supplies row (l % 16) of A and column (l % 16) of B, codes
// 32*(l/16) .. +32; element r of lane l is C[4*(l/16) + r][l % 16].
__device__ __forceinline__ f32x4 mfma_e4m3(i32x8 a, i32x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 127, 0, 127);
}

// The lane's 32 codes as four bf16 fragments of 8 (both operands take the
// same k in the same order, so which k a fragment holds does not matter).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
struct Wide {
  bf16x8 f[4];
};
__device__ __forceinline__ Wide widen(i32x8 q) {
  Wide w;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * j + i], 1.0f, false);
      const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(q[2 * j + i], 1.0f, true);
      w.f[j][4 * i] = lo[0];
      w.f[j][4 * i + 1] = lo[1];
      w.f[j][4 * i + 2] = hi[0];
      w.f[j][4 * i + 3] = hi[1];
    }
  return w;
}
__device__ __forceinline__ f32x4 mfma_wide(const Wide& a, const Wide& b, f32x4 c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = mfma16x16x32(a.f[j], b.f[j], c);
  return c;
}

// Swizzle of a tile row's eight 16-byte chunks: chunk c of row r lies in place
// c ^ key(r) of the row's 128 bytes, rows 2i and 2i + 1 in the two halves of
// the LDS banks' 256 bytes.  A fragment's reads of 16 bytes a lane (row l % 16,
// chunk 2 (l / 16)) go through in groups of 16 lanes, {0-3, 12-15, 20-27},
// {4-11, 16-19, 28-31} and the same 32 further on: rows 0-3 and 12-15 of one
// chunk with rows 4-11 of the chunk two further.  So the keys of one half of
// these row pairs are 4 .. 7 and those of the other 0 .. 3, a set that ^ 2 maps
// to itself: every group's 16 places differ.  (With key = i every read took
// twice its cycles, 43% of all that the LDS spent in a large product.)  The
// key repeats every 16 rows, so one lane offset serves every fragment.
__device__ __forceinline__ int key(int row) {
  return ((row >> 1) & 3) | ((~((row >> 3) ^ (row >> 2)) & 1) << 2);
}

// The lane's codes of a 16-row fragment starting at tile row `row0`: its row
// l % 16, the 32 codes from 32 (l / 16) of the block.
__device__ __forceinline__ i32x8 frag(const unsigned char* tile, int row0, int lane) {
  const int row = row0 + lane % 16, c = 2 * (lane / 16);
  const unsigned char* p = tile + row * kRow;
  const u32x4 lo = *reinterpret_cast<const u32x4*>(p + ((c ^ key(row)) << 4));
  const u32x4 hi = *reinterpret_cast<const u32x4*>(p + (((c + 1) ^ key(row)) << 4));
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
               (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

// As dma16, from a buffer at byte offset voff + soff (soff uniform).
__device__ __forceinline__ void buf_dma16(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff, void* lds) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, voff, soff,
                                           0, 0);
}

// Scale words with any layout: word (row, block) at p[row * r + block * k].
struct Scales {
  const float* p;
  int64_t r, k;
};

// Four neighbouring values of a row to LDS.
__device__ __forceinline__ void put4(float* p, float a, float b, float c, float d) {
  *reinterpret_cast<f32x4*>(p) = f32x4{a, b, c, d};
}
__device__ __forceinline__ void put4(uint16_t* p, float a, float b, float c, float d) {
  *reinterpret_cast<uint2*>(p) =
      make_uint2(f32_to_bf16_bits(a) | static_cast<uint32_t>(f32_to_bf16_bits(b)) << 16,
                 f32_to_bf16_bits(c) | static_cast<uint32_t>(f32_to_bf16_bits(d)) << 16);
}

// A wave's fragments to y, 32 rows at a time through its own room in LDS, so
// that they leave as whole runs of y's rows (a lane's own values lie in one
// row, a column apart from its neighbour's: stored directly they took a third
// of the time of a large product).  The wave's part starts at row rw, column
// cw of the tile at (m0, n0), whose last row and column are mr and nr.
template <int FM, int FN, int TN, typename OUT>
__device__ __forceinline__ void store_tile(OUT* room, int lane, const f32x4 (&acc)[FN][FM], OUT* y,
                                           int64_t m0, int rw, int mr, int64_t N, int64_t n0, int cw,
                                           int nr) {
  constexpr int kVec = 16 / static_cast<int>(sizeof(OUT)), kPitch = TN + kVec, kChunks = TN / kVec;
  const bool vec = N % kVec == 0;  // every row of y then starts 16-byte aligned
#pragma unroll
  for (int m = 0; m < FM; m += 2) {
    const int rows = m + 1 < FM ? 32 : 16;  // known once unrolled
#pragma unroll
    for (int i = 0; i < rows / 16; ++i)
#pragma unroll
      for (int n = 0; n < FN; ++n)
        put4(room + (16 * i + lane % 16) * kPitch + 16 * n + 4 * (lane / 16), acc[n][m + i][0],
             acc[n][m + i][1], acc[n][m + i][2], acc[n][m + i][3]);
    wave_order();
    const int row0 = rw + 16 * m;
    if (vec) {
#pragma unroll
      for (int i = 0; i < rows * kChunks / kWave; ++i) {
        const int r = (i * kWave + lane) / kChunks, c = (i * kWave + lane) % kChunks * kVec;
        const u32x4 v = *reinterpret_cast<const u32x4*>(room + r * kPitch + c);
        // N % kVec == 0: a chunk that starts inside the row ends inside it
        if (row0 + r <= mr && cw + c <= nr) st16(y + (m0 + row0 + r) * N + n0 + cw + c, v);
      }
    } else {
      for (int i = 0; i < rows * TN / kWave; ++i) {
        const int r = (i * kWave + lane) / TN, c = (i * kWave + lane) % TN;
        const OUT v = room[r * kPitch + c];
        if (row0 + r <= mr && cw + c <= nr) y[(m0 + row0 + r) * N + n0 + cw + c] = v;
      }
    }
    wave_order();
  }
}

// A BM x BN tile of y.  The workgroup's waves form KS groups of WM x WN, each
// wave with a (BM/WM) x (BN/WN) part of the tile; group g takes the blocks g,
// g + KS, ... along k, so that small tiles still have many waves and long
// copies (the groups' sums meet in LDS at the end, added in group order).
// The b matrix is the matrix cores' row operand, so a lane holds outputs of
// one row of y: the row's scale is one register, and the columns' scales are
// uniform over a wave (sb for 128 x 128 blocks) or lie in LDS (ROWS: sb for
// each row of b).  Tiles and scale words are copied straight to LDS through a
// ring of ST stages of KS blocks, ST - 1 of them in flight while one is
// multiplied.  Each group copies its own block; a wave issues the same number
// of copies for every block, so "a stage has landed" is a count of
// outstanding copies.
// Few rows are bound by that chain (fill the ring, five or ten stages, join the
// groups, store), not by the host: called back to back from C, 1 x 5,120 x
// 5,120 takes 7.7 us on one set of operands, which stay in the last-level cache
// (3.4 TB/s), and 8.7 over sixteen; 64 x 5,125 x 2,560, 161 workgroups, 6.7 and
// 7.5 (6.3 and 7.1 with 5,120 outputs, whose rows are stored in whole pieces).
template <int BM, int BN, int KS, int WM, int WN, int ST, bool ROWS, typename OUT>
__global__ __launch_bounds__(64 * KS * WM * WN) void matmul_tile(
    const uint8_t* __restrict__ a, Scales sa, const uint8_t* __restrict__ b, Scales sb,
    OUT* __restrict__ y, int64_t M, int64_t N, int64_t K) {
  constexpr int G = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int kScales = (BM + BN) * kRow;                    // scale words after the tiles
  constexpr int kWords = ((BM + BN + 63) / 64) * 64;           // copied 64 at a time
  constexpr int kBlock = kScales + kWords * 4, kStage = KS * kBlock;
  constexpr int kPart = FN * FM * 4 * kWave * G * 4;          // a group's sums
  constexpr int kRoom = 32 * (TN * static_cast<int>(sizeof(OUT)) + 16);  // a wave's, to store from
  constexpr int kLds = std::max({ST * kStage, (KS - 1) * kPart, G * kRoom});
  static_assert(TM % 32 == 0 && TN % 16 == 0 && TN <= 128, "tile shape");
  __shared__ __attribute__((aligned(16))) unsigned char lds[kLds];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int g = wave / G, wg = wave % G, wm = wg / WN, wn = wg % WN;
  const uint32_t nt = static_cast<uint32_t>((N + BN - 1) / BN);
  const int64_t m0 = static_cast<int64_t>(blockIdx.x / nt) * BM, n0 = static_cast<int64_t>(blockIdx.x % nt) * BN;
  const int nkb = static_cast<int>(K / 128);

  // rows past the matrices' ends repeat the last one (whole 8-row regions of
  // a past it are not copied); nothing of them is stored
  const int mr = static_cast<int>(min(M - m0, static_cast<int64_t>(BM))) - 1;
  const int nr = static_cast<int>(min(N - n0, static_cast<int64_t>(BN))) - 1;
  constexpr int NA = (BM / 8 + G - 1) / G, NB = (BN / 8 + G - 1) / G, NS = (kWords / 64 + G - 1) / G;
  const uint8_t* at0 = a + m0 * K;
  const uint8_t* bt0 = b + n0 * K;
  uint32_t aoff[NA], boff[NB];
  const float* soff[NS];
  int64_t sstep[NS];
  int copies = 0;
#pragma unroll
  for (int i = 0; i < NA; ++i) {
    const int row = 8 * (wg + i * G) + lane / 8;
    aoff[i] = static_cast<uint32_t>(min(row, mr)) * static_cast<uint32_t>(K) + (((lane % 8) ^ key(row)) << 4);
    copies += (8 * (wg + i * G) <= mr) ? 1 : 0;
  }
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int row = 8 * (wg + i * G) + lane / 8;
    boff[i] = static_cast<uint32_t>(min(row, nr)) * static_cast<uint32_t>(K) + (((lane % 8) ^ key(row)) << 4);
    copies += (8 * (wg + i * G) < BN) ? 1 : 0;
  }
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const int w = 64 * (wg + i * G) + lane;  // tile rows of a, then of b
    const int64_t r = w < BM ? m0 + min(w, mr) : n0 + min(w - BM, nr);
    soff[i] = w < BM ? sa.p + r * sa.r + g * sa.k : sb.p + (ROWS ? r : r / 128) * sb.r + g * sb.k;
    sstep[i] = (w < BM ? sa.k : sb.k) * KS;  // from one of the group's blocks to its next
    copies += (64 * (wg + i * G) < kWords) ? 1 : 0;
  }
  auto copy = [&](int st, int kb) {
    unsigned char* at = lds + st * kStage + g * kBlock;
    unsigned char* bt = at + BM * kRow;
#pragma unroll
    for (int i = 0; i < NB; ++i)
      if (8 * (wg + i * G) < BN) dma16(bt0 + (boff[i] + kb * 128), bt + (wg + i * G) * 1024);
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (8 * (wg + i * G) <= mr) dma16(at0 + (aoff[i] + kb * 128), at + (wg + i * G) * 1024);
#pragma unroll
    for (int i = 0; i < NS; ++i)
      if (64 * (wg + i * G) < kWords) {
        dma4(soff[i], at + kScales + (wg + i * G) * 256);
        soff[i] += sstep[i];  // the blocks are copied in order
      }
  };

  constexpr bool kWide = sizeof(OUT) == 4;  // binary32 results: binary32 sums
  using Frag = std::conditional_t<kWide, Wide, i32x8>;
  auto operand = [](i32x8 q) {
    if constexpr (kWide) return widen(q);
    else return q;
  };
  auto product = [](const Frag& x, const Frag& w) {
    if constexpr (kWide) return mfma_wide(x, w, f32x4{});
    else return mfma_e4m3(x, w, f32x4{});
  };
  f32x4 acc[FN][FM];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[n][m] = f32x4{};

  const int stages = (nkb + KS - 1) / KS;
  // copies of this wave's block of stage s (none where the last stage has no block for it)
  auto issued = [&](int s) { return s < stages && s * KS + g < nkb ? copies : 0; };
#pragma unroll
  for (int s = 0; s < ST - 1; ++s)
    if (s * KS + g < nkb) copy(s, s * KS + g);
  {
    int later = 0;
#pragma unroll
    for (int s = 1; s < ST - 1; ++s) later += issued(s);
    tile::ring_barrier(later);
  }
  int st = 0;
  for (int s = 0; s < stages; ++s) {
    const int kn = (s + ST - 1) * KS + g;
    if (kn < nkb) copy(st == 0 ? ST - 1 : st - 1, kn);  // the stage multiplied last time
    if (s * KS + g < nkb) {
      const unsigned char* at = lds + st * kStage + g * kBlock;
      const unsigned char* bt = at + BM * kRow;
      const float* sat = reinterpret_cast<const float*>(at + kScales) + wm * TM;
      const float* sbt = reinterpret_cast<const float*>(at + kScales) + BM + wn * TN;
      Frag bf[FN];
#pragma unroll
      for (int n = 0; n < FN; ++n) bf[n] = operand(frag(bt, wn * TN + 16 * n, lane));
      // Products of row fragment m beside the multiply-adds of fragment m - 1
      // (one product, then four of those), its successor's codes on their way.
      f32x4 p[2][FN];
      float sc[2];
      auto add = [&](int m, int n) {
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float sr = ROWS ? sc[m & 1] * sbt[16 * n + 4 * (lane / 16) + r] : sc[m & 1];
          acc[n][m][r] = __builtin_fmaf(p[m & 1][n][r], sr, acc[n][m][r]);
        }
      };
      i32x8 next = frag(at, wm * TM, lane);
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const Frag af = operand(next);
        if (m + 1 < FM) next = frag(at, wm * TM + 16 * (m + 1), lane);
        sc[m & 1] = sat[16 * m + lane % 16] * (ROWS ? 1.0f : sbt[0]);
#pragma unroll
        for (int n = 0; n < FN; ++n) {
          p[m & 1][n] = product(bf[n], af);
          if (m > 0) add(m - 1, n);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int n = 0; n < FN; ++n) add(FM - 1, n);
    }
    int later = 0;
#pragma unroll
    for (int i = 2; i < ST; ++i) later += issued(s + i);
    tile::ring_barrier(later);  // stage s + 1 has landed, stage s is read
    st = (st == ST - 1) ? 0 : st + 1;
  }

  if constexpr (KS > 1) {
    f32x4* part = reinterpret_cast<f32x4*>(lds);
    if (g > 0) {
#pragma unroll
      for (int n = 0; n < FN; ++n)
#pragma unroll
        for (int m = 0; m < FM; ++m)
          part[((((g - 1) * G + wg) * FN + n) * FM + m) * kWave + lane] = acc[n][m];
    }
    __syncthreads();
    if (g == 0)
#pragma unroll
      for (int o = 0; o < KS - 1; ++o)
#pragma unroll
        for (int n = 0; n < FN; ++n)
#pragma unroll
          for (int m = 0; m < FM; ++m)
            acc[n][m] += part[(((o * G + wg) * FN + n) * FM + m) * kWave + lane];
    __syncthreads();
    if (g > 0) return;
  }
  store_tile<FM, FN, TN>(reinterpret_cast<OUT*>(lds + wg * kRoom), lane, acc, y, m0, wm * TM, mr, N, n0,
                         wn * TN, nr);
}

// ---- many rows -------------------------------------------------------------
// 256-column tiles of BM rows, eight waves of BM/2 x 64, one
// workgroup per compute unit, two stages of one block.  The next stage's
// copies are spread over the products (nine instructions a wave: issued
// together they fill the unit's texture path and hold up every wave's LDS
// reads).
//
// 8,192 x 5,120 x 5,120 in bf16: 207 us on one set of operands, 217 over three
// (2.0 PFLOP/s; the instruction alone runs at 4.0), the matrix cores busy 42% of
// the cycles: copies, scaling and the wait at a block's end delay products
// instead of running beside them.  With any one of them left out, on codes of
// zero, so that the clock stays: 141, 152 and 139 us against 174.  Real codes
// cost the clock under power another 23.
//
// Order of the tiles: workgroups are dealt round-robin to the 8 XCDs, each
// with its own L2, so workgroup b takes the (b / 8) % 32-th tile of chunk
// b % 8 of its round of 256 (one tile per compute unit), a chunk being about
// 4 tiles along m by 8 along n that share their operands in one L2.  The last
// round's tiles, when they are at most a half or a quarter of the compute
// units, are cut into halves or quarters along m, so that every unit has a
// piece of it.
struct TileGrid {
  int full;     // workgroups of whole rounds of 256 tiles
  int rest;     // tiles of the last round
  int split;    // pieces each is cut into: 1, 2 or 4
  int nt, mt;   // tiles along n and m
};

template <int BM, bool ROWS, typename OUT>
struct Many {
  static constexpr bool kWide = sizeof(OUT) == 4;
  static constexpr int BN = 256, TN = 64, FN = TN / 16, W = 8;
  static constexpr int AR = (BM + 63) / 64 * 64;  // rows of room for a's part: copies are of 64
  static constexpr int kScales = (AR + BN) * kRow, kStage = kScales + (AR + BN) * 4;
  static constexpr int kRoom = 32 * (TN * static_cast<int>(sizeof(OUT)) + 16);
  static constexpr int kLds = std::max(2 * kStage, W * kRoom);
  using Frag = std::conditional_t<kWide, Wide, i32x8>;

  // FM: 16-row fragments of a wave (its share of 2 * 16 FM rows).
  template <int FM>
  static __device__ __forceinline__ void run(unsigned char* lds, const uint8_t* a, Scales sa,
                                             const uint8_t* b, Scales sb, OUT* y, int64_t M,
                                             int64_t N, int64_t K, int64_t m0, int64_t n0) {
    constexpr int R = 32 * FM, TM = 16 * FM;  // rows of the piece, of a wave
    constexpr int NA = (R + 63) / 64, NB = BN / 64;  // copies of 8 rows a wave
    const int lane = threadIdx.x % kWave;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int wm = wave / 4, wn = wave % 4;
    const int nkb = static_cast<int>(K / 128);
    // rows past the matrices' ends repeat the last one; nothing of them is stored
    const int mr = static_cast<int>(min(M - m0, static_cast<int64_t>(R))) - 1;
    const int nr = static_cast<int>(min(N - n0, static_cast<int64_t>(BN))) - 1;
    // One lane offset serves every copy of an operand: copy c's rows are 64 c
    // further, a scalar offset, and the buffer's extent ends with the last
    // row (what stands in LDS beyond it is not stored).  The extent is
    // compared with the lane's offset after subtracting the scalar one, so a
    // copy of only missing rows repeats the first instead.
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(a + m0 * K, static_cast<uint32_t>(mr + 1) * static_cast<uint32_t>(K));
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(b + n0 * K, static_cast<uint32_t>(nr + 1) * static_cast<uint32_t>(K));
    const int crow = 8 * wave + lane / 8;
    const uint32_t coff = static_cast<uint32_t>(crow) * static_cast<uint32_t>(K) + (((lane % 8) ^ key(crow)) << 4);
    uint32_t astep[NA], bstep[NB];
#pragma unroll
    for (int i = 0; i < NA; ++i) astep[i] = 64 * i <= mr ? 64u * i * static_cast<uint32_t>(K) : 0u;
#pragma unroll
    for (int i = 0; i < NB; ++i) bstep[i] = 64 * i <= nr ? 64u * i * static_cast<uint32_t>(K) : 0u;
    // scale words: waves 0-3 of the b rows, the others of the a rows (where
    // there are fewer, two waves copy the same)
    const int sw = wave < 4 ? wave : (wave - 4) % (AR / 64), srow = 64 * sw + lane;
    const float* soff;
    if (wave < 4) {
      const int64_t r = n0 + min(srow, nr);
      soff = sb.p + (ROWS ? r : r / 128) * sb.r;
    } else {
      soff = sa.p + (m0 + min(srow, mr)) * sa.r;
    }
    const int64_t sstep = wave < 4 ? sb.k : sa.k;
    const int sdst = kScales + (wave < 4 ? AR * 4 : 0) + sw * 256;
    auto copy = [&](int st, int kb, int c) {
      unsigned char* t = lds + st * kStage;
      if (c < NB) buf_dma16(rb, coff, bstep[c < NB ? c : 0] + kb * 128, t + AR * kRow + (wave + W * c) * 1024);
      else if (c < NB + NA) buf_dma16(ra, coff, astep[c < NB ? 0 : c - NB < NA ? c - NB : 0] + kb * 128, t + (wave + W * (c - NB)) * 1024);
      else dma4(soff + kb * sstep, t + sdst);
    };
    auto operand = [](i32x8 q) {
      if constexpr (kWide) return widen(q);
      else return q;
    };
    f32x4 acc[FN][FM];
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int m = 0; m < FM; ++m) acc[n][m] = f32x4{};
    constexpr int kCopies = NA + NB + 1, kEach = (kCopies + FM * FN - 1) / (FM * FN);
    constexpr int kLag = 3;  // products between a product and its multiply-adds
    if (nkb > 0)
#pragma unroll
      for (int c = 0; c < kCopies; ++c) copy(0, 0, c);
    __syncthreads();
    // the lane's place in its fragments: chunks 2 (l / 16) and the next one
    const int f0 = (lane % 16) * kRow + ((2 * (lane / 16) ^ key(lane % 16)) << 4);
    auto codes = [&](const unsigned char* t) {
      const u32x4 lo = *reinterpret_cast<const u32x4*>(t + f0);
      const u32x4 hi = *reinterpret_cast<const u32x4*>(t + (f0 ^ 16));
      return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
                   (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
    };
    for (int kb = 0; kb < nkb; ++kb) {
      const unsigned char* at = lds + (kb & 1) * kStage + wm * TM * kRow;
      const unsigned char* bt = lds + (kb & 1) * kStage + (AR + wn * TN) * kRow;
      const float* sat = reinterpret_cast<const float*>(lds + (kb & 1) * kStage + kScales) + wm * TM + lane % 16;
      const float* sbt = reinterpret_cast<const float*>(lds + (kb & 1) * kStage + kScales) + AR + wn * TN;
      const int kn = min(kb + 1, nkb - 1);  // the last stage's copies are not used
      Frag bf[FN];
      f32x4 sr[ROWS ? FN : 1];
      float sc[2];
      i32x8 next = codes(at);
      sc[0] = sat[0] * (ROWS ? 1.0f : sbt[0]);
#pragma unroll
      for (int n = 0; n < FN; ++n) bf[n] = operand(codes(bt + 16 * n * kRow));
      if (ROWS) {
#pragma unroll
        for (int n = 0; n < FN; ++n)
          sr[ROWS ? n : 0] = *reinterpret_cast<const f32x4*>(sbt + 16 * n + 4 * (lane / 16));
      }
      constexpr int kHeld = kWide ? 2 * FN : kLag + 1;
      f32x4 p[kHeld];
      auto add = [&](int i) {  // the block's sums of product i into the result's
        const int m = i / FN, n = i % FN;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          acc[n][m][r] = __builtin_fmaf(p[i % kHeld][r],
                                        ROWS ? sc[m & 1] * sr[ROWS ? n : 0][r] : sc[m & 1], acc[n][m][r]);
      };
#pragma unroll
      for (int m = 0; m < FM; ++m) {
        const Frag af = operand(next);
        float scn = 0.0f;
        if constexpr (kWide) {
          // A product is four dependent instructions: those of the row
          // fragment's FN products take turns, the multiply-adds of the
          // fragment before beside them (224 rows: 117 us for 5,120 x 2,560 x
          // 4,224 against 120 with them behind their own products).
          static_assert(FN == 4, "one product's multiply-adds beside each turn");
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int i = m * 4 + j;
#pragma unroll
            for (int n = 0; n < FN; ++n)
              p[(m * FN + n) % kHeld] =
                  mfma16x16x32(bf[n].f[j], af.f[j], j ? p[(m * FN + n) % kHeld] : f32x4{});
            __builtin_amdgcn_sched_barrier(0);
            if (m > 0) add(i - FN);
            if (j == 0 && m + 1 < FM) {
              next = codes(at + 16 * (m + 1) * kRow);
              scn = sat[16 * (m + 1)];
            }
#pragma unroll
            for (int c = i * kEach; c < (i + 1) * kEach && c < kCopies; ++c) copy((kb + 1) & 1, kn, c);
            __builtin_amdgcn_sched_barrier(0);
          }
          if (m == FM - 1)
#pragma unroll
            for (int n = 0; n < FN; ++n) add(m * FN + n);
          if (m + 1 < FM) sc[(m + 1) & 1] = scn * (ROWS ? 1.0f : sbt[0]);
          __builtin_amdgcn_sched_barrier(0);
        } else {
          // Beside each product the multiply-adds of the third one before it
          // (whose sums are ready by then), the next row fragment's codes and
          // the next stage's copies on their way.
#pragma unroll
          for (int n = 0; n < FN; ++n) {
            const int i = m * FN + n;
            p[i % kHeld] = mfma_e4m3(bf[n], af, f32x4{});
            __builtin_amdgcn_sched_barrier(0);
            if (n == 0 && m + 1 < FM) {
              next = codes(at + 16 * (m + 1) * kRow);
              scn = sat[16 * (m + 1)];
            }
            if (i >= kLag) add(i - kLag);
#pragma unroll
            for (int c = i * kEach; c < (i + 1) * kEach && c < kCopies; ++c) copy((kb + 1) & 1, kn, c);
            if (n == FN - 1 && m + 1 < FM) sc[(m + 1) & 1] = scn * (ROWS ? 1.0f : sbt[0]);
            __builtin_amdgcn_sched_barrier(0);
          }
        }
      }
      if (!kWide)
#pragma unroll
        for (int i = FM * FN - kLag; i < FM * FN; ++i) add(i);
      __syncthreads();  // waits for this wave's copies, then for every wave
    }
    store_tile<FM, FN, TN>(reinterpret_cast<OUT*>(lds + wave * kRoom), lane, acc, y, m0, wm * TM, mr, N,
                           n0, wn * TN, nr);
  }
};

template <int BM, bool ROWS, typename OUT>
__global__ __launch_bounds__(512, 2) void matmul_many(
    const uint8_t* __restrict__ a, Scales sa, const uint8_t* __restrict__ b, Scales sb,
    OUT* __restrict__ y, int64_t M, int64_t N, int64_t K, TileGrid t) {
  using T = Many<BM, ROWS, OUT>;
  __shared__ __attribute__((aligned(16))) unsigned char lds[T::kLds];
  int L = blockIdx.x, piece = 0, split = 1;
  if (L < t.full) {
    L = (L / 256 * 8 + L % 8) * 32 + L / 8 % 32;
  } else {
    const int u = L - t.full, per = (t.rest * t.split + 7) / 8;  // an XCD's pieces
    const int i = u % 8 * per + u / 8;
    if (u / 8 >= per || i >= t.rest * t.split) return;
    split = t.split;
    L = t.full + i / split;
    piece = i % split;
  }
  const int band = L / (4 * t.nt), gm = min(4, t.mt - 4 * band), j = L - band * 4 * t.nt;
  const int quad = j / (gm * 8), rem = j - quad * gm * 8;
  const int64_t n0 = static_cast<int64_t>(quad * 8 + rem / gm) * T::BN;
  const int64_t m0 = static_cast<int64_t>(4 * band + rem % gm) * BM + piece * (BM / split);
  if (m0 >= M) return;
  constexpr int FM = BM / 32;
  if (split == 1) T::template run<FM>(lds, a, sa, b, sb, y, M, N, K, m0, n0);
  if constexpr (FM % 2 == 0)
    if (split == 2) T::template run<FM / 2>(lds, a, sa, b, sb, y, M, N, K, m0, n0);
  if constexpr (FM % 4 == 0)
    if (split == 4) T::template run<FM / 4>(lds, a, sa, b, sb, y, M, N, K, m0, n0);
}

// Maximum over a row of 16 lanes, in each of them, by data-parallel moves.
__device__ __forceinline__ float row_max(float v) {
  auto step = [&](int o) { v = fmaxf(v, __builtin_bit_cast(float, o)); };
  step(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, false));   // neighbours
  step(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, false));   // pairs
  step(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xF, 0xF, false));  // half rows
  step(__builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xF, 0xF, false));  // the row
  return v;
}

// ---- quantisation in both orientations --------------------------------------
// One workgroup per 128 x 128 tile of v; thread (rg, cg) holds rows 4 rg .. +4
// and columns 8 cg .. +8, packed as they lie in memory.  A scale covers 128
// columns of a row and, for the transposed codes, 128 rows of a column (BLOCK:
// the whole tile, both ways).  The transposed codes cross the tile through
// LDS, so v is read once and both codes leave in whole lines.  Rows and
// columns past v's end count as zeros.  The scales of rows and columns leave
// block-major, 128 consecutive words a tile, as the products' copies read
// them.  4,099 x 5,120 bf16 both ways, 84 MB: 22.5 us (27 with the columns'
// maxima of the eight waves read by every thread, 38 with the plain division
// and half the threads).  Rows that are not a multiple of 8 columns are read
// value by value: 4,099 x 5,125 takes 41 us.
template <typename IO, bool BLOCK, bool VEC>
__global__ __launch_bounds__(512) void quant_2d(const IO* __restrict__ v, int64_t rows,
                                                int64_t cols, int64_t ncb, uint8_t* __restrict__ q,
                                                float* __restrict__ s, uint8_t* __restrict__ qt,
                                                float* __restrict__ st) {
  constexpr int P = 4, kWaves = 8;
  __shared__ __attribute__((aligned(16))) uint32_t tile[128][32];
  __shared__ __attribute__((aligned(16))) uint32_t top[128];  // columns' maxima (bits of floats >= 0)
  __shared__ float sh[kWaves];
  const int tid = threadIdx.x, cg = tid % 16, rg = tid / 16, wave = tid / kWave;
  if (!BLOCK) {
    if (tid < 128) top[tid] = 0;
    __syncthreads();
  }
  const int64_t rb = blockIdx.x / ncb, cb = blockIdx.x % ncb;
  const int64_t nrb = (rows + 127) / 128;
  const int64_t r0 = rb * 128 + P * rg, c0 = cb * 128 + 8 * cg;
  constexpr int kWords = sizeof(IO) == 2 ? 1 : 2;
  u32x4 raw[P][kWords];
#pragma unroll
  for (int p = 0; p < P; ++p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) raw[p][i] = u32x4{0, 0, 0, 0};
    if (r0 + p >= rows) continue;
    const IO* src = v + (r0 + p) * cols + c0;
    if (VEC) {
      if (c0 < cols)
#pragma unroll
        for (int i = 0; i < kWords; ++i) raw[p][i] = ld16(src + i * 4);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c0 + j < cols) {
          if constexpr (sizeof(IO) == 2) raw[p][0][j / 2] |= static_cast<uint32_t>(src[j]) << (16 * (j % 2));
          else raw[p][j / 4][j % 4] = __float_as_uint(src[j]);
        }
    }
  }
  auto value = [&](int p, int j) {
    if constexpr (sizeof(IO) == 2) {
      const uint32_t w = raw[p][0][j / 2];
      return __uint_as_float(j % 2 ? w & 0xFFFF0000u : w << 16);
    } else {
      return __uint_as_float(raw[p][j / 4][j % 4]);
    }
  };
  float rmax[P], cmax[8];
#pragma unroll
  for (int p = 0; p < P; ++p) rmax[p] = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) cmax[j] = 0.0f;
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float m = fabsf(value(p, j));
      rmax[p] = fmaxf(rmax[p], m);
      cmax[j] = fmaxf(cmax[j], m);
    }
  if (BLOCK) {
    float m = fmaxf(fmaxf(rmax[0], rmax[1]), fmaxf(rmax[2], rmax[3]));
    m = row_max(m);
    m = fmaxf(m, __shfl_xor(m, 16));
    m = fmaxf(m, __shfl_xor(m, 32));
    if (tid % kWave == 0) sh[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sh[w]);
#pragma unroll
    for (int p = 0; p < P; ++p) rmax[p] = m;
#pragma unroll
    for (int j = 0; j < 8; ++j) cmax[j] = m;
  } else {
#pragma unroll
    for (int p = 0; p < P; ++p) rmax[p] = row_max(rmax[p]);
    if (qt) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        cmax[j] = fmaxf(cmax[j], __shfl_xor(cmax[j], 16));
        cmax[j] = fmaxf(cmax[j], __shfl_xor(cmax[j], 32));
      }
      if (tid % kWave < 16)
#pragma unroll
        for (int j = 0; j < 8; ++j) atomicMax(&top[8 * cg + j], __float_as_uint(cmax[j]));
    }
  }
  if (q) {
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const BlockDivisor d(rmax[p]);
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = value(p, j);
      const uint2 code = d.codes(x);
      if (r0 + p < rows) {
        *reinterpret_cast<uint2*>(q + (r0 + p) * (ncb * 128) + c0) = code;
        if (!BLOCK && cg == 0) s[cb * rows + r0 + p] = d.s;
      }
    }
    if (BLOCK && tid == 0) s[rb * ncb + cb] = e4m3_scale(rmax[0]);
  }
  if (qt) {
    if (!BLOCK) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) cmax[j] = __uint_as_float(top[8 * cg + j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const BlockDivisor d(cmax[j]);
      const float x[P] = {value(0, j), value(1, j), value(2, j), value(3, j)};
      tile[8 * cg + j][rg ^ (2 * cg)] = d.codes(x);  // spread over the banks
      if (!BLOCK && rg == 0 && c0 + j < cols) st[rb * cols + c0 + j] = d.s;
    }
    if (BLOCK && tid == 0) st[cb * nrb + rb] = e4m3_scale(cmax[0]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = tid / 8 + 64 * i, ch = tid % 8, g = c / 8;
      if (cb * 128 + c >= cols) continue;
      const u32x4 w = *reinterpret_cast<const u32x4*>(&tile[c][(4 * ch) ^ ((2 * g) & 28)]);
      st16(qt + (cb * 128 + c) * (nrb * 128) + rb * 128 + 16 * ch,
           g % 2 ? u32x4{w[2], w[3], w[0], w[1]} : w);
    }
  }
}

// The form of a product: the one whose tiles are estimated to take least time,
// rounds of 256 tiles (one per compute unit) times the time of a tile's
// 128-deep block.  Microseconds a block, from products with N = K = 5120 (bf16
// results: 1 row 8.5 us, 64 rows 12.4, 128 rows 16.7, 256 rows 23, 512 rows 37,
// 1,024 rows 48, 2,048 rows 61, 8,192 rows 215; binary32 results: 64 rows 15.7,
// 256 rows 37, 512 rows 61, 8,192 rows 404):
struct Form {
  int bm, bn;
  float us, wide;      // bf16 results, binary32 results (a negative time: not built)
  float half, quarter; // of the 256-column tiles' halves and quarters in the last round
};
constexpr Form kForms[] = {
    {32, 16, 0.09f, 0.14f, 0, 0},     {32, 32, 0.14f, 0.22f, 0, 0},
    {64, 16, 0.16f, 0.24f, 0, 0},     {64, 32, 0.24f, 0.32f, 0, 0},
    {64, 64, 0.34f, 0.51f, 0, 0},     {128, 64, 0.52f, 0.85f, 0, 0},
    {128, 128, 0.85f, 1.45f, 0, 0},   {128, 256, -1.0f, 2.1f, 1.5f, 1.2f},
    {192, 256, 1.52f, -1.0f, 1.2f, 0}, {224, 256, 1.75f, 3.5f, 0, 0},
    {256, 256, 1.9f, -1.0f, 1.27f, 1.0f}};
constexpr int kFormTiles = 7;  // the forms before are matmul_tile's

TileGrid tile_grid(int64_t M, int64_t N, const Form& f) {
  TileGrid t;
  t.nt = static_cast<int>(ceil_div(N, 256));
  t.mt = static_cast<int>(ceil_div(M, f.bm));
  const int64_t tiles = static_cast<int64_t>(t.nt) * t.mt;
  t.full = static_cast<int>(tiles / 256 * 256);
  t.rest = static_cast<int>(tiles - t.full);
  t.split = 1;
  if (f.half > 0 && t.rest * 2 <= 256) t.split = 2;
  if (f.quarter > 0 && t.rest * 4 <= 256) t.split = 4;
  return t;
}

int choose_form(int64_t M, int64_t N, bool wide) {
  int best = 0;
  float least = 0.0f;
  for (int i = 0; i < static_cast<int>(sizeof(kForms) / sizeof(kForms[0])); ++i) {
    const Form& f = kForms[i];
    const float each = wide ? f.wide : f.us;
    if (each < 0) continue;
    float us;
    if (i < kFormTiles) {
      us = static_cast<float>(ceil_div(ceil_div(M, f.bm) * ceil_div(N, f.bn), 256)) * each;
    } else {
      const TileGrid t = tile_grid(M, N, f);
      us = static_cast<float>(t.full / 256) * each;
      if (t.rest) us += t.split == 1 ? each : t.split == 2 ? f.half : f.quarter;
    }
    if (i == 0 || us < least) {
      least = us;
      best = i;
    }
  }
  return best;
}

template <bool ROWS, typename OUT>
void launch_product(int64_t M, int64_t N, int64_t K, const uint8_t* a, Scales sa,
                    const uint8_t* b, Scales sb, void* y, hipStream_t s) {
  OUT* out = static_cast<OUT*>(y);
  constexpr bool kWide = sizeof(OUT) == 4;
  const int form = choose_form(M, N, kWide);
  if (form >= kFormTiles) {
    const TileGrid t = tile_grid(M, N, kForms[form]);
    const dim3 grid(static_cast<unsigned>(t.full + ceil_div(t.rest * t.split, 8) * 8));
#define BEAM_MANY(BM)                                                                           \
  hipLaunchKernelGGL((matmul_many<BM, ROWS, OUT>), grid, dim3(512), 0, s, a, sa, b, sb, out, M, \
                     N, K, t)
    if constexpr (kWide) {
      if (form == 7) BEAM_MANY(128);
      else BEAM_MANY(224);
    } else {
      if (form == 8) BEAM_MANY(192);
      else if (form == 9) BEAM_MANY(224);
      else BEAM_MANY(256);
    }
#undef BEAM_MANY
    return;
  }
#define BEAM_TILE(BM, BN, KS, WM, WN, ST)                                                       \
  hipLaunchKernelGGL((matmul_tile<BM, BN, KS, WM, WN, ST, ROWS, OUT>),                          \
                     dim3(static_cast<unsigned>(ceil_div(N, BN) * ceil_div(M, BM))),            \
                     dim3(64 * KS * WM * WN), 0, s, a, sa, b, sb, out, M, N, K)
  switch (form) {
    case 0: BEAM_TILE(32, 16, 8, 1, 1, 3); break;
    case 1: BEAM_TILE(32, 32, 4, 1, 1, 3); break;
    case 2: BEAM_TILE(64, 16, 4, 2, 1, 3); break;
    case 3: BEAM_TILE(64, 32, 4, 2, 2, 3); break;
    case 4: BEAM_TILE(64, 64, 2, 2, 2, 3); break;
    case 5: BEAM_TILE(128, 64, 2, 4, 1, 3); break;
    default: BEAM_TILE(128, 128, 1, 2, 4, 3); break;
  }
#undef BEAM_TILE
}

}  // namespace

hipError_t launch_quant_2d(int64_t rows, int64_t cols, int32_t dtype, bool block, const void* v,
                           uint8_t* q, float* s, uint8_t* qt, float* st, hipStream_t stream) {
  const int64_t ncb = ceil_div(cols, 128);
  const dim3 grid(static_cast<unsigned>(ceil_div(rows, 128) * ncb));
  const bool vec = cols % 8 == 0;  // every row then starts 16-byte aligned
#define BEAM_Q3(IO, B, V)                                                                     \
  hipLaunchKernelGGL((quant_2d<IO, B, V>), grid, dim3(512), 0, stream,                        \
                     static_cast<const IO*>(v), rows, cols, ncb, q, s, qt, st)
#define BEAM_Q2(IO, B)              \
  do {                              \
    if (vec) BEAM_Q3(IO, B, true);  \
    else BEAM_Q3(IO, B, false);     \
  } while (0)
#define BEAM_Q1(IO)                 \
  do {                              \
    if (block) BEAM_Q2(IO, true);   \
    else BEAM_Q2(IO, false);        \
  } while (0)
  if (dtype == BEAM_BF16) BEAM_Q1(uint16_t);
  else BEAM_Q1(float);
#undef BEAM_Q1
#undef BEAM_Q2
#undef BEAM_Q3
  return hipGetLastError();
}

hipError_t launch_matmul_e4m3(int64_t M, int64_t N, int64_t K, const uint8_t* a, const float* sa,
                              const int64_t* sa_stride, const uint8_t* b, const float* sb,
                              const int64_t* sb_stride, bool rows, int32_t dtype, void* y,
                              hipStream_t s) {
  const Scales za{sa, sa_stride[0], sa_stride[1]}, zb{sb, sb_stride[0], sb_stride[1]};
  if (dtype == BEAM_BF16) {
    if (rows) launch_product<true, uint16_t>(M, N, K, a, za, b, zb, y, s);
    else launch_product<false, uint16_t>(M, N, K, a, za, b, zb, y, s);
  } else {
    if (rows) launch_product<true, float>(M, N, K, a, za, b, zb, y, s);
    else launch_product<false, float>(M, N, K, a, za, b, zb, y, s);
  }
  return hipGetLastError();
}

}  // namespace beam
