// The product of two e4m3 matrices with a scale for each block of 128 along
// the reduction, y[m,n] = sum_kb sa[m,kb] sb[n,kb] sum_{k in kb} a[m,k] b[n,k],
// dense (the expert path's grouped products are its own kernels), and the
// quantiser that makes its operands in both orientations.
//
// Each 128-deep block's products are summed by the matrix cores into fresh
// registers and added to the result's with one fused multiply-add by the
// block's scale: no ratio of scales is formed, so scales of any size mix.
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
#include <type_traits>

#include "common.h"
#include "internal.h"

namespace beam {
namespace {

constexpr int kRow = 128;  // bytes of a tile row: one block of 128 codes

// D = A(32x64) * B(64x32) + C on e4m3 codes (format 0, unit E8M0 scales).
// Lane l supplies row (l % 32) of A and column (l % 32) of B, codes
// 32*(l/32) .. +32 of the 64-deep slice; element r of lane l is
// C[8*(r/4) + 4*(l/32) + r%4][l % 32].
__device__ __forceinline__ f32x16 mfma_e4m3(i32x8 a, i32x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 127, 0, 127);
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
__device__ __forceinline__ f32x16 mfma_wide(const Wide& a, const Wide& b, f32x16 c) {
#pragma unroll
  for (int j = 0; j < 4; ++j) c = mfma32x32x16(a.f[j], b.f[j], c);
  return c;
}

// Swizzle of a tile row's eight 16-byte chunks: the chunks of any 8
// consecutive rows, and of the even or odd rows of any 16, lie on distinct
// bank groups.
__device__ __forceinline__ int key(int row) { return (row ^ (row >> 3)) & 7; }

// Codes of half h (64 deep) of the lane's row of a 32-row fragment starting
// at tile row `row0`.
__device__ __forceinline__ i32x8 frag(const unsigned char* tile, int row0, int lane, int h) {
  const int row = row0 + lane % 32, c = 4 * h + 2 * (lane / 32);
  const unsigned char* p = tile + row * kRow;
  const u32x4 lo = *reinterpret_cast<const u32x4*>(p + ((c ^ key(row)) << 4));
  const u32x4 hi = *reinterpret_cast<const u32x4*>(p + (((c + 1) ^ key(row)) << 4));
  return i32x8{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3],
               (int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
}

__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(uint16_t* p, float v) { *p = f32_to_bf16_bits(v); }

// A BM x BN tile of y by WM x WN waves of (BM/WM) x (BN/WN).  The b matrix is
// the matrix cores' row operand, so a lane holds outputs of one row of y:
// the row's scale is one register, and the columns' scales are uniform over a
// wave (sb for 128 x 128 blocks) or lie in LDS (ROWS: sb for each row of b).
// Tiles and scale words are copied straight to LDS, two stages of one block
// each: stage kb + 1 is on its way while stage kb is multiplied.
template <int BM, int BN, int WM, int WN, bool ROWS, typename OUT>
__global__ __launch_bounds__(64 * WM * WN) void matmul_tile(
    const uint8_t* __restrict__ a, const float* __restrict__ sa, const uint8_t* __restrict__ b,
    const float* __restrict__ sb, OUT* __restrict__ y, int64_t M, int64_t N, int64_t K) {
  constexpr int W = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 32, FN = TN / 32;
  constexpr int kScales = (BM + BN) * kRow, kStage = kScales + (BM + BN) * 4;
  __shared__ __attribute__((aligned(16))) unsigned char lds[2][kStage];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave / WN, wn = wave % WN;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * BM, n0 = static_cast<int64_t>(blockIdx.x) * BN;
  const int nkb = static_cast<int>(K / 128);

  // rows past the matrices' ends repeat the last one; nothing of them is stored
  const int mr = static_cast<int>(min(M - m0, static_cast<int64_t>(BM))) - 1;
  const int nr = static_cast<int>(min(N - n0, static_cast<int64_t>(BN))) - 1;
  auto copy = [&](int st, int kb) {
#pragma unroll
    for (int i = wave; i < BM / 8; i += W) {
      const int row = 8 * i + lane / 8;
      dma16(a + (m0 + min(row, mr)) * K + kb * 128 + (((lane % 8) ^ key(row)) << 4),
            &lds[st][i * 1024]);
    }
#pragma unroll
    for (int i = wave; i < BN / 8; i += W) {
      const int row = 8 * i + lane / 8;
      dma16(b + (n0 + min(row, nr)) * K + kb * 128 + (((lane % 8) ^ key(row)) << 4),
            &lds[st][BM * kRow + i * 1024]);
    }
#pragma unroll
    for (int i = wave; i < (BM + BN) / 64; i += W) {
      const int row = 64 * i + lane;
      const int64_t r = i < BM / 64 ? m0 + min(row, mr) : n0 + min(row - BM, nr);
      const float* s = i < BM / 64 ? sa + r * nkb : sb + (ROWS ? r : r / 128) * nkb;
      dma4(s + kb, &lds[st][kScales + 256 * i]);
    }
  };

  constexpr bool kWide = sizeof(OUT) == 4;  // binary32 results: binary32 sums
  using Frag = std::conditional_t<kWide, Wide, i32x8>;
  auto operand = [](i32x8 q) {
    if constexpr (kWide) return widen(q);
    else return q;
  };
  auto product = [](const Frag& x, const Frag& w, f32x16 c) {
    if constexpr (kWide) return mfma_wide(x, w, c);
    else return mfma_e4m3(x, w, c);
  };
  f32x16 acc[FN][FM];
#pragma unroll
  for (int n = 0; n < FN; ++n)
#pragma unroll
    for (int m = 0; m < FM; ++m) acc[n][m] = f32x16{};
  if (nkb > 0) copy(0, 0);
  __syncthreads();
  for (int kb = 0; kb < nkb; ++kb) {
    const unsigned char* at = lds[kb & 1];
    const unsigned char* bt = at + BM * kRow;
    const float* sat = reinterpret_cast<const float*>(at + kScales) + wm * TM;
    const float* sbt = reinterpret_cast<const float*>(at + kScales) + BM + wn * TN;
    if (kb + 1 < nkb) copy((kb + 1) & 1, kb + 1);
    Frag bf[FN][2];
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) bf[n][h] = operand(frag(bt, wn * TN + 32 * n, lane, h));
#pragma unroll
    for (int m = 0; m < FM; ++m) {
      const Frag a0 = operand(frag(at, wm * TM + 32 * m, lane, 0));
      const Frag a1 = operand(frag(at, wm * TM + 32 * m, lane, 1));
      const float s = sat[32 * m + lane % 32] * (ROWS ? 1.0f : sbt[0]);
#pragma unroll
      for (int n = 0; n < FN; ++n) {
        f32x16 p = product(bf[n][0], a0, f32x16{});
        p = product(bf[n][1], a1, p);
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const float sr = ROWS ? s * sbt[32 * n + 8 * (r / 4) + 4 * (lane / 32) + r % 4] : s;
          acc[n][m][r] = __builtin_fmaf(p[r], sr, acc[n][m][r]);
        }
      }
    }
    __syncthreads();  // waits for this wave's copies, then for every wave
  }

#pragma unroll
  for (int m = 0; m < FM; ++m) {
    const int row = wm * TM + 32 * m + lane % 32;
    if (row > mr) continue;
    OUT* yr = y + (m0 + row) * N + n0;
#pragma unroll
    for (int n = 0; n < FN; ++n)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int col = wn * TN + 32 * n + 8 * (r / 4) + 4 * (lane / 32) + r % 4;
        if (col <= nr) put(yr + col, acc[n][m][r]);
      }
  }
}

// ---- quantisation in both orientations --------------------------------------
// One workgroup per 128 x 128 tile of v; thread (rg, cg) holds rows 8 rg .. +8
// and columns 8 cg .. +8.  A scale covers 128 columns of a row and, for the
// transposed codes, 128 rows of a column (BLOCK: the whole tile, both ways).
// The transposed codes cross the tile through LDS, so v is read once and both
// codes leave in whole lines.  Rows and columns past v's end count as zeros.
template <typename IO, bool BLOCK, bool VEC>
__global__ __launch_bounds__(256) void quant_2d(const IO* __restrict__ v, int64_t rows,
                                                int64_t cols, int64_t ncb, uint8_t* __restrict__ q,
                                                float* __restrict__ s, uint8_t* __restrict__ qt,
                                                float* __restrict__ st) {
  __shared__ __attribute__((aligned(16))) uint2 tile[128][16];
  __shared__ float sh[4][128];
  const int tid = threadIdx.x, cg = tid % 16, rg = tid / 16, wave = tid / kWave;
  const int64_t rb = blockIdx.x / ncb, cb = blockIdx.x % ncb;
  const int64_t nrb = (rows + 127) / 128;
  const int64_t r0 = rb * 128 + 8 * rg, c0 = cb * 128 + 8 * cg;
  float x[8][8];
#pragma unroll
  for (int p = 0; p < 8; ++p) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[p][j] = 0.0f;
    if (r0 + p >= rows) continue;
    const IO* src = v + (r0 + p) * cols + c0;
    if (VEC) {
      if (c0 < cols) {
        if constexpr (sizeof(IO) == 2) {
          const u32x4 w = ld16(src);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[p][2 * j] = __uint_as_float(w[j] << 16);
            x[p][2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
          }
        } else {
          const u32x4 w0 = ld16(src), w1 = ld16(src + 4);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[p][j] = __uint_as_float(w0[j]);
            x[p][4 + j] = __uint_as_float(w1[j]);
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c0 + j < cols) {
          if constexpr (sizeof(IO) == 2) x[p][j] = bf16_bits_to_f32(src[j]);
          else x[p][j] = src[j];
        }
    }
  }
  float rmax[8], cmax[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) rmax[p] = cmax[p] = 0.0f;
#pragma unroll
  for (int p = 0; p < 8; ++p)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float m = fabsf(x[p][j]);
      rmax[p] = fmaxf(rmax[p], m);
      cmax[j] = fmaxf(cmax[j], m);
    }
  if (BLOCK) {
    float m = 0.0f;
#pragma unroll
    for (int p = 0; p < 8; ++p) m = fmaxf(m, rmax[p]);
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) m = fmaxf(m, __shfl_xor(m, off));
    if (tid % kWave == 0) sh[0][wave] = m;
    __syncthreads();
    m = fmaxf(fmaxf(sh[0][0], sh[0][1]), fmaxf(sh[0][2], sh[0][3]));
#pragma unroll
    for (int p = 0; p < 8; ++p) rmax[p] = cmax[p] = m;
  } else {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
#pragma unroll
      for (int off = 8; off >= 1; off >>= 1) rmax[p] = fmaxf(rmax[p], __shfl_xor(rmax[p], off));
#pragma unroll
      for (int off = 32; off >= 16; off >>= 1) cmax[p] = fmaxf(cmax[p], __shfl_xor(cmax[p], off));
    }
    if (tid % kWave < 16)
#pragma unroll
      for (int j = 0; j < 8; ++j) sh[wave][8 * cg + j] = cmax[j];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j)
      cmax[j] = fmaxf(fmaxf(sh[0][8 * cg + j], sh[1][8 * cg + j]),
                      fmaxf(sh[2][8 * cg + j], sh[3][8 * cg + j]));
  }
  if (q) {
#pragma unroll
    for (int p = 0; p < 8; ++p) {
      const float sc = e4m3_scale(rmax[p]);
      const uint32_t lo = e4m3x4(x[p][0] / sc, x[p][1] / sc, x[p][2] / sc, x[p][3] / sc);
      const uint32_t hi = e4m3x4(x[p][4] / sc, x[p][5] / sc, x[p][6] / sc, x[p][7] / sc);
      if (r0 + p < rows) {
        *reinterpret_cast<uint2*>(q + (r0 + p) * (ncb * 128) + c0) = make_uint2(lo, hi);
        if (!BLOCK && cg == 0) s[(r0 + p) * ncb + cb] = sc;
      }
    }
    if (BLOCK && tid == 0) s[rb * ncb + cb] = e4m3_scale(rmax[0]);
  }
  if (qt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float sc = e4m3_scale(cmax[j]);
      const uint32_t lo = e4m3x4(x[0][j] / sc, x[1][j] / sc, x[2][j] / sc, x[3][j] / sc);
      const uint32_t hi = e4m3x4(x[4][j] / sc, x[5][j] / sc, x[6][j] / sc, x[7][j] / sc);
      tile[8 * cg + j][rg ^ cg] = make_uint2(lo, hi);  // spread over the banks
      if (!BLOCK && rg == 0 && c0 + j < cols) st[(c0 + j) * nrb + rb] = sc;
    }
    if (BLOCK && tid == 0) st[cb * nrb + rb] = e4m3_scale(cmax[0]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = tid / 8 + 32 * i, ch = tid % 8, g = c / 8;
      if (cb * 128 + c >= cols) continue;
      const uint2 lo = tile[c][(2 * ch) ^ g], hi = tile[c][(2 * ch + 1) ^ g];
      st16(qt + (cb * 128 + c) * (nrb * 128) + rb * 128 + 16 * ch, u32x4{lo.x, lo.y, hi.x, hi.y});
    }
  }
}

}  // namespace

hipError_t launch_quant_2d(int64_t rows, int64_t cols, int32_t dtype, bool block, const void* v,
                           uint8_t* q, float* s, uint8_t* qt, float* st, hipStream_t stream) {
  const int64_t ncb = ceil_div(cols, 128);
  const dim3 grid(static_cast<unsigned>(ceil_div(rows, 128) * ncb));
  const bool vec = cols % 8 == 0;  // every row then starts 16-byte aligned
#define BEAM_Q3(IO, B, V)                                                                     \
  hipLaunchKernelGGL((quant_2d<IO, B, V>), grid, dim3(256), 0, stream,                        \
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
                              const uint8_t* b, const float* sb, bool rows, int32_t dtype,
                              void* y, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(ceil_div(N, 128)), static_cast<unsigned>(ceil_div(M, 128)));
#define BEAM_MM2(R, OUT)                                                                      \
  hipLaunchKernelGGL((matmul_tile<128, 128, 2, 2, R, OUT>), grid, dim3(256), 0, s, a, sa, b,  \
                     sb, static_cast<OUT*>(y), M, N, K)
#define BEAM_MM1(OUT)             \
  do {                            \
    if (rows) BEAM_MM2(true, OUT); \
    else BEAM_MM2(false, OUT);    \
  } while (0)
  if (dtype == BEAM_BF16) BEAM_MM1(uint16_t);
  else BEAM_MM1(float);
#undef BEAM_MM1
#undef BEAM_MM2
  return hipGetLastError();
}

}  // namespace beam
