// Declarations shared by the operators around a paged key-value cache
// (serve.cpp, rope.hip, attention.hip, pages.hip, score.hip).
#pragma once

#include <type_traits>

#include "common.h"
#include "internal.h"

namespace beam {

// A paged cache: keys and values, strides in elements.
struct Cache {
  void* k;
  void* v;
  int64_t page_stride, token_stride, head_stride;
  const int32_t* tables;  // [seqs, cols]
  int64_t seqs;
  int32_t pages, cols;
  int32_t shift;  // page_size = 1 << shift
};

constexpr int kMaxHeadDim = 256;

// rope.hip: norms and rotation of attention heads
struct RopeArgs {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;  // elements between tokens
  const float* wq;
  const float* wk;
  const int32_t* pos;
  const double* inv_freq;
  void* q_out;
  void* k_out;
  Cache cache;  // k null: none
  const int32_t* rows;
  int64_t T;
  int32_t Hq, Hkv, D, rot;
  float eps, temp_length, temp_exponent;
  bool interleaved;
};
struct RopeGradArgs {
  RopeArgs f;  // the forward's inputs
  const void* dq_out;
  const void* dk_out;
  void* dq;
  void* dk;
  float* part;  // workspace [groups][2][D]
};
int rope_grad_groups(int64_t T);
hipError_t launch_qk_norm_rope(const RopeArgs& a, int32_t dtype, hipStream_t s);
hipError_t launch_qk_norm_rope_backward(const RopeGradArgs& a, int32_t dtype, float* d_wq,
                                        float* d_wk, hipStream_t s);

// attention.hip: attention of one token of each sequence over a paged cache
struct AttendArgs {
  const void* q;     // [seqs, Hq, D]
  const void* gate;  // [seqs, Hq, D] or null
  Cache cache;
  const int32_t* lengths;
  void* out;
  float* lse;
  float* part;  // workspace
  int32_t Hq, Hkv, D;
  int32_t window;  // 0: none
  float scale;
};
size_t attend_workspace(int64_t seqs, int Hq, int Hkv, int D);
hipError_t launch_paged_attention(const AttendArgs& a, int32_t dtype, hipStream_t s);

// pages.hip: the cache's page tables
struct PageArgs {
  int64_t old_rows, rows, cols, pages;
  int32_t shift;
  const int32_t* tables;
  const int32_t* lengths;
  const int32_t* refs;
  const int32_t* parents;
  const int32_t* grow;
  int32_t* tables_out;
  int32_t* lengths_out;
  int32_t* refs_out;
  int32_t* new_id;  // compaction
  int32_t* count;   // missing pages, or used ones
};
size_t pages_workspace(int64_t pages, int64_t rows);
hipError_t launch_pages_copy(const beam_moe_pools& p, int64_t pages, int64_t n, const int32_t* src,
                             const int32_t* dst, hipStream_t s);
hipError_t launch_pages_update(const PageArgs& a, const beam_moe_pools& p, void* ws, hipStream_t s);
hipError_t launch_pages_compact(const PageArgs& a, const beam_moe_pools& p, void* ws,
                                hipStream_t s);

// score.hip: log probabilities of tokens
struct ScoreArgs {
  const void* logits;
  int64_t stride;
  const int64_t* targets;
  float softcap, scale;
  float* logprobs;
  float* entropy;
  float* lse;
  int32_t* top_ids;
  float* top_logprobs;
  int64_t T;
  int32_t V, top;
};
struct ScoreGradArgs {
  const void* logits;
  int64_t stride;
  const int64_t* targets;
  float softcap, scale;
  const float* lse;
  const float* entropy;
  const float* d_logprobs;
  const float* d_entropy;
  void* d_logits;
  int64_t d_stride;
  int64_t T;
  int32_t V;
};
constexpr int kMaxTop = 16;
int64_t score_pieces_count(int64_t T, int64_t V);  // workgroups of a call
size_t score_workspace(int64_t T, int64_t V, int top);
hipError_t launch_token_logprobs(const ScoreArgs& a, int32_t dtype, void* ws, hipStream_t s);
hipError_t launch_token_logprobs_backward(const ScoreGradArgs& a, int32_t dtype, hipStream_t s);

// Eight values of a type as they lie in memory, and as binary32.
template <typename IO>
struct Eight {
  static constexpr int kWords = static_cast<int>(sizeof(IO)) / 2;
  u32x4 w[kWords];
  __device__ __forceinline__ void load(const IO* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = ld16(p + i * (8 / kWords));
  }
  // (Past the caches' usual order: head norms of 16,381 tokens 101 us instead of
  // 106, a training step of 8,191 119 instead of 128.)
  __device__ __forceinline__ void store(IO* p) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i)
      __builtin_nontemporal_store(w[i], reinterpret_cast<u32x4*>(p + i * (8 / kWords)));
  }
  // Makes the compiler forget values it has unpacked (it would rather keep them,
  // in twice the registers, than unpack again).
  __device__ __forceinline__ void repack() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) asm volatile("" : "+v"(w[i]));
  }
  __device__ __forceinline__ float get(int j) const {
    if constexpr (sizeof(IO) == 2)
      return __uint_as_float(j % 2 ? w[0][j / 2] & 0xFFFF0000u : w[0][j / 2] << 16);
    else
      return __uint_as_float(w[j / 4][j % 4]);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    if constexpr (sizeof(IO) == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        w[0][j] = f32_to_bf16_bits(v[2 * j]) |
                  static_cast<uint32_t>(f32_to_bf16_bits(v[2 * j + 1])) << 16;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j / 4][j % 4] = __float_as_uint(v[j]);
    }
  }
};

}  // namespace beam
