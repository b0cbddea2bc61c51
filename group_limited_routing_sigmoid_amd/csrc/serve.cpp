// C ABI of the operators around a paged key-value cache: host-side checks, then
// the launches.  See include/beam_moe.h for the contract of every entry point.
#include <float.h>
#include <math.h>

#include "serve.h"

using namespace beam;

namespace {

bool is_dtype(int32_t t) { return t == BEAM_F32 || t == BEAM_BF16; }
bool power_of_two(int64_t n) { return n > 0 && (n & (n - 1)) == 0; }
int32_t log2_of(int64_t n) {
  int32_t i = 0;
  while ((int64_t{1} << i) < n) ++i;
  return i;
}
template <typename... P>
bool all_aligned(P... p) {
  return (aligned16(p) && ...);
}
// Strides in elements that keep 16-byte alignment.
bool stride_ok(int64_t n, int32_t dtype) { return n >= 0 && n % (dtype == BEAM_BF16 ? 8 : 4) == 0; }

int check_heads(int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype) {
  if (Hq < 1 || Hkv < 1 || !is_dtype(dtype)) return BEAM_ERR_INVALID_ARG;
  if (Hq > 4096 || Hkv > 4096 || D < 8 || D > kMaxHeadDim || D % 8) return BEAM_ERR_UNSUPPORTED;
  return BEAM_OK;
}

int check_rope(int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype, int32_t rot,
               int32_t interleaved, float eps, float temp_length, float temp_exponent) {
  const int st = check_heads(Hq, Hkv, D, dtype);
  if (st != BEAM_OK) return st;
  if (T < 0 || rot < 0 || rot > D || (interleaved != 0 && interleaved != 1))
    return BEAM_ERR_INVALID_ARG;
  if (!(eps > 0.0f) || !isfinite(eps) || !(temp_length >= 0.0f) || !isfinite(temp_length) ||
      !isfinite(temp_exponent))
    return BEAM_ERR_INVALID_ARG;
  // the inverse root of a number below binary32's normal ones is infinite, and NaN times
  // a head of zeros
  if (eps < FLT_MIN) return BEAM_ERR_UNSUPPORTED;
  // a launch holds fewer than 2^32 threads, 64 a token
  if (rot % 16 || T >= (int64_t{1} << 25) || T * (Hq + 2 * Hkv) >= (int64_t{1} << 31))
    return BEAM_ERR_UNSUPPORTED;
  return BEAM_OK;
}

// A cache's shape; its pointers are the caller's to check.
int make_cache(void* k, void* v, int64_t page_stride, int64_t token_stride, int64_t head_stride,
               int64_t pages, int64_t page_size, const int32_t* tables, int64_t seqs,
               int64_t cols, int32_t dtype, Cache* c) {
  if (pages < 1 || seqs < 0 || cols < 0) return BEAM_ERR_INVALID_ARG;
  if (!stride_ok(page_stride, dtype) || !stride_ok(token_stride, dtype) ||
      !stride_ok(head_stride, dtype))
    return BEAM_ERR_INVALID_ARG;
  if (!power_of_two(page_size) || page_size > (1 << 30) || pages > 0x7FFFFFFF ||
      cols > 0x7FFFFFFF || cols * page_size > 0x7FFFFFFF || token_stride >= (1 << 25))
    return BEAM_ERR_UNSUPPORTED;
  c->k = k;
  c->v = v;
  c->page_stride = page_stride;
  c->token_stride = token_stride;
  c->head_stride = head_stride;
  c->tables = tables;
  c->seqs = seqs;
  c->pages = static_cast<int32_t>(pages);
  c->cols = static_cast<int32_t>(cols);
  c->shift = log2_of(page_size);
  return BEAM_OK;
}

int check_workspace(const void* ws, size_t have, size_t need) {
  if (need && (!ws || have < need)) return BEAM_ERR_WORKSPACE;
  return reinterpret_cast<uintptr_t>(ws) % 256 ? BEAM_ERR_INVALID_ARG : BEAM_OK;
}

constexpr int32_t kMaxLayers = 65536;  // arrays times layers are counted in 32 bits

int check_pools(const beam_moe_pools* p) {
  if (!p || p->count < 0 || p->count > 8 || p->layers < 0) return BEAM_ERR_INVALID_ARG;
  if (p->layers > kMaxLayers) return BEAM_ERR_UNSUPPORTED;
  for (int i = 0; i < p->count; ++i) {
    if (p->layers && (!p->base[i] || !aligned16(p->base[i]))) return BEAM_ERR_INVALID_ARG;
    if (p->bytes[i] < 0 || p->bytes[i] % 16 || p->layer_stride[i] % 16 || p->page_stride[i] % 16)
      return BEAM_ERR_INVALID_ARG;
  }
  return BEAM_OK;
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr int64_t kMaxPages = int64_t{1} << 24, kMaxRows = 65536;

int check_tables(int64_t old_rows, int64_t rows, int64_t cols, int64_t pages, int64_t page_size) {
  if (old_rows < 0 || rows < 0 || cols < 0 || pages < 0) return BEAM_ERR_INVALID_ARG;
  if (old_rows > kMaxRows || rows > kMaxRows || pages >= kMaxPages || !power_of_two(page_size) ||
      page_size > (1 << 30) || cols > 0x7FFFFFFF || cols * page_size > 0x7FFFFFFF ||
      rows * cols > 0x7FFFFFFF || old_rows * cols > 0x7FFFFFFF)
    return BEAM_ERR_UNSUPPORTED;
  return BEAM_OK;
}

int check_score(int64_t T, int64_t V, int32_t dtype, int64_t stride, float softcap, float scale) {
  if (T < 0 || V < 1 || !is_dtype(dtype) || (T > 1 && stride < V)) return BEAM_ERR_INVALID_ARG;
  if (!(softcap >= 0.0f) || !isfinite(softcap) || !(scale > 0.0f) || !isfinite(scale))
    return BEAM_ERR_INVALID_ARG;
  // what the kernels multiply with, in base 2
  if (!isfinite(kLog2E * scale) ||
      (softcap > 0.0f && (!isfinite(2.0f * kLog2E * scale * softcap) || !isfinite(2.0f * kLog2E / softcap))))
    return BEAM_ERR_UNSUPPORTED;
  // 256 threads a piece, fewer than 2^32 in all
  if (V > (1 << 24) || T >= (1 << 23) || score_pieces_count(T, V) >= (1 << 24))
    return BEAM_ERR_UNSUPPORTED;
  return BEAM_OK;
}

}  // namespace

extern "C" {

int beam_moe_qk_norm_rope(int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype,
                          const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                          const void* v, int64_t v_stride, const float* q_weight,
                          const float* k_weight, float eps, const int32_t* positions,
                          const double* inv_freq, int32_t rot, int32_t interleaved,
                          float temp_length, float temp_exponent, void* q_out, void* k_out,
                          void* k_cache, void* v_cache, int64_t page_stride, int64_t token_stride,
                          int64_t head_stride, int64_t pages, int64_t page_size,
                          const int32_t* tables, int64_t seqs, int64_t table_cols,
                          const int32_t* rows, void* stream) {
  int st = check_rope(T, Hq, Hkv, D, dtype, rot, interleaved, eps, temp_length, temp_exponent);
  if (st != BEAM_OK) return st;
  RopeArgs a = {};
  const bool cached = k_cache || v_cache;
  if (cached) {
    st = make_cache(k_cache, v_cache, page_stride, token_stride, head_stride, pages, page_size,
                    tables, seqs, table_cols, dtype, &a.cache);
    if (st != BEAM_OK) return st;
  }
  if (T == 0) return BEAM_OK;
  if (!q || !k || !q_weight || !k_weight || !q_out || (!k_out && !cached))
    return BEAM_ERR_INVALID_ARG;
  if (cached && (!k_cache || !v_cache || !v || (!tables && seqs * table_cols > 0)))
    return BEAM_ERR_INVALID_ARG;
  if (!positions && (rot || temp_length != 0.0f || cached)) return BEAM_ERR_INVALID_ARG;
  if (rot && !inv_freq) return BEAM_ERR_INVALID_ARG;
  if (!all_aligned(q, k, v, q_weight, k_weight, positions, inv_freq, q_out, k_out, k_cache,
                   v_cache, tables, rows))
    return BEAM_ERR_INVALID_ARG;
  if (!stride_ok(q_stride, dtype) || !stride_ok(k_stride, dtype) ||
      (cached && !stride_ok(v_stride, dtype)))
    return BEAM_ERR_INVALID_ARG;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.wq = q_weight;
  a.wk = k_weight;
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.q_out = q_out;
  a.k_out = k_out;
  a.rows = rows;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.rot = rot;
  a.eps = eps;
  a.temp_length = temp_length;
  a.temp_exponent = temp_exponent;
  a.interleaved = interleaved != 0;
  return hip_status(launch_qk_norm_rope(a, dtype, static_cast<hipStream_t>(stream)));
}

int beam_moe_qk_norm_rope_workspace_bytes(int64_t T, int32_t Hq, int32_t Hkv, int32_t D,
                                          size_t* bytes) {
  if (!bytes) return BEAM_ERR_INVALID_ARG;
  const int st = check_rope(T, Hq, Hkv, D, BEAM_BF16, 0, 0, 1.0f, 0.0f, 0.0f);
  if (st != BEAM_OK) return st;
  *bytes = static_cast<size_t>(rope_grad_groups(T)) * 2 * static_cast<size_t>(D) *
           sizeof(float);
  return BEAM_OK;
}

int beam_moe_qk_norm_rope_backward(int64_t T, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype,
                                   const void* d_q_out, const void* d_k_out, const void* q,
                                   int64_t q_stride, const void* k, int64_t k_stride,
                                   const float* q_weight, const float* k_weight, float eps,
                                   const int32_t* positions, const double* inv_freq, int32_t rot,
                                   int32_t interleaved, float temp_length, float temp_exponent,
                                   void* d_q, void* d_k, float* d_q_weight, float* d_k_weight,
                                   void* workspace, size_t ws_bytes, void* stream) {
  int st = check_rope(T, Hq, Hkv, D, dtype, rot, interleaved, eps, temp_length, temp_exponent);
  if (st != BEAM_OK) return st;
  if (!d_q_weight || !d_k_weight) return BEAM_ERR_INVALID_ARG;
  if (T > 0) {
    if (!d_q_out || !d_k_out || !q || !k || !q_weight || !k_weight || !d_q || !d_k)
      return BEAM_ERR_INVALID_ARG;
    if (!positions && (rot || temp_length != 0.0f)) return BEAM_ERR_INVALID_ARG;
    if (rot && !inv_freq) return BEAM_ERR_INVALID_ARG;
    if (!stride_ok(q_stride, dtype) || !stride_ok(k_stride, dtype)) return BEAM_ERR_INVALID_ARG;
  }
  if (!all_aligned(d_q_out, d_k_out, q, k, q_weight, k_weight, positions, inv_freq, d_q, d_k,
                   d_q_weight, d_k_weight))
    return BEAM_ERR_INVALID_ARG;
  size_t need = 0;
  st = beam_moe_qk_norm_rope_workspace_bytes(T, Hq, Hkv, D, &need);
  if (st != BEAM_OK) return st;
  st = check_workspace(workspace, ws_bytes, need);
  if (st != BEAM_OK) return st;
  RopeGradArgs g = {};
  RopeArgs& a = g.f;
  a.q = q;
  a.k = k;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.wq = q_weight;
  a.wk = k_weight;
  a.pos = positions;
  a.inv_freq = inv_freq;
  a.T = T;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.rot = rot;
  a.eps = eps;
  a.temp_length = temp_length;
  a.temp_exponent = temp_exponent;
  a.interleaved = interleaved != 0;
  g.dq_out = d_q_out;
  g.dk_out = d_k_out;
  g.dq = d_q;
  g.dk = d_k;
  g.part = static_cast<float*>(workspace);
  return hip_status(launch_qk_norm_rope_backward(g, dtype, d_q_weight, d_k_weight,
                                                 static_cast<hipStream_t>(stream)));
}

int beam_moe_paged_attention_workspace_bytes(int64_t seqs, int32_t Hq, int32_t Hkv, int32_t D,
                                             size_t* bytes) {
  if (!bytes || seqs < 0) return BEAM_ERR_INVALID_ARG;
  const int st = check_heads(Hq, Hkv, D, BEAM_BF16);
  if (st != BEAM_OK) return st;
  if (Hq % Hkv) return BEAM_ERR_INVALID_ARG;
  if (seqs >= (1 << 24) || seqs * Hq >= (1 << 24)) return BEAM_ERR_UNSUPPORTED;
  *bytes = attend_workspace(seqs, Hq, Hkv, D);
  return BEAM_OK;
}

int beam_moe_paged_attention(int64_t seqs, int32_t Hq, int32_t Hkv, int32_t D, int32_t dtype,
                             const void* q, const void* gate, const void* k_cache,
                             const void* v_cache, int64_t page_stride, int64_t token_stride,
                             int64_t head_stride, int64_t pages, int64_t page_size,
                             const int32_t* tables, int64_t table_cols, const int32_t* lengths,
                             float scale, int64_t window, void* out, float* lse, void* workspace,
                             size_t ws_bytes, void* stream) {
  int st = check_heads(Hq, Hkv, D, dtype);
  if (st != BEAM_OK) return st;
  size_t need = 0;
  st = beam_moe_paged_attention_workspace_bytes(seqs, Hq, Hkv, D, &need);
  if (st != BEAM_OK) return st;
  if (!(scale > 0.0f) || !isfinite(scale) || window < 0) return BEAM_ERR_INVALID_ARG;
  AttendArgs a = {};
  st = make_cache(const_cast<void*>(k_cache), const_cast<void*>(v_cache), page_stride,
                  token_stride, head_stride, pages, page_size, tables, seqs, table_cols, dtype,
                  &a.cache);
  if (st != BEAM_OK) return st;
  // tokens are counted in 31 bits up to 64 steps of 256 past a sequence's end, units
  // of work in 32
  if (table_cols * page_size > 0x7FFF0000 ||
      seqs * (table_cols * page_size) >= (int64_t{1} << 36) || !isfinite(kLog2E * scale))
    return BEAM_ERR_UNSUPPORTED;
  if (seqs == 0) return BEAM_OK;
  if (!q || !k_cache || !v_cache || !lengths || !out || (!tables && table_cols > 0))
    return BEAM_ERR_INVALID_ARG;
  if (!all_aligned(q, gate, k_cache, v_cache, tables, lengths, out, lse))
    return BEAM_ERR_INVALID_ARG;
  st = check_workspace(workspace, ws_bytes, need);
  if (st != BEAM_OK) return st;
  a.q = q;
  a.gate = gate;
  a.lengths = lengths;
  a.out = out;
  a.lse = lse;
  a.part = static_cast<float*>(workspace);
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.D = D;
  a.window = window > 0x7FFFFFFF ? 0 : static_cast<int32_t>(window);  // longer than any table
  a.scale = scale;
  return hip_status(launch_paged_attention(a, dtype, static_cast<hipStream_t>(stream)));
}

int beam_moe_pages_copy(const beam_moe_pools* pools, int64_t pages, int64_t n, const int32_t* src,
                        const int32_t* dst, void* stream) {
  const int st = check_pools(pools);
  if (st != BEAM_OK) return st;
  if (pages < 0 || n < 0) return BEAM_ERR_INVALID_ARG;
  if (pages > 0x7FFFFFFF || n > 0x7FFFFFFF) return BEAM_ERR_UNSUPPORTED;
  if (n == 0) return BEAM_OK;
  if (!src || !dst || !all_aligned(src, dst)) return BEAM_ERR_INVALID_ARG;
  return hip_status(
      launch_pages_copy(*pools, pages, n, src, dst, static_cast<hipStream_t>(stream)));
}

int beam_moe_pages_workspace_bytes(int64_t pages, int64_t rows, size_t* bytes) {
  if (!bytes || pages < 0 || rows < 0) return BEAM_ERR_INVALID_ARG;
  if (pages >= kMaxPages || rows > kMaxRows) return BEAM_ERR_UNSUPPORTED;
  *bytes = pages_workspace(pages, rows);
  return BEAM_OK;
}

int beam_moe_pages_update(int64_t old_rows, int64_t rows, int64_t cols, int64_t pages,
                          int64_t page_size, const int32_t* tables, const int32_t* lengths,
                          const int32_t* refs, const int32_t* parents, const int32_t* grow,
                          int32_t* tables_out, int32_t* lengths_out, int32_t* refs_out,
                          int32_t* missing, const beam_moe_pools* pools, void* workspace,
                          size_t ws_bytes, void* stream) {
  int st = check_tables(old_rows, rows, cols, pages, page_size);
  if (st != BEAM_OK) return st;
  st = check_pools(pools);
  if (st != BEAM_OK) return st;
  if ((!parents && rows != old_rows && rows > 0) || !missing) return BEAM_ERR_INVALID_ARG;
  if (pages > 0 && (!refs || !refs_out || refs == refs_out)) return BEAM_ERR_INVALID_ARG;
  if (old_rows > 0 && (!lengths || (cols > 0 && !tables))) return BEAM_ERR_INVALID_ARG;
  if (rows > 0 && (!lengths_out || lengths_out == lengths ||
                   (cols > 0 && (!tables_out || tables_out == tables))))
    return BEAM_ERR_INVALID_ARG;
  if (!all_aligned(tables, lengths, refs, parents, grow, tables_out, lengths_out, refs_out,
                   missing))
    return BEAM_ERR_INVALID_ARG;
  st = check_workspace(workspace, ws_bytes, pages_workspace(pages, rows));
  if (st != BEAM_OK) return st;
  PageArgs a = {};
  a.old_rows = old_rows;
  a.rows = rows;
  a.cols = cols;
  a.pages = pages;
  a.shift = log2_of(page_size);
  a.tables = tables;
  a.lengths = lengths;
  a.refs = refs;
  a.parents = parents;
  a.grow = grow;
  a.tables_out = tables_out;
  a.lengths_out = lengths_out;
  a.refs_out = refs_out;
  a.count = missing;
  return hip_status(
      launch_pages_update(a, *pools, workspace, static_cast<hipStream_t>(stream)));
}

int beam_moe_pages_compact(int64_t rows, int64_t cols, int64_t pages, int64_t page_size,
                           const int32_t* tables, const int32_t* lengths, const int32_t* refs,
                           int32_t* tables_out, int32_t* refs_out, int32_t* new_id, int32_t* live,
                           const beam_moe_pools* pools, void* workspace, size_t ws_bytes,
                           void* stream) {
  int st = check_tables(rows, rows, cols, pages, page_size);
  if (st != BEAM_OK) return st;
  st = check_pools(pools);
  if (st != BEAM_OK) return st;
  if (!live || (pages > 0 && (!refs || !refs_out || !new_id || refs == refs_out)))
    return BEAM_ERR_INVALID_ARG;
  if (rows > 0 && (!lengths || (cols > 0 && (!tables || !tables_out))))
    return BEAM_ERR_INVALID_ARG;
  if (!all_aligned(tables, lengths, refs, tables_out, refs_out, new_id, live))
    return BEAM_ERR_INVALID_ARG;
  st = check_workspace(workspace, ws_bytes, pages_workspace(pages, rows));
  if (st != BEAM_OK) return st;
  PageArgs a = {};
  a.old_rows = a.rows = rows;
  a.cols = cols;
  a.pages = pages;
  a.shift = log2_of(page_size);
  a.tables = tables;
  a.lengths = lengths;
  a.refs = refs;
  a.tables_out = tables_out;
  a.refs_out = refs_out;
  a.new_id = new_id;
  a.count = live;
  return hip_status(
      launch_pages_compact(a, *pools, workspace, static_cast<hipStream_t>(stream)));
}

int beam_moe_token_logprobs_workspace_bytes(int64_t T, int64_t V, int32_t top, size_t* bytes) {
  if (!bytes) return BEAM_ERR_INVALID_ARG;
  const int st = check_score(T, V, BEAM_F32, V, 0.0f, 1.0f);
  if (st != BEAM_OK) return st;
  if (top < 0 || top > V) return BEAM_ERR_INVALID_ARG;
  if (top > kMaxTop) return BEAM_ERR_UNSUPPORTED;
  *bytes = T == 0 ? 0 : score_workspace(T, V, top);
  return BEAM_OK;
}

int beam_moe_token_logprobs(int64_t T, int64_t V, int32_t dtype, const void* logits,
                            int64_t row_stride, const int64_t* targets, float softcap, float scale,
                            int32_t top, float* logprobs, float* entropy, float* lse,
                            int32_t* top_ids, float* top_logprobs, void* workspace,
                            size_t ws_bytes, void* stream) {
  int st = check_score(T, V, dtype, row_stride, softcap, scale);
  if (st != BEAM_OK) return st;
  size_t need = 0;
  st = beam_moe_token_logprobs_workspace_bytes(T, V, top, &need);
  if (st != BEAM_OK) return st;
  if (T == 0) return BEAM_OK;
  if (!logits || !entropy || !lse || !targets != !logprobs) return BEAM_ERR_INVALID_ARG;
  if (top > 0 && (!top_ids || !top_logprobs)) return BEAM_ERR_INVALID_ARG;
  if (!all_aligned(logits, targets, logprobs, entropy, lse, top_ids, top_logprobs))
    return BEAM_ERR_INVALID_ARG;
  st = check_workspace(workspace, ws_bytes, need);
  if (st != BEAM_OK) return st;
  ScoreArgs a = {};
  a.logits = logits;
  a.stride = row_stride;
  a.targets = targets;
  a.softcap = softcap;
  a.scale = scale;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.lse = lse;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.T = T;
  a.V = static_cast<int32_t>(V);
  a.top = top;
  return hip_status(
      launch_token_logprobs(a, dtype, workspace, static_cast<hipStream_t>(stream)));
}

int beam_moe_token_logprobs_backward(int64_t T, int64_t V, int32_t dtype, const void* logits,
                                     int64_t row_stride, const int64_t* targets, float softcap,
                                     float scale, const float* lse, const float* entropy,
                                     const float* d_logprobs, const float* d_entropy,
                                     void* d_logits, int64_t d_row_stride, void* stream) {
  const int st = check_score(T, V, dtype, row_stride, softcap, scale);
  if (st != BEAM_OK) return st;
  if (T > 1 && d_row_stride < V) return BEAM_ERR_INVALID_ARG;
  if (T == 0) return BEAM_OK;
  if (!logits || !lse || !entropy || !d_logits || (!d_logprobs && !d_entropy) ||
      (d_logprobs && !targets) || (d_logits == logits && row_stride != d_row_stride))
    return BEAM_ERR_INVALID_ARG;
  if (!all_aligned(logits, targets, lse, entropy, d_logprobs, d_entropy, d_logits))
    return BEAM_ERR_INVALID_ARG;
  ScoreGradArgs a = {};
  a.logits = logits;
  a.stride = row_stride;
  a.targets = targets;
  a.softcap = softcap;
  a.scale = scale;
  a.lse = lse;
  a.entropy = entropy;
  a.d_logprobs = d_logprobs;
  a.d_entropy = d_entropy;
  a.d_logits = d_logits;
  a.d_stride = d_row_stride;
  a.T = T;
  a.V = static_cast<int32_t>(V);
  return hip_status(
      launch_token_logprobs_backward(a, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
