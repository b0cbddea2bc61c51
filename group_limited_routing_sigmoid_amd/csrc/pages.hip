// The page tables of a cache between two decode steps: rows that go on from a
// parent's pages, shared pages copied before they are written, new pages, pages
// of rows that went away; the packing of used pages to a pool's front; and the
// copies of pages themselves.
//
// Everything is decided by integers: references by counts (integer atomics,
// whose order changes nothing), pages by their rank among the free ones, wants
// by their place in the rows' order.  The tables' part is bound by its few
// dependent launches, the copies' by reading and writing the pages once.
#include <algorithm>
#include <climits>

#include "serve.h"

namespace beam {
namespace {

constexpr int kThreads = 256;
constexpr int kEach = 8;                    // pages of a thread
constexpr int kBlock = kThreads * kEach;    // pages of a workgroup
constexpr int64_t kCopyBlocks = 1 << 16;    // workgroups of a copy, which take turns
constexpr int kDemand = 1024;               // threads that count the rows' wants

struct Space {  // workspace
  int32_t* writers;   // [pages] rows that would write to a page that they hold in part
  int32_t* lowest;    // [pages] the lowest of them
  int32_t* counts;    // [blocks] free (or used) pages of a block
  int32_t* begin;     // [rows + 1] a row's first want among all
  int32_t* copied;    // [rows] the page that a row copies, or -1
  int32_t* children;  // [old rows]
  int32_t* over;      // [1] pages wanted past the columns
};

struct Row {  // what a new row has and wants
  int parent;  // or -1
  int held, grow;
  int have, need;  // pages
};

__device__ __forceinline__ int held_tokens(const PageArgs& a, int r) {
  return min(max(a.lengths[r], 0), static_cast<int>(a.cols << a.shift));
}
__device__ __forceinline__ int pages_for(const PageArgs& a, int64_t tokens) {
  return static_cast<int>((tokens + (int64_t{1} << a.shift) - 1) >> a.shift);
}
__device__ __forceinline__ Row row_of(const PageArgs& a, int i) {
  Row r;
  r.parent = a.parents ? a.parents[i] : i;
  if (r.parent < 0 || r.parent >= a.old_rows) r.parent = -1;
  r.held = r.parent < 0 ? 0 : held_tokens(a, r.parent);
  r.grow = a.grow ? max(a.grow[i], 0) : 0;
  r.have = pages_for(a, r.held);
  r.need = pages_for(a, static_cast<int64_t>(r.held) + r.grow);
  return r;
}
// The unfilled last page that the row is going to write to, or -1.
__device__ __forceinline__ int open_page(const PageArgs& a, const Row& r) {
  if (r.grow == 0 || (r.held & ((1 << a.shift) - 1)) == 0) return -1;
  const int p = a.tables[r.parent * a.cols + r.have - 1];
  return p >= 0 && p < a.pages ? p : -1;
}

__device__ __forceinline__ void copy_page(const beam_moe_pools& p, int part, int src, int dst) {
  const int i = part / p.layers, layer = part % p.layers;
  char* base = static_cast<char*>(p.base[i]) + layer * p.layer_stride[i];
  const char* from = base + src * p.page_stride[i];
  char* to = base + dst * p.page_stride[i];
  const int64_t n = p.bytes[i];
  int64_t at = static_cast<int64_t>(threadIdx.x) * 16;
  const int64_t step = static_cast<int64_t>(blockDim.x) * 16;
  for (; at + 3 * step < n; at += 4 * step) {
    const u32x4 v0 = ld16(from + at), v1 = ld16(from + at + step), v2 = ld16(from + at + 2 * step),
                v3 = ld16(from + at + 3 * step);
    st16(to + at, v0);
    st16(to + at + step, v1);
    st16(to + at + 2 * step, v2);
    st16(to + at + 3 * step, v3);
  }
  for (; at < n; at += step) st16(to + at, ld16(from + at));
}

// Sum over the workgroup's threads before this one; *total the sum over all.
template <int kN>
__device__ __forceinline__ int scan(int v, int* total) {
  __shared__ int waves[kN / kWave];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  int sum = v;
#pragma unroll
  for (int i = 1; i < kWave; i *= 2) {
    const int x = __shfl_up(sum, i);
    if (lane >= i) sum += x;
  }
  __syncthreads();
  if (lane == kWave - 1) waves[wave] = sum;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kN / kWave; ++i) {
    if (i < wave) before += waves[i];
    all += waves[i];
  }
  *total = all;
  return before + sum - v;
}
// Sum of v over the workgroup.
__device__ __forceinline__ int sum_all(int v) {
  int total;
  scan<kThreads>(v, &total);
  return total;
}

__global__ __launch_bounds__(kThreads) void update_prepare(PageArgs a, Space w) {
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t p = id; p < a.pages; p += step) {
    a.refs_out[p] = a.refs[p];
    w.writers[p] = 0;
    w.lowest[p] = INT_MAX;
  }
  // rows that go on from each old one
  const int lane = threadIdx.x % kWave;
  for (int64_t r = id / kWave; r < a.old_rows; r += step / kWave) {
    int n = a.rows ? 1 : 0;  // without parents each goes on from itself
    if (a.parents) {
      n = 0;
      for (int64_t i = lane; i - lane < a.rows; i += kWave)
        n += __popcll(__ballot(i < a.rows && a.parents[i] == r));
    }
    if (lane == 0) w.children[r] = n;
  }
}

// A workgroup for each new row, then one for each old row.
__global__ __launch_bounds__(kThreads) void update_rows(PageArgs a, Space w) {
  if (blockIdx.x < a.rows) {
    const int i = blockIdx.x;
    const Row r = row_of(a, i);
    const int32_t* from = a.tables + max(r.parent, 0) * a.cols;
    int32_t* to = a.tables_out + i * a.cols;
    for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) to[c] = c < r.have ? from[c] : -1;
    if (threadIdx.x) return;
    const int p = open_page(a, r);
    if (p < 0) return;
    atomicAdd(&w.writers[p], 1);
    atomicMin(&w.lowest[p], i);
    return;
  }
  const int r = blockIdx.x - static_cast<int>(a.rows);
  const int by = w.children[r] - 1;
  if (by == 0) return;
  const int have = pages_for(a, held_tokens(a, r));
  for (int64_t c = threadIdx.x; c < have; c += kThreads) {
    const int p = a.tables[r * a.cols + c];
    if (p >= 0 && p < a.pages) atomicAdd(&a.refs_out[p], by);
  }
}

// Workgroup 0: every row's first want, the page it copies, its new length.  The
// others: free pages of their block.
__global__ __launch_bounds__(kDemand) void update_count(PageArgs a, Space w) {
  int total;
  if (blockIdx.x) {
    const int64_t p0 = (blockIdx.x - 1) * static_cast<int64_t>(kBlock);
    int n = 0;
    for (int64_t p = p0 + threadIdx.x; p < min<int64_t>(p0 + kBlock, a.pages); p += kDemand)
      n += a.refs_out[p] <= 0;
    scan<kDemand>(n, &total);
    if (threadIdx.x == 0) w.counts[blockIdx.x - 1] = total;
    return;
  }
  int before = 0, over = 0;
  for (int64_t i0 = 0; i0 < a.rows; i0 += kDemand) {
    const int64_t i = i0 + threadIdx.x;
    int want = 0;
    if (i < a.rows) {
      const Row r = row_of(a, static_cast<int>(i));
      const int p = open_page(a, r), most = static_cast<int>(a.cols);
      int copy = -1;
      if (p >= 0) {
        const int refs = a.refs_out[p];
        if (refs != 1 && !(refs == w.writers[p] && w.lowest[p] == i)) copy = p;
      }
      w.copied[i] = copy;
      if (copy >= 0) a.tables_out[i * a.cols + r.have - 1] = -1;  // until it has one
      want = (copy >= 0) + min(r.need, most) - r.have;
      over += max(r.need - most, 0);
      const int64_t size = static_cast<int64_t>(r.held) + r.grow;
      a.lengths_out[i] = static_cast<int>(min<int64_t>(size, a.cols << a.shift));
    }
    const int first = scan<kDemand>(want, &total);
    if (i < a.rows) w.begin[i] = before + first;
    before += total;
  }
  scan<kDemand>(over, &total);
  if (threadIdx.x == 0) {
    w.begin[a.rows] = before;
    *w.over = total;
  }
}

// Each free page goes to the want of its rank.  (A copied page keeps at least
// one reference, so giving one of its references up here frees none.)
__global__ __launch_bounds__(kThreads) void update_give(PageArgs a, Space w, int blocks) {
  const int rows = static_cast<int>(a.rows), wants = w.begin[rows];
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  for (int64_t i = id; i < rows; i += static_cast<int64_t>(gridDim.x) * kThreads)
    if (w.copied[i] >= 0) atomicSub(&a.refs_out[w.copied[i]], 1);
  int n = 0;
  if (blockIdx.x == 0) {
    for (int b = threadIdx.x; b < blocks; b += kThreads) n += w.counts[b];
    n = sum_all(n);
    if (threadIdx.x == 0) *a.count = max(wants - n, 0) + *w.over;
  }
  n = 0;
  for (int b = threadIdx.x; b < static_cast<int>(blockIdx.x); b += kThreads) n += w.counts[b];
  const int before = sum_all(n);
  if (before >= wants) return;
  const int64_t p0 = id * kEach;
  bool free[kEach];
  n = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    free[j] = p0 + j < a.pages && a.refs_out[p0 + j] <= 0;
    n += free[j];
  }
  int total;
  int rank = before + scan<kThreads>(n, &total);
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    if (!free[j]) continue;
    if (rank >= wants) break;
    int lo = 0, hi = rows - 1;  // the last row whose first want is no later
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (w.begin[mid] <= rank) lo = mid;
      else hi = mid - 1;
    }
    const Row r = row_of(a, lo);
    const int slot = r.have + rank - w.begin[lo] - (w.copied[lo] >= 0);
    a.tables_out[lo * a.cols + slot] = static_cast<int>(p0 + j);
    a.refs_out[p0 + j] = 1;
    ++rank;
  }
}

// A workgroup takes rows' copies in one layer of one array.
__global__ __launch_bounds__(kThreads) void update_copy(PageArgs a, Space w, beam_moe_pools p) {
  const int parts = p.count * p.layers;
  for (int64_t x = blockIdx.x; x < a.rows * parts; x += gridDim.x) {
    const int i = static_cast<int>(x / parts), src = w.copied[i];
    if (src < 0) continue;
    const int dst = a.tables_out[i * a.cols + row_of(a, i).have - 1];
    if (dst >= 0) copy_page(p, static_cast<int>(x % parts), src, dst);
  }
}

__global__ __launch_bounds__(kThreads) void copy_list(beam_moe_pools p, int64_t pages, int64_t n,
                                                       const int32_t* src, const int32_t* dst) {
  const int parts = p.count * p.layers;
  for (int64_t x = blockIdx.x; x < n * parts; x += gridDim.x) {
    const int s = src[x / parts], d = dst[x / parts];
    if (s >= 0 && s < pages && d >= 0 && d < pages) copy_page(p, static_cast<int>(x % parts), s, d);
  }
}

struct PackSpace {
  int32_t* counts;  // [blocks] used pages
  int32_t* from;    // [pages] pages that move
  int32_t* to;      // [pages] where to
  int32_t* rank;    // [pages] of a page that moves among them, else -1
  int32_t* moves;   // [1]
};

__global__ __launch_bounds__(kThreads) void pack_count(PageArgs a, PackSpace w) {
  const int64_t p0 = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * kEach;
  int n = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) n += p0 + j < a.pages && a.refs[p0 + j] > 0;
  n = sum_all(n);
  if (threadIdx.x == 0) w.counts[blockIdx.x] = n;
}

__global__ __launch_bounds__(kThreads) void pack_rank(PageArgs a, PackSpace w, int blocks) {
  // used pages of all blocks, before this one, and below the front's end n
  int all = 0, mine = 0;
  for (int b = threadIdx.x; b < blocks; b += kThreads) {
    const int c = w.counts[b];
    all += c;
    if (b < static_cast<int>(blockIdx.x)) mine += c;
  }
  const int n = sum_all(all), before = sum_all(mine);
  const int cut = n / kBlock;
  int front = 0;
  for (int b = threadIdx.x; b < cut; b += kThreads) front += w.counts[b];
  for (int64_t p = static_cast<int64_t>(cut) * kBlock + threadIdx.x; p < n; p += kThreads)
    front += a.refs[p] > 0;
  front = sum_all(front);
  if (blockIdx.x == 0 && threadIdx.x == 0) {
    *w.moves = n - front;
    *a.count = n;
  }
  const int64_t p0 = (static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x) * kEach;
  int refs[kEach], used = 0;
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    refs[j] = p0 + j < a.pages ? a.refs[p0 + j] : 0;
    used += refs[j] > 0;
  }
  int total;
  int rank = before + scan<kThreads>(used, &total);  // used pages before p
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int p = static_cast<int>(p0) + j;
    if (p >= a.pages) break;
    int r = -1, to = -1;
    if (refs[j] > 0) {
      if (p < n) to = p;
      else {
        r = rank - front;
        w.from[r] = p;
      }
      ++rank;
    } else if (p < n) {
      w.to[p - rank] = p;
    }
    w.rank[p] = r;
    if (r < 0) a.new_id[p] = to;
    if (p >= n || refs[j] > 0) a.refs_out[p] = p < n ? refs[j] : 0;
  }
}

__global__ __launch_bounds__(kThreads) void pack_move(PageArgs a, PackSpace w, beam_moe_pools p) {
  const int moves = *w.moves, n = *a.count;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
  for (int64_t i = id; i < moves; i += step) {
    a.new_id[w.from[i]] = w.to[i];
    a.refs_out[w.to[i]] = a.refs[w.from[i]];
  }
  for (int64_t i = blockIdx.x; i < a.rows; i += gridDim.x) {
    const int have = pages_for(a, held_tokens(a, static_cast<int>(i)));
    for (int64_t c = threadIdx.x; c < a.cols; c += kThreads) {
      int v = c < have ? a.tables[i * a.cols + c] : -1;
      if (v < 0 || v >= a.pages) v = -1;
      else if (w.rank[v] >= 0) v = w.to[w.rank[v]];
      else if (v >= n || a.refs[v] <= 0) v = -1;
      a.tables_out[i * a.cols + c] = v;
    }
  }
  const int parts = p.count * p.layers;
  const int64_t items = static_cast<int64_t>(moves) * parts;
  for (int64_t x = blockIdx.x; x < items; x += gridDim.x) {
    const int i = static_cast<int>(x / parts);
    copy_page(p, static_cast<int>(x % parts), w.from[i], w.to[i]);
  }
}

template <typename P>
int32_t* carve(P*& at, int64_t n) {
  int32_t* p = at;
  at += ceil_div(n, 64) * 64;
  return p;
}

}  // namespace

size_t pages_workspace(int64_t pages, int64_t rows) {
  auto room = [](int64_t n) { return ceil_div(n, 64) * 64; };
  // from, to and rank of a packing; writers and lowest of an update
  return sizeof(int32_t) * static_cast<size_t>(3 * room(pages) + room(ceil_div(pages, kBlock)) +
                                               2 * room(rows + 1) + room(65536) + room(1));
}

hipError_t launch_pages_copy(const beam_moe_pools& p, int64_t pages, int64_t n, const int32_t* src,
                             const int32_t* dst, hipStream_t s) {
  const int64_t blocks = std::min(n * p.count * p.layers, kCopyBlocks);
  if (blocks == 0) return hipSuccess;
  hipLaunchKernelGGL(copy_list, dim3(blocks), dim3(kThreads), 0, s, p, pages, n, src, dst);
  return hipGetLastError();
}

hipError_t launch_pages_update(const PageArgs& a, const beam_moe_pools& p, void* ws,
                               hipStream_t s) {
  int32_t* at = static_cast<int32_t*>(ws);
  const int blocks = static_cast<int>(ceil_div(a.pages, kBlock));
  Space w;
  w.writers = carve(at, a.pages);
  w.lowest = carve(at, a.pages);
  w.counts = carve(at, blocks);
  w.begin = carve(at, a.rows + 1);
  w.copied = carve(at, a.rows);
  w.children = carve(at, a.old_rows);
  w.over = carve(at, 1);
  const int64_t work = std::max(a.pages, a.old_rows * kWave);
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(ceil_div(work, kThreads), 2048));
  hipLaunchKernelGGL(update_prepare, dim3(grid), dim3(kThreads), 0, s, a, w);
  if (a.rows + a.old_rows)
    hipLaunchKernelGGL(update_rows, dim3(a.rows + a.old_rows), dim3(kThreads), 0, s, a, w);
  hipLaunchKernelGGL(update_count, dim3(blocks + 1), dim3(kDemand), 0, s, a, w);
  hipLaunchKernelGGL(update_give, dim3(std::max(blocks, 1)), dim3(kThreads), 0, s, a, w, blocks);
  const int64_t copies = std::min(a.rows * p.count * p.layers, kCopyBlocks);
  if (copies)
    hipLaunchKernelGGL(update_copy, dim3(copies), dim3(kThreads), 0, s, a, w, p);
  return hipGetLastError();
}

hipError_t launch_pages_compact(const PageArgs& a, const beam_moe_pools& p, void* ws,
                                hipStream_t s) {
  int32_t* at = static_cast<int32_t*>(ws);
  const int blocks = static_cast<int>(ceil_div(a.pages, kBlock));
  PackSpace w;
  w.from = carve(at, a.pages);
  w.to = carve(at, a.pages);
  w.rank = carve(at, a.pages);
  w.counts = carve(at, blocks);
  w.moves = carve(at, 1);
  const int grid = std::max(blocks, 1);
  hipLaunchKernelGGL(pack_count, dim3(grid), dim3(kThreads), 0, s, a, w);
  hipLaunchKernelGGL(pack_rank, dim3(grid), dim3(kThreads), 0, s, a, w, blocks);
  const int64_t work = std::max<int64_t>({1, a.rows, a.pages * p.count * p.layers});
  hipLaunchKernelGGL(pack_move, dim3(std::min<int64_t>(work, 4096)), dim3(kThreads), 0, s, a, w, p);
  return hipGetLastError();
}

}  // namespace beam
