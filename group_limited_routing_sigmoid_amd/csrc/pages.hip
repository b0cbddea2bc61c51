// The page tables of a cache between two decode steps: rows that go on from a
// parent's pages, shared pages copied before they are written, new pages, pages
// of rows that went away; the packing of used pages to a pool's front; and the
// copies of pages themselves.
//
// Everything is decided by integers: references by counts (integer atomics,
// whose order changes nothing), pages by their rank among the free ones, wants
// by their place in the rows' order.  The tables' part is a chain of short steps,
// each of which needs the one before whole: four launches and the copies', or,
// for a pool and a batch that one workgroup holds in LDS, one (32 rows of 189 pages,
// a pool of 1,000: 7 us, where the four launches took 18; 512 rows, a pool of
// 28,000: 18 us in four, and 24 for copies of 130 MB).  The copies are bound by
// reading and writing the pages once (2.8 GB in 505 us).
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
  int32_t* list;      // [pages] free pages in order, as many as are wanted
  int32_t* given;     // [1] how many those are
  int32_t* children;  // [old rows]
  int32_t* over;      // [1] pages wanted past the columns
};

struct Row {  // what a new row has and wants
  int parent;  // or -1
  int held, grow;
  int have, need;  // pages; need: at most the columns
  int64_t over;    // pages past those
};

__device__ __forceinline__ int held_tokens(const PageArgs& a, int r) {
  return min(max(a.lengths[r], 0), static_cast<int>(a.cols << a.shift));
}
__device__ __forceinline__ int64_t pages_for(const PageArgs& a, int64_t tokens) {
  return (tokens + (int64_t{1} << a.shift) - 1) >> a.shift;
}
__device__ __forceinline__ int held_pages(const PageArgs& a, int r) {
  return static_cast<int>(pages_for(a, held_tokens(a, r)));
}
__device__ __forceinline__ Row row_of(const PageArgs& a, int i) {
  Row r;
  r.parent = a.parents ? a.parents[i] : i;
  if (r.parent < 0 || r.parent >= a.old_rows) r.parent = -1;
  r.held = r.parent < 0 ? 0 : held_tokens(a, r.parent);
  r.grow = a.grow ? max(a.grow[i], 0) : 0;
  r.have = static_cast<int>(pages_for(a, r.held));
  const int64_t need = pages_for(a, static_cast<int64_t>(r.held) + r.grow);
  r.need = static_cast<int>(min<int64_t>(need, a.cols));
  r.over = need - r.need;
  return r;
}
// The unfilled last page that the row is going to write to, or -1.
__device__ __forceinline__ int open_page(const PageArgs& a, const Row& r) {
  if (r.grow == 0 || (r.held & ((1 << a.shift) - 1)) == 0) return -1;
  const int p = a.tables[r.parent * a.cols + r.have - 1];
  return p >= 0 && p < a.pages ? p : -1;
}

// ONCE: past the caches' usual order, where many pages move (549 us instead of 563
// for 2.8 GB; a copied page that is read again soon stays in them).  A workgroup
// for each page of a layer, so that it reads the whole of an ordinary one before it
// writes (511 us; 4,096 workgroups that take turns 546, by fours 549).
constexpr int kBurst = 8;
template <bool ONCE>
__device__ __forceinline__ void copy_page(const beam_moe_pools& p, int part, int src, int dst) {
  const int i = part / p.layers, layer = part % p.layers;
  char* base = static_cast<char*>(p.base[i]) + layer * p.layer_stride[i];
  const char* from = base + src * p.page_stride[i];
  char* to = base + dst * p.page_stride[i];
  const int64_t n = p.bytes[i];
  auto read = [&](int64_t at) {
    const u32x4* x = reinterpret_cast<const u32x4*>(from + at);
    return ONCE ? __builtin_nontemporal_load(x) : *x;
  };
  auto write = [&](int64_t at, u32x4 v) {
    u32x4* x = reinterpret_cast<u32x4*>(to + at);
    if (ONCE) __builtin_nontemporal_store(v, x);
    else *x = v;
  };
  int64_t at = static_cast<int64_t>(threadIdx.x) * 16;
  const int64_t step = static_cast<int64_t>(blockDim.x) * 16;
  for (; at + (kBurst - 1) * step < n; at += kBurst * step) {
    u32x4 v[kBurst];
#pragma unroll
    for (int u = 0; u < kBurst; ++u) v[u] = read(at + u * step);
#pragma unroll
    for (int u = 0; u < kBurst; ++u) write(at + u * step, v[u]);
  }
  for (; at < n; at += step) write(at, read(at));
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
// Sum of v over the workgroup, held to an int32.
template <int kN>
__device__ __forceinline__ int sum_long(int64_t v) {
  __shared__ int64_t waves[kN / kWave];
#pragma unroll
  for (int i = 1; i < kWave; i *= 2) v += __shfl_xor(v, i);
  __syncthreads();
  if (threadIdx.x % kWave == 0) waves[threadIdx.x / kWave] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int i = 0; i < kN / kWave; ++i) v += waves[i];
  return static_cast<int>(min<int64_t>(v, INT_MAX));
}
__device__ __forceinline__ int add_held(int a, int b) {  // of two counts
  return static_cast<int>(min<int64_t>(static_cast<int64_t>(a) + b, INT_MAX));
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
  const int have = held_pages(a, r);
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
  int before = 0;
  int64_t over = 0;
  for (int64_t i0 = 0; i0 < a.rows; i0 += kDemand) {
    const int64_t i = i0 + threadIdx.x;
    int want = 0;
    if (i < a.rows) {
      const Row r = row_of(a, static_cast<int>(i));
      const int p = open_page(a, r);
      int copy = -1;
      if (p >= 0) {
        const int refs = a.refs_out[p];
        if (refs != 1 && !(refs == w.writers[p] && w.lowest[p] == i)) copy = p;
      }
      w.copied[i] = copy;
      want = (copy >= 0) + r.need - r.have;
      over += r.over;
      const int64_t size = static_cast<int64_t>(r.held) + r.grow;
      a.lengths_out[i] = static_cast<int>(min<int64_t>(size, a.cols << a.shift));
    }
    const int first = scan<kDemand>(want, &total);
    if (i < a.rows) w.begin[i] = before + first;
    before += total;
  }
  const int overs = sum_long<kDemand>(over);
  if (threadIdx.x == 0) {
    w.begin[a.rows] = before;
    *w.over = overs;
  }
}

// The free pages in order, as far as they are wanted.  (A copied page keeps at
// least one reference, so giving one of its references up here frees none.)
__global__ __launch_bounds__(kThreads) void update_list(PageArgs a, Space w, int blocks) {
  const int rows = static_cast<int>(a.rows), wants = w.begin[rows];
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  const int64_t p0 = id * kEach;
  int refs[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) refs[j] = p0 + j < a.pages ? a.refs_out[p0 + j] : 1;
  int all = 0, mine = 0;  // free pages of every block, of those before this one
  for (int b = threadIdx.x; b < blocks; b += kThreads) {
    const int n = w.counts[b];
    all += n;
    if (b < static_cast<int>(blockIdx.x)) mine += n;
  }
  const int before = sum_all(mine);
  if (blockIdx.x == 0) {
    all = sum_all(all);
    if (threadIdx.x == 0) {
      *a.count = add_held(max(wants - all, 0), *w.over);
      *w.given = min(wants, all);
    }
  }
  int n = 0, total;
#pragma unroll
  for (int j = 0; j < kEach; ++j) n += refs[j] <= 0;
  int rank = before + scan<kThreads>(n, &total);
#pragma unroll
  for (int j = 0; j < kEach; ++j)
    if (refs[j] <= 0) {
      if (rank < wants) {
        w.list[rank] = static_cast<int>(p0 + j);
        a.refs_out[p0 + j] = 1;
      }
      ++rank;
    }
  for (int64_t i = id; i < rows; i += static_cast<int64_t>(gridDim.x) * kThreads)
    if (w.copied[i] >= 0) atomicSub(&a.refs_out[w.copied[i]], 1);
}

// A row's new entries (`fill`), and its copy in one layer of one array: a
// workgroup for each, which take turns.
__global__ __launch_bounds__(kThreads) void update_copy(PageArgs a, Space w, beam_moe_pools p,
                                                         bool fill) {
  const int parts = max(p.count * p.layers, 1);
  for (int64_t x = blockIdx.x; x < a.rows * parts; x += gridDim.x) {
    const int i = static_cast<int>(x / parts), part = static_cast<int>(x % parts);
    const int src = w.copied[i], begin = w.begin[i], given = *w.given;
    const bool copies = src >= 0;
    if (fill && part == 0) {
      const int n = w.begin[i + 1] - begin, have = n > 0 ? row_of(a, i).have : 0;
      for (int j = threadIdx.x; j < n; j += kThreads)
        a.tables_out[i * a.cols + have + j - copies] = begin + j < given ? w.list[begin + j] : -1;
    }
    if (copies && begin < given && p.count * p.layers > 0) copy_page<false>(p, part, src, w.list[begin]);
  }
}

// All of the tables' part in one workgroup: references and who writes where in LDS.
constexpr int kSmallPages = 8192, kSmallRows = kDemand, kSmallEntries = 1 << 16;
__global__ __launch_bounds__(kDemand) void update_small(PageArgs a, Space w) {
  extern __shared__ int32_t lds[];
  const int pages = static_cast<int>(a.pages), rows = static_cast<int>(a.rows);
  const int old_rows = static_cast<int>(a.old_rows), cols = static_cast<int>(a.cols);
  int32_t* const refs = lds;
  int32_t* const writers = refs + pages;  // later the list of free pages
  int32_t* const lowest = writers + pages;
  int32_t* const children = lowest + pages;
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave;
  constexpr int kWaves = kDemand / kWave;
  // the thread's row
  const bool mine = tid < rows;
  Row r = {};
  if (mine) r = row_of(a, tid);
  const int open = mine ? open_page(a, r) : -1;
  for (int p = tid; p < pages; p += kDemand) {
    refs[p] = a.refs[p];
    writers[p] = 0;
    lowest[p] = INT_MAX;
  }
  if (tid < old_rows) children[tid] = a.parents || rows == 0 ? 0 : 1;
  __syncthreads();
  if (a.parents && mine && r.parent >= 0) atomicAdd(&children[r.parent], 1);
  if (open >= 0) {
    atomicAdd(&writers[open], 1);
    atomicMin(&lowest[open], tid);
  }
  for (int i = wave; i < rows; i += kWaves) {
    const Row x = row_of(a, i);
    const int32_t* from = a.tables + max(x.parent, 0) * cols;
    for (int c = lane; c < cols; c += kWave) a.tables_out[i * cols + c] = c < x.have ? from[c] : -1;
  }
  __syncthreads();
  for (int i = wave; i < old_rows; i += kWaves) {
    const int by = children[i] - 1;
    if (by == 0) continue;
    const int have = held_pages(a, i);
    for (int c = lane; c < have; c += kWave) {
      const int p = a.tables[i * cols + c];
      if (p >= 0 && p < pages) atomicAdd(&refs[p], by);
    }
  }
  __syncthreads();
  int copy = -1, want = 0, wants;
  int64_t over = 0;
  if (mine) {
    if (open >= 0 && refs[open] != 1 && !(refs[open] == writers[open] && lowest[open] == tid)) copy = open;
    want = (copy >= 0) + r.need - r.have;
    over = r.over;
    a.lengths_out[tid] =
        static_cast<int>(min<int64_t>(static_cast<int64_t>(r.held) + r.grow, a.cols << a.shift));
  }
  const int begin = scan<kDemand>(want, &wants);
  const int overs = sum_long<kDemand>(over);
  // free pages: eight neighbours a thread
  int n = 0, all;
  bool free[kEach];
#pragma unroll
  for (int j = 0; j < kEach; ++j) {
    const int p = tid * kEach + j;
    free[j] = p < pages && refs[p] <= 0;
    n += free[j];
  }
  int rank = scan<kDemand>(n, &all);
#pragma unroll
  for (int j = 0; j < kEach; ++j)
    if (free[j]) {
      if (rank < wants) {
        writers[rank] = tid * kEach + j;
        refs[tid * kEach + j] = 1;
      }
      ++rank;
    }
  __syncthreads();
  const int given = min(wants, all);
  if (copy >= 0) atomicSub(&refs[copy], 1);
  if (mine) {
    for (int j = 0; j < want; ++j)
      a.tables_out[tid * cols + r.have + j - (copy >= 0)] = begin + j < given ? writers[begin + j] : -1;
    w.copied[tid] = copy;
    w.begin[tid] = begin;
    if (copy >= 0 && begin < given) w.list[begin] = writers[begin];
  }
  if (tid == 0) {
    *w.given = given;
    *a.count = add_held(max(wants - all, 0), overs);
  }
  __syncthreads();
  for (int p = tid; p < pages; p += kDemand) a.refs_out[p] = refs[p];
}

__global__ __launch_bounds__(kThreads) void copy_list(beam_moe_pools p, int64_t pages, int64_t n,
                                                       const int32_t* src, const int32_t* dst) {
  const int parts = p.count * p.layers;
  for (int64_t x = blockIdx.x; x < n * parts; x += gridDim.x) {
    const int s = src[x / parts], d = dst[x / parts];
    if (s >= 0 && s < pages && d >= 0 && d < pages) copy_page<true>(p, static_cast<int>(x % parts), s, d);
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
    const int have = held_pages(a, static_cast<int>(i));
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
    copy_page<true>(p, static_cast<int>(x % parts), w.from[i], w.to[i]);
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
  // from, to and rank of a packing; writers, lowest and list of an update
  return sizeof(int32_t) * static_cast<size_t>(3 * room(pages) + room(ceil_div(pages, kBlock)) +
                                               2 * room(rows + 1) + room(65536) + 2 * room(1));
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
  w.given = carve(at, 1);
  w.list = carve(at, a.pages);
  const int64_t copies = std::min(a.rows * p.count * p.layers, kCopyBlocks);
  if (a.pages <= kSmallPages && std::max(a.rows, a.old_rows) <= kSmallRows &&
      std::max(a.rows, a.old_rows) * a.cols <= kSmallEntries) {
    const size_t shared = static_cast<size_t>(3 * a.pages + a.old_rows) * sizeof(int32_t);
    hipLaunchKernelGGL(update_small, dim3(1), dim3(kDemand), shared, s, a, w);
    if (copies)
      hipLaunchKernelGGL(update_copy, dim3(copies), dim3(kThreads), 0, s, a, w, p, false);
    return hipGetLastError();
  }
  const int64_t work = std::max(a.pages, a.old_rows * kWave);
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>(ceil_div(work, kThreads), 2048));
  hipLaunchKernelGGL(update_prepare, dim3(grid), dim3(kThreads), 0, s, a, w);
  if (a.rows + a.old_rows)
    hipLaunchKernelGGL(update_rows, dim3(a.rows + a.old_rows), dim3(kThreads), 0, s, a, w);
  hipLaunchKernelGGL(update_count, dim3(blocks + 1), dim3(kDemand), 0, s, a, w);
  hipLaunchKernelGGL(update_list, dim3(std::max(blocks, 1)), dim3(kThreads), 0, s, a, w, blocks);
  if (a.rows)
    hipLaunchKernelGGL(update_copy, dim3(std::max(copies, std::min(a.rows, kCopyBlocks))),
                       dim3(kThreads), 0, s, a, w, p, true);
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
  hipLaunchKernelGGL(pack_move, dim3(std::min(work, kCopyBlocks)), dim3(kThreads), 0, s, a, w, p);
  return hipGetLastError();
}

}  // namespace beam
