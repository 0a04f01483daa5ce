// Operations on whole pages of the paged caches: copy, fork, free, compact.
//
// A pool of NB pages is described by ref_counts [NB]: a page is in use while
// its count is positive.  Block-table rows hold page ids; the page operations
// move page contents in every tensor whose first dimension is the page (any
// element type, any layout of the other dimensions), counts and table entries.
//
// Copies are bound by memory (twice the page bytes).  The bookkeeping of fork,
// free and compact is a few passes over small integer arrays in which every
// step needs the one before (claims before updates, counts before ranks); it
// runs in one cluster of eight blocks, whose hardware barrier and shared
// counts take the place of separate launches.
#include <cooperative_groups.h>

#include "pa_device.cuh"
#include "pa_host.h"

#include <algorithm>

namespace cg = cooperative_groups;

namespace pa {

constexpr int kMaxPageTensors = 48;      // tensors of one copy launch (kernel parameters of 4 KB)
constexpr int kMaxCaches = 1024;         // tensors of one call
constexpr int kItemBytes = 1024;         // one warp's share of a page of one tensor: 2 x 16 bytes a lane
constexpr int kWindow = 8;               // pages of the pool a warp looks at together (compaction)
constexpr int kClusterCtas = 8;
constexpr int kClusterThreads = 1024;
constexpr uint32_t kErrPageOp = 32u;

// One tensor's pages: `n2 x n1` runs of `run` contiguous bytes.
struct PageTensor {
  uint8_t* base;
  int64_t page_stride, s1, s2;   // bytes
  int32_t run, n1, n2;
  int32_t vec;                   // bytes a lane moves at once (16, 8, 4, 2 or 1)
  int32_t item0;                 // first item of this tensor within a page's items
  int32_t pad;
};

enum PairSource { kPairsListed, kPairsFork, kPairsCompact };

struct CopyParams {
  PageTensor t[kMaxPageTensors];
  int32_t num_tensors, items;    // items of one page
  int64_t pairs;                 // copies to look at
  int32_t num_pages;
  const int32_t *src, *dst;      // listed pairs; fork: dst = the new pages; compact: dst = the page map
  const int32_t *parents, *seq_lens, *tables;   // fork
  int64_t table_stride;
  const int32_t* num_used;       // compact
  uint32_t* err;
};

// Source and destination page of copy k; false: nothing to do.
template <PairSource SRC>
__device__ __forceinline__ bool pair_of(const CopyParams& p, int64_t k, int& src, int& dst, bool report) {
  if constexpr (SRC == kPairsListed) {
    src = p.src[k];
    dst = p.dst[k];
    if (src < 0 || dst < 0) return false;                  // padding
    if (src >= p.num_pages || dst >= p.num_pages) {
      if (report) atomicOr(p.err, kErrPageRange);
      return false;
    }
  } else {
    dst = __ldcg(p.dst + k);                               // -1 where the fork took no page
    if (dst < 0) return false;
    const int row = p.parents[k];
    src = p.tables[static_cast<int64_t>(row) * p.table_stride + p.seq_lens[row] / kPage];
    if (src < 0 || src >= p.num_pages) return false;       // reported by the fork kernel
  }
  return src != dst;
}

// Byte `x` of a page of several runs: its offset from the page's start.
__device__ __forceinline__ int64_t run_offset(const PageTensor& t, int x) {
  const int i = x / t.run;
  const int i2 = i / t.n1;
  return i2 * t.s2 + (i - i2 * t.n1) * t.s1 + (x - i * t.run);
}

// `bytes` (at most kItemBytes) starting at byte `off` of a page, one warp:
// U loads of a lane are issued before any is stored.
template <typename V>
__device__ __forceinline__ void copy_item(const PageTensor& t, int64_t src, int64_t dst, int off, int bytes, int lane) {
  constexpr int W = static_cast<int>(sizeof(V));
  const uint8_t* a = t.base + src * t.page_stride;
  uint8_t* b = t.base + dst * t.page_stride;
  if (t.n1 == 1 && t.n2 == 1) {
    constexpr int U = 2;
    for (int o = lane * W; o < bytes; o += U * 32 * W) {
      V v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (o + u * 32 * W < bytes) v[u] = *reinterpret_cast<const V*>(a + off + o + u * 32 * W);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (o + u * 32 * W < bytes) *reinterpret_cast<V*>(b + off + o + u * 32 * W) = v[u];
    }
  } else {
    constexpr int U = 2;
    for (int o = lane * W; o < bytes; o += U * 32 * W) {
      V v[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (o + u * 32 * W < bytes) v[u] = *reinterpret_cast<const V*>(a + run_offset(t, off + o + u * 32 * W));
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (o + u * 32 * W < bytes) *reinterpret_cast<V*>(b + run_offset(t, off + o + u * 32 * W)) = v[u];
    }
  }
}

// Item `item` of page src to page dst.
__device__ __forceinline__ void copy_page_item(const CopyParams& p, int item, int64_t src, int64_t dst, int lane) {
  int lo = 0, hi = p.num_tensors - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.t[mid].item0 <= item) lo = mid; else hi = mid - 1;
  }
  const PageTensor& t = p.t[lo];
  const int off = (item - t.item0) * kItemBytes;
  const int bytes = min(kItemBytes, t.run * t.n1 * t.n2 - off);
  switch (t.vec) {
    case 16: copy_item<uint4>(t, src, dst, off, bytes, lane); break;
    case 8: copy_item<uint2>(t, src, dst, off, bytes, lane); break;
    case 4: copy_item<uint32_t>(t, src, dst, off, bytes, lane); break;
    case 2: copy_item<uint16_t>(t, src, dst, off, bytes, lane); break;
    default: copy_item<uint8_t>(t, src, dst, off, bytes, lane); break;
  }
}

// A warp takes one item (at most 1 KB of one tensor of one page) at a time, the
// items of a page side by side.  Bound by memory: 604 MB of random 18 KB pages take
// 96 us, torch's copy of as many consecutive bytes 95.  Small items and a grid of
// four waves keep the load even: 4 KB items in one wave took 134 us, 1 KB items in
// one wave 110, a warp an item (a launch of every item's warp) 100.
template <PairSource SRC>
__global__ void __launch_bounds__(256, 8) pa_page_copy_kernel(const __grid_constant__ CopyParams p) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (blockDim.x / 32);
  const int64_t first = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  if constexpr (SRC == kPairsCompact) {
    // (window of kWindow pages, item): the pages that move have ids from num_used on
    const int64_t base = __ldcg(p.num_used);
    const int64_t total = (p.num_pages - base + kWindow - 1) / kWindow * p.items;
    for (int64_t i = first; i < total; i += warps) {
      const int64_t w = i / p.items;
      const int64_t page = base + w * kWindow + lane;
      const int to = lane < kWindow && page < p.num_pages ? __ldcg(p.dst + page) : -1;
      for (uint32_t m = __ballot_sync(0xffffffffu, to >= 0); m != 0u; m &= m - 1u) {
        const int b = __ffs(m) - 1;
        copy_page_item(p, static_cast<int>(i - w * p.items), base + w * kWindow + b, __shfl_sync(0xffffffffu, to, b), lane);
      }
    }
  } else {
    const int64_t total = p.pairs * p.items;
    for (int64_t i = first; i < total; i += warps) {
      const int64_t k = i / p.items;
      const int item = static_cast<int>(i - k * p.items);
      int src, dst;
      if (pair_of<SRC>(p, k, src, dst, item == 0 && lane == 0)) copy_page_item(p, item, src, dst, lane);
    }
  }
}

// Table entries after a compaction: every entry that names a page in use.  (As a
// part of the copy kernel it cost that kernel's registers: 126 us against 116 for a
// compaction that reads and writes 579 MB; as a part of the numbering cluster it gained
// nothing on 120 entries and lost 4 us on 65536.)
__global__ void __launch_bounds__(256) pa_table_remap_kernel(int32_t* tables, int64_t stride, int64_t rows,
                                                             int64_t cols, const int32_t* map, int32_t num_pages) {
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t total = rows * cols, step = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
    const int64_t r = i / cols;
    int32_t* e = tables + r * stride + (i - r * cols);
    const int32_t id = *e;
    if (id < 0 || id >= num_pages) continue;
    const int32_t to = __ldcg(map + id);
    if (to >= 0 && to != id) *e = to;
  }
}

// ------------------------------------------------------------ bookkeeping
struct PoolParams {
  int32_t* tables;
  int64_t table_stride;
  int32_t rows, cols;
  int32_t* seq_lens;
  int32_t* ref;
  int32_t num_pages;
  const int32_t *parents, *children;
  int32_t* pages;        // fork: new pages; free: the free list; compact: the page map
  int32_t* count;        // free: entries of the list; compact: pages in use
  int32_t n;             // entries of the call's lists
  const int32_t* list;   // free: rows
  uint32_t* err;
};

// (The bookkeeping kernels are bound by dependent steps, not by bytes.  Device time as
// profiled, with cold caches: forking 256 rows of 32 to 256 pages 12.9 us, freeing them
// and listing their pool 15.2, numbering a pool of 32768 pages 13.)

// Fork: a warp decides one entry (every check reads state that no entry's
// update changes: lengths of the children, counts of the new pages), then,
// after the cluster's barrier, applies it.
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kClusterThreads, 1)
    pa_page_fork_kernel(const PoolParams p) {
  constexpr int W = kClusterThreads / 32;
  static_assert(kMaxSeqsHost <= 32 * kClusterCtas * W, "a warp's verdicts fit one word");
  uint32_t accepted = 0u;                         // bit j: this warp's j-th entry
  grid_dependency_wait();
  grid_launch_dependents();
  cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w0 = static_cast<int>(cluster.block_rank()) * W + warp;
  int j = 0;
  for (int k = w0; k < p.n; k += kClusterCtas * W, ++j) {
    const int par = p.parents[k], chi = p.children[k], page = p.pages[k];
    if (par < 0 || chi < 0) continue;             // padding
    bool ok = par < p.rows && chi < p.rows;
    if (ok) {
      const int len = p.seq_lens[par];
      const int full = len / kPage;
      const bool part = len % kPage != 0;
      ok = len >= 0 && full + (part ? 1 : 0) <= p.cols && p.seq_lens[chi] == 0;
      if (ok && part) ok = page >= 0 && page < p.num_pages && p.ref[page] == 0;
      bool clash = false;
      for (int x = lane; x < p.n; x += 32) {
        const int xp = p.parents[x], xc = p.children[x];
        if (xp < 0 || xc < 0) continue;
        clash |= xp == chi;                                     // the child is itself forked from
        clash |= x < k && (xc == chi || (part && p.pages[x] == page));   // an earlier entry has it
      }
      ok = !__any_sync(0xffffffffu, clash) && ok;
    }
    if (ok) accepted |= 1u << j;
    else if (lane == 0) atomicOr(p.err, kErrPageOp);
  }
  cluster.sync();
  j = 0;
  for (int k = w0; k < p.n; k += kClusterCtas * W, ++j) {
    if (!((accepted >> j) & 1u)) {
      if (lane == 0) p.pages[k] = -1;
      continue;
    }
    const int par = p.parents[k], chi = p.children[k];
    const int len = p.seq_lens[par], full = len / kPage;
    const int32_t* from = p.tables + static_cast<int64_t>(par) * p.table_stride;
    int32_t* to = p.tables + static_cast<int64_t>(chi) * p.table_stride;
    for (int x0 = lane; x0 < full; x0 += 4 * 32) {
      int id[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) id[u] = x0 + 32 * u < full ? from[x0 + 32 * u] : 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (x0 + 32 * u >= full) break;
        to[x0 + 32 * u] = id[u];
        if (id[u] >= 0 && id[u] < p.num_pages) atomicAdd(p.ref + id[u], 1);
        else atomicOr(p.err, kErrPageRange);
      }
    }
    if (lane == 0) {
      if (len % kPage != 0) {
        const int page = p.pages[k];
        to[full] = page;
        atomicAdd(p.ref + page, 1);     // was 0; a damaged table may share it in the same call
        if (from[full] < 0 || from[full] >= p.num_pages) atomicOr(p.err, kErrPageRange);
      } else {
        p.pages[k] = -1;
      }
      p.seq_lens[chi] = len;
    }
  }
}

// Pages [lo, hi) of a warp: the pool cut into equal runs of 32-page words.
__device__ __forceinline__ void warp_pages(int num_pages, int w, int warps, int64_t& lo, int64_t& hi) {
  const int64_t words = (static_cast<int64_t>(num_pages) + 31) / 32;
  lo = min(static_cast<int64_t>(num_pages), words * w / warps * 32);
  hi = min(static_cast<int64_t>(num_pages), words * (w + 1) / warps * 32);
}

// One bit a page: the pages of a warp's run that are in use (count positive), a word
// of 32 at a time.  The first look at the counts leaves the words in shared memory
// (eight loads in flight); runs of more than kMaskWords words are read again.
constexpr int kMaskWords = 256;          // a warp: pools of up to 2 million pages

template <typename F>
__device__ __forceinline__ void read_words(const int32_t* ref, int64_t lo, int64_t hi, int lane, uint32_t* words, F each) {
  for (int64_t b0 = lo; b0 < hi; b0 += 8 * 32) {
    int r[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t id = b0 + 32 * u + lane;
      r[u] = id < hi ? __ldcg(ref + id) : 0;
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int64_t b = b0 + 32 * u;
      if (b >= hi) break;
      const uint32_t m = __ballot_sync(0xffffffffu, r[u] > 0);
      const int64_t w = (b - lo) / 32;
      if (lane == 0 && w < kMaskWords) words[w] = m;
      each(b, m, r[u]);
    }
  }
  __syncwarp();
}

// The word of pages b .. b + 31 of a run that starts at lo.
__device__ __forceinline__ uint32_t word_of(const int32_t* ref, int64_t lo, int64_t hi, int64_t b, int lane,
                                            const uint32_t* words) {
  const int64_t w = (b - lo) / 32;
  if (w < kMaskWords) return words[w];
  return __ballot_sync(0xffffffffu, b + lane < hi && __ldcg(ref + b + lane) > 0);
}

// Bits of a word's pages b .. b + 31 with ids below n.
__device__ __forceinline__ uint32_t below(int64_t b, int64_t n) {
  return n <= b ? 0u : (n >= b + 32 ? 0xffffffffu : (1u << (n - b)) - 1u);
}

// Exclusive prefix of one value per warp over the cluster's warps, in (block,
// warp) order, and the total.  `s` holds this block's warps' values.
__device__ __forceinline__ int cluster_prefix(cg::cluster_group& cluster, int v, int* s_warp, int* s_total, int& total) {
  constexpr int W = kClusterThreads / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (lane == 0) s_warp[warp] = v;
  __syncthreads();
  const int wv = s_warp[lane % W];
  int inc = wv;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += y;
  }
  if (threadIdx.x == 31) *s_total = inc;
  const int before = __shfl_sync(0xffffffffu, inc - wv, warp);
  cluster.sync();
  const int rank = static_cast<int>(cluster.block_rank());
  int off = 0;
  total = 0;
  for (int b = 0; b < kClusterCtas; ++b) {
    const int c = *cluster.map_shared_rank(s_total, b);
    if (b < rank) off += c;
    total += c;
  }
  return off + before;
}

// Free: a warp releases one row at a time; then the pages whose count is 0 are
// listed in ascending order.
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kClusterThreads, 1)
    pa_page_free_kernel(const PoolParams p) {
  constexpr int W = kClusterThreads / 32;
  __shared__ int s_warp[W];
  __shared__ int s_total;
  __shared__ uint32_t s_words[W][kMaskWords];
  grid_dependency_wait();
  grid_launch_dependents();
  cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = static_cast<int>(cluster.block_rank()) * W + warp;
  for (int k = w; k < p.n; k += kClusterCtas * W) {
    const int row = p.list[k];
    if (row < 0) continue;                        // padding
    if (row >= p.rows) {
      if (lane == 0) atomicOr(p.err, kErrPageOp);
      continue;
    }
    // the exchange makes a row listed twice release its pages once
    int len = 0;
    if (lane == 0) len = atomicExch(p.seq_lens + row, 0);
    len = __shfl_sync(0xffffffffu, len, 0);
    if (len <= 0) continue;
    int held = (len - 1) / kPage + 1;
    if (held > p.cols) {
      if (lane == 0) atomicOr(p.err, kErrSeqLen);
      held = p.cols;
    }
    const int32_t* from = p.tables + static_cast<int64_t>(row) * p.table_stride;
    // four pages a lane in flight: ids, then counts
    for (int x0 = lane; x0 < held; x0 += 4 * 32) {
      int id[4], old[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) id[u] = x0 + 32 * u < held ? from[x0 + 32 * u] : -2;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const bool valid = id[u] >= 0 && id[u] < p.num_pages;
        if (!valid && x0 + 32 * u < held) atomicOr(p.err, kErrPageRange);
        old[u] = valid ? atomicSub(p.ref + id[u], 1) : 1;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (old[u] <= 0) {                        // was free already: its count stays
          atomicAdd(p.ref + id[u], 1);
          atomicOr(p.err, kErrPageOp);
        }
    }
  }
  cluster.sync();
  int64_t lo, hi;
  warp_pages(p.num_pages, w, kClusterCtas * W, lo, hi);
  int mine = 0;
  read_words(p.ref, lo, hi, lane, s_words[warp],
             [&](int64_t b, uint32_t m, int) { mine += __popc(~m & below(b, hi)); });
  int total;
  int at = cluster_prefix(cluster, mine, s_warp, &s_total, total);
  for (int64_t b = lo; b < hi; b += 32) {
    const uint32_t m = ~word_of(p.ref, lo, hi, b, lane, s_words[warp]) & below(b, hi);
    if (m >> lane & 1u) p.pages[at + __popc(m & ((1u << lane) - 1u))] = static_cast<int32_t>(b + lane);
    at += __popc(m);
  }
  if (w == 0 && lane == 0) *p.count = total;
  for (int64_t i = total + static_cast<int64_t>(w) * 32 + lane; i < p.num_pages; i += kClusterCtas * W * 32)
    p.pages[i] = -1;
  cluster.sync();                                  // no block leaves while its total may still be read
}

// Compact, the bookkeeping: U pages are in use; the k-th page in use with id
// >= U ("high") moves to the k-th free page with id < U ("hole").  The holes'
// list lives in map[U ..] until the high pages have read it (there are at most
// NB - U holes), a high page's target in its own count, negated, until the map
// is written.
__global__ void __cluster_dims__(kClusterCtas, 1, 1) __launch_bounds__(kClusterThreads, 1)
    pa_page_compact_kernel(const PoolParams p) {
  constexpr int W = kClusterThreads / 32;
  __shared__ int s_warp[W];
  __shared__ int s_total, s_low;                  // s_low: pages in use with ids below U
  __shared__ uint32_t s_words[W][kMaskWords];
  grid_dependency_wait();
  grid_launch_dependents();
  cg::cluster_group cluster = cg::this_cluster();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w = static_cast<int>(cluster.block_rank()) * W + warp;
  uint32_t* const words = s_words[warp];
  int64_t lo, hi;
  warp_pages(p.num_pages, w, kClusterCtas * W, lo, hi);
  int mine = 0;
  bool negative = false;
  read_words(p.ref, lo, hi, lane, words, [&](int64_t, uint32_t m, int r) {
    mine += __popc(m);
    negative |= r < 0;
  });
  if (negative) atomicOr(p.err, kErrPageOp);
  int U;
  const int used = cluster_prefix(cluster, mine, s_warp, &s_total, U);     // pages in use before lo
  // before a page x there are x - (pages in use before it) free pages, and from U on
  // (pages in use before x) - (pages in use before U) high ones: the warp whose run
  // holds U tells every block the latter
  if (lo <= U && U < hi) {
    int before = used;
    for (int64_t b = lo; b < U; b += 32) before += __popc(word_of(p.ref, lo, hi, b, lane, words) & below(b, U));
    if (lane < kClusterCtas) *cluster.map_shared_rank(&s_low, lane) = before;
  }
  int at_hole = static_cast<int>(lo) - used;
  for (int64_t b = lo; b < min(hi, static_cast<int64_t>(U)); b += 32) {
    const uint32_t in = below(b, min(hi, static_cast<int64_t>(U)));
    const uint32_t m = word_of(p.ref, lo, hi, b, lane, words);
    const int64_t id = b + lane;
    if (in >> lane & 1u) p.pages[id] = m >> lane & 1u ? static_cast<int32_t>(id) : -1;
    if ((in & ~m) >> lane & 1u) p.pages[U + at_hole + __popc(in & ~m & ((1u << lane) - 1u))] = static_cast<int32_t>(id);
    at_hole += __popc(in & ~m);
  }
  cluster.sync();
  int at_high = lo < U ? 0 : used - s_low;
  for (int64_t b = lo; b < hi; b += 32) {
    const int64_t id = b + lane;
    const uint32_t m = word_of(p.ref, lo, hi, b, lane, words) & ~below(b, U);
    if (m >> lane & 1u) {
      const int to = __ldcg(p.pages + U + at_high + __popc(m & ((1u << lane) - 1u)));
      p.ref[to] = __ldcg(p.ref + id);
      p.ref[id] = -1 - to;
    } else if (id < hi) {
      if (id >= U) p.ref[id] = 0;
    }
    at_high += __popc(m);
    __syncwarp();
  }
  cluster.sync();
#pragma unroll 4
  for (int64_t b = lo; b < hi; b += 32) {
    const int64_t id = b + lane;
    if (id >= hi || id < U) continue;
    const int r = p.ref[id];
    p.pages[id] = r < 0 ? -1 - r : -1;
    p.ref[id] = 0;
  }
  if (w == 0 && lane == 0) *p.count = U;
}

namespace {

template <typename K, typename... A>
cudaError_t launch_pdl(K kernel, dim3 grid, int threads, cudaStream_t stream, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

int elem_bytes(int dtype) {
  switch (dtype) {
    case PA_BF16: return 2;
    case PA_FP8_E4M3: case PA_FP4_E2M1X2: return 1;
    case PA_F32: case PA_I32: return 4;
    default: return 0;
  }
}

// Geometry of one cache tensor [NB, ...]: its pages as n2 x n1 contiguous runs.
int page_tensor(const pa_tensor_t& c, int index, int64_t nb, PageTensor* out, int64_t* page_bytes) {
  if (c.data == nullptr) return host_fail(PA_ERR_INVALID_ARG, "caches[%d]: data pointer is NULL", index);
  if (c.ndim < 2 || c.ndim > 4) return host_fail(PA_ERR_INVALID_ARG, "caches[%d]: ndim %d not in 2..4", index, c.ndim);
  const int64_t es = elem_bytes(c.dtype);
  if (es == 0) return host_fail(PA_ERR_INVALID_ARG, "caches[%d]: unknown element type", index);
  if (c.shape[0] != nb)
    return host_fail(PA_ERR_INVALID_ARG, "caches[%d] has %lld pages, expected %lld", index,
                     static_cast<long long>(c.shape[0]), static_cast<long long>(nb));
  int64_t bytes = es;
  for (int d = 0; d < c.ndim; ++d) {
    if (c.shape[d] < 1 && d > 0) return host_fail(PA_ERR_INVALID_ARG, "caches[%d]: empty dimension", index);
    if (c.stride[d] < 0 || (c.stride[d] == 0 && c.shape[d] > 1))
      return host_fail(PA_ERR_INVALID_ARG, "caches[%d]: strides must be positive", index);
    if (d > 0) {
      if (c.shape[d] > (int64_t(1) << 28) || bytes * c.shape[d] > (int64_t(1) << 28))
        return host_fail(PA_ERR_UNSUPPORTED, "caches[%d]: a page of more than 256 MiB", index);
      bytes *= c.shape[d];
    }
  }
  if (!host_aligned(c.data, static_cast<size_t>(es)))
    return host_fail(PA_ERR_INVALID_ARG, "caches[%d]: data not aligned to its element", index);
  // dimensions inside the page, innermost first, merged where contiguous
  int64_t run = es, n[3] = {1, 1, 1}, s[3] = {0, 0, 0};
  int m = 0;
  for (int d = c.ndim - 1; d >= 1; --d) {
    if (c.shape[d] == 1) continue;
    const int64_t sb = c.stride[d] * es;
    if (m == 0 && sb == run) {
      run *= c.shape[d];
    } else if (m > 0 && sb == n[m - 1] * s[m - 1]) {
      n[m - 1] *= c.shape[d];
    } else {
      n[m] = c.shape[d];
      s[m] = sb;
      ++m;
    }
  }
  if (m == 3) return host_fail(PA_ERR_UNSUPPORTED, "caches[%d]: a page layout with no contiguous run", index);
  PageTensor t = {};
  t.base = static_cast<uint8_t*>(c.data);
  t.page_stride = c.stride[0] * es;
  t.run = static_cast<int32_t>(run);
  t.n1 = static_cast<int32_t>(n[0]);
  t.s1 = s[0];
  t.n2 = static_cast<int32_t>(n[1]);
  t.s2 = s[1];
  uint64_t bits = reinterpret_cast<uint64_t>(c.data) | static_cast<uint64_t>(t.page_stride) |
                  static_cast<uint64_t>(run) | static_cast<uint64_t>(t.s1) | static_cast<uint64_t>(t.s2);
  t.vec = 16;
  while (bits % static_cast<uint64_t>(t.vec) != 0) t.vec /= 2;
  *out = t;
  *page_bytes = bytes;
  return PA_OK;
}

struct CacheList {
  const pa_tensor_t* caches;
  int32_t count;
};

int check_caches(const CacheList& c, int64_t nb) {
  if (c.count < 0 || c.count > kMaxCaches)
    return host_fail(PA_ERR_UNSUPPORTED, "num_caches %d not in [0, %d]", c.count, kMaxCaches);
  if (c.count > 0 && c.caches == nullptr) return host_fail(PA_ERR_INVALID_ARG, "caches: pointer is NULL");
  PageTensor t;
  int64_t bytes;
  for (int i = 0; i < c.count; ++i) {
    const int st = page_tensor(c.caches[i], i, nb, &t, &bytes);
    if (st != PA_OK) return st;
  }
  return PA_OK;
}

// The copies of `p` (pairs set by the caller) in every tensor, up to
// kMaxPageTensors a launch.
template <PairSource SRC>
int launch_copies(CopyParams& p, const CacheList& c, int64_t nb, int num_sms, cudaStream_t stream) {
  for (int first = 0; first < c.count; first += kMaxPageTensors) {
    p.num_tensors = std::min(kMaxPageTensors, c.count - first);
    int64_t items = 0;
    for (int i = 0; i < p.num_tensors; ++i) {
      int64_t bytes;
      const int st = page_tensor(c.caches[first + i], first + i, nb, &p.t[i], &bytes);
      if (st != PA_OK) return st;
      p.t[i].item0 = static_cast<int32_t>(items);
      items += (bytes + kItemBytes - 1) / kItemBytes;
    }
    p.items = static_cast<int32_t>(items);
    const int64_t units = SRC == kPairsCompact ? (p.pairs + kWindow - 1) / kWindow : p.pairs;
    const int64_t blocks = (units * items + 7) / 8;
    const dim3 grid(static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>(blocks, int64_t(num_sms) * 32))), 1, 1);
    const cudaError_t e = launch_pdl(pa_page_copy_kernel<SRC>, grid, 256, stream, p);
    if (e != cudaSuccess) return host_cuda_fail(e, "page copy launch");
  }
  return PA_OK;
}

// A contiguous int32 vector.
int check_ints(const pa_tensor_t* t, const char* name, int64_t n) {
  const int st = host_check_tensor(t, name, 1, n == 0);
  if (st != PA_OK) return st;
  if (t->data == nullptr) return PA_OK;
  if (t->dtype != PA_I32) return host_fail(PA_ERR_INVALID_ARG, "%s must be int32", name);
  if (t->shape[0] != n)
    return host_fail(PA_ERR_INVALID_ARG, "%s has %lld entries, expected %lld", name,
                     static_cast<long long>(t->shape[0]), static_cast<long long>(n));
  if (n > 1 && t->stride[0] != 1) return host_fail(PA_ERR_INVALID_ARG, "%s must be contiguous", name);
  if (!host_aligned(t->data, 4)) return host_fail(PA_ERR_INVALID_ARG, "%s must be 4-byte aligned", name);
  return PA_OK;
}

int64_t length_of(const pa_tensor_t* t) { return t != nullptr && t->ndim >= 1 ? t->shape[0] : -1; }

// Block tables [B, max_blocks] whose rows do not overlap, and ref_counts [NB].
int check_pool(const pa_tensor_t* bt, const pa_tensor_t* ref, PoolParams* p) {
  int st;
  if ((st = host_check_tensor(bt, "block_tables", 2, false)) != PA_OK) return st;
  if (bt->dtype != PA_I32) return host_fail(PA_ERR_INVALID_ARG, "block_tables must be int32");
  if ((bt->shape[1] > 1 && bt->stride[1] != 1) || (bt->shape[0] > 1 && bt->stride[0] < bt->shape[1]))
    return host_fail(PA_ERR_INVALID_ARG, "block_tables rows must be contiguous and must not overlap");
  if (!host_aligned(bt->data, 4)) return host_fail(PA_ERR_INVALID_ARG, "block_tables must be 4-byte aligned");
  if (bt->shape[0] > kMaxSeqsHost || bt->shape[1] > (int64_t(1) << 27))
    return host_fail(PA_ERR_UNSUPPORTED, "block table too large");
  const int64_t nb = length_of(ref);
  if (nb < 0) return host_fail(PA_ERR_INVALID_ARG, "ref_counts must be a vector");
  if (nb < 1 || nb > (int64_t(1) << 31) - 64)
    return host_fail(PA_ERR_UNSUPPORTED, "ref_counts: %lld pages", static_cast<long long>(nb));
  if ((st = check_ints(ref, "ref_counts", nb)) != PA_OK) return st;
  p->tables = static_cast<int32_t*>(bt->data);
  p->table_stride = bt->stride[0];
  p->rows = static_cast<int32_t>(bt->shape[0]);
  p->cols = static_cast<int32_t>(bt->shape[1]);
  p->ref = static_cast<int32_t*>(ref->data);
  p->num_pages = static_cast<int32_t>(nb);
  return PA_OK;
}

int pages_copy(const CacheList& c, const pa_tensor_t* src, const pa_tensor_t* dst, cudaStream_t stream) {
  int st;
  const int64_t n = length_of(src);
  if (n < 0 || n > (int64_t(1) << 30)) return host_fail(PA_ERR_INVALID_ARG, "src_pages must be a vector");
  if ((st = check_ints(src, "src_pages", n)) || (st = check_ints(dst, "dst_pages", n))) return st;
  if (c.count < 1) return host_fail(PA_ERR_INVALID_ARG, "num_caches %d < 1", c.count);
  if (c.caches == nullptr) return host_fail(PA_ERR_INVALID_ARG, "caches: pointer is NULL");
  const int64_t nb = c.caches[0].ndim >= 1 ? c.caches[0].shape[0] : 0;
  if (nb < 0 || nb > (int64_t(1) << 31) - 64) return host_fail(PA_ERR_UNSUPPORTED, "tensor extents too large");
  if ((st = check_caches(c, nb)) != PA_OK) return st;
  if (n == 0) return PA_OK;
  auto lock = host_lock();
  HostDevice dev;
  if ((st = host_device(&dev)) != PA_OK) return st;
  CopyParams p = {};
  p.pairs = n;
  p.num_pages = static_cast<int32_t>(nb);
  p.src = static_cast<const int32_t*>(src->data);
  p.dst = static_cast<const int32_t*>(dst->data);
  p.err = dev.status;
  return launch_copies<kPairsListed>(p, c, nb, dev.num_sms, stream);
}

int pages_fork(const CacheList& c, const pa_tensor_t* bt, const pa_tensor_t* sl, const pa_tensor_t* ref,
               const pa_tensor_t* parents, const pa_tensor_t* children, const pa_tensor_t* pages,
               cudaStream_t stream) {
  int st;
  PoolParams p = {};
  if ((st = check_pool(bt, ref, &p)) != PA_OK) return st;
  if ((st = check_ints(sl, "seq_lens", p.rows)) != PA_OK) return st;
  const int64_t n = length_of(parents);
  if (n < 0) return host_fail(PA_ERR_INVALID_ARG, "parents must be a vector");
  if (n > kMaxSeqsHost)
    return host_fail(PA_ERR_UNSUPPORTED, "parents: %lld entries > %d", static_cast<long long>(n),
                     kMaxSeqsHost);
  if ((st = check_ints(parents, "parents", n)) || (st = check_ints(children, "children", n)) ||
      (st = check_ints(pages, "new_pages", n)) || (st = check_caches(c, p.num_pages)))
    return st;
  if (n == 0) return PA_OK;
  auto lock = host_lock();
  HostDevice dev;
  if ((st = host_device(&dev)) != PA_OK) return st;
  p.seq_lens = static_cast<int32_t*>(sl->data);
  p.parents = static_cast<const int32_t*>(parents->data);
  p.children = static_cast<const int32_t*>(children->data);
  p.pages = static_cast<int32_t*>(pages->data);
  p.n = static_cast<int32_t>(n);
  p.err = dev.status;
  const cudaError_t e = launch_pdl(pa_page_fork_kernel, dim3(kClusterCtas, 1, 1), kClusterThreads, stream, p);
  if (e != cudaSuccess) return host_cuda_fail(e, "page fork launch");
  CopyParams cp = {};
  cp.pairs = n;
  cp.num_pages = p.num_pages;
  cp.dst = p.pages;
  cp.parents = p.parents;
  cp.seq_lens = p.seq_lens;
  cp.tables = p.tables;
  cp.table_stride = p.table_stride;
  cp.err = dev.status;
  return launch_copies<kPairsFork>(cp, c, p.num_pages, dev.num_sms, stream);
}

int pages_free(const pa_tensor_t* bt, const pa_tensor_t* sl, const pa_tensor_t* ref, const pa_tensor_t* rows,
               const pa_tensor_t* pages, const pa_tensor_t* count, cudaStream_t stream) {
  int st;
  PoolParams p = {};
  if ((st = check_pool(bt, ref, &p)) != PA_OK) return st;
  if ((st = check_ints(sl, "seq_lens", p.rows)) != PA_OK) return st;
  const int64_t n = length_of(rows);
  if (n < 0) return host_fail(PA_ERR_INVALID_ARG, "rows must be a vector");
  if (n > kMaxSeqsHost)
    return host_fail(PA_ERR_UNSUPPORTED, "rows: %lld entries > %d", static_cast<long long>(n), kMaxSeqsHost);
  if ((st = check_ints(rows, "rows", n)) || (st = check_ints(pages, "free_pages", p.num_pages)) ||
      (st = check_ints(count, "num_free", 1)))
    return st;
  auto lock = host_lock();
  HostDevice dev;
  if ((st = host_device(&dev)) != PA_OK) return st;
  p.seq_lens = static_cast<int32_t*>(sl->data);
  p.list = static_cast<const int32_t*>(rows->data);
  p.pages = static_cast<int32_t*>(pages->data);
  p.count = static_cast<int32_t*>(count->data);
  p.n = static_cast<int32_t>(n);
  p.err = dev.status;
  const cudaError_t e = launch_pdl(pa_page_free_kernel, dim3(kClusterCtas, 1, 1), kClusterThreads, stream, p);
  return e == cudaSuccess ? PA_OK : host_cuda_fail(e, "page free launch");
}

int pages_compact(const CacheList& c, const pa_tensor_t* bt, const pa_tensor_t* ref, const pa_tensor_t* map,
                  const pa_tensor_t* count, cudaStream_t stream) {
  int st;
  PoolParams p = {};
  if ((st = check_pool(bt, ref, &p)) != PA_OK) return st;
  if ((st = check_ints(map, "page_map", p.num_pages)) || (st = check_ints(count, "num_used", 1)) ||
      (st = check_caches(c, p.num_pages)))
    return st;
  auto lock = host_lock();
  HostDevice dev;
  if ((st = host_device(&dev)) != PA_OK) return st;
  p.pages = static_cast<int32_t*>(map->data);
  p.count = static_cast<int32_t*>(count->data);
  p.err = dev.status;
  cudaError_t e = launch_pdl(pa_page_compact_kernel, dim3(kClusterCtas, 1, 1), kClusterThreads, stream, p);
  if (e != cudaSuccess) return host_cuda_fail(e, "page compaction launch");
  CopyParams cp = {};
  cp.pairs = p.num_pages;
  cp.num_pages = p.num_pages;
  cp.dst = p.pages;
  cp.num_used = p.count;
  cp.err = dev.status;
  if ((st = launch_copies<kPairsCompact>(cp, c, p.num_pages, dev.num_sms, stream)) != PA_OK) return st;
  const int64_t entries = int64_t(p.rows) * p.cols;
  if (entries == 0) return PA_OK;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>((entries + 255) / 256, int64_t(dev.num_sms) * 8)), 1, 1);
  e = launch_pdl(pa_table_remap_kernel, grid, 256, stream, p.tables, p.table_stride, static_cast<int64_t>(p.rows),
                 static_cast<int64_t>(p.cols), static_cast<const int32_t*>(p.pages), p.num_pages);
  return e == cudaSuccess ? PA_OK : host_cuda_fail(e, "table remap launch");
}

}  // namespace
}  // namespace pa

extern "C" int paged_attn_pages_copy(const pa_tensor_t* caches, int32_t num_caches, const pa_tensor_t* src_pages,
                                     const pa_tensor_t* dst_pages, pa_stream_t stream) {
  return pa::host_entry([&] {
    return pa::pages_copy({caches, num_caches}, src_pages, dst_pages, reinterpret_cast<cudaStream_t>(stream));
  });
}

extern "C" int paged_attn_pages_fork(const pa_tensor_t* caches, int32_t num_caches, const pa_tensor_t* block_tables,
                                     const pa_tensor_t* seq_lens, const pa_tensor_t* ref_counts,
                                     const pa_tensor_t* parents, const pa_tensor_t* children,
                                     const pa_tensor_t* new_pages, pa_stream_t stream) {
  return pa::host_entry([&] {
    return pa::pages_fork({caches, num_caches}, block_tables, seq_lens, ref_counts, parents, children, new_pages,
                          reinterpret_cast<cudaStream_t>(stream));
  });
}

extern "C" int paged_attn_pages_free(const pa_tensor_t* block_tables, const pa_tensor_t* seq_lens,
                                     const pa_tensor_t* ref_counts, const pa_tensor_t* rows,
                                     const pa_tensor_t* free_pages, const pa_tensor_t* num_free, pa_stream_t stream) {
  return pa::host_entry([&] {
    return pa::pages_free(block_tables, seq_lens, ref_counts, rows, free_pages, num_free,
                          reinterpret_cast<cudaStream_t>(stream));
  });
}

extern "C" int paged_attn_pages_compact(const pa_tensor_t* caches, int32_t num_caches,
                                        const pa_tensor_t* block_tables, const pa_tensor_t* ref_counts,
                                        const pa_tensor_t* page_map, const pa_tensor_t* num_used,
                                        pa_stream_t stream) {
  return pa::host_entry([&] {
    return pa::pages_compact({caches, num_caches}, block_tables, ref_counts, page_map, num_used,
                             reinterpret_cast<cudaStream_t>(stream));
  });
}
