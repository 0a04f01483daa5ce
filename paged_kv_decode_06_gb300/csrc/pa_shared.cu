// Decode attention for batches that share prefixes: the plan of the shared part and its
// attention, all of a group's query rows against the pages its sequences have in common.
//
// Plan (one block): the pages that a group shares are those of shared_lens, cut to what
// every member sees whole ((L_i - q_i) / 16 pages, so that a sequence keeps a page of its
// own and no mask is needed), none for a group with fewer than two members; and each
// group's place in the order of steps and partial rows (pa_shared.h).
//
// Attention (tcgen05): with R rows a head the products cost 4 R D flops a key against
// 4 D bytes (bf16), so from about 280 rows on the tensor cores bound it, below that
// memory does; a softmax thread a row has 128 exponentials a block, half of what the two
// products of the block take.  A CTA holds two 128-row tiles ("slots") of query rows in
// shared memory and S / P (128 columns) and O (128 columns) of each in tensor memory, all
// 512 columns; blocks of 128 keys, K and V apart, pass through a ring.  One thread
// issues P V of slot 0, Q K^T of slot 0's next block, then the same for slot 1, so that
// one slot's softmax runs while the tensor cores work for the other.
//
// Warps: 0 issues the products and owns tensor memory, 1-3 load pages (a warp's TMA issue
// is serial, about 90 ns a 2 KB box, and a block has 32 boxes), 4-7 and 8-11 are the
// slots' softmax, thread = query row = tensor-memory lane.  P overwrites its S in
// 16 bits; O is rescaled only where the running maximum grew by more than 2^8.
//
// Order in the tensor pipe: one thread issues every product, and they run in that order,
// so S of a slot's next block may overwrite the P that the slot's P V before it reads.
// A commit covers all earlier products: once a softmax warp sees S of block b, P V of the
// slot's block before it has left O complete, and O may be rescaled.
//
// Waits are bounded, and each is made once a phase in order, so its barrier is never more
// than one phase behind (mbarrier parities cannot tell further).
#include "pa_device.cuh"
#include "pa_kernels.h"
#include "pa_pack.cuh"
#include "pa_shared.h"
#include "pa_split_tc.cuh"

namespace pa {
namespace {

// ---------------------------------------------------------------- plan kernel
constexpr int kPlanThreads = 1024;

// Inclusive sum over the block of one value a thread; *total gets the sum of all.
__device__ __forceinline__ int64_t block_scan(int64_t v, int64_t* s_warp, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) s_warp[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int64_t x = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    s_warp[lane] = x;
  }
  __syncthreads();
  if (warp > 0) v += s_warp[warp - 1];
  *total = s_warp[31];
  __syncthreads();
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) pa_shared_plan_kernel(const SharedParams p) {
  __shared__ int64_t s_warp[32];
  grid_dependency_wait();
  grid_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  for (int i = tid; i < p.num_seqs; i += kPlanThreads) {
    p.skip[i] = 0;
    p.seq_group[i] = -1;
  }
  // Groups are consecutive ranges of sequences; with any other list nothing is shared.
  bool bad = false;
  for (int g = tid; g < p.num_groups; g += kPlanThreads) {
    const int a = p.group_start[g], b = p.group_start[g + 1];
    bad |= a < 0 || b < a || b > p.num_seqs;
  }
  // A query_start_loc that is no cumulative sum could spread a group's tokens (each
  // partial row has its place by them).
  for (int i = tid; i < p.num_seqs; i += kPlanThreads) {
    const int a = p.qsl != nullptr ? p.qsl[i] : i, b = p.qsl != nullptr ? p.qsl[i + 1] : i + 1;
    bad |= a < 0 || b < a || b > p.num_tokens || b - a > p.max_qlen;
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) atomicOr(p.err, kErrQueryLen);
  for (int g = warp; g < p.num_groups; g += kPlanThreads / 32) {
    const int a = bad ? 0 : p.group_start[g], b = bad ? 0 : p.group_start[g + 1];
    // members: sequences with query tokens, all at positions of their own
    int pages = max(0, p.shared_lens[g]) / kPage, members = 0, t_lo = INT_MAX, t_hi = 0, first = INT_MAX;
    pages = min(pages, p.max_blocks);
    for (int i = a + lane; i < b; i += 32) {
      const int L = p.seq_lens[i];
      const int t0 = p.qsl != nullptr ? p.qsl[i] : i, t1 = p.qsl != nullptr ? p.qsl[i + 1] : i + 1;
      const bool in = t1 > t0 && L >= t1 - t0;
      if (!in) continue;
      ++members;
      first = min(first, i);
      pages = min(pages, (L - (t1 - t0)) / kPage);
      t_lo = min(t_lo, t0);
      t_hi = max(t_hi, t1);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      members += __shfl_xor_sync(0xffffffffu, members, o);
      pages = min(pages, __shfl_xor_sync(0xffffffffu, pages, o));
      first = min(first, __shfl_xor_sync(0xffffffffu, first, o));
      t_lo = min(t_lo, __shfl_xor_sync(0xffffffffu, t_lo, o));
      t_hi = max(t_hi, __shfl_xor_sync(0xffffffffu, t_hi, o));
    }
    if (members < 2 || pages < p.min_pages) pages = 0;
    SharedGroup sg = {};
    sg.seq = first;
    sg.pages = pages;
    if (pages > 0) {
      sg.t0 = t_lo;
      sg.rows = (t_hi - t_lo) * p.G;
      sg.pairs = (sg.rows + kSharedPair - 1) / kSharedPair;
      sg.last_rows = sg.rows - kSharedPair * (sg.pairs - 1);
      sg.blocks = (pages + kSharedBlockPages - 1) / kSharedBlockPages;
      const bool single = sg.last_rows <= kSharedTile;
      sg.steps_head = (sg.pairs - 1) * sg.blocks + shared_steps(sg, sg.pairs - 1);
      sg.rows_head = kSharedPair * (sg.pairs - 1) + (single ? 2 * sg.last_rows : sg.last_rows);
    }
    if (lane == 0) p.groups[g] = sg;
    if (pages == 0) continue;
    for (int i = a + lane; i < b; i += 32) {
      const int L = p.seq_lens[i];
      const int t0 = p.qsl != nullptr ? p.qsl[i] : i, t1 = p.qsl != nullptr ? p.qsl[i + 1] : i + 1;
      const bool in = t1 > t0 && L >= t1 - t0;
      if (in) {
        p.skip[i] = pages;
        p.seq_group[i] = g;
      }
    }
  }
  __syncthreads();
  int64_t step0 = 0, row0 = 0;
  for (int g0 = 0; g0 < p.num_groups; g0 += kPlanThreads) {
    const int g = g0 + tid;
    int64_t steps = 0, rows = 0;
    if (g < p.num_groups) {
      steps = static_cast<int64_t>(p.groups[g].steps_head) * p.Hkv;
      rows = static_cast<int64_t>(p.groups[g].rows_head) * p.Hkv;
    }
    int64_t all_steps, all_rows;
    const int64_t s1 = block_scan(steps, s_warp, &all_steps), r1 = block_scan(rows, s_warp, &all_rows);
    if (g < p.num_groups) {
      p.groups[g].step0 = step0 + s1 - steps;
      p.groups[g].row0 = row0 + r1 - rows;
    }
    step0 += all_steps;
    row0 += all_rows;
  }
  if (tid == 0) {
    p.totals->steps = step0;
    p.totals->rows = row0;
  }
}

// ------------------------------------------------------------- prefix kernel
constexpr int kThreads = 384;
constexpr int kLoaders = 3;               // warps 1 .. 3
constexpr int kSoftmaxWarp0 = 4;          // two warpgroups, a slot each
constexpr int kBlockPages = kSharedBlockPages;
constexpr int kKeys = 16 * kBlockPages;
constexpr uint32_t kHalf = kKeys * 128u;  // 64 features (128 bytes) of a block's keys, or of a tile's rows
constexpr uint32_t kCols = 512;
constexpr uint32_t kColS = 0;             // + 128 slot: S, its P over the first 64 columns
constexpr uint32_t kColO = 256;           // + 128 slot

template <int D>
struct PrefixGeo {
  static constexpr uint32_t TILE = (D / 64) * kHalf;     // bytes of a query tile, a K or a V block
  static constexpr int RING = D == 128 ? 5 : 10;
  static constexpr uint32_t SMEM = 1024 + 2 * TILE + RING * TILE + 1024;
};

// A piece: consecutive steps of one (group, head, pair) in this CTA.
struct Piece {
  int g, head, pair;
  int s0, s1;          // steps of the pair, [s0, s1)
  bool single;
};

// Walks this CTA's steps piece by piece; every warp runs one.
struct PieceWalker {
  int64_t x, end;
  int g;
  SharedGroup sg;
  __device__ __forceinline__ void start(const SharedParams& p, int64_t from, int64_t to) {
    x = from;
    end = to;
    // the last group that starts at or before x and has steps
    int lo = 0;
    for (int base = 0; base < p.num_groups; base += 32) {
      const int gg = base + (threadIdx.x & 31);
      const bool before = gg < p.num_groups && p.groups[gg].step0 <= x && p.groups[gg].pages > 0;
      const unsigned m = __ballot_sync(0xffffffffu, before);
      if (m != 0) lo = base + 31 - __clz(m);
    }
    g = lo;
    sg = p.groups[g];
  }
  __device__ __forceinline__ bool more() const { return x < end; }
  __device__ __forceinline__ Piece next(const SharedParams& p) {
    while (sg.pages == 0 || x >= sg.step0 + static_cast<int64_t>(sg.steps_head) * p.Hkv) sg = p.groups[++g];
    Piece c;
    c.g = g;
    const int64_t off = x - sg.step0;
    c.head = static_cast<int>(off / sg.steps_head);
    const int in_head = static_cast<int>(off - static_cast<int64_t>(c.head) * sg.steps_head);
    c.pair = min(in_head / sg.blocks, sg.pairs - 1);
    c.s0 = in_head - c.pair * sg.blocks;
    c.single = shared_single(sg, c.pair);
    const int n = shared_steps(sg, c.pair);
    c.s1 = static_cast<int>(min(static_cast<int64_t>(n), c.s0 + (end - x)));
    x += c.s1 - c.s0;
    return c;
  }
};

// 32 consecutive 32-bit columns of this thread's tensor-memory lane.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
// Waits for this thread's loads; the registers pass through, so that no use of them is
// moved before the wait.
template <int N>
__device__ __forceinline__ void after_wait(uint32_t (&r)[N]) {
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < N; ++e) asm volatile("" : "+r"(r[e]));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) { after_wait<16>(r); }
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) { after_wait<32>(r); }

// Block of `slot` in step s of a piece, or -1.
__device__ __forceinline__ int block_of(const Piece& c, const SharedGroup& sg, int s, int slot) {
  const int b = c.single ? 2 * s + slot : s;
  return b < sg.blocks ? b : -1;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    pa_shared_prefix_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                            const SharedParams p) {
  using GG = PrefixGeo<D>;
  constexpr int NH = D / 64;
  constexpr int RING = GG::RING;
  extern __shared__ uint8_t smem_raw[];
  __shared__ uint32_t s_tmem;
  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  const uint32_t ring0 = base + 2 * GG::TILE;
  const uint32_t bar0 = ring0 + RING * GG::TILE;
  auto full_bar = [&](int e) { return bar0 + 8u * e; };
  auto empty_bar = [&](int e) { return bar0 + 8u * (RING + e); };
  const uint32_t xb = bar0 + 8u * (2 * RING);
  auto sfull_bar = [&](int slot) { return xb + 8u * slot; };
  auto pfull_bar = [&](int slot) { return xb + 8u * (2 + slot); };
  auto qfull_bar = [&](int slot) { return xb + 8u * (4 + slot); };
  auto odone_bar = [&](int slot) { return xb + 8u * (6 + slot); };
  const uint32_t drain_bar = xb + 8u * 8;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
    for (int e = 0; e < RING; ++e) {
      mbar_init(full_bar(e), kLoaders);
      mbar_init(empty_bar(e), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(sfull_bar(s), 1);
      mbar_init(pfull_bar(s), 4);
      mbar_init(qfull_bar(s), 4);
      mbar_init(odone_bar(s), 1);
    }
    mbar_init(drain_bar, 1);
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t X = p.totals->steps;
  const int ng = X > 0 ? shared_ctas(X, gridDim.x, p.min_steps) : 0;
  const int cta = blockIdx.x;
  if (cta >= ng) return;
  const int64_t from = cta * X / ng, to = (cta + 1) * X / ng;
  if (from >= to) return;
  if (warp == 0) tmem_alloc(smem_addr(&s_tmem), kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = warp_uniform(s_tmem);
  PieceWalker wk;
  wk.start(p, from, to);

  if (warp >= 1 && warp < kSoftmaxWarp0) {
    // =============================== loaders =================================
    const int me = warp - 1;
    int e = 0;
    uint32_t round = 0;
    bool ok = true;
    while (ok && wk.more()) {
      const Piece c = wk.next(p);
      const SharedGroup& sg = wk.sg;
      const int32_t* row = p.block_tables + static_cast<int64_t>(sg.seq) * p.bt_stride;
      for (int s = c.s0; ok && s < c.s1; ++s) {
        // the step's K blocks, then its V blocks
        const int b0 = block_of(c, sg, s, 0), nb = c.single && block_of(c, sg, s, 1) >= 0 ? 2 : 1;
        for (int k = 0; k < 2 * nb; ++k) {
          const bool is_v = k >= nb;
          const int b = b0 + (is_v ? k - nb : k);
          const int np = min(kBlockPages, sg.pages - b * kBlockPages);
          // box x = (page, half): dealt over the three warps, a lane each
          const int x = kLoaders * lane + me, pg = x / NH, h = x - pg * NH;
          const int page = pg < np ? row[b * kBlockPages + pg] : 0;
          if (round > 0 && !warp_wait(empty_bar(e), (round - 1) & 1u, p.wait_ns)) {
            if (lane == 0) atomicOr(p.err, kErrTimeout);
            ok = false;
            break;
          }
          const int mine = np * NH > me ? (np * NH - me + kLoaders - 1) / kLoaders : 0;
          if (lane == 0) mbar_arrive_expect_tx(full_bar(e), static_cast<uint32_t>(mine) * kTcBox);
          __syncwarp();
          if (pg < np) {
            if ((page < 0 || page >= p.num_pages) && h == 0) atomicOr(p.err, kErrPageRange);
            // (a page id out of range reads as zeros: TMA fills outside the tensor)
            tma_load_4d(ring0 + static_cast<uint32_t>(e) * GG::TILE + h * kHalf + static_cast<uint32_t>(pg) * kTcBox,
                        is_v ? &tmap_v : &tmap_k, h * 64, 0, c.head, page, full_bar(e));
          }
          if (++e == RING) {
            e = 0;
            ++round;
          }
        }
      }
    }
  } else if (warp == 0) {
    // ============================ product issuer =============================
    const uint32_t idesc_o = umma_idesc_bf16(128, D, true);
    const uint32_t idesc_s = umma_idesc_bf16(128, 16, false) & ~(0x3Fu << 17);
    struct Cur {
      Piece c;
      int s, blocks, pages;
      uint32_t e;          // ring entry (counted on) of the step's first K block
      bool has[2];
    };
    uint32_t pn[2] = {0, 0}, qn[2] = {0, 0};                 // P and Q phases waited for
    uint32_t entries = 0;
    Cur cur = {}, nxt = {};
    auto fetch = [&](Cur& t, const Cur* before) -> bool {
      // the step after `before` (or the first)
      if (before != nullptr && before->s + 1 < before->c.s1) {
        t = *before;
        ++t.s;
      } else {
        if (!wk.more()) return false;
        t.c = wk.next(p);
        t.s = t.c.s0;
        t.blocks = wk.sg.blocks;
        t.pages = wk.sg.pages;
      }
      const int b1 = 2 * t.s + 1;
      t.has[0] = true;
      t.has[1] = !t.c.single || b1 < t.blocks;
      t.e = entries;
      entries += t.c.single && t.has[1] ? 4 : 2;
      return true;
    };
    auto np_of = [&](const Cur& t, int slot) {
      const int b = t.c.single ? 2 * t.s + slot : t.s;
      return min(kBlockPages, t.pages - b * kBlockPages);
    };
    // whether slot has a block in the piece at all / in a later step of it
    auto last_of = [&](const Cur& t, int slot) {
      return t.s + 1 == t.c.s1 || (slot == 1 && t.c.single && 2 * t.s + 3 >= t.blocks);
    };
    auto issue_s = [&](const Cur& t, int slot) -> bool {
      if (!t.has[slot]) return true;
      const uint32_t e = t.e + (t.c.single ? slot : 0);
      const uint32_t at = e % RING;
      if (t.s == t.c.s0 && !warp_wait(qfull_bar(slot), qn[slot]++ & 1u, p.wait_ns)) return false;
      if (!(slot == 1 && !t.c.single) && !warp_wait(full_bar(at), (e / RING) & 1u, p.wait_ns)) return false;
      tc_fence_after();
      const uint64_t kd = umma_sdesc_sw128(warp_uniform(ring0 + at * GG::TILE), 16u, 1024u);
      const uint64_t qd = umma_sdesc_sw128(warp_uniform(base + slot * GG::TILE), 16u, 1024u);
      const uint32_t idesc = warp_uniform(idesc_s | (static_cast<uint32_t>(2 * np_of(t, slot)) << 17));
      const uint32_t tS = warp_uniform(tbase + kColS + 128u * slot);
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k) {
          const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32u) >> 4;
          umma_ss(tS, qd + off, kd + off, idesc, k > 0);
        }
        umma_commit(sfull_bar(slot));
        if (t.c.single || slot == 1) umma_commit(empty_bar(at));
      }
      __syncwarp();
      return true;
    };
    auto issue_pv = [&](const Cur& t, int slot) -> bool {
      if (!t.has[slot]) return true;
      const uint32_t e = t.e + (t.c.single ? (t.has[1] ? 2 : 1) + slot : 1);
      const uint32_t at = e % RING;
      if (!warp_wait(pfull_bar(slot), pn[slot]++ & 1u, p.wait_ns)) return false;
      if (!(slot == 1 && !t.c.single) && !warp_wait(full_bar(at), (e / RING) & 1u, p.wait_ns)) return false;
      tc_fence_after();
      const uint64_t vd = umma_sdesc_sw128(warp_uniform(ring0 + at * GG::TILE), kHalf, 1024u);
      const uint32_t tO = warp_uniform(tbase + kColO + 128u * slot), tP = warp_uniform(tbase + kColS + 128u * slot);
      const int np = np_of(t, slot);
      const bool fresh = t.s == t.c.s0;                       // a piece's first block overwrites O
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < kBlockPages; ++k)
          if (k < np)
            umma_ts(tO, tP + 8u * k, vd + static_cast<uint64_t>((k * kTcBox) >> 4), idesc_o, !(fresh && k == 0));
        if (t.c.single || slot == 1) umma_commit(empty_bar(at));
        if (last_of(t, slot)) umma_commit(odone_bar(slot));
      }
      __syncwarp();
      return true;
    };
    bool ok = fetch(cur, nullptr) && issue_s(cur, 0) && issue_s(cur, 1);
    bool have = true;
    while (ok && have) {
      have = fetch(nxt, &cur);
      ok = issue_pv(cur, 0) && (!have || issue_s(nxt, 0)) && issue_pv(cur, 1) && (!have || issue_s(nxt, 1));
      cur = nxt;
    }
    if (!ok && lane == 0) atomicOr(p.err, kErrTimeout);
    // every product must be complete before tensor memory is freed
    if (lane == 0) umma_commit(drain_bar);
    __syncwarp();
    if (!warp_wait(drain_bar, 0u, p.wait_ns) && lane == 0) atomicOr(p.err, kErrTimeout);
  } else {
    // ================================ softmax ================================
    const int slot = (warp - kSoftmaxWarp0) >> 2;
    const int rho = 32 * (warp & 3) + lane;                   // row of the tile = tensor-memory lane
    const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tS = tbase + lane_off + kColS + 128u * slot, tO = tbase + lane_off + kColO + 128u * slot;
    uint32_t sn = 0, on = 0;
    bool ok = true;
    // this thread's query row of a piece into the slot's tile (rows past the pair's are zero)
    auto stage_q = [&](const Piece& c, const SharedGroup& sg) {
      const int r = c.pair * kSharedPair + (c.single ? 0 : slot * kSharedTile) + rho;
      const bool have = r < sg.rows;
      const uint4* src = nullptr;
      if (have)
        src = reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(sg.t0 + r / p.G) * p.q_stride_t +
                                             static_cast<int64_t>(c.head * p.G + r % p.G) * D);
      uint8_t* dst = gbase + slot * GG::TILE;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = have ? src[8 * h + k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int k = 0; k < 8; ++k) *reinterpret_cast<uint4*>(dst + h * kHalf + swz<128>(rho, k)) = v[k];
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull_bar(slot));
    };
    // blocks of this slot in a piece
    auto blocks_in = [&](const Piece& c, const SharedGroup& sg) {
      return c.single ? max(0, min(c.s1, (sg.blocks - slot + 1) / 2) - c.s0) : c.s1 - c.s0;
    };
    Piece c = wk.next(p);
    SharedGroup sg = wk.sg;
    if (blocks_in(c, sg) > 0) stage_q(c, sg);
    for (;;) {
      const int n = blocks_in(c, sg);
      float m = -INFINITY, l = 0.f, lr = 0.f;                 // running maximum (log2 units), sums of the weights and
      for (int k = 0; ok && k < n; ++k) {                     // of the weights as rounded into P
        const int b = c.single ? 2 * (c.s0 + k) + slot : c.s0 + k;
        const int np = min(kBlockPages, sg.pages - b * kBlockPages);
        if (!warp_wait(sfull_bar(slot), sn++ & 1u, p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // The scale (of either sign, or zero) joins the exponent's FMA where it is positive,
        // and the maximum is taken over the raw scores.  S is read twice, 32 columns at a
        // time, rather than held in 128 registers.
        const float cs = p.scale_log2, mult = cs > 0.f ? cs : 1.f;
        const bool plain = np == kBlockPages && cs > 0.f;
        auto scores = [&](int k2, float (&sv)[32]) {
          uint32_t r[32];
          tmem_ld32(tS + 32u * k2, r);
          tmem_wait_ld32(r);
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[e] = __uint_as_float(r[e]);
          if (!plain) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              if (!(cs > 0.f)) sv[e] *= cs;
              if (32 * k2 + e >= 16 * np) sv[e] = -INFINITY;
            }
          }
        };
        float mb = -INFINITY;
#pragma unroll
        for (int k2 = 0; k2 < kKeys / 32; ++k2) {
          float sv[32];
          scores(k2, sv);
          mb = fmaxf(mb, Max3Tree<32>::run(sv));
        }
        mb *= mult;
        const float m_new = fmaxf(m, mb);
        const bool grow = m_new > m + 8.f;                    // also from -inf to anything
        if (k > 0 && __any_sync(0xffffffffu, grow)) {
          const float alpha = grow ? fast_exp2(m - m_new) : 1.f;
#pragma unroll
          for (int ch = 0; ch < D / 16; ++ch) {
            uint32_t r[16];
            tmem_ld16(tO + 16u * ch, r);
            tmem_wait_ld16(r);
#pragma unroll
            for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * alpha);
            tmem_st16(tO + 16u * ch, r);
          }
          if (grow) {
            l *= alpha;
            lr *= alpha;
          }
        }
        if (grow) m = m_new;
        const float mneg = m == -INFINITY ? 0.f : -m;
        const uint64_t mult2 = f2_pack(mult, mult), mneg2 = f2_pack(mneg, mneg);
        uint64_t lsum = f2_pack(0.f, 0.f), rsum = lsum;
#pragma unroll
        for (int k2 = 0; k2 < kKeys / 32; ++k2) {
          // (P's columns 16 k2 .. lie in the 32-column chunks read so far)
          uint32_t w[16];
          float sv[32];
          scores(k2, sv);
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x0, x1;
            f2_unpack(ffma2(f2_pack(sv[2 * e], sv[2 * e + 1]), mult2, mneg2), x0, x1);
            const float a0 = fast_exp2(x0), a1 = fast_exp2(x1);
            w[e] = pack_bf16(a0, a1);
            lsum = fadd2(lsum, f2_pack(a0, a1));
            rsum = fadd2(rsum, f2_pack(bf16_lo(w[e]), bf16_hi(w[e])));
          }
          tmem_st16(tS + 16u * k2, w);
        }
        {
          float s0, s1;
          f2_unpack(lsum, s0, s1);
          l += s0 + s1;
          f2_unpack(rsum, s0, s1);
          lr += s0 + s1;
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull_bar(slot));
      }
      if (!ok) break;
      // the next piece's rows while this one's last product runs: its Q K^T products are
      // complete (S of the last block was read)
      const Piece pc = c;
      const SharedGroup pg = sg;
      const bool more = wk.more();
      if (more) {
        c = wk.next(p);
        sg = wk.sg;
        if (blocks_in(c, sg) > 0) stage_q(c, sg);
      }
      const int in_pair = pg.rows - pc.pair * kSharedPair;    // rows from the pair's first on
      const int r = pc.single ? rho : slot * kSharedTile + rho;
      const bool mine = r < in_pair && (pc.single || r < kSharedPair);
      const int64_t prow = pg.row0 + static_cast<int64_t>(pc.head) * pg.rows_head +
                           static_cast<int64_t>(pc.pair) * kSharedPair + static_cast<int64_t>(cta) * kSharedPair +
                           (pc.single ? slot * pg.last_rows + rho : r);
      if (n == 0) {
        if (mine) p.ws_ml[prow] = make_float2(-INFINITY, 0.f);
      } else {
        if (!warp_wait(odone_bar(slot), on++ & 1u, p.wait_ns)) {
          ok = false;
          break;
        }
        tc_fence_after();
        // O / l is the weighted mean of V rows: O is normalised by the rounded weights' sum
        const float ps = lr > 0.f ? l / lr : (lr != lr ? lr : 0.f);
        float* orow = p.ws_o + prow * D;
#pragma unroll
        for (int ch = 0; ch < D / 16; ++ch) {
          uint32_t o[16];
          tmem_ld16(tO + 16u * ch, o);
          tmem_wait_ld16(o);
          if (mine) {
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<float4*>(orow + 16 * ch + e) =
                  make_float4(__uint_as_float(o[e]) * ps, __uint_as_float(o[e + 1]) * ps,
                              __uint_as_float(o[e + 2]) * ps, __uint_as_float(o[e + 3]) * ps);
          }
        }
        if (mine) p.ws_ml[prow] = make_float2(m, l);
        // the slot's next P V, which overwrites O, is issued after this thread's next P
        tc_fence_before();
      }
      if (!more) break;
    }
    if (!ok && lane == 0) atomicOr(p.err, kErrTimeout);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tbase, kCols);
}

cudaLaunchConfig_t config(int grid, int threads, size_t smem, bool pdl, cudaStream_t stream,
                          cudaLaunchAttribute* attr) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cfg;
}

}  // namespace

cudaError_t launch_shared_plan(const SharedParams& p, bool pdl, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(1, kPlanThreads, 0, pdl, stream, attr);
  return cudaLaunchKernelEx(&cfg, pa_shared_plan_kernel, p);
}

cudaError_t launch_shared_prefix(int head_dim, const CUtensorMap& tk, const CUtensorMap& tv, const SharedParams& p,
                                 int grid, bool pdl, cudaStream_t stream) {
  cudaLaunchAttribute attr[1];
  if (head_dim == 128) {
    const cudaLaunchConfig_t cfg = config(grid, kThreads, PrefixGeo<128>::SMEM, pdl, stream, attr);
    return cudaLaunchKernelEx(&cfg, pa_shared_prefix_kernel<128>, tk, tv, p);
  }
  if (head_dim == 64) {
    const cudaLaunchConfig_t cfg = config(grid, kThreads, PrefixGeo<64>::SMEM, pdl, stream, attr);
    return cudaLaunchKernelEx(&cfg, pa_shared_prefix_kernel<64>, tk, tv, p);
  }
  return cudaErrorInvalidValue;
}

cudaError_t set_shared_smem_limits() {
  cudaError_t e = cudaFuncSetAttribute(pa_shared_prefix_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(PrefixGeo<128>::SMEM));
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(pa_shared_prefix_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(PrefixGeo<64>::SMEM));
  return e;
}

}  // namespace pa
