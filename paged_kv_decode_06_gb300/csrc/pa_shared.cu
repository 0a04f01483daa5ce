// Decode attention for batches that share prefixes: the plan of the shared part and its
// attention, all of a group's query rows against the pages its sequences have in common.
//
// Plan (one block): the pages that a group shares are those of shared_lens, cut to what
// every member sees whole ((L_i - q_i) / 16 pages, so that a sequence keeps a page of its
// own and no mask is needed), none for a group with fewer than two members; each group's
// place in the order of steps and partial rows (pa_shared.h); and the SMs for each part.
//
// Attention (tcgen05): with R rows a head the products cost 4 R D flops a key against
// 4 D bytes (bf16), so from about 280 rows on the tensor cores bound it, below that
// memory does.  A CTA holds two 128-row tiles ("slots") of query rows in
// shared memory and S / P (128 columns) and O (128 columns) of each in tensor memory, all
// 512 columns; blocks of 128 keys pass through a ring of K and a ring of V.  While one
// slot's softmax runs, the tensor cores work for the other.
//
// Warps: 0 and 1 issue a slot's S each, 2 and 3 its P V (a product takes its issuer 90 to 130
// cycles, most of it the tensor pipe's: one warp for both of a slot 1.9 us a step, one for
// both slots 2.8, these four 1.6) and 0 owns tensor memory; 4 loads K pages, 5 V pages; of
// an fp8 cache 8 to 15 convert codes to f16 (exact); the last eight are the slots' softmax,
// thread = row of tensor memory.  Registers are dealt by role.  S of 64 keys, twice in each
// slot, P over it in 16 bits (f16 beside an fp8 cache): S of the next 64 keys is there when a
// softmax ends.  O is rescaled only where the running maximum grew by more than 2^8.
//
// What bounds a step of 128 keys (1.6 us at 1.9 GHz, D 128, bf16): 2048 cycles of products;
// 2500 of shared memory, as S of 64 keys reads Q anew (fp8: 3000, and 2.3 us); per slot and 64
// keys about 1200 of softmax, of which 256 are exponentials.  256 sequences behind 32768
// tokens, 277 GFLOP: 215 us on 128 SMs where nothing else runs.
//
// S of a sub-block overwrites the P of two before once P V has read it; so a softmax warp
// that sees S of sub-block b knows P V of b - 2 in O.
//
// Waits are bounded, and each is made once a phase in order (every K and every V block by both
// slots' issuers, by its loader and its converters), so its barrier is never more than one
// phase behind (mbarrier parities cannot tell further).
#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_kernels.h"
#include "pa_pack.cuh"
#include "pa_quant.cuh"
#include "pa_shared.h"
#include "pa_split_tc.cuh"

namespace pa {
namespace {

// ---------------------------------------------------------------- plan kernel
constexpr int kPlanThreads = 1024;        // at most
constexpr int kPlanInts = 7;              // shared memory a sequence

// Sum over the block (in a fixed order).
__device__ __forceinline__ float2 block_sum(float2 v, float2* s_warp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  if (lane == 0) s_warp[warp] = v;
  __syncthreads();
  v = lane < warps ? s_warp[lane] : make_float2(0.f, 0.f);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
    v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
  }
  return v;
}

// Bound by latency: the arrays are read once, everything after that is in shared memory.
__global__ void __launch_bounds__(kPlanThreads) pa_shared_plan_kernel(const SharedParams p) {
  __shared__ float2 s_sum[32];
  extern __shared__ int32_t s_plan[];
  const int B = p.num_seqs, NG = p.num_groups;
  int32_t* const s_len = s_plan;                  // [B] each
  int32_t* const s_t0 = s_len + B;
  int32_t* const s_t1 = s_t0 + B;
  int32_t* const s_skip = s_t1 + B;
  int32_t* const s_group = s_skip + B;
  int32_t* const s_steps = s_group + B;           // of a group (NG <= B), a head
  int32_t* const s_rows = s_steps + B;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x;
  grid_dependency_wait();
  grid_launch_dependents();
  // Groups are consecutive ranges of sequences; with any other list nothing is shared.
  bool bad = false;
  for (int g = tid; g < NG; g += threads) {
    const int a = p.group_start[g], b = p.group_start[g + 1];
    bad |= a < 0 || b < a || b > B;
  }
  // A query_start_loc that is no cumulative sum could spread a group's tokens (each
  // partial row has its place by them).
  for (int i = tid; i < B; i += threads) {
    const int a = p.qsl != nullptr ? p.qsl[i] : i, b = p.qsl != nullptr ? p.qsl[i + 1] : i + 1;
    s_len[i] = p.seq_lens[i];
    s_t0[i] = a;
    s_t1[i] = b;
    s_skip[i] = 0;
    s_group[i] = -1;
    bad |= a < 0 || b < a || b > p.num_tokens || b - a > p.max_qlen;
  }
  bad = __syncthreads_or(bad);
  if (bad && tid == 0) atomicOr(p.err, kErrQueryLen);
  for (int g = warp; g < NG; g += threads / 32) {
    const int a = bad ? 0 : p.group_start[g], b = bad ? 0 : p.group_start[g + 1];
    // members: sequences with query tokens, all at positions of their own
    int pages = max(0, p.shared_lens[g]) / kPage, members = 0, t_lo = INT_MAX, t_hi = 0, first = INT_MAX;
    pages = min(pages, p.max_blocks);
    auto member = [&](int i) { return s_t1[i] > s_t0[i] && s_len[i] >= s_t1[i] - s_t0[i]; };
    for (int i = a + lane; i < b; i += 32) {
      if (!member(i)) continue;
      ++members;
      first = min(first, i);
      pages = min(pages, (s_len[i] - (s_t1[i] - s_t0[i])) / kPage);
      t_lo = min(t_lo, s_t0[i]);
      t_hi = max(t_hi, s_t1[i]);
    }
    members = __reduce_add_sync(0xffffffffu, members);
    pages = __reduce_min_sync(0xffffffffu, pages);
    first = __reduce_min_sync(0xffffffffu, first);
    t_lo = __reduce_min_sync(0xffffffffu, t_lo);
    t_hi = __reduce_max_sync(0xffffffffu, t_hi);
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
    if (lane == 0) {
      p.groups[g] = sg;
      s_steps[g] = sg.steps_head;
      s_rows[g] = sg.rows_head;
    }
    for (int i = a + lane; pages > 0 && i < b; i += 32)
      if (member(i)) {
        s_skip[i] = pages;
        s_group[i] = g;
      }
  }
  __syncthreads();
  // What the sequences' own pages cost (x), and what the shared ones would if nothing were
  // shared (y): where that is little, it is less than the shared part's own start and end.
  float2 cost = make_float2(0.f, 0.f);
  if (p.beside) {
    for (int i = tid; i < B; i += threads) {
      const int n = (s_len[i] > 0 ? min((s_len[i] - 1) / kPage + 1, p.max_blocks) : 0) - s_skip[i];
      if (n > 0) cost.x += static_cast<float>(n) * p.page_cost + p.unit_cost;
      cost.y += static_cast<float>(s_skip[i]) * p.page_cost;
    }
    cost = block_sum(cost, s_sum);
  }
  const bool alone = p.beside && cost.y * p.Hkv < static_cast<float>(p.alone_cost) * p.ctas;
  for (int i = tid; i < B; i += threads) {
    p.skip[i] = alone ? 0 : s_skip[i];
    p.seq_group[i] = alone ? -1 : s_group[i];
  }
  if (alone)
    for (int g = tid; g < NG; g += threads) p.groups[g] = SharedGroup{};
  __syncthreads();                                // (all of it before the release at the end)
  if (warp != 0) return;
  // The groups' places, 32 at a time.
  int64_t steps = 0, rows = 0;
  for (int g0 = 0; g0 < NG && !alone; g0 += 32) {
    const int g = g0 + lane;
    const int64_t n = g < NG ? static_cast<int64_t>(s_steps[g]) * p.Hkv : 0;
    const int64_t r = g < NG ? static_cast<int64_t>(s_rows[g]) * p.Hkv : 0;
    int64_t ns = n, rs = r;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, ns, o), z = __shfl_up_sync(0xffffffffu, rs, o);
      if (lane >= o) {
        ns += y;
        rs += z;
      }
    }
    if (g < NG) {
      p.groups[g].step0 = steps + ns - n;
      p.groups[g].row0 = rows + rs - r;
    }
    steps += __shfl_sync(0xffffffffu, ns, 31);
    rows += __shfl_sync(0xffffffffu, rs, 31);
  }
  if (lane != 0) return;
  // The SMs for each part, in proportion to its work; some more for the sequences' own pages,
  // whose many short walks pay more for memory the longer the other part runs, and four at
  // least (8 sequences of 500 tokens behind 65536, in a graph: 50 us with one, 40 with four, 43
  // with 28).
  int n = p.ctas;
  if (cost.x > 0.f && steps > 0) {
    const float a = static_cast<float>(steps) * p.step_cost, b = cost.x * p.Hkv;
    const float each = (a + b) / p.ctas;                     // ns
    const float more = 0.2f * a / (a + b) * fmaxf(0.f, each - 20000.f);
    n = min(max(1, p.ctas - 4), max(1, p.ctas - static_cast<int>(b / (each - more) + 0.5f)));
  }
  if (n > steps) n = static_cast<int>(steps);
  p.totals->steps = steps;
  p.totals->ctas = n;
  const int own = p.beside ? max(1, min(p.own_ctas, p.ctas - n)) : p.own_ctas;
  store_release(p.ready, (p.call << kReadyBits) | static_cast<uint64_t>(own));
}

// ------------------------------------------------------------- prefix kernel
constexpr int kIssuers = 4;               // warps 0, 1: a slot's S = Q K^T each, 2, 3: its P V
constexpr int kLoaders = 2;               // warps 4, 5 (6, 7: none)
constexpr int kConverter0 = 8, kConverters = 8;   // fp8 caches: warps 8 .. 11 for K, 12 .. 15 for V
constexpr int kSoftmaxWarps = 8;          // the last: a slot's four, a thread a row
constexpr int kBlockPages = kSharedBlockPages;   // K or V of 128 keys in a place of its ring
constexpr int kKeys = 16 * kBlockPages;
constexpr int kSubPages = 4;              // a product and its softmax: 64 keys
constexpr uint32_t kCols = 512;
constexpr uint32_t kColS = 0;             // + 128 slot + 64 (sub-block % 2): S, its P over the first 32 columns
constexpr uint32_t kColO = 256;           // + 128 slot

// Rows of 64 features (128 bytes, 128-byte swizzle) in groups of eight: a block's key rows
// r = 16 page + slot, or a tile's query rows, at group r / 8, then feature half, then r % 8.
// A page of a block is then one run of 16 D elements, one TMA box (128 features: of five
// dimensions), and a product's operand has groups NH KB apart.
template <int D>
struct Geo2 {
  static constexpr int NH = D / 64;
  static constexpr uint32_t GROUP = NH * 1024u;
  static constexpr uint32_t PAGE = 2 * GROUP;
  static constexpr uint32_t TILE = kBlockPages * PAGE;   // bytes of a query tile, a K or a V block
};

template <int D, bool FP8>
struct PrefixGeo {
  static constexpr uint32_t TILE = Geo2<D>::TILE;
  static constexpr int KR = D == 128 ? (FP8 ? 1 : 2) : 4, VR = D == 128 ? 2 : 4;   // blocks of K, of V
  static constexpr int SOFT0 = FP8 ? kConverter0 + kConverters : kConverter0;
  static constexpr int THREADS = 32 * (SOFT0 + kSoftmaxWarps);
  // Registers a thread of each role's warps; together what the launch has (4 x 128 and 6 x 80
  // of 128 threads: an increase beyond that would wait for ever)
  static constexpr int R_ISSUE = FP8 ? 64 : 80, R_LOAD = FP8 ? 48 : 80, R_CONVERT = 56, R_SOFT = FP8 ? 128 : 176;
  static constexpr int R_LAUNCH = FP8 ? 80 : 128;
  static_assert(R_ISSUE + R_LOAD + (FP8 ? 2 * R_CONVERT : 0) + 2 * R_SOFT == THREADS / 128 * R_LAUNCH, "register shares");
  static constexpr uint32_t OFF_RING = 2 * TILE;
  static constexpr uint32_t RAW = kKeys * D;             // fp8: codes of a block
  static constexpr int RAWS = FP8 ? (D == 128 ? 2 : 4) : 0;   // code blocks of K, as many of V
  static constexpr uint32_t OFF_RAW = OFF_RING + (KR + VR) * TILE;
  static constexpr uint32_t OFF_BAR = OFF_RAW + 2 * RAWS * RAW;
  static constexpr uint32_t SMEM = OFF_BAR + 512;
};

// A piece: consecutive blocks of one (group, head, pair) in this CTA.
struct Piece {
  int head, pair;
  int b0, b1;          // blocks, [b0, b1)
  bool single;
  int64_t row0;        // padded rows before the pair's
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
    const int64_t off = x - sg.step0;
    c.head = static_cast<int>(off / sg.steps_head);
    int at = static_cast<int>(off - static_cast<int64_t>(c.head) * sg.steps_head);
    c.pair = min(at / sg.blocks, sg.pairs - 1);
    at -= c.pair * sg.blocks;
    c.single = shared_single(sg, c.pair);
    const int n = static_cast<int>(min(static_cast<int64_t>(shared_steps(sg, c.pair) - at), end - x));
    c.b0 = c.single ? 2 * at : at;
    c.b1 = c.single ? min(2 * (at + n), sg.blocks) : at + n;
    c.row0 = sg.row0 + static_cast<int64_t>(c.head) * sg.rows_head + static_cast<int64_t>(c.pair) * kSharedPair;
    x += n;
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

// Page ids of a group's blocks for a warp: those of four blocks, a lane each, and the four
// after them on their way.
struct PageIds {
  const int32_t* row;
  int pages, batch, ids, next;
  __device__ __forceinline__ int entry(int at) const { return at < pages ? row[at] : 0; }
  __device__ __forceinline__ void start(const SharedParams& p, const SharedGroup& sg) {
    row = p.block_tables + static_cast<int64_t>(sg.seq) * p.bt_stride;
    pages = sg.pages;
    batch = -2;
  }
  __device__ __forceinline__ void turn_to(int want) {
    if (want == batch) return;
    const int lane = threadIdx.x & 31;
    ids = want == batch + 1 ? next : entry(32 * want + lane);
    next = entry(32 * (want + 1) + lane);
    batch = want;
  }
  // page pg of block b (of the batch turned to); every lane calls it
  __device__ __forceinline__ int of(int b, int pg) const { return __shfl_sync(0xffffffffu, ids, (8 * b + pg) & 31); }
};

// Sub-blocks of a slot in a piece, and the pages of the last one.  A single tile's slots
// take a half of each block's pages.
__device__ __forceinline__ int subs_in(const Piece& c, const SharedGroup& sg, int slot, int& last) {
  const int n = c.b1 - c.b0;
  const int np = min(kBlockPages, sg.pages - (c.b1 - 1) * kBlockPages);
  if (!c.single) {
    last = np > kSubPages ? np - kSubPages : np;
    return 2 * n - (np > kSubPages ? 0 : 1);
  }
  last = kSubPages;
  if (slot == 0) last = min(np, kSubPages);
  else if (np > kSubPages) last = np - kSubPages;
  return slot == 1 && np <= kSubPages ? n - 1 : n;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// kind::f16 with f16 A and B and an fp32 accumulator.
__device__ __forceinline__ uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return umma_idesc_bf16(M, N, b_mn_major) & ~((1u << 7) | (1u << 10));
}

template <int N>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

template <int D, bool FP8>
__global__ void __launch_bounds__(PrefixGeo<D, FP8>::THREADS, 1)
    pa_shared_prefix_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                            const SharedParams p) {
  using GG = PrefixGeo<D, FP8>;
  constexpr int NH = D / 64;
  constexpr int RING = GG::KR + GG::VR, RAWS = GG::RAWS;
  constexpr uint32_t TILE = GG::TILE, PAGE = Geo2<D>::PAGE, GROUP = Geo2<D>::GROUP;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const gbase = smem_raw;
  const uint32_t base = smem_addr(smem_raw);
  const uint32_t ring0 = base + GG::OFF_RING;
  const uint32_t bar0 = base + GG::OFF_BAR;
  auto full_bar = [&](int e) { return bar0 + 8u * e; };             // rings' places: K blocks, V blocks
  auto empty_bar = [&](int e) { return bar0 + 8u * (RING + e); };
  // place of the n-th K or V block of this CTA, and the phase of its barriers
  auto place = [&](int is_v, uint32_t n) -> uint32_t { return is_v ? GG::KR + n % GG::VR : n % GG::KR; };
  auto phase = [&](int is_v, uint32_t n) -> uint32_t { return is_v ? n / GG::VR : n / GG::KR; };
  const uint32_t xb = bar0 + 8u * (2 * RING);
  // of a slot: S of a sub-block (by its parity), its P, its P V done; query rows staged; all drained
  auto sfull_bar = [&](int slot, uint32_t n) { return xb + 8u * (2 * slot + (n & 1)); };
  auto pfull_bar = [&](int slot, uint32_t n) { return xb + 8u * (4 + 2 * slot + (n & 1)); };
  auto odone_bar = [&](int slot, uint32_t n) { return xb + 8u * (8 + 2 * slot + (n & 1)); };
  auto qfull_bar = [&](int slot) { return xb + 8u * (12 + slot); };
  auto drain_bar = [&](int issuer) { return xb + 8u * (14 + issuer); };
  auto rawfull_bar = [&](int e) { return xb + 8u * (18 + e); };     // fp8: codes of K blocks, of V blocks
  auto rawempty_bar = [&](int e) { return xb + 8u * (18 + 2 * RAWS + e); };
  static_assert(2 * RING + 18 + 4 * RAWS <= 63, "barriers");
  uint32_t* const s_tmem = reinterpret_cast<uint32_t*>(gbase + GG::OFF_BAR + 504);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
    for (int e = 0; e < RING; ++e) {
      mbar_init(full_bar(e), FP8 ? kConverters / 2 : 1);
      mbar_init(empty_bar(e), 2);
    }
    for (int e = 0; e < 2 * RAWS; ++e) {
      mbar_init(rawfull_bar(e), 1);
      mbar_init(rawempty_bar(e), kConverters / 2);
    }
    for (int s = 0; s < 2; ++s) {
      for (int k = 0; k < 2; ++k) {
        mbar_init(sfull_bar(s, k), 1);
        mbar_init(pfull_bar(s, k), kSoftmaxWarps / 2);
        mbar_init(odone_bar(s, k), 1);
      }
      mbar_init(qfull_bar(s), kSoftmaxWarps / 2);
      mbar_init(drain_bar(s), 1);
      mbar_init(drain_bar(2 + s), 1);
    }
    fence_mbar_init();
  }
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t X = p.totals->steps;
  const int ng = p.totals->ctas;
  const int cta = blockIdx.x;
  if (cta >= ng) return;
  const int64_t from = cta * X / ng, to = (cta + 1) * X / ng;
  if (from >= to) return;
  if ((base & 1023u) != 0) {              // the swizzle and the operands need the alignment declared above
    if (tid == 0) atomicOr(p.err, kErrTimeout);
    return;
  }
  if (warp == 0) tmem_alloc(smem_addr(s_tmem), kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = warp_uniform(*s_tmem);
  PieceWalker wk;
  wk.start(p, from, to);

  if (warp >= kIssuers && warp < kConverter0) {
    // =============================== loaders =================================
    registers_down<GG::R_LOAD>();
    if (warp < kIssuers + kLoaders) {
      // One warp loads the K blocks, the other the V blocks.
      const int is_v = warp - kIssuers;
      constexpr int kRaws = RAWS > 0 ? RAWS : 1;
      const CUtensorMap* const map = is_v ? &tmap_v : &tmap_k;
      // boxes, a lane each: a page, or (split boxes: heads that are not contiguous) eight
      // slots and 64 features of one
      const int per = !FP8 && NH == 2 && ((p.split_boxes >> is_v) & 1) ? 4 : 1;
      const int pg = lane / per, part = lane - pg * per;
      const uint32_t bytes = (FP8 ? 16u * D : PAGE) / per;
      const uint32_t to = FP8 ? base + GG::OFF_RAW + pg * bytes : ring0 + pg * PAGE + part * 1024u;
      uint32_t n = 0;                                          // blocks before
      bool ok = true;
      PageIds ids;
      while (ok && wk.more()) {
        const Piece c = wk.next(p);
        ids.start(p, wk.sg);
        for (int b = c.b0; b < c.b1; ++b, ++n) {
          const int np = min(kBlockPages, wk.sg.pages - b * kBlockPages);
          ids.turn_to(b >> 2);
          const int page = ids.of(b, pg);
          const uint32_t e = FP8 ? is_v * RAWS + n % kRaws : place(is_v, n);
          const uint32_t round = FP8 ? n / kRaws : phase(is_v, n);
          const uint32_t full = FP8 ? rawfull_bar(e) : full_bar(e);
          if (round > 0 && !warp_wait(FP8 ? rawempty_bar(e) : empty_bar(e), (round - 1) & 1u, p.wait_ns)) {
            if (lane == 0) atomicOr(p.err, kErrTimeout);
            ok = false;
            break;
          }
          if (lane == 0) mbar_arrive_expect_tx(full, static_cast<uint32_t>(np * per) * bytes);
          __syncwarp();
          if (pg < np) {
            if ((page < 0 || page >= p.num_pages) && part == 0) atomicOr(p.err, kErrPageRange);
            // (a page id out of range reads as zeros: TMA fills outside the tensor)
            if constexpr (FP8) {
              tma_load_4d(to + e * GG::RAW, map, 0, 0, c.head, page, full);
            } else {
              if (NH == 1)
                tma_load_4d(to + e * TILE, map, 0, 0, c.head, page, full);
              else if (per == 1)
                tma_load_5d(to + e * TILE, map, 0, 0, NH * c.head, 0, page, full);
              else                                              // part = 2 (slot / 8) + half
                tma_load_4d(to + e * TILE, map, 64 * (part & 1), 8 * (part >> 1), c.head, page, full);
            }
          }
        }
      }
      // No copy may be on its way when the CTA ends (one is only where a wait ran out, which
      // a caller's limit may be too short for).
      const uint32_t places = FP8 ? kRaws : is_v ? GG::VR : GG::KR;
      for (uint32_t k = n > places ? n - places : 0; k < n; ++k)
        warp_wait(FP8 ? rawfull_bar(is_v * RAWS + k % kRaws) : full_bar(place(is_v, k)),
                  (FP8 ? k / kRaws : phase(is_v, k)) & 1u, kDrainNs);
    }
  } else if (FP8 && warp >= kConverter0 && warp < GG::SOFT0) {
    // ============================== converters ===============================
    // e4m3 codes to f16 (exact), into the products' layout.  A thread takes 16 codes of a
    // row at a time.  Eight lanes (a phase of 128 bytes of the loads and stores) take four
    // chunks of two rows, of 128 features different halves of them: no bank conflict on
    // either side.  The codes' place is given back after the proxy fence: the copy that
    // fills it next is not ordered behind plain loads without one.
    registers_down<GG::R_CONVERT>();
    const int is_v = warp >= kConverter0 + kConverters / 2;
    const int ct = (tid - 32 * kConverter0) & (16 * kConverters - 1);
    constexpr int ITER = kKeys * (D / 16) / (16 * kConverters), HALF = ITER / 2;
    constexpr int kRaws = RAWS > 0 ? RAWS : 1;
    const int cc = ct & 3, odd = (ct >> 2) & 1;
    uint32_t n = 0;                                          // blocks before
    bool ok = true;
    while (ok && wk.more()) {
      const Piece c = wk.next(p);
      for (int b = c.b0; b < c.b1; ++b, ++n) {
        const int np = min(kBlockPages, wk.sg.pages - b * kBlockPages);
        const uint32_t er = is_v * RAWS + n % kRaws, e = place(is_v, n);
        ok = warp_wait(rawfull_bar(er), (n / kRaws) & 1u, p.wait_ns);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok) break;
          const uint8_t* src = gbase + GG::OFF_RAW + er * GG::RAW;
          uint8_t* dst = gbase + GG::OFF_RING + e * TILE;
          auto row_of = [&](int i) { return NH == 2 ? 32 * (i >> 1) + 2 * (ct >> 3) + (odd ^ (i & 1)) : 32 * i + (ct >> 2); };
          const int half = NH == 2 ? odd : 0;
          uint4 v[HALF];
#pragma unroll
          for (int i = 0; i < HALF; ++i)
            v[i] = *reinterpret_cast<const uint4*>(src + row_of(h * HALF + i) * D + 64 * half + 16 * cc);
          if (h == 0 && phase(is_v, n) > 0) ok = warp_wait(empty_bar(e), (phase(is_v, n) - 1) & 1u, p.wait_ns);
          if (!ok) break;
#pragma unroll
          for (int i = 0; i < HALF; ++i) {
            const int row = row_of(h * HALF + i);
            if ((row >> 4) >= np) continue;
            uint8_t* g = dst + (row >> 3) * GROUP + half * 1024u;
            *reinterpret_cast<uint4*>(g + swz<128>(row & 7, 2 * cc)) =
                make_uint4(e4m3x2_to_f16x2(v[i].x), e4m3x2_to_f16x2(v[i].x >> 16), e4m3x2_to_f16x2(v[i].y),
                           e4m3x2_to_f16x2(v[i].y >> 16));
            *reinterpret_cast<uint4*>(g + swz<128>(row & 7, 2 * cc + 1)) =
                make_uint4(e4m3x2_to_f16x2(v[i].z), e4m3x2_to_f16x2(v[i].z >> 16), e4m3x2_to_f16x2(v[i].w),
                           e4m3x2_to_f16x2(v[i].w >> 16));
          }
        }
        if (!ok) {
          if (lane == 0) atomicOr(p.err, kErrTimeout);
          break;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full_bar(e));
          mbar_arrive(rawempty_bar(er));
        }
      }
    }
  } else if (warp < kIssuers) {
    // =========================== product issuers =============================
    registers_down<GG::R_ISSUE>();
    const int slot = warp & 1, is_v = warp >> 1;
    const uint32_t idesc = !is_v ? (FP8 ? idesc_f16(128, 16, false) : umma_idesc_bf16(128, 16, false)) & ~(0x3Fu << 17)
                                 : (FP8 ? idesc_f16(128, D, true) : umma_idesc_bf16(128, D, true));
    const uint64_t qd = umma_sdesc_sw128(warp_uniform(base + slot * TILE), 16u, GROUP);
    const uint32_t tS = warp_uniform(tbase + kColS + 128u * slot), tO = warp_uniform(tbase + kColO + 128u * slot);
    uint32_t before = 0;           // blocks of the pieces before
    uint32_t tiles = 0, n = 0;     // query tiles seen, sub-blocks
    bool ok = true;
    while (ok && wk.more()) {
      const Piece c = wk.next(p);
      int last = 0;
      const int subs = subs_in(c, wk.sg, slot, last);
      if (subs > 0 && !is_v) ok = warp_wait(qfull_bar(slot), tiles++ & 1u, p.wait_ns);
      for (int i = 0; ok && i < subs; ++i, ++n) {
        // The sub-block's block; its place is free once both slots' products have read it:
        // each commits at its last sub-block of the block.
        const uint32_t b = before + static_cast<uint32_t>(c.single ? i : i >> 1), at = place(is_v, b);
        const int part = c.single ? slot : i & 1;
        const bool opens = c.single || (i & 1) == 0, closes = c.single || (i & 1) == 1 || i == subs - 1;
        if (opens) ok = warp_wait(full_bar(at), phase(is_v, b) & 1u, p.wait_ns);
        const int np = static_cast<int>(warp_uniform(static_cast<uint32_t>(i == subs - 1 ? last : kSubPages)));
        const uint32_t sp = warp_uniform(tS + 64u * (n & 1u));
        const uint32_t src = warp_uniform(ring0 + at * TILE + part * (kSubPages * PAGE));
        if (!is_v) {
          // over P of two sub-blocks ago, which its P V has read
          if (ok && n >= 2) ok = warp_wait(odone_bar(slot, n), ((n >> 1) - 1) & 1u, p.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint64_t kd = umma_sdesc_sw128(src, 16u, GROUP);
          const uint32_t id = warp_uniform(idesc | (static_cast<uint32_t>(2 * np) << 17));
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
              const uint32_t off = ((k >> 2) * 1024u + (k & 3) * 32u) >> 4;
              umma_ss(sp, qd + off, kd + off, id, k > 0);
            }
            umma_commit(sfull_bar(slot, n));
            if (closes) umma_commit(empty_bar(at));
          }
        } else {
          if (ok) ok = warp_wait(pfull_bar(slot, n), (n >> 1) & 1u, p.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint64_t vd = umma_sdesc_sw128(src, 1024u, GROUP);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kSubPages; ++k)              // (a piece's first overwrites O)
              if (k < np) umma_ts(tO, sp + 8u * k, vd + static_cast<uint64_t>((k * PAGE) >> 4), idesc, k > 0 || i > 0);
            umma_commit(odone_bar(slot, n));
            if (closes) umma_commit(empty_bar(at));
          }
        }
        __syncwarp();
      }
      const uint32_t blocks = c.b1 - c.b0;
      if (ok && c.single && static_cast<uint32_t>(subs) < blocks) {
        // a last block without pages for this slot
        const uint32_t b = before + static_cast<uint32_t>(subs), at = place(is_v, b);
        ok = warp_wait(full_bar(at), phase(is_v, b) & 1u, p.wait_ns);
        if (ok && lane == 0) mbar_arrive(empty_bar(at));
      }
      before += blocks;
    }
    if (!ok && lane == 0) atomicOr(p.err, kErrTimeout);
    // every product must be complete before tensor memory is freed
    if (elect_one()) umma_commit(drain_bar(warp));
    __syncwarp();
    if (!warp_wait(drain_bar(warp), 0u, kDrainNs) && lane == 0) atomicOr(p.err, kErrTimeout);
  } else {
    // ================================ softmax ================================
    registers_up<GG::R_SOFT>();
    const int slot = (warp - GG::SOFT0) >> 2;
    const int quarter = warp & 3;
    const int rho = 32 * quarter + lane;                      // row of the tile = tensor-memory lane
    const uint32_t lane_off = static_cast<uint32_t>(32 * quarter) << 16;
    const uint32_t tS0 = tbase + lane_off + kColS + 128u * slot, tO = tbase + lane_off + kColO + 128u * slot;
    uint32_t n = 0;                                           // sub-blocks of the pieces before
    float next_scale = 1.f;                                   // fp8: what the staged row was divided by
    bool ok = cta != p.give_up_cta || slot != 0;              // (testing aid: this slot's warps give up at once)
    // this thread's query row of a piece into the slot's tile (rows past the pair's are
    // zero).  fp8 caches: in f16, divided by a power of two that leaves the largest element
    // in [1, 2).
    auto stage_q = [&](const Piece& c, const SharedGroup& sg) {
      const int r = c.pair * kSharedPair + (c.single ? 0 : slot * kSharedTile) + rho;
      const bool have = r < sg.rows;
      const uint4* src = nullptr;
      if (have)
        src = reinterpret_cast<const uint4*>(p.q + static_cast<int64_t>(sg.t0 + r / p.G) * p.q_stride_t +
                                             static_cast<int64_t>(c.head * p.G + r % p.G) * D);
      uint4 v[D / 8];
#pragma unroll
      for (int ch = 0; ch < D / 8; ++ch) v[ch] = have ? src[ch] : make_uint4(0u, 0u, 0u, 0u);   // 8 features
      if constexpr (FP8) {
        uint32_t mx = 0;
#pragma unroll
        for (int ch = 0; ch < D / 8; ++ch)
          mx = max_u16x2(mx, max_u16x2(max_u16x2(v[ch].x & 0x7FFF7FFFu, v[ch].y & 0x7FFF7FFFu),
                                       max_u16x2(v[ch].z & 0x7FFF7FFFu, v[ch].w & 0x7FFF7FFFu)));
        const int ex = static_cast<int>((max(mx & 0xFFFFu, mx >> 16) >> 7) & 0xFFu) - 127;
        const int e2 = ex == 128 ? 0 : min(126, max(-100, ex));   // (NaN and infinities stay as they are)
        next_scale = __uint_as_float(static_cast<uint32_t>(e2 + 127) << 23);
        const float div = __uint_as_float(static_cast<uint32_t>(127 - e2) << 23);
#pragma unroll
        for (int ch = 0; ch < D / 8; ++ch)
          v[ch] = make_uint4(pack_f16(bf16_lo(v[ch].x) * div, bf16_hi(v[ch].x) * div),
                             pack_f16(bf16_lo(v[ch].y) * div, bf16_hi(v[ch].y) * div),
                             pack_f16(bf16_lo(v[ch].z) * div, bf16_hi(v[ch].z) * div),
                             pack_f16(bf16_lo(v[ch].w) * div, bf16_hi(v[ch].w) * div));
      }
      uint8_t* dst = gbase + slot * TILE + (rho >> 3) * GROUP;
#pragma unroll
      for (int ch = 0; ch < D / 8; ++ch)
        *reinterpret_cast<uint4*>(dst + (ch >> 3) * 1024u + swz<128>(rho & 7, ch & 7)) = v[ch];
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(qfull_bar(slot));
    };
    Piece c = wk.next(p);
    SharedGroup sg = wk.sg;
    int last = 0, subs = subs_in(c, sg, slot, last);
    if (subs > 0) stage_q(c, sg);
    for (;;) {
      // The scale (of either sign, or zero) joins the exponent's FMA where it is positive,
      // and the maximum is taken over the raw scores.
      const float cs = p.scale_log2 * next_scale;
      const bool positive = p.scale_log2 > 0.f;
      const float mult = positive ? cs : 1.f;
      const int in_pair = sg.rows - c.pair * kSharedPair;     // rows from the pair's first on
      const int r = c.single ? rho : slot * kSharedTile + rho;
      const bool mine = r < in_pair && r < kSharedPair;
      const bool idle = !__any_sync(0xffffffffu, mine);       // no row of this warp exists
      float m = -INFINITY, l = 0.f;                           // running maximum (log2 units), sum
      for (int k = 0; ok && k < subs; ++k) {
        const uint32_t nk = n + k;
        if (!warp_wait(sfull_bar(slot, nk), (nk >> 1) & 1u, p.wait_ns)) {
          ok = false;
          break;
        }
        if (idle) {
          // (what its rows' P and O hold reaches nobody)
          if (lane == 0) mbar_arrive(pfull_bar(slot, nk));
          continue;
        }
        tc_fence_after();
        const uint32_t tS = tS0 + 64u * (nk & 1u);
        const int np = k == subs - 1 ? last : kSubPages;
        uint32_t w[64];
        tmem_ld32(tS, *reinterpret_cast<uint32_t(*)[32]>(&w[0]));
        tmem_ld32(tS + 32u, *reinterpret_cast<uint32_t(*)[32]>(&w[32]));
        after_wait<64>(w);
        if (np < kSubPages || !positive) {
#pragma unroll
          for (int e = 0; e < 64; ++e) {
            float x = __uint_as_float(w[e]);
            if (!positive) x *= cs;
            w[e] = __float_as_uint(e < 16 * np ? x : -INFINITY);
          }
        }
        float mx[64];
#pragma unroll
        for (int e = 0; e < 64; ++e) mx[e] = __uint_as_float(w[e]);
        const float m_new = fmaxf(m, Max3Tree<64>::run(mx) * mult);
        const bool grow = m_new > m + 8.f;                    // also from -inf to anything
        if (k > 0 && __any_sync(0xffffffffu, grow)) {
          // O must hold P V of the sub-block before (the one before that is complete: S of
          // this one was issued behind it)
          if (!warp_wait(odone_bar(slot, nk - 1), ((nk - 1) >> 1) & 1u, p.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const float alpha = grow ? fast_exp2(m - m_new) : 1.f;
#pragma unroll
          for (int ch = 0; ch < D / 16; ++ch) {
            uint32_t o[16];
            tmem_ld16(tO + 16u * ch, o);
            after_wait<16>(o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st16(tO + 16u * ch, o);
          }
          if (grow) l *= alpha;
        }
        if (grow) m = m_new;
        const float mneg = m == -INFINITY ? 0.f : -m;
        const uint64_t mult2 = f2_pack(mult, mult), mneg2 = f2_pack(mneg, mneg);
        uint64_t lsum = f2_pack(0.f, 0.f), lsum2 = lsum;
#pragma unroll
        for (int k2 = 0; k2 < 2; ++k2) {
          uint32_t pw[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            float x0, x1;
            f2_unpack(ffma2(f2_pack(__uint_as_float(w[32 * k2 + 2 * e]), __uint_as_float(w[32 * k2 + 2 * e + 1])), mult2,
                            mneg2), x0, x1);
            const float a0 = fast_exp2(x0), a1 = fast_exp2(x1);
            pw[e] = FP8 ? pack_f16(a0, a1) : pack_bf16(a0, a1);
            if (e & 1) lsum2 = fadd2(lsum2, f2_pack(a0, a1));
            else lsum = fadd2(lsum, f2_pack(a0, a1));
          }
          tmem_st16(tS + 16u * k2, pw);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(pfull_bar(slot, nk));
        float s0, s1;
        f2_unpack(fadd2(lsum, lsum2), s0, s1);
        l += s0 + s1;
      }
      if (!ok) break;
      n += subs;
      const int done = subs;
      // the slot's tile of partial rows: chunk d / 4 of all its rows, then the next chunk (a
      // warp's stores are whole lines)
      const int64_t tile0 = c.row0 + static_cast<int64_t>(cta) * kSharedPair +
                            slot * (c.single ? sg.last_rows : kSharedTile);
      const int tile_rows = shared_tile_rows(sg, c.pair, slot);
      // the next piece's rows while this one's last products run: its Q K^T products are
      // complete (S of the last sub-block was read)
      const bool more = wk.more();
      if (more) {
        c = wk.next(p);
        sg = wk.sg;
        subs = subs_in(c, sg, slot, last);
        if (subs > 0) stage_q(c, sg);
      }
      if (done == 0) {
        if (mine) p.ws_ml[tile0 + rho] = make_float2(-INFINITY, 0.f);
      } else {
        if (!warp_wait(odone_bar(slot, n - 1), ((n - 1) >> 1) & 1u, p.wait_ns)) {
          ok = false;
          break;
        }
        if (!idle) {
          tc_fence_after();
          float* orow = p.ws_o + tile0 * D + 4 * rho;
#pragma unroll
          for (int ch = 0; ch < D / 16; ++ch) {
            uint32_t o[16];
            tmem_ld16(tO + 16u * ch, o);
            after_wait<16>(o);
            if (mine) {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<uint4*>(orow + (16 * ch + e) * tile_rows) =
                    make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            }
          }
          if (mine) p.ws_ml[tile0 + rho] = make_float2(m, l);
          // (the slot's next P V, which overwrites O, is issued after this thread's next P)
          tc_fence_before();
        }
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
  const int threads = min(kPlanThreads, max(128, (max(p.num_seqs, 32 * p.num_groups) + 31) / 32 * 32));
  const cudaLaunchConfig_t cfg = config(1, threads, 4 * kPlanInts * static_cast<size_t>(p.num_seqs), pdl, stream, attr);
  return cudaLaunchKernelEx(&cfg, pa_shared_plan_kernel, p);
}

namespace {

using PrefixKernel = void (*)(CUtensorMap, CUtensorMap, SharedParams);
struct PrefixForm {
  PrefixKernel kernel;
  int threads, registers;
  uint32_t smem;
};
template <int D, bool FP8>
PrefixForm prefix_form() {
  using GG = PrefixGeo<D, FP8>;
  return {pa_shared_prefix_kernel<D, FP8>, GG::THREADS, GG::R_LAUNCH, GG::SMEM};
}
PrefixForm prefix_form_of(int head_dim, bool fp8) {
  if (head_dim == 128) return fp8 ? prefix_form<128, true>() : prefix_form<128, false>();
  return fp8 ? prefix_form<64, true>() : prefix_form<64, false>();
}

}  // namespace

cudaError_t launch_shared_prefix(int head_dim, bool fp8, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const SharedParams& p, int grid, bool pdl, cudaStream_t stream) {
  const PrefixForm f = prefix_form_of(head_dim, fp8);
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = config(grid, f.threads, f.smem, pdl, stream, attr);
  return cudaLaunchKernelEx(&cfg, f.kernel, tk, tv, p);
}

cudaError_t set_shared_smem_limits() {
  const cudaError_t plan = cudaFuncSetAttribute(reinterpret_cast<const void*>(pa_shared_plan_kernel),
                                                cudaFuncAttributeMaxDynamicSharedMemorySize, 4 * kPlanInts * kMaxSeqsHost);
  if (plan != cudaSuccess) return plan;
  for (int form = 0; form < 4; ++form) {
    const PrefixForm f = prefix_form_of(form & 1 ? 128 : 64, form & 2);
    const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(f.kernel),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(f.smem));
    if (e != cudaSuccess) return e;
    // a build that launches with fewer registers than the roles are dealt would never end
    cudaFuncAttributes attr;
    const cudaError_t a = cudaFuncGetAttributes(&attr, reinterpret_cast<const void*>(f.kernel));
    if (a != cudaSuccess) return a;
    if (attr.numRegs < f.registers) return cudaErrorInvalidKernelImage;
  }
  return cudaSuccess;
}

}  // namespace pa
