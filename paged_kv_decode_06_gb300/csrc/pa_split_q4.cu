// Split-KV decode attention over a 4-bit paged cache (pa_q4.cuh has the format).
//
// Work decomposition, workspace and merge are those of the bf16 / fp8 split
// kernel: CTA g takes a range of the (sequence, head chunk, page) order; a unit cut
// by a range boundary leaves fp32 partials for the merge kernel.  The ranges are
// equal in pages plus a few for the start and end of every unit that has pages.
//
// At 4.5 bits a cached feature the walk is bound by what a warp issues per
// feature, so everything that does not depend on the query rows is done once a
// key and row tile (a KV head of up to 16 rows, or 32 of 64 features in a large batch, has one tile;
// more tiles fetch and convert the pages once each), and nothing is done for rows that
// do not exist:
//   * scores are computed transposed, S^T = K Q^T with mma.sync m16n8k16: the
//     16 keys of a page are the M rows and the N side is 8 query rows (the usual
//     4 to 8 rows of a KV head fill it; the other orientation pads them to 16);
//   * a K fragment is two codes -> one f16 pair (cvt), times the group's scale
//     (one f16x2 multiply): both exact.  A lane reads 32 (D = 128) or 16 (D = 64)
//     consecutive features of its key with one load: feature order inside the
//     contraction is free as long as the query fragments follow it;
//   * S^T's accumulator layout (keys down, rows across) becomes the B operand
//     of O^T = V^T P^T by one 8x8 transpose of f16 pairs a half page, and the
//     output accumulators carry the same query rows as the lane's scores, so
//     rescaling needs no exchange;
//   * a V fragment wants the same feature of two consecutive keys in a pair:
//     two words of codes (8 features of each key) are interleaved nibble-wise
//     with four logical operations, then converted and scaled like K;
//   * the running maximum moves only when a score exceeds it by 2^8 (one vote a
//     step); P is then at most 256, a warp's largest P at least 1, and the rounding
//     to f16 2^-11 relative, or 2^-25 absolute for P below 2^-14 (the sums take P
//     unrounded).  The maximum is over keys: a sink joins at the end of its piece.
// Query rows are scaled by a power of two into f16's range (exact except for
// elements 2^-14 below the row's largest), and the power goes into the row's logit factor.
//
// A CTA is eight warps, two CTAs an SM for at most 8 query rows a KV head (128
// registers a thread), else one (255).  KW x MT x HC warps are in use: HC KV heads,
// MT tiles of 8 NT query rows, and KW warps that take a head's pages in turn and meet
// in shared memory at the end of a segment (a sequence's pages in this CTA).  The
// host's plan has the rules for NT, HC and KW with what each side measured.
//
// Every warp feeds itself: it copies the 2.3 KB (D = 128) of its head's codes and
// scales of a page with five 16-byte cp.async a lane into its own ring, S pages
// ahead, so no warp ever waits for another or polls a barrier.  The form before it,
// producer warps with bulk tensor copies of whole pages into a ring of the CTA's,
// ran 153 us on the batch of 256 (673 MB): a third of the issue slots went to the
// producers, to polling and to register spills (a producer warpgroup's registers
// are not the consumers'), and a copy instruction held a producer for 280 to 540
// cycles beside warps that compute.
//
// Measured: 256 sequences of 128 to 8192 tokens, 32 / 8 heads of 128 (673 MB): 134 us,
// 5.0 TB/s, 74% of the copy bandwidth (long sequences alone: 5.6 TB/s).  Bound by warp
// instructions, 330 a page and head of 2.3 KB (172 in the compute loop, the rest in the
// fetch, at the segments' ends and in the prologue), and the latencies between them: four
// warps a scheduler fill 57% of the issue slots (counters of a batch of 96), and more
// warps (85 registers: spills), deeper rings or more independent sums do not help.  32
// sequences of 4 tokens and 64 rows of 8 heads, window 4096 (117 MB): 70 us, bound by
// the two warps a scheduler that 246 registers leave (issue 42%, tensor pipe 26%).  One
// sequence of 32768 tokens, 64 features, its 19 MB in L2: 14.9 us, of which the two
// kernels' start-up and the dependent loads (lengths, page ids, pages; descriptor,
// partials) are about 12.  A batch padded with empty sequences (8 of 4096 tokens, 32 / 8
// heads, in a batch of 256): 25 us, without the padding 21.
#include "pa_q4.cuh"
#include "pa_split.cuh"

namespace pa {

constexpr int kQ4Warps = 8;                                         // of a CTA
constexpr int q4_ctas_per_sm(int nt) { return nt == 1 ? 2 : 1; }
// Pages in flight a warp: about 9 KB, 150 KB an SM where two CTAs are on it.
constexpr int q4_stages(int d) { return d == 128 ? 4 : 8; }
// What a segment's start and end cost, in pages of a warp: the CTAs' shares count them
// (0, 5 and 16 pages: the batch of 256 141, 134 and 142 us; 256 sequences of up to 1000
// tokens 34, 24 and 31; 64 sequences of up to 3000 tokens, 16 rows: 0, 5 and 8 pages 36,
// 31 and 30).
constexpr int q4_segment_pages(int nt) { return nt == 1 ? 5 : 8; }
// A team's query fragments (D x 8 NT x 2 bytes) in shared memory.  Its KW warps write
// the same values; the barriers at a segment's end keep one segment's apart from the
// next one's.
constexpr uint32_t q4_query_bytes(int d, int nt) { return static_cast<uint32_t>(d * 8 * nt * 2); }

template <int D>
struct GeoQ4 {
  static constexpr int ROWB = D / 2;        // bytes of a row's codes
  static constexpr int TILE = 16 * ROWB;    // codes of one page of one head
  static constexpr int SROW = D / 16;       // bytes of a row's scales
  static constexpr int STILE = 16 * SROW;   // scales of one page and head
  static constexpr int KS = D / 16;         // k-steps of K Q^T; also 16-feature tiles of V^T
  static constexpr int LW = D / 32;         // words of codes a lane reads of its key
  // a page and head in a warp's ring: K codes, V codes, K scales, V scales
  static constexpr int V = TILE, KSC = 2 * TILE, VSC = 2 * TILE + STILE, PAGE = 2 * (TILE + STILE);
};

// Slot of tile row t (0 .. 7; rows 8 .. 15 add 8): a permutation that makes the
// values' reads (tile rows 2 tig, 2 tig + 1 of four lanes) free of bank conflicts.
template <int D>
__device__ __forceinline__ int slot_of(int t) {
  return D == 128 ? t ^ ((t >> 1) & 1) : t ^ ((t >> 2) & 1);
}

// Byte offset of byte b of a slot's codes: 64-byte rows (D = 128) have their four
// 16-byte chunks permuted by the pair of rows, 32-byte rows lie as they are.
template <int D>
__device__ __forceinline__ uint32_t code_off(int slot, int b) {
  const uint32_t off = static_cast<uint32_t>(slot * (D / 2) + b);
  return D == 128 ? off ^ (((off >> 7) & 3u) << 4) : off;
}

// 16 bytes global -> shared, asynchronous.
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}

// The last key that a query row of a segment sees (rows past the segment's: as its first).
struct RowsQ4 {
  int min_lim;               // of the first query token
  int row0, R;               // first row of the warp's tiles, rows of the segment
  uint32_t g_inv;
  __device__ __forceinline__ int last(int rl) const {
    const int rho = row0 + rl;
    return min_lim + (rho < R ? static_cast<int>(static_cast<uint32_t>(rho) * g_inv >> 16) : 0);
  }
};

// What a lane reads of every page (offsets into the page's place in the ring) and
// the slots of its keys.
struct LaneQ4 {
  uint32_t ka, va, dva;      // codes: scores' first key; values' first key, from it to the second
  uint32_t ksa, vsa, dvs;    // scales, likewise
  uint32_t slots;            // the scores' key | the values' keys << 8, << 16
};

// (a & mask) | (b & ~mask)
__device__ __forceinline__ uint32_t bitsel(uint32_t a, uint32_t b, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xE2;" : "=r"(r) : "r"(a), "r"(mask), "r"(b));
  return r;
}

// A row's running maximum before its first score (no finite score is below
// it, and 2^(kUnsetMax - score) is 0), and how far a score may exceed the
// maximum before it moves.
constexpr float kUnsetMax = -3e38f;
constexpr float kMoveMax = 8.f;
// The largest maximum that a sink sets (differences with it stay finite).
constexpr float kMaxSink = 3e38f;

// One warp's state: 8 NT query rows of one KV head.  Lane (gq = lane / 4, tig =
// lane % 4) holds the query rows 8 n + 2 tig + e (n < NT, e < 2) of the scores
// and the outputs.
// The query fragments stay in shared memory (qs: this lane's, 512 bytes a pair of
// k-steps and row tile): registers do not hold them beside the outputs.
template <int D, int NT>
struct StateQ4 {
  using GG = GeoQ4<D>;
  float O[GG::KS][NT][4];      // O^T: [feature tile][row tile]; elements (feature 2 i, rows e), (2 i + 1, rows e)
  uint32_t qs;
  float m[NT][2], l[NT][2];    // running maximum (log2 units), this lane's share of the sum
  float fac[NT][2];            // logit factor of the row (log2 units per raw score)

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = kUnsetMax;
        l[n][e] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < GG::KS; ++i) O[i][n][0] = O[i][n][1] = O[i][n][2] = O[i][n][3] = 0.f;
    }
  }

  // Query row `row` (bf16, D features; nullptr: no such row) of tile n: this lane's
  // features D/4 tig .. D/4 tig + D/4 - 1.
  static __device__ __forceinline__ void read_query(uint2 (&w)[GG::KS], const uint16_t* row, int tig) {
#pragma unroll
    for (int ks = 0; ks < GG::KS; ++ks)
      w[ks] = row != nullptr ? *reinterpret_cast<const uint2*>(row + (D / 4) * tig + 4 * ks) : make_uint2(0u, 0u);
  }

  // ... and into fragments of tile n.
  __device__ __forceinline__ void set_query(int n, const uint2 (&w)[GG::KS], int tig, float scale_log2) {
    float amax = 0.f;
#pragma unroll
    for (int ks = 0; ks < GG::KS; ++ks)
      amax = fmaxf(fmaxf(fmaxf(fabsf(bf16_lo(w[ks].x)), fabsf(bf16_hi(w[ks].x))),
                         fmaxf(fabsf(bf16_lo(w[ks].y)), fabsf(bf16_hi(w[ks].y)))), amax);
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // exponent of the row's largest element, kept where 2^-e and 2^e are normal (a
    // subnormal row then lies 2^-7 and less, above f16's subnormals, and elements of
    // 2^127 at 2^12)
    int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
    ex = max(-126, min(115, ex));
    const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
#pragma unroll
    for (int ks = 0; ks < GG::KS; ks += 2) {
      uint32_t f[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        f[2 * u] = pack_f16(bf16_lo(w[ks + u].x) * down, bf16_hi(w[ks + u].x) * down);
        f[2 * u + 1] = pack_f16(bf16_lo(w[ks + u].y) * down, bf16_hi(w[ks + u].y) * down);
      }
      asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(qs + (ks / 2 * NT + n) * 512), "r"(f[0]),
                   "r"(f[1]), "r"(f[2]), "r"(f[3])
                   : "memory");
    }
    const float f = scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
    fac[n][0] = __shfl_sync(0xffffffffu, f, 8 * tig);
    fac[n][1] = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
  }

  // NP pages of this warp's head, at ring addresses `at`.  EDGE (one page): some row
  // does not see all 16 keys.
  template <bool EDGE, int NP>
  __device__ __forceinline__ void page(const LaneQ4& ln, const uint32_t (&at)[NP], int tb, int L, int window,
                                       const RowsQ4& rows, int tig) {
    static_assert(!EDGE || NP == 1, "edge pages one at a time");
    constexpr int CH = 8 * GG::ROWB, SH = 8 * GG::SROW;   // from a key to the one 8 rows on
    // ---- S^T = K Q^T: NP x NA independent sums
    constexpr int NA = NT == 1 && NP == 1 ? 2 : 1;
    float S[NP][NA][NT][4];
#pragma unroll
    for (int g = 0; g < NP; ++g)
#pragma unroll
      for (int z = 0; z < NA; ++z)
#pragma unroll
        for (int n = 0; n < NT; ++n) S[g][z][n][0] = S[g][z][n][1] = S[g][z][n][2] = S[g][z][n][3] = 0.f;
    {
      uint32_t c0[NP][GG::LW], c1[NP][GG::LW], s0[NP], s1[NP];   // codes and scales of the lane's two keys
#pragma unroll
      for (int g = 0; g < NP; ++g) {
        const uint32_t ka = at[g] + ln.ka, ksa = at[g] + ln.ksa;
        if constexpr (D == 128) {
          const uint4 a = lds128(ka), b = lds128(ka + CH);
          c0[g][0] = a.x; c0[g][1] = a.y; c0[g][2] = a.z; c0[g][3] = a.w;
          c1[g][0] = b.x; c1[g][1] = b.y; c1[g][2] = b.z; c1[g][3] = b.w;
          s0[g] = e4m3x2_to_f16x2(lds16(ksa));
          s1[g] = e4m3x2_to_f16x2(lds16(ksa + SH));
        } else {
          const uint2 a = lds64(ka), b = lds64(ka + CH);
          c0[g][0] = a.x; c0[g][1] = a.y;
          c1[g][0] = b.x; c1[g][1] = b.y;
          s0[g] = e4m3x2_to_f16x2(lds8(ksa));
          s1[g] = e4m3x2_to_f16x2(lds8(ksa + SH));
        }
      }
#pragma unroll
      for (int j = 0; j < GG::LW; ++j) {
        uint32_t f[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const uint4 v = lds128(qs + (j * NT + n) * 512);
          f[n][0] = v.x; f[n][1] = v.y; f[n][2] = v.z; f[n][3] = v.w;
        }
#pragma unroll
        for (int g = 0; g < NP; ++g) {
          const uint32_t t0 = j < 2 ? half_lo2(s0[g]) : half_hi2(s0[g]), t1 = j < 2 ? half_lo2(s1[g]) : half_hi2(s1[g]);
          uint32_t h0[4], h1[4];
          e2m1x8_to_f16(c0[g][j], h0);
          e2m1x8_to_f16(c1[g][j], h1);
          const uint32_t a0[4] = {hmul2(h0[0], t0), hmul2(h1[0], t1), hmul2(h0[1], t0), hmul2(h1[1], t1)};
          const uint32_t a1[4] = {hmul2(h0[2], t0), hmul2(h1[2], t1), hmul2(h0[3], t0), hmul2(h1[3], t1)};
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_f16(S[g][0][n], a0, f[n][0], f[n][1]);
            mma_f16(S[g][NA - 1][n], a1, f[n][2], f[n][3]);
          }
        }
      }
      if constexpr (NA == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) S[0][0][0][k] += S[0][1][0][k];
      }
    }
    // ---- softmax weights.  S[n]: (key t0, rows e), (key t0 + 8, rows e).
    const int t0 = EDGE ? tb + static_cast<int>(ln.slots & 255u) : 0;
    auto hidden = [&](int n, int k) {
      const int tok = t0 + 8 * (k >> 1), lm = EDGE ? rows.last(8 * n + 2 * tig + (k & 1)) : 0;
      return EDGE && (tok > lm || (window > 0 && tok <= lm - window));
    };
    float x[NP][NT][4];
    float top = -INFINITY;
#pragma unroll
    for (int g = 0; g < NP; ++g)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[g][n][k] = fmaf(S[g][0][n][k], fac[n][k & 1], -m[n][k & 1]);
          if (hidden(n, k)) x[g][n][k] = -INFINITY;
        }
        top = fmax3(top, x[g][n][0], x[g][n][1]);
        top = fmax3(top, x[g][n][2], x[g][n][3]);
      }
    if (__any_sync(0xffffffffu, top > kMoveMax)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mn = -INFINITY;
#pragma unroll
          for (int g = 0; g < NP; ++g)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              x[g][n][2 * h + e] = hidden(n, 2 * h + e) ? -INFINITY : S[g][0][n][2 * h + e] * fac[n][e];
              mn = fmaxf(mn, x[g][n][2 * h + e]);
            }
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
          mn = fmaxf(m[n][e], mn);
          const float al = fast_exp2(m[n][e] - mn);
          m[n][e] = mn;
          l[n][e] *= al;
#pragma unroll
          for (int i = 0; i < GG::KS; ++i) {
            O[i][n][e] *= al;
            O[i][n][2 + e] *= al;
          }
#pragma unroll
          for (int g = 0; g < NP; ++g) {
            x[g][n][e] -= mn;
            x[g][n][2 + e] -= mn;
          }
        }
    }
    uint32_t Pb[NP][NT][2];           // P^T as B fragments: keys 2 tig, 2 tig + 1 (+ 8) of row gq
#pragma unroll
    for (int g = 0; g < NP; ++g)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[g][n][k] = fast_exp2(x[g][n][k]);
        l[n][0] += x[g][n][0] + x[g][n][2];
        l[n][1] += x[g][n][1] + x[g][n][3];
        Pb[g][n][0] = transpose8x8(pack_f16(x[g][n][0], x[g][n][1]));
        Pb[g][n][1] = transpose8x8(pack_f16(x[g][n][2], x[g][n][3]));
      }
    // ---- O^T += V^T P^T.  This lane's keys: tile rows 2 tig, 2 tig + 1, + 8; its
    // features: D/8 gq .. D/8 gq + D/8 - 1, of one scale group.
#pragma unroll
    for (int g = 0; g < NP; ++g) {
      const uint32_t va = at[g] + ln.va, vsa = at[g] + ln.vsa;
      const uint32_t vsb = vsa + ln.dvs, vb = va + ln.dva;
      uint32_t sc[4] = {lds8(vsa), lds8(vsb), lds8(vsa + SH), lds8(vsb + SH)};
      if constexpr (EDGE) {
        // Keys that no row sees take scale 0, so that nothing they hold meets
        // P = 0.  A NaN scale of a key that only some rows see is set aside: its
        // value is 0 here, and the rows that do see it become NaN.
        const int v0 = static_cast<int>(ln.slots >> 8 & 255u), v1 = static_cast<int>(ln.slots >> 16);
        const int tok[4] = {tb + v0, tb + v1, tb + v0 + 8, tb + v1 + 8};
        bool bad = false;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool nan = (sc[k] & 0x7Fu) == 0x7Fu;
          bad |= nan && tok[k] < L;
          if (nan || tok[k] >= L) sc[k] = 0u;
        }
        if (__any_sync(0xffffffffu, bad)) {
          const uint32_t col = vsa - static_cast<uint32_t>(v0 * GG::SROW);   // slot 0 of the lane's group
          for (int s = 0; s < kPage && tb + s < L; ++s) {
            if ((lds8(col + s * GG::SROW) & 0x7Fu) != 0x7Fu) continue;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int lm = rows.last(8 * n + 2 * tig + e);
                if (tb + s <= lm && !(window > 0 && tb + s <= lm - window)) {
#pragma unroll
                  for (int i = 0; i < GG::KS; ++i) {
                    O[i][n][e] = __uint_as_float(0x7FC00000u);
                    O[i][n][2 + e] = __uint_as_float(0x7FC00000u);
                  }
                }
              }
          }
        }
      }
      const uint32_t sa = e4m3x2_to_f16x2(prmt(sc[0], sc[1], 0x0040u));
      const uint32_t sb = e4m3x2_to_f16x2(prmt(sc[2], sc[3], 0x0040u));
      constexpr int VW = D / 64;        // words of codes a lane reads of each key
      uint32_t w[4][VW];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t row = (k & 1 ? vb : va) + (k >> 1) * CH;
        if constexpr (D == 128) {
          const uint2 v = lds64(row);
          w[k][0] = v.x;
          w[k][1] = v.y;
        } else {
          w[k][0] = lds32(row);
        }
      }
#pragma unroll
      for (int j = 0; j < VW; ++j) {
        uint32_t a0[4], a1[4], a2[4], a3[4];
        // even features of two keys side by side, then odd features
        e2m1x8_to_f16(bitsel(w[0][j], w[1][j] * 16u, 0x0F0F0F0Fu), a0);
        e2m1x8_to_f16(bitsel(w[0][j] >> 4, w[1][j], 0x0F0F0F0Fu), a1);
        e2m1x8_to_f16(bitsel(w[2][j], w[3][j] * 16u, 0x0F0F0F0Fu), a2);
        e2m1x8_to_f16(bitsel(w[2][j] >> 4, w[3][j], 0x0F0F0F0Fu), a3);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint32_t a[4] = {hmul2(a0[u], sa), hmul2(a1[u], sa), hmul2(a2[u], sb), hmul2(a3[u], sb)};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(O[4 * j + u][n], a, Pb[g][n][0], Pb[g][n][1]);
        }
      }
    }
  }
};

// Barrier of the KW warps of a team (all of them come by at every segment's end).
__device__ __forceinline__ void team_sync(int team, int kw_warps) {
  asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "r"(32 * kw_warps) : "memory");
}

// The order in which the CTAs take their shares: a unit with n > 0 pages is W + n long,
// the W first (its start and end; a cut there is before its first page).  pos[i], the
// prologue's prefix, is the sum of W + n over the sequences before i that have pages.
struct OrderQ4 {
  const int32_t* pos;
  int B, NC, W;
  __device__ __forceinline__ uint32_t at(int i) const { return static_cast<uint32_t>(pos[i]); }
  __device__ __forceinline__ int64_t start(int i) const { return static_cast<int64_t>(NC) * at(i); }
  __device__ __forceinline__ int pages(int i) const {
    const uint32_t d = at(i + 1) - at(i);
    return static_cast<int>(d == 0u ? 0u : d - static_cast<uint32_t>(W));
  }
  // The unit at coordinate y < start(B), its page there (j), and the coordinate at which
  // its pages begin.
  __device__ __forceinline__ Cursor unit(int64_t y, int64_t& first) const {
    int lo = 0, hi = B - 1;                        // the last sequence that starts at y or before has pages
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start(mid) <= y) lo = mid; else hi = mid - 1;
    }
    Cursor cu;
    cu.i = lo;
    cu.n = pages(lo);
    cu.c = static_cast<int>((y - start(lo)) / (cu.n + W));
    first = start(lo) + static_cast<int64_t>(cu.c) * (cu.n + W) + W;
    cu.j = static_cast<int>(max(static_cast<int64_t>(0), y - first));
    return cu;
  }
  // The unit after cu's, which is not the last.
  __device__ __forceinline__ void next(Cursor& cu) const {
    cu.j = 0;
    if (++cu.c < NC) return;
    cu.c = 0;
    const uint32_t here = at(++cu.i);
    if (at(cu.i + 1) == here) {                    // no pages: to the last sequence that starts here
      int lo = cu.i + 1, hi = B - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (at(mid) == here) lo = mid; else hi = mid - 1;
      }
      cu.i = lo;
    }
    cu.n = pages(cu.i);
  }
};

// A segment: the pages [j0, j1) of unit (sequence i, head chunk c) in a CTA's range.
struct SegmentQ4 {
  int i, c, n;      // sequence, head chunk, pages of the sequence
  int j0, j1;
};

// `left`: the range's end, from the unit's first page on (it may lie behind the unit).
__device__ __forceinline__ SegmentQ4 segment_at(const Cursor& cu, int64_t left) {
  SegmentQ4 s;
  s.i = cu.i;
  s.c = cu.c;
  s.n = cu.n;
  s.j0 = cu.j;
  s.j1 = static_cast<int>(min(static_cast<int64_t>(cu.n), left));
  return s;
}

template <bool V>
struct Bool {
  static constexpr bool value = V;
};

// A warp's fetch state between segments.
struct FetchQ4 {
  Cursor cu;             // the unit after the segment
  int64_t left;          // the end of the CTA's range, from that unit's first page on
  int n, i, j;           // pages of the segment whose ids are yet to come, its sequence, the first of them
  int ahead_i, ahead_j;  // sequence and page of the ids loaded ahead (-1: none)
};

template <int D, int NT, bool WINDOW>
__global__ void __launch_bounds__(32 * kQ4Warps, q4_ctas_per_sm(NT))
    pa_split_q4_kernel(const __grid_constant__ SplitQ4Params p) {
  using GG = GeoQ4<D>;
  constexpr int S = q4_stages(D);
  const int window = WINDOW ? p.window : 0;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_scan[kQ4Warps];
  __shared__ int s_total;
  int32_t* const s_pre = reinterpret_cast<int32_t*>(smem + p.off_prefix);
  int32_t* const s_len = s_pre + (p.num_seqs + 1);
  int32_t* const s_qsl = s_len + p.num_seqs;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.num_seqs, HC = p.HC, NC = p.NC, MT = p.MT, KW = p.KW;
  grid_dependency_wait();
  const int W = q4_segment_pages(NT) * KW;
  const int active = page_prefix<true>(p, window, s_pre, s_len, s_qsl, s_scan, &s_total, W);
  __syncthreads();

  const OrderQ4 order = {s_pre, B, NC, W};
  const int64_t XW = order.start(B);
  const int64_t X = XW - static_cast<int64_t>(NC) * active * W;     // pages
  int64_t ng64 = (X + p.min_pages - 1) / p.min_pages;
  if (ng64 < 1) ng64 = 1;
  const int NG = static_cast<int>(ng64 < gridDim.x ? ng64 : gridDim.x);
  if (blockIdx.x == 0)   // units without pages: nothing for the merge
    for (int64_t u = tid; u < static_cast<int64_t>(B) * NC; u += blockDim.x)
      if (order.pages(static_cast<int>(u / NC)) == 0) p.ws_unit[u] = make_int4(0, 0, 0, 0);
  grid_launch_dependents();

  const int g = blockIdx.x;
  if (g >= NG || X == 0) return;
  // CTAs take equal shares of the order
  int64_t first_page;
  Cursor cu = order.unit(g * XW / NG, first_page);
  int64_t left = (g + 1 == NG ? XW : (g + 1) * XW / NG) - first_page;
  const int teams = HC * MT;
  if (left <= cu.j || warp >= teams * KW) return;
  const int team = warp % teams, kw = warp / teams, lg_kw = __ffs(KW) - 1;
  const int hh = team / MT, wt = team - hh * MT;
  const int gq = lane >> 2, tig = lane & 3;
  const int G = p.G, row0 = 8 * NT * wt;
  const uint32_t ring = smem_addr(smem) + static_cast<uint32_t>(warp * S * GG::PAGE);

  // ---- the fetch side: this warp's pages (kw, kw + KW, ... of every segment) in
  // order, S of them ahead of the computation.  `ids` holds 32 page ids, one a
  // lane; the 32 that follow are loaded ahead.  What only a new segment or a new 32
  // ids need waits in shared memory (every lane stores the same values).
  FetchQ4* const fst = reinterpret_cast<FetchQ4*>(smem + p.off_state) + warp;
  fst->cu = cu;
  fst->left = left;
  fst->n = 0;
  fst->ahead_i = -1;
  __syncwarp();
  int ids = 0, nids = 0, flane = 0, fstop = 0;   // the next id's lane, and the lanes that hold one (< 0: no page left)
  // this lane's part of a page: rows lane / CPR (and RPI on, ...) of the codes, 16 bytes;
  // the scales' copy takes the first SL lanes for K and the next for V
  constexpr int CPR = GG::ROWB / 16, RPI = 32 / CPR, SL = GG::STILE / 16;
  const uint32_t dlane = code_off<D>(lane / CPR, lane % CPR * 16);
  const uint8_t *kp = nullptr, *vp = nullptr, *sp = nullptr;   // in page 0, of the segment's head
  auto ids_of = [&](int i, int j) {
    const int x = j + lane * KW;
    return x < order.pages(i)
               ? p.block_tables[static_cast<int64_t>(i) * p.bt_stride + x +
                                first_visible_page(s_len[i], s_qsl[i + 1] - s_qsl[i], window)]
               : 0;
  };
  auto refill = [&]() {             // the next ids of the segment, or those of the next segment with pages for this warp
    int n = fst->n, i = fst->i, j = fst->j;      // pages of the segment not yet in `ids`, from page j on
    Cursor c = fst->cu;
    int64_t rest = fst->left;
    if (n == 0) {
      SegmentQ4 s;
      while (n == 0 && rest > 0) {
        s = segment_at(c, rest);
        rest -= s.n + W;
        if (rest > 0) order.next(c);
        n = (s.j1 - s.j0 - kw + KW - 1) >> lg_kw;
      }
      if (n == 0) {
        fstop = -1;
        return;
      }
      i = s.i;
      j = s.j0 + kw;
      const int head = s.c * HC + hh;
      kp = p.k_codes + lane / CPR * p.kc_stride_slot + lane % CPR * 16 + head * p.kc_stride_head;
      vp = p.v_codes + lane / CPR * p.vc_stride_slot + lane % CPR * 16 + head * p.vc_stride_head;
      sp = (lane < SL ? p.k_sc + lane * 16 : p.v_sc + (lane - SL) * 16) + static_cast<int64_t>(head) * GG::STILE;
    }
    ids = fst->ahead_i == i && fst->ahead_j == j ? nids : ids_of(i, j);
    flane = 0;
    fstop = min(n, 32);
    if (lane < fstop && static_cast<uint32_t>(ids) >= static_cast<uint32_t>(p.num_pages)) {
      atomicOr(p.err, kErrPageRange);             // no such page: page 0's contents instead
      ids = 0;
    }
    n -= fstop;
    j += 32 * KW;
    const int ni = n > 0 ? i : (rest > 0 ? c.i : -1), nj = n > 0 ? j : kw;
    if (ni >= 0) nids = ids_of(ni, nj);
    __syncwarp();
    fst->cu = c;
    fst->left = rest;
    fst->n = n;
    fst->i = i;
    fst->j = j;
    fst->ahead_i = ni;
    fst->ahead_j = nj;
    __syncwarp();
  };
  const uint32_t s_page = lane < SL ? p.k_sc_page : p.v_sc_page;
  auto fetch = [&](uint32_t dst) {                // one page (or none: an empty group)
    if (flane == fstop) refill();
    if (fstop >= 0) {
      const uint32_t id = static_cast<uint32_t>(__shfl_sync(0xffffffffu, ids, flane));
      ++flane;
      const uint8_t* k = kp + static_cast<uint64_t>(id) * p.kc_stride_page;
      const uint8_t* v = vp + static_cast<uint64_t>(id) * p.vc_stride_page;
#pragma unroll
      for (int r = 0; r < 16; r += RPI) {
        copy16(dst + dlane + r * GG::ROWB, k + r * p.kc_stride_slot);
        copy16(dst + dlane + GG::V + r * GG::ROWB, v + r * p.vc_stride_slot);
      }
      if (lane < 2 * SL) copy16(dst + GG::KSC + lane * 16, sp + static_cast<uint64_t>(id) * s_page);
    }
    copy_commit();
  };

  // ---- the compute side
  LaneQ4 ln;
  {
    const int r0 = slot_of<D>(gq), v0 = slot_of<D>(2 * tig), v1 = slot_of<D>(2 * tig + 1);
    ln.ka = code_off<D>(r0, D / 8 * tig);
    ln.va = GG::V + code_off<D>(v0, D / 16 * gq);
    ln.dva = GG::V + code_off<D>(v1, D / 16 * gq) - ln.va;
    ln.ksa = GG::KSC + r0 * GG::SROW + (D == 128 ? 2 * tig : tig);
    ln.vsa = GG::VSC + v0 * GG::SROW + (D == 128 ? gq : gq >> 1);
    ln.dvs = static_cast<uint32_t>((v1 - v0) * GG::SROW);
    ln.slots = static_cast<uint32_t>(r0 | v0 << 8 | v1 << 16);
  }
  StateQ4<D, NT> cs;
  cs.qs = smem_addr(smem) + p.off_q + static_cast<uint32_t>(team) * q4_query_bytes(D, NT) + 16u * lane;
  // rows of a KV head are numbered (query token, head of the group): row / G by a
  // product (exact for the at most 128 rows of a head's tiles)
  const uint32_t g_inv = (65536u + G - 1u) / static_cast<uint32_t>(G);
  auto token_of = [&](int rho) { return static_cast<int>(static_cast<uint32_t>(rho) * g_inv >> 16); };
  SegmentQ4 sg = segment_at(cu, left);
  SeqInfo si = seq_info(p, s_len, s_qsl, sg.i, lane == 0 && warp == 0, window);
  auto row_at = [&](const SegmentQ4& s, const SeqInfo& q, int n) {
    const int rho = row0 + 8 * n + gq, t = token_of(rho);
    return t < q.qn ? p.q + static_cast<int64_t>(q.t0 + t) * p.q_stride_t + ((s.c * HC + hh) * G + rho - t * G) * D
                    : nullptr;
  };
  // the next segment's query rows on their way towards L2 (a load that misses it takes 2
  // to 5 us beside the page stream)
  auto query_ahead = [&](const SegmentQ4& s, const SeqInfo& q) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint16_t* row = row_at(s, q, n);
      if (row != nullptr) prefetch_l2(row + (D / 4) * tig);
    }
  };
  query_ahead(sg, si);
  const uint32_t ring_end = ring + static_cast<uint32_t>(S * GG::PAGE);
  for (uint32_t a = ring; a < ring_end; a += GG::PAGE) fetch(a);
  uint32_t at = ring;               // the page to compute
  bool first = true;
  for (;;) {
    left -= sg.n + W;
    const int R = G * si.qn, min_lim = si.L - si.qn;
    const bool active = row0 < R;
    const RowsQ4 rows = {min_lim, row0, R, g_inv};
    const int hq_base = (sg.c * HC + hh) * G;
    if (sg.j0 == 0 && warp == 0 && lane == 0) {
      // this CTA holds the unit's first page: describe the unit for the merge
      const int64_t a = order.start(sg.i) + static_cast<int64_t>(sg.c) * (sg.n + W);
      const int last_cta = static_cast<int>(((a + W + sg.n) * NG - 1) / XW);
      p.ws_unit[static_cast<int64_t>(sg.i) * NC + sg.c] =
          make_int4(g, (last_cta - g + 1) | (first ? 0 : (1 << 30)), si.t0, si.qn);
    }
    if (active) {
      cs.reset();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        uint2 w[GG::KS];
        cs.read_query(w, row_at(sg, si, n), tig);
        cs.set_query(n, w, tig, p.scale_log2);
      }
      __syncwarp();
    }
    SegmentQ4 ns = sg;
    SeqInfo ni = si;
    if (left > 0) {
      order.next(cu);
      ns = segment_at(cu, left);
      ni = seq_info(p, s_len, s_qsl, ns.i, lane == 0 && warp == 0, window);
      query_ahead(ns, ni);
    }
    {
      // this warp's pages by their first tokens: below `lo` or from `hi` on some row
      // does not see all keys
      const int t_end = kPage * (si.js + sg.j1);
      const int lo = WINDOW ? min(t_end, si.L - window) : 0, hi = min(t_end, min_lim - (kPage - 2));
      int t = kPage * (si.js + sg.j0 + kw);
      auto after = [&](uint32_t a) { return a + GG::PAGE == ring_end ? ring : a + GG::PAGE; };
      auto run = [&](auto edge, int stop) {
        for (; t < stop; t += kPage * KW) {
          copy_wait<S - 1>();
          __syncwarp();
          const uint32_t one[1] = {at};
          if (active) cs.template page<decltype(edge)::value, 1>(ln, one, t, si.L, window, rows, tig);
          __syncwarp();
          fetch(at);
          at = after(at);
        }
      };
      if (WINDOW) run(Bool<true>{}, lo);
      // two at once while there are two: their chains of dependent steps overlap
      for (; t + kPage * KW < hi; t += 2 * kPage * KW) {
        copy_wait<S - 2>();
        __syncwarp();
        const uint32_t two[2] = {at, after(at)};
        if (active) cs.template page<false, 2>(ln, two, t, si.L, window, rows, tig);
        __syncwarp();
        fetch(two[0]);
        fetch(two[1]);
        at = after(two[1]);
      }
      run(Bool<false>{}, hi);
      run(Bool<true>{}, t_end);
    }
    // ---- end of the segment
    const bool complete = sg.j0 == 0 && sg.j1 == sg.n;
    const bool sinks_here = p.sinks != nullptr && sg.j0 == 0;
    float sk[NT][2];                  // this lane's rows' sinks (log2 units)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rho = row0 + 8 * n + 2 * tig + e;
        sk[n][e] = sinks_here && rho < R ? p.sinks[hq_base + rho - token_of(rho) * G] * 1.4426950408889634f : 0.f;
      }
    const int64_t ws_row = (static_cast<int64_t>(2 * g + (first ? 0 : 1)) * HC + hh) * p.R_max + row0;
    const int t_first = si.t0;
    first = false;
    sg = ns;
    si = ni;
    constexpr int FPL = D / 8;        // features a lane holds of each of its rows
    if (active) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) cs.l[n][e] += __shfl_xor_sync(0xffffffffu, cs.l[n][e], o);
    }
    // KW warps of a team meet: warp kw gathers the features of the lanes with
    // gq / (8 / KW) == kw, so every warp leaves the other lanes' rows in shared
    // memory: [rows of the tile][features it does not gather].
    const int per = 8 >> lg_kw;                                  // gq values a warp gathers
    const bool gathers = gq >> (3 - lg_kw) == kw;
    if (KW > 1) {
      constexpr int WROWS = 8 * NT;
      const int cols = FPL * (8 - per) + 4;                      // floats between rows (16-byte aligned)
      const uint32_t warp_bytes = static_cast<uint32_t>(WROWS * cols * 4 + WROWS * 8);
      auto ml_of = [&](int k) {
        return reinterpret_cast<float2*>(smem + p.off_xchg + (team + k * teams) * warp_bytes);
      };
      // features of lane row q in warp k's rows (k does not gather them)
      auto row_of = [&](int k, int rl, int q) {
        return reinterpret_cast<float*>(ml_of(k) + WROWS) + rl * cols + FPL * (q >> (3 - lg_kw) > k ? q - per : q);
      };
      if (active) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rl = 8 * n + 2 * tig + e;
            if (gq == 0) ml_of(kw)[rl] = make_float2(cs.m[n][e], cs.l[n][e]);
            if (gathers) continue;
            float* o = row_of(kw, rl, gq);
#pragma unroll
            for (int i = 0; i < GG::KS; i += 2)
              *reinterpret_cast<float4*>(o + 2 * i) =
                  make_float4(cs.O[i][n][e], cs.O[i][n][2 + e], cs.O[i + 1][n][e], cs.O[i + 1][n][2 + e]);
          }
      }
      team_sync(team, KW);
      if (active && gathers) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rl = 8 * n + 2 * tig + e;
            float mx = cs.m[n][e];
            for (int k = 0; k < KW; ++k) mx = fmaxf(mx, ml_of(k)[rl].x);
            const float a = fast_exp2(cs.m[n][e] - mx);
            float lt = a * cs.l[n][e];
#pragma unroll
            for (int i = 0; i < GG::KS; ++i) {
              cs.O[i][n][e] *= a;
              cs.O[i][n][2 + e] *= a;
            }
            for (int k = 0; k < KW; ++k) {
              if (k == kw) continue;
              const float2 ml = ml_of(k)[rl];
              const float b = fast_exp2(ml.x - mx);
              lt += b * ml.y;
              const float* o = row_of(k, rl, gq);
#pragma unroll
              for (int i = 0; i < GG::KS; i += 2) {
                const float4 v = *reinterpret_cast<const float4*>(o + 2 * i);
                cs.O[i][n][e] += b * v.x;
                cs.O[i][n][2 + e] += b * v.y;
                cs.O[i + 1][n][e] += b * v.z;
                cs.O[i + 1][n][2 + e] += b * v.w;
              }
            }
            cs.m[n][e] = mx;
            cs.l[n][e] = lt;
          }
      }
      team_sync(team, KW);             // read: the next segment may write
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rl = 8 * n + 2 * tig + e, rho = row0 + rl;
        if (rho >= R || !gathers) continue;
        const int tk = token_of(rho), t = t_first + tk, hq = hq_base + rho - tk * G;
        float lt = cs.l[n][e], mm = cs.m[n][e];
        if (sinks_here) {
          // The sink, a virtual key with a zero value row, joins the sum of the unit's
          // first piece here, in fp32: the keys' f16 weights stay relative to the keys'
          // own maximum, however far the sink lies above it.  The maximum moves only
          // where the sum would leave fp32's range; an infinite sink makes the sum
          // infinite (output 0), a NaN one NaN.
          float mx = mm;
          if (sk[n][e] - mm > 64.f) {
            mx = fminf(sk[n][e], kMaxSink);
            const float al = fast_exp2(mm - mx);
            lt *= al;
#pragma unroll
            for (int i = 0; i < GG::KS; ++i) {
              cs.O[i][n][e] *= al;
              cs.O[i][n][2 + e] *= al;
            }
          }
          lt += fast_exp2(sk[n][e] - mx);
          mm = mx;
        }
        if (complete) {
          const float inv = lt == 0.f ? 0.f : __fdividef(p.v_scale, lt);
          uint16_t* o = p.out + static_cast<int64_t>(t) * p.out_stride_t + static_cast<int64_t>(hq) * p.out_stride_h +
                        FPL * gq;
#pragma unroll
          for (int i = 0; i < GG::KS; i += 2)
            *reinterpret_cast<uint2*>(o + 2 * i) =
                make_uint2(pack_bf16(cs.O[i][n][e] * inv, cs.O[i][n][2 + e] * inv),
                           pack_bf16(cs.O[i + 1][n][e] * inv, cs.O[i + 1][n][2 + e] * inv));
          if (p.lse != nullptr && gq == 0)
            p.lse[static_cast<int64_t>(t) * p.lse_stride_t + static_cast<int64_t>(hq) * p.lse_stride_h] =
                lt == 0.f ? -INFINITY : (mm + fast_log2(lt)) * 0.69314718055994530942f;
        } else {
          float* o = p.ws_o + (ws_row + rl) * D + FPL * gq;
#pragma unroll
          for (int i = 0; i < GG::KS; i += 2)
            *reinterpret_cast<float4*>(o + 2 * i) =
                make_float4(cs.O[i][n][e], cs.O[i][n][2 + e], cs.O[i + 1][n][e], cs.O[i + 1][n][2 + e]);
          if (gq == 0) p.ws_ml[ws_row + rl] = make_float2(mm, lt);
        }
      }
    if (left <= 0) return;
  }
}

namespace {

template <int D, int NT>
cudaError_t launch_nt(cudaLaunchConfig_t* cfg, const SplitQ4Params& p) {
  cfg->blockDim = dim3(32 * kQ4Warps, 1, 1);
  return p.window > 0 ? cudaLaunchKernelEx(cfg, pa_split_q4_kernel<D, NT, true>, p)
                      : cudaLaunchKernelEx(cfg, pa_split_q4_kernel<D, NT, false>, p);
}

template <int D, int NT>
cudaError_t limit_nt(int smem) {
  const cudaError_t e = cudaFuncSetAttribute(pa_split_q4_kernel<D, NT, false>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(pa_split_q4_kernel<D, NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

}  // namespace

int split_q4_warps() { return kQ4Warps; }
int split_q4_ctas_per_sm(int nt) { return q4_ctas_per_sm(nt); }
int split_q4_stages(int head_dim) { return q4_stages(head_dim); }
uint32_t split_q4_state_bytes() { return kQ4Warps * sizeof(FetchQ4); }
uint32_t split_q4_query_bytes(int head_dim, int nt) { return q4_query_bytes(head_dim, nt); }

cudaError_t launch_split_q4(int head_dim, int nt, const SplitQ4Params& p, int grid, int smem, bool pdl,
                            cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (head_dim == 128 && nt == 1) return launch_nt<128, 1>(&cfg, p);
  if (head_dim == 128 && nt == 2) return launch_nt<128, 2>(&cfg, p);
  if (head_dim == 64 && nt == 1) return launch_nt<64, 1>(&cfg, p);
  if (head_dim == 64 && nt == 2) return launch_nt<64, 2>(&cfg, p);
  if (head_dim == 64 && nt == 4) return launch_nt<64, 4>(&cfg, p);
  return cudaErrorInvalidValue;
}

cudaError_t set_split_smem_limits_q4(int smem) {
  cudaError_t e;
  if ((e = limit_nt<128, 1>(smem)) || (e = limit_nt<128, 2>(smem)) || (e = limit_nt<64, 1>(smem)) ||
      (e = limit_nt<64, 2>(smem)) || (e = limit_nt<64, 4>(smem)))
    return e;
  return cudaSuccess;
}

}  // namespace pa
