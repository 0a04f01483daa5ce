// Split-KV decode attention over a 4-bit paged cache (pa_q4.cuh has the format).
//
// Work decomposition, workspace and merge are those of the bf16 / fp8 split
// kernel: CTA g takes an equal range of the (sequence, head chunk, page) order;
// a unit cut by a range boundary leaves fp32 partials for the merge kernel.
//
// At 4.5 bits a cached feature the walk is bound by what a warp issues per
// feature, so everything that does not depend on the query rows is done once a
// key, and nothing is done for rows that do not exist:
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
//     page); P is then at most 256 and its rounding to f16 is 2^-12 relative.
// Query rows are scaled by a power of two into f16's range (exact except for
// elements 2^-14 below the row's largest), and the power goes into the row's logit factor.
//
// CTA (one an SM): a warpgroup of producers, then CW = 16
// consumer warps for 8 query rows a warp or 8 for more, with the registers split
// between the two kinds (setmaxnreg).  KW x MT x HC consumer warps are in use:
// HC KV heads, MT tiles of 8 NT query rows, and KW warps that take a head's pages
// (a stage of the ring, BP pages, at a time) in turn and meet in shared memory at
// the end of a segment (a sequence's pages in this CTA).  All waits are bounded.
#include "pa_q4.cuh"
#include "pa_split.cuh"

namespace pa {

// Consumer warps of a CTA and the registers of a consumer / producer thread:
// with 128 producer threads the two shares add up to what the CTA is launched
// with (96 x 640 and 168 x 384).
constexpr int q4_warps(int nt) { return nt == 1 ? 16 : 8; }
// Query fragments in shared memory (D x 8 NT f16 of a warp) or in registers.
constexpr bool q4_query_in_smem(int nt) { return nt == 4; }
constexpr uint32_t q4_query_bytes(int d, int nt) { return q4_query_in_smem(nt) ? static_cast<uint32_t>(d * 8 * nt * 2) : 0u; }
template <int NT>
struct RegsQ4 {
  static constexpr int CONS = NT == 1 ? 112 : 232, PROD = NT == 1 ? 32 : 40;
  static constexpr int LAUNCH = NT == 1 ? 96 : 168;
  static_assert(q4_warps(NT) * CONS + 4 * PROD <= (q4_warps(NT) + 4) * LAUNCH, "register split");
};

template <int D>
struct GeoQ4 {
  static constexpr int ROWB = D / 2;        // bytes of a row's codes
  static constexpr int TILE = 16 * ROWB;    // codes of one page of one head
  static constexpr int SROW = D / 16;       // bytes of a row's scales
  static constexpr int STILE = 16 * SROW;   // scales of one page and head
  static constexpr int KS = D / 16;         // k-steps of K Q^T; also 16-feature tiles of V^T
  static constexpr int LW = D / 32;         // words of codes a lane reads of its key
};

// A page's codes lie in shared memory as in the cache, [16 slots][HC heads][D / 2
// bytes], in TMA box rows of IB = 128, 64 or 32 bytes (the largest that divides a
// slot's bytes: the copy engine's time goes by box rows; with a head's 64-byte row
// a box row it took 3.7 cycles a row, twice the time of 128-byte rows) and the
// swizzle of that span: address bits [4, 4 + k) XOR bits [7, 7 + k).
__device__ __forceinline__ uint32_t code_off(int slot, int byte, int slot_bytes, int ib) {
  const uint32_t off = static_cast<uint32_t>(slot * slot_bytes + byte);
  const uint32_t mask = ib == 128 ? 7u : ib == 64 ? 3u : 0u;
  return off ^ (((off >> 7) & mask) << 4);
}

// Slot of tile row t (bits t2 t1 t0; rows 8 .. 15 add 8).  A warp reads the scores'
// keys eight lanes (D = 128: rows t0) or sixteen (D = 64: rows t1 t0) at a time and
// the values' keys by rows t2 t1: the slot bits that reach the bank of a read,
// directly or through the swizzle, must differ there.  Which bits these are goes
// by the bytes of a slot (free of conflicts for 32 to 256 bytes; values two-way at
// 512, more above).
template <int D>
__device__ __forceinline__ int slot_of(int t, int slot_bytes) {
  const int t0 = t & 1, t1 = (t >> 1) & 1, t2 = (t >> 2) & 1;
  if (slot_bytes == 256 || slot_bytes == 32) return t1 | (t0 ^ t2) << 1 | t2 << 2;
  if (slot_bytes == 128) return t2 | t1 << 1 | (t0 ^ t2) << 2;
  if (D == 64 && slot_bytes == 64) return t1 | t2 << 1 | (t0 ^ t2) << 2;
  return t ^ t1;
}

// What a lane reads of every page (offsets into a stage) and the slots of its keys.
struct LaneQ4 {
  uint32_t ka, va, dva;      // codes: scores' first key; values' first key, from it to the second
  uint32_t ksa, vsa, dvs;    // scales, likewise
  uint32_t slots;            // the scores' key | the values' keys << 8, << 16
};

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

// One warp's state: 8 NT query rows of one KV head.  Lane (gq = lane / 4, tig =
// lane % 4) holds the query rows 8 n + 2 tig + e (n < NT, e < 2) of the scores
// and the outputs.
// QS: the query fragments stay in shared memory (qs: this lane's, 512 bytes a pair
// of k-steps and row tile) instead of registers.
template <int D, int NT, bool QS>
struct StateQ4 {
  using GG = GeoQ4<D>;
  float O[GG::KS][NT][4];      // O^T: [feature tile][row tile]; elements (feature 2 i, rows e), (2 i + 1, rows e)
  uint32_t Qf[QS ? 1 : GG::KS][NT][2];  // query rows as B fragments
  uint32_t qs;
  float m[NT][2], l[NT][2];    // running maximum (log2 units), this lane's share of the sum
  float fac[NT][2];            // logit factor of the row (log2 units per raw score)
  int lim[NT][2];              // last key the row sees

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

  // Query row `row` (bf16, D features; nullptr: no such row) of tile n into
  // fragments: this lane's features are D/4 tig .. D/4 tig + D/4 - 1.
  __device__ __forceinline__ void load_query(int n, const uint16_t* row, int tig, float scale_log2) {
    uint2 w[GG::KS];
    float amax = 0.f;
#pragma unroll
    for (int ks = 0; ks < GG::KS; ++ks)
      w[ks] = row != nullptr ? *reinterpret_cast<const uint2*>(row + (D / 4) * tig + 4 * ks) : make_uint2(0u, 0u);
#pragma unroll
    for (int ks = 0; ks < GG::KS; ++ks)
      amax = fmaxf(fmaxf(fmaxf(fabsf(bf16_lo(w[ks].x)), fabsf(bf16_hi(w[ks].x))),
                         fmaxf(fabsf(bf16_lo(w[ks].y)), fabsf(bf16_hi(w[ks].y)))), amax);
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // exponent of the row's largest element, kept where 2^-e and scale * 2^e are normal
    int ex = static_cast<int>(__float_as_uint(amax) >> 23) - 127;
    ex = max(-100, min(115, ex));
    const float down = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
#pragma unroll
    for (int ks = 0; ks < GG::KS; ks += 2) {
      uint32_t f[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        f[2 * u] = pack_f16(bf16_lo(w[ks + u].x) * down, bf16_hi(w[ks + u].x) * down);
        f[2 * u + 1] = pack_f16(bf16_lo(w[ks + u].y) * down, bf16_hi(w[ks + u].y) * down);
      }
      if constexpr (QS) {
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(qs + (ks / 2 * NT + n) * 512), "r"(f[0]),
                     "r"(f[1]), "r"(f[2]), "r"(f[3])
                     : "memory");
      } else {
        Qf[ks][n][0] = f[0];
        Qf[ks][n][1] = f[1];
        Qf[ks + 1][n][0] = f[2];
        Qf[ks + 1][n][1] = f[3];
      }
    }
    const float f = scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
    fac[n][0] = __shfl_sync(0xffffffffu, f, 8 * tig);
    fac[n][1] = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
  }

  // One page of this warp's head: its codes at `co`, its scales at `so`, CH bytes
  // of codes from a key to the one 8 rows on.  EDGE: some row does not see all 16
  // keys.
  template <bool EDGE>
  __device__ __forceinline__ void page(const LaneQ4& ln, uint32_t co, uint32_t so, uint32_t CH, int tb, int L,
                                       int window) {
    constexpr int SH = 8 * GG::SROW;
    const uint32_t ka = co + ln.ka, ksa = so + ln.ksa, va = co + ln.va, vsa = so + ln.vsa;
    // ---- S^T = K Q^T, in NA independent sums
    constexpr int NA = NT == 1 ? 2 : 1;
    float S[NA][NT][4];
#pragma unroll
    for (int z = 0; z < NA; ++z)
#pragma unroll
      for (int n = 0; n < NT; ++n) S[z][n][0] = S[z][n][1] = S[z][n][2] = S[z][n][3] = 0.f;
    {
      uint32_t c0[GG::LW], c1[GG::LW], s0, s1;   // codes and scales of the lane's two keys
      if constexpr (D == 128) {
        const uint4 a = lds128(ka), b = lds128(ka + CH);
        c0[0] = a.x; c0[1] = a.y; c0[2] = a.z; c0[3] = a.w;
        c1[0] = b.x; c1[1] = b.y; c1[2] = b.z; c1[3] = b.w;
        s0 = e4m3x2_to_f16x2(lds16(ksa));
        s1 = e4m3x2_to_f16x2(lds16(ksa + SH));
      } else {
        const uint2 a = lds64(ka), b = lds64(ka + CH);
        c0[0] = a.x; c0[1] = a.y;
        c1[0] = b.x; c1[1] = b.y;
        s0 = e4m3x2_to_f16x2(lds8(ksa));
        s1 = e4m3x2_to_f16x2(lds8(ksa + SH));
      }
#pragma unroll
      for (int j = 0; j < GG::LW; ++j) {
        const uint32_t t0 = j < 2 ? half_lo2(s0) : half_hi2(s0), t1 = j < 2 ? half_lo2(s1) : half_hi2(s1);
        uint32_t h0[4], h1[4];
        e2m1x8_to_f16(c0[j], h0);
        e2m1x8_to_f16(c1[j], h1);
        const uint32_t a0[4] = {hmul2(h0[0], t0), hmul2(h1[0], t1), hmul2(h0[1], t0), hmul2(h1[1], t1)};
        const uint32_t a1[4] = {hmul2(h0[2], t0), hmul2(h1[2], t1), hmul2(h0[3], t0), hmul2(h1[3], t1)};
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (QS) {
            const uint4 f = lds128(qs + (j * NT + n) * 512);
            mma_f16(S[0][n], a0, f.x, f.y);
            mma_f16(S[NA - 1][n], a1, f.z, f.w);
          } else {
            mma_f16(S[0][n], a0, Qf[2 * j][n][0], Qf[2 * j][n][1]);
            mma_f16(S[NA - 1][n], a1, Qf[2 * j + 1][n][0], Qf[2 * j + 1][n][1]);
          }
        }
      }
      if constexpr (NA == 2) {
#pragma unroll
        for (int k = 0; k < 4; ++k) S[0][0][k] += S[1][0][k];
      }
    }
    // ---- softmax weights.  S[n]: (key t0, rows e), (key t0 + 8, rows e).
    const int t0 = EDGE ? tb + static_cast<int>(ln.slots & 255u) : 0;
    auto hidden = [&](int n, int k) {
      const int tok = t0 + 8 * (k >> 1), lm = lim[n][k & 1];
      return EDGE && (tok > lm || (window > 0 && tok <= lm - window));
    };
    float x[NT][4];
    float top = -INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        x[n][k] = fmaf(S[0][n][k], fac[n][k & 1], -m[n][k & 1]);
        if (hidden(n, k)) x[n][k] = -INFINITY;
      }
      top = fmax3(top, x[n][0], x[n][1]);
      top = fmax3(top, x[n][2], x[n][3]);
    }
    if (__any_sync(0xffffffffu, top > kMoveMax)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float a = hidden(n, e) ? -INFINITY : S[0][n][e] * fac[n][e];
          const float b = hidden(n, 2 + e) ? -INFINITY : S[0][n][2 + e] * fac[n][e];
          float mn = fmaxf(a, b);
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
          x[n][e] = a - mn;
          x[n][2 + e] = b - mn;
        }
    }
    uint32_t Pb[NT][2];               // P^T as B fragments: keys 2 tig, 2 tig + 1 (+ 8) of row gq
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) x[n][k] = fast_exp2(x[n][k]);
      l[n][0] += x[n][0] + x[n][2];
      l[n][1] += x[n][1] + x[n][3];
      Pb[n][0] = transpose8x8(pack_f16(x[n][0], x[n][1]));
      Pb[n][1] = transpose8x8(pack_f16(x[n][2], x[n][3]));
    }
    // ---- O^T += V^T P^T.  This lane's keys: tile rows 2 tig, 2 tig + 1, + 8; its
    // features: D/8 gq .. D/8 gq + D/8 - 1, of one scale group.
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
            for (int e = 0; e < 2; ++e)
              if (tb + s <= lim[n][e] && !(window > 0 && tb + s <= lim[n][e] - window)) {
#pragma unroll
                for (int i = 0; i < GG::KS; ++i) {
                  O[i][n][e] = __uint_as_float(0x7FC00000u);
                  O[i][n][2 + e] = __uint_as_float(0x7FC00000u);
                }
              }
        }
      }
    }
    const uint32_t sa = e4m3x2_to_f16x2(prmt(sc[0], sc[1], 0x0040u)), sb = e4m3x2_to_f16x2(prmt(sc[2], sc[3], 0x0040u));
    constexpr int VW = D / 64;        // words of codes a lane reads of each key
    uint32_t w[4][VW];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t at = (k & 1 ? vb : va) + (k >> 1) * CH;
      if constexpr (D == 128) {
        const uint2 v = lds64(at);
        w[k][0] = v.x;
        w[k][1] = v.y;
      } else {
        w[k][0] = lds32(at);
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
        for (int n = 0; n < NT; ++n) mma_f16(O[4 * j + u][n], a, Pb[n][0], Pb[n][1]);
      }
    }
  }
};

// mbar_wait that sleeps about NS nanoseconds between tries: a try takes about 27
// cycles, and warps that poll without a pause took a third of the CTA's issue slots.
template <int NS>
__device__ __forceinline__ bool mbar_poll(uint32_t bar, uint32_t parity, uint64_t limit_ns) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    __nanosleep(NS);
    if (mbar_try_wait(bar, parity)) return true;
    if (global_timer_ns() - t0 > limit_ns) return false;
  }
}

// A segment: the pages [j0, j1) of unit (sequence i, head chunk c) in a CTA's range.
struct SegmentQ4 {
  int i, c, n;      // sequence, head chunk, pages of the sequence
  int j0, j1;
};

__device__ __forceinline__ SegmentQ4 segment_at(const Cursor& cu, int64_t left) {
  SegmentQ4 s;
  s.i = cu.i;
  s.c = cu.c;
  s.n = cu.n;
  s.j0 = cu.j;
  s.j1 = static_cast<int>(min(static_cast<int64_t>(cu.n), cu.j + left));
  return s;
}

// The cursor after a segment (its last page was the sequence's, or the range ended).
__device__ __forceinline__ void next_unit(Cursor& cu, const int32_t* pre, int B, int NC) {
  cu.j = cu.n - 1;
  advance(cu, pre, B, NC);
}

template <int D, int NT, bool WINDOW>
__global__ void __launch_bounds__(32 * (4 + q4_warps(NT)), 1)
    pa_split_q4_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const __grid_constant__ SplitQ4Params p) {
  using GG = GeoQ4<D>;
  constexpr int CW = q4_warps(NT);
  const int window = WINDOW ? p.window : 0;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_scan[4 + CW];
  __shared__ int s_total;

  const uint32_t raw = smem_addr(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* const gbase = smem_raw + (base - raw);
  int32_t* const s_pre = reinterpret_cast<int32_t*>(gbase + p.off_prefix);
  int32_t* const s_len = s_pre + (p.num_seqs + 1);
  int32_t* const s_qsl = s_len + p.num_seqs;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int B = p.num_seqs, HC = p.HC, NC = p.NC, MT = p.MT, KW = p.KW, BP = p.block_pages;
  const int nstage = p.nstage, ncw = HC * MT * KW;
  const uint32_t bar0 = base + p.off_bar;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (nstage + s); };
  // teams (the KW warps of a head and row tile): partials written / read
  auto put_bar = [&](int t) { return bar0 + 8u * (2 * nstage + t); };
  auto got_bar = [&](int t) { return bar0 + 8u * (2 * nstage + CW + t); };
  if (tid == 0) {
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
    for (int s = 0; s < nstage; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), HC * MT);   // one kw's warps
    }
    for (int t = 0; t < HC * MT; ++t) {
      mbar_init(put_bar(t), KW);
      mbar_init(got_bar(t), KW);
    }
    fence_mbar_init();
  }
  grid_dependency_wait();
  page_prefix(p, window, s_pre, s_len, s_qsl, s_scan, &s_total, true);
  __syncthreads();

  const int64_t X = static_cast<int64_t>(NC) * s_pre[B];
  int64_t ng64 = (X + p.min_pages - 1) / p.min_pages;
  if (ng64 < 1) ng64 = 1;
  const int NG = static_cast<int>(ng64 < gridDim.x ? ng64 : gridDim.x);
  if (blockIdx.x == 0)   // units without pages: nothing for the merge
    for (int64_t u = tid; u < static_cast<int64_t>(B) * NC; u += blockDim.x)
      if (pages_of(s_pre, static_cast<int>(u / NC)) == 0) p.ws_unit[u] = make_int4(0, 0, 0, 0);
  grid_launch_dependents();

  const int g = blockIdx.x;
  if (g >= NG || X == 0) return;
  const int64_t start = static_cast<int64_t>(g) * X / NG;
  const int64_t end = static_cast<int64_t>(g + 1) * X / NG;
  int64_t left = end - start;
  if (left <= 0) return;
  const uint32_t code_page = static_cast<uint32_t>(HC * GG::TILE), scale_page = static_cast<uint32_t>(HC * GG::STILE);

  if (warp < 4) {
    // ============================ producers ================================
    // Four warps share the stages, warp w those with s % 4 == w (issuing one copy
    // holds a warp for 280 to 540 cycles beside warps that compute: one producer
    // fed 5.0 TB/s at most).  A stage has one warp for good, so that its waiter has
    // seen every earlier phase of its barrier: a parity wait cannot tell a phase
    // that is two behind from one that is complete.  One lane issues a group's
    // copies.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(RegsQ4<NT>::PROD));
    if (warp >= nstage) return;
    const int box_rows = static_cast<int>(code_page) / (kPage * p.box_bytes);
    Cursor cu = locate(s_pre, B, NC, start);
    int mine = warp;                   // this warp's next stage, ...
    uint32_t turn = 0;                 // its turn, ...
    int next = warp;                   // and the groups until then, from the segment's first
    while (left > 0) {
      const SegmentQ4 sg = segment_at(cu, left);
      left -= sg.j1 - sg.j0;
      next_unit(cu, s_pre, B, NC);
      const int pages = sg.j1 - sg.j0, groups = (pages + BP - 1) / BP;
      const int32_t* row = p.block_tables + static_cast<int64_t>(sg.i) * p.bt_stride + sg.j0 +
                           first_visible_page(s_len[sg.i], s_qsl[sg.i + 1] - s_qsl[sg.i], window);
      // page ids of a group, one a lane, loaded a group ahead
      int ids = lane < BP && next * BP + lane < pages ? row[next * BP + lane] : 0;
      while (next < groups) {
        const int now = ids, np = min(BP, pages - next * BP);
        const int at_stage = mine;
        const uint32_t at_turn = turn;
        // the next group of this warp: its next stage, or its first of the next turn
        mine += 4;
        next += 4;
        if (mine >= nstage) {
          next += nstage - mine + warp;
          mine = warp;
          ++turn;
        }
        if (lane < BP && next * BP + lane < pages) ids = row[next * BP + lane];
        if (at_turn > 0 && !mbar_poll<100>(empty_bar(at_stage), (at_turn - 1) & 1u, p.wait_ns)) {
          if (lane == 0) atomicOr(p.err, kErrTimeout);
          return;
        }
        const uint32_t bar = full_bar(at_stage);
        uint32_t dst = base + p.off_stage + static_cast<uint32_t>(at_stage) * p.stage_bytes, dst_sc = dst + p.off_ks;
        if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(np) * 2u * (code_page + scale_page));
        for (int pg = 0; pg < np; ++pg) {
          const int phys = __shfl_sync(0xffffffffu, now, pg);
          if (lane == 0) {
            // an out-of-range page reads as zero codes (TMA fill) and page 0's scales
            const bool bad = phys < 0 || phys >= p.num_pages;
            if (bad) atomicOr(p.err, kErrPageRange);
            const int64_t id = bad ? 0 : phys, at = static_cast<int64_t>(sg.c) * scale_page;
            tma_load_4d(dst, &tmap_k, 0, sg.c * box_rows, 0, phys, bar);
            tma_load_4d(dst + p.off_v, &tmap_v, 0, sg.c * box_rows, 0, phys, bar);
            bulk_load(dst_sc, p.k_sc + id * p.k_sc_page + at, scale_page, bar);
            bulk_load(dst_sc + (p.off_vs - p.off_ks), p.v_sc + id * p.v_sc_page + at, scale_page, bar);
          }
          dst += code_page;
          dst_sc += scale_page;
        }
      }
      next -= groups;
    }
    return;
  }

  // ============================== consumers ================================
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(RegsQ4<NT>::CONS));
  const int cw = warp - 4;
  if (cw >= ncw) return;
  Cursor cu = locate(s_pre, B, NC, start);
  const int team = cw % (HC * MT), kw = cw / (HC * MT);
  const int hh = team / MT, wt = team - hh * MT;
  const int gq = lane >> 2, tig = lane & 3;
  const int G = p.G, row0 = 8 * NT * wt;
  const int slot_bytes = HC * GG::ROWB;
  const uint32_t CH = static_cast<uint32_t>(8 * slot_bytes);
  LaneQ4 ln;
  {
    const int r0 = slot_of<D>(gq, slot_bytes), v0 = slot_of<D>(2 * tig, slot_bytes), v1 = slot_of<D>(2 * tig + 1, slot_bytes);
    ln.ka = code_off(r0, hh * GG::ROWB + D / 8 * tig, slot_bytes, p.box_bytes);
    ln.va = p.off_v + code_off(v0, hh * GG::ROWB + D / 16 * gq, slot_bytes, p.box_bytes);
    ln.dva = p.off_v + code_off(v1, hh * GG::ROWB + D / 16 * gq, slot_bytes, p.box_bytes) - ln.va;
    ln.ksa = p.off_ks + hh * GG::STILE + r0 * GG::SROW + (D == 128 ? 2 * tig : tig);
    ln.vsa = p.off_vs + hh * GG::STILE + v0 * GG::SROW + (D == 128 ? gq : gq >> 1);
    ln.dvs = static_cast<uint32_t>((v1 - v0) * GG::SROW);
    ln.slots = static_cast<uint32_t>(r0 | v0 << 8 | v1 << 16);
  }
  StateQ4<D, NT, q4_query_in_smem(NT)> cs;
  cs.qs = base + p.off_q + static_cast<uint32_t>(cw) * q4_query_bytes(D, NT) + 16u * lane;
  bool first = true;
  int mine = kw, next = kw;     // this warp's next stage, and the groups until then
  uint32_t turn = 0, seg_no = 0;
  while (left > 0) {
    const SegmentQ4 sg = segment_at(cu, left);
    left -= sg.j1 - sg.j0;
    next_unit(cu, s_pre, B, NC);
    const SeqInfo si = seq_info(p, s_len, s_qsl, sg.i, lane == 0 && cw == 0, window);
    const int R = G * si.qn, min_lim = si.L - si.qn;
    const bool active = row0 < R;
    const int hq_base = (sg.c * HC + hh) * G;
    if (sg.j0 == 0 && cw == 0 && lane == 0) {
      // this CTA holds the unit's first page: describe the unit for the merge
      const int64_t a = static_cast<int64_t>(NC) * s_pre[sg.i] + static_cast<int64_t>(sg.c) * sg.n;
      const int last_cta = static_cast<int>(((a + sg.n) * NG - 1) / X);
      p.ws_unit[static_cast<int64_t>(sg.i) * NC + sg.c] =
          make_int4(g, (last_cta - g + 1) | (first ? 0 : (1 << 30)), si.t0, si.qn);
    }
    if (active) {
      cs.reset();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int rho = row0 + 8 * n + gq;
        const uint16_t* row = nullptr;
        if (rho < R) row = p.q + static_cast<int64_t>(si.t0 + rho / G) * p.q_stride_t + (hq_base + rho % G) * D;
        cs.load_query(n, row, tig, p.scale_log2);
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int r2 = row0 + 8 * n + 2 * tig + e;
          cs.lim[n][e] = min_lim + (r2 < R ? r2 / G : 0);
          if (p.sinks != nullptr && sg.j0 == 0 && kw == 0 && r2 < R) {
            // the sink: a virtual first key with a zero value row
            const float sk = p.sinks[hq_base + r2 % G] * 1.4426950408889634f;
            cs.m[n][e] = fmaxf(sk, kUnsetMax);
            cs.l[n][e] = gq == 0 && sk != -INFINITY ? 1.f : 0.f;
          }
        }
      }
    }
    {
      // the segment's pages in groups of BP, a stage each; this warp's groups are
      // those in the stages s with s % KW == kw (nstage is a multiple of KW), so
      // that it waits for every phase of their barriers.  edge_lo .. edge_hi: the
      // pages (by first token) whose keys every row sees
      const int tb0 = kPage * (si.js + sg.j0), tb_end = kPage * (si.js + sg.j1);
      const int groups = (sg.j1 - sg.j0 + BP - 1) / BP;
      const int edge_hi = min_lim - (kPage - 1), edge_lo = WINDOW ? si.L - window : 0;
      for (; next < groups; next += KW) {
        if (!mbar_poll<40>(full_bar(mine), turn & 1u, p.wait_ns)) {
          if (lane == 0) atomicOr(p.err, kErrTimeout);
          return;
        }
        if (active) {
          uint32_t co = base + p.off_stage + static_cast<uint32_t>(mine) * p.stage_bytes, so = co;
          int t = tb0 + kPage * BP * next;
          const int tb_stop = min(t + kPage * BP, tb_end);
          for (; t < tb_stop; t += kPage) {
            if (t > edge_hi || (WINDOW && t < edge_lo))
              cs.template page<true>(ln, co, so, CH, t, si.L, window);
            else
              cs.template page<false>(ln, co, so, CH, t, si.L, window);
            co += code_page;
            so += scale_page;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty_bar(mine));
        mine += KW;
        if (mine >= nstage) {
          mine = kw;
          ++turn;
        }
      }
      next -= groups;
    }
    // ---- end of the segment
    const bool complete = sg.j0 == 0 && sg.j1 == sg.n;
    const int which = first ? 0 : 1;
    first = false;
    const int64_t ws_row = (static_cast<int64_t>(2 * g + which) * HC + hh) * p.R_max + row0;
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
    const int per = 8 / (KW > 8 ? 8 : KW);                       // gq values a warp gathers
    const bool mine = KW == 1 || gq / per == kw;
    if (KW > 1) {
      constexpr int WROWS = 8 * NT;
      const int cols = FPL * (8 - per) + 4;                      // floats between rows (16-byte aligned)
      const uint32_t warp_bytes = static_cast<uint32_t>(WROWS * cols * 4 + WROWS * 8);
      auto ml_of = [&](int k) {
        return reinterpret_cast<float2*>(gbase + p.off_xchg + (team + k * HC * MT) * warp_bytes);
      };
      // features of lane row q in warp k's rows (k does not gather them)
      auto row_of = [&](int k, int rl, int q) {
        return reinterpret_cast<float*>(ml_of(k) + WROWS) + rl * cols + FPL * (q / per > k ? q - per : q);
      };
      if (seg_no > 0 && !mbar_poll<40>(got_bar(team), (seg_no - 1) & 1u, p.wait_ns)) {
        if (lane == 0) atomicOr(p.err, kErrTimeout);
        return;
      }
      if (active) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int rl = 8 * n + 2 * tig + e;
            if (gq == 0) ml_of(kw)[rl] = make_float2(cs.m[n][e], cs.l[n][e]);
            if (mine) continue;
            float* o = row_of(kw, rl, gq);
#pragma unroll
            for (int i = 0; i < GG::KS; i += 2)
              *reinterpret_cast<float4*>(o + 2 * i) =
                  make_float4(cs.O[i][n][e], cs.O[i][n][2 + e], cs.O[i + 1][n][e], cs.O[i + 1][n][2 + e]);
          }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(put_bar(team));
      if (!mbar_poll<40>(put_bar(team), seg_no & 1u, p.wait_ns)) {
        if (lane == 0) atomicOr(p.err, kErrTimeout);
        return;
      }
      if (active && mine) {
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
      __syncwarp();
      if (lane == 0) mbar_arrive(got_bar(team));
      ++seg_no;
    }
    if (!active || !mine) continue;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rl = 8 * n + 2 * tig + e, rho = row0 + rl;
        if (rho >= R) continue;
        const float lt = cs.l[n][e], mm = cs.m[n][e];
        if (complete) {
          const int t = si.t0 + rho / G, hq = hq_base + rho % G;
          const float inv = lt == 0.f ? 0.f : p.v_scale / lt;
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
  }
}

namespace {

template <int D, int NT>
cudaError_t launch_nt(cudaLaunchConfig_t* cfg, const CUtensorMap& tk, const CUtensorMap& tv, const SplitQ4Params& p) {
  cfg->blockDim = dim3(32 * (4 + q4_warps(NT)), 1, 1);
  return p.window > 0 ? cudaLaunchKernelEx(cfg, pa_split_q4_kernel<D, NT, true>, tk, tv, p)
                      : cudaLaunchKernelEx(cfg, pa_split_q4_kernel<D, NT, false>, tk, tv, p);
}

template <int D>
cudaError_t launch_d(cudaLaunchConfig_t* cfg, int nt, const CUtensorMap& tk, const CUtensorMap& tv,
                     const SplitQ4Params& p) {
  if (nt == 1) return launch_nt<D, 1>(cfg, tk, tv, p);
  if (nt == 2) return launch_nt<D, 2>(cfg, tk, tv, p);
  if (nt == 4) return launch_nt<D, 4>(cfg, tk, tv, p);
  return cudaErrorInvalidValue;
}

template <int D, int NT>
cudaError_t limit_nt(int smem) {
  const cudaError_t e = cudaFuncSetAttribute(pa_split_q4_kernel<D, NT, false>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(pa_split_q4_kernel<D, NT, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

}  // namespace

int split_q4_warps(int nt) { return q4_warps(nt); }
uint32_t split_q4_query_bytes(int head_dim, int nt) { return q4_query_bytes(head_dim, nt); }

cudaError_t launch_split_q4(int head_dim, int nt, const CUtensorMap& tk, const CUtensorMap& tv, const SplitQ4Params& p,
                            int grid, int smem, bool pdl, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (head_dim == 128) return launch_d<128>(&cfg, nt, tk, tv, p);
  if (head_dim == 64) return launch_d<64>(&cfg, nt, tk, tv, p);
  return cudaErrorInvalidValue;
}

cudaError_t set_split_smem_limits_q4(int smem) {
  cudaError_t e;
  if ((e = limit_nt<128, 1>(smem)) || (e = limit_nt<128, 2>(smem)) || (e = limit_nt<128, 4>(smem)) ||
      (e = limit_nt<64, 1>(smem)) || (e = limit_nt<64, 2>(smem)) || (e = limit_nt<64, 4>(smem)))
    return e;
  return cudaSuccess;
}

}  // namespace pa
