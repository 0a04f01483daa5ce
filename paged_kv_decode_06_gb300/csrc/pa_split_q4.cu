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
// CTA: warp 0 is the producer, then KW x MT x HC consumer warps: HC KV heads, MT
// tiles of 8 NT query rows, and KW warps that take every KW-th page of a head and
// meet in shared memory at the end of a segment (a sequence's pages in this CTA).
// All waits are bounded.
//
// A row's partial whose sum is NaN carries a finite maximum, so that the merge
// does not take it for an empty one.
#include "pa_q4.cuh"
#include "pa_split.cuh"

namespace pa {

constexpr int kQ4MaxWarps = 8;

template <int D>
struct GeoQ4 {
  static constexpr int ROWB = D / 2;        // bytes of a row's codes
  static constexpr int TILE = 16 * ROWB;    // codes of one page and head
  static constexpr int SROW = D / 16;       // bytes of a row's scales
  static constexpr int STILE = 16 * SROW;   // scales of one page and head
  static constexpr int KS = D / 16;         // k-steps of K Q^T; also 16-feature tiles of V^T
  static constexpr int LW = D / 32;         // words of codes a lane reads of its key
};

// Slot of tile row t (0 .. 7; rows 8 .. 15 add 8): a permutation that makes the
// V reads (rows 2 tig, 2 tig + 1 of four lanes) free of bank conflicts.
template <int D>
__device__ __forceinline__ int slot_of(int t) {
  return D == 128 ? t ^ ((t >> 1) & 1) : t ^ ((t >> 2) & 1);
}

// Byte offset of byte b of a row's codes: D = 128 rows are 64 bytes in the
// 64-byte swizzle, D = 64 rows are 32 bytes unswizzled.
template <int D>
__device__ __forceinline__ uint32_t code_off(int row, int b) {
  if constexpr (D == 128) {
    const uint32_t off = static_cast<uint32_t>(row * 64 + b);
    return off ^ (((off >> 7) & 3u) << 4);
  } else {
    return static_cast<uint32_t>(row * 32 + b);
  }
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

// (a & mask) | (b & ~mask)
__device__ __forceinline__ uint32_t bitsel(uint32_t a, uint32_t b, uint32_t mask) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xE2;" : "=r"(r) : "r"(a), "r"(mask), "r"(b));
  return r;
}

// One warp's state: 8 NT query rows of one KV head.  Lane (gq = lane / 4, tig =
// lane % 4) holds the query rows 8 n + 2 tig + e (n < NT, e < 2) of the scores
// and the outputs.
template <int D, int NT>
struct StateQ4 {
  using GG = GeoQ4<D>;
  float O[GG::KS][NT][4];      // O^T: [feature tile][row tile]; elements (feature 2 i, rows e), (2 i + 1, rows e)
  uint32_t Qf[GG::KS][NT][2];  // query rows as B fragments
  float m[NT][2], l[NT][2];    // running maximum (log2 units), this lane's share of the sum
  float fac[NT][2];            // logit factor of the row (log2 units per raw score)
  int lim[NT][2];              // last key the row sees

  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[n][e] = -INFINITY;
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
    for (int ks = 0; ks < GG::KS; ++ks) {
      Qf[ks][n][0] = pack_f16(bf16_lo(w[ks].x) * down, bf16_hi(w[ks].x) * down);
      Qf[ks][n][1] = pack_f16(bf16_lo(w[ks].y) * down, bf16_hi(w[ks].y) * down);
    }
    const float f = scale_log2 * __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
    fac[n][0] = __shfl_sync(0xffffffffu, f, 8 * tig);
    fac[n][1] = __shfl_sync(0xffffffffu, f, 8 * tig + 4);
  }

  // One page of this warp's head: kb, vb the codes, ks, vs the scales (shared
  // memory addresses of the head's tiles), tb the page's first token.
  __device__ __forceinline__ void page(uint32_t kb, uint32_t vb, uint32_t ksb, uint32_t vsb, int tb, int L, int min_lim,
                                       int window, int lane) {
    const int gq = lane >> 2, tig = lane & 3;
    float S[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) S[n][0] = S[n][1] = S[n][2] = S[n][3] = 0.f;
    const int r0 = slot_of<D>(gq);
    // ---- S^T = K Q^T
    {
      uint32_t c0[GG::LW], c1[GG::LW], s0, s1;   // codes and scales of keys r0 and r0 + 8
      if constexpr (D == 128) {
        const uint4 a = lds128(kb + code_off<D>(r0, 16 * tig)), b = lds128(kb + code_off<D>(r0 + 8, 16 * tig));
        c0[0] = a.x; c0[1] = a.y; c0[2] = a.z; c0[3] = a.w;
        c1[0] = b.x; c1[1] = b.y; c1[2] = b.z; c1[3] = b.w;
        s0 = e4m3x2_to_f16x2(lds16(ksb + r0 * 8 + 2 * tig));
        s1 = e4m3x2_to_f16x2(lds16(ksb + (r0 + 8) * 8 + 2 * tig));
      } else {
        const uint2 a = lds64(kb + code_off<D>(r0, 8 * tig)), b = lds64(kb + code_off<D>(r0 + 8, 8 * tig));
        c0[0] = a.x; c0[1] = a.y;
        c1[0] = b.x; c1[1] = b.y;
        s0 = e4m3x2_to_f16x2(lds8(ksb + r0 * 4 + tig));
        s1 = e4m3x2_to_f16x2(lds8(ksb + (r0 + 8) * 4 + tig));
      }
#pragma unroll
      for (int j = 0; j < GG::LW; ++j) {
        const uint32_t sel = j < 2 ? 0x1010u : 0x3232u;   // the group of these 8 features
        const uint32_t t0 = prmt(s0, 0u, sel), t1 = prmt(s1, 0u, sel);
        uint32_t h0[4], h1[4];
        e2m1x8_to_f16(c0[j], h0);
        e2m1x8_to_f16(c1[j], h1);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          h0[u] = hmul2(h0[u], t0);
          h1[u] = hmul2(h1[u], t1);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const uint32_t a[4] = {h0[2 * u], h1[2 * u], h0[2 * u + 1], h1[2 * u + 1]};
#pragma unroll
          for (int n = 0; n < NT; ++n) mma_f16(S[n], a, Qf[2 * j + u][n][0], Qf[2 * j + u][n][1]);
        }
      }
    }
    // ---- softmax weights.  S[n]: (key r0, rows e), (key r0 + 8, rows e).
    const bool edge = tb + kPage - 1 > min_lim || (window > 0 && tb < L - window);
    uint32_t hidden = 0u;             // bit 4 n + 2 h + e: key r0 + 8 h is not seen by row (n, e)
    if (edge) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int tok = tb + r0 + 8 * h;
            if (tok > lim[n][e] || (window > 0 && tok <= lim[n][e] - window)) hidden |= 1u << (4 * n + 2 * h + e);
          }
    }
    float x[NT][4];
    float top = -INFINITY;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float base = m[n][k & 1] == -INFINITY ? 0.f : m[n][k & 1];
        x[n][k] = fmaf(S[n][k], fac[n][k & 1], -base);
        if (hidden >> (4 * n + k) & 1u) x[n][k] = -INFINITY;
        // scores above an unset maximum count from -inf: any of them moves it
        top = fmaxf(top, m[n][k & 1] == -INFINITY && x[n][k] != -INFINITY ? INFINITY : x[n][k]);
      }
    }
    if (__any_sync(0xffffffffu, top > 8.f)) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float a = hidden >> (4 * n + e) & 1u ? -INFINITY : S[n][e] * fac[n][e];
          const float b = hidden >> (4 * n + 2 + e) & 1u ? -INFINITY : S[n][2 + e] * fac[n][e];
          float mx = fmaxf(a, b);
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
          const float mn = fmaxf(m[n][e], mx);
          const float base = mn == -INFINITY ? 0.f : mn;
          const float al = fast_exp2(m[n][e] - base);
          m[n][e] = mn;
          l[n][e] *= al;
#pragma unroll
          for (int i = 0; i < GG::KS; ++i) {
            O[i][n][e] *= al;
            O[i][n][2 + e] *= al;
          }
          x[n][e] = a - base;
          x[n][2 + e] = b - base;
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
    const int v0 = slot_of<D>(2 * tig), v1 = slot_of<D>(2 * tig + 1);
    const int rows[4] = {v0, v1, v0 + 8, v1 + 8};
    const int grp = D == 128 ? gq : gq >> 1;
    uint32_t sc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) sc[k] = lds8(vsb + rows[k] * GG::SROW + grp);
    if (edge) {
      // Keys that no row sees take scale 0, so that nothing they hold meets
      // P = 0.  A NaN scale of a key that only some rows see is set aside: its
      // value is 0 here, and NaN is added to the rows that do see it.
      bool bad = false;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tok = tb + rows[k];
        if (tok >= L) sc[k] = 0u;
        else if ((sc[k] & 0x7Fu) == 0x7Fu) {
          bad = true;
          sc[k] = 0u;
        }
      }
      if (__any_sync(0xffffffffu, bad)) {
        for (int s = 0; s < kPage; ++s) {
          const int tok = tb + s;
          if (tok >= L || (lds8(vsb + s * GG::SROW + grp) & 0x7Fu) != 0x7Fu) continue;
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (tok <= lim[n][e] && !(window > 0 && tok <= lim[n][e] - window)) {
#pragma unroll
                for (int i = 0; i < GG::KS; ++i) {
                  O[i][n][e] = __uint_as_float(0x7FC00000u);
                  O[i][n][2 + e] = __uint_as_float(0x7FC00000u);
                }
              }
        }
      }
    }
    const uint32_t sa = e4m3x2_to_f16x2(sc[0] | (sc[1] << 8)), sb = e4m3x2_to_f16x2(sc[2] | (sc[3] << 8));
    constexpr int VW = D / 64;        // words of codes a lane reads of each key
    uint32_t w[4][VW];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (D == 128) {
        const uint2 v = lds64(vb + code_off<D>(rows[k], 8 * gq));
        w[k][0] = v.x;
        w[k][1] = v.y;
      } else {
        w[k][0] = lds32(vb + code_off<D>(rows[k], 4 * gq));
      }
    }
#pragma unroll
    for (int j = 0; j < VW; ++j) {
      uint32_t a0[4], a1[4], a2[4], a3[4];
      // even features of two keys side by side, then odd features
      e2m1x8_to_f16(bitsel(w[0][j], w[1][j] << 4, 0x0F0F0F0Fu), a0);
      e2m1x8_to_f16(bitsel(w[0][j] >> 4, w[1][j], 0x0F0F0F0Fu), a1);
      e2m1x8_to_f16(bitsel(w[2][j], w[3][j] << 4, 0x0F0F0F0Fu), a2);
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

template <int D, int NT, bool WINDOW, int MINB>
__global__ void __launch_bounds__(32 * (1 + kQ4MaxWarps), MINB)
    pa_split_q4_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const __grid_constant__ SplitQ4Params p) {
  using GG = GeoQ4<D>;
  const int window = WINDOW ? p.window : 0;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_scan[1 + kQ4MaxWarps];
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
  auto got_bar = [&](int t) { return bar0 + 8u * (2 * nstage + kQ4MaxWarps + t); };
  if (tid == 0) {
    prefetch_tensormap(&tmap_k);
    prefetch_tensormap(&tmap_v);
    for (int s = 0; s < nstage; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), ncw);
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
  Cursor cu = locate(s_pre, B, NC, start);
  int stage = 0;
  uint32_t round = 0;
  const uint32_t code_page = static_cast<uint32_t>(HC * GG::TILE), scale_page = static_cast<uint32_t>(HC * GG::STILE);

  if (warp == 0) {
    // ============================ producer =================================
    // block-table entries [wj, wj + 32) of sequence wi, one a lane; the entries
    // needed after them (ni, nj) are loaded ahead
    int wi = -1, wj = 0, wval = 0, ni = -1, nj = 0, nval = 0;
    auto window_of = [&](int i, int j) {
      const int jj = j + lane;
      const int js = first_visible_page(s_len[i], s_qsl[i + 1] - s_qsl[i], window);
      return jj < pages_of(s_pre, i) ? p.block_tables[static_cast<int64_t>(i) * p.bt_stride + js + jj] : 0;
    };
    while (left > 0) {
      const SegmentQ4 sg = segment_at(cu, left);
      left -= sg.j1 - sg.j0;
      next_unit(cu, s_pre, B, NC);
      for (int jb = sg.j0; jb < sg.j1; jb += BP) {
        if (wi != sg.i || jb < wj || jb + BP > wj + 32) {
          wval = ni == sg.i && nj == jb ? nval : window_of(sg.i, jb);
          wi = sg.i;
          wj = jb;
          ni = -1;
          if (jb + 32 < sg.j1) {
            ni = sg.i;
            nj = jb + 32;
          } else if (left > 0) {
            ni = cu.i;
            nj = 0;
          }
          if (ni >= 0) nval = window_of(ni, nj);
        }
        const int np = min(BP, sg.j1 - jb);
        if (round > 0 && !mbar_wait(empty_bar(stage), (round - 1) & 1u, p.wait_ns)) {
          if (lane == 0) atomicOr(p.err, kErrTimeout);
          return;
        }
        if (lane == 0)
          mbar_arrive_expect_tx(full_bar(stage), static_cast<uint32_t>(np) * 2u * (code_page + scale_page));
        __syncwarp();
        const uint32_t st = base + p.off_stage + static_cast<uint32_t>(stage) * p.stage_bytes;
        for (int k0 = 0; k0 < 4 * BP; k0 += 32) {      // four copies a page, one a lane
          const int k = k0 + lane, pg = k >> 2;
          const int phys0 = __shfl_sync(0xffffffffu, wval, (jb - wj + pg) & 31);
          if (pg >= np) continue;
          const bool bad = phys0 < 0 || phys0 >= p.num_pages;
          if (bad && (k & 3) == 0) atomicOr(p.err, kErrPageRange);
          switch (k & 3) {     // an out-of-range page reads as zero codes (TMA fill) and page 0's scales
            case 0: tma_load_4d(st + pg * code_page, &tmap_k, 0, 0, sg.c * HC, phys0, full_bar(stage)); break;
            case 1: tma_load_4d(st + p.off_v + pg * code_page, &tmap_v, 0, 0, sg.c * HC, phys0, full_bar(stage)); break;
            case 2:
              bulk_load(st + p.off_ks + pg * scale_page,
                        p.k_sc + (bad ? 0 : phys0) * p.k_sc_page + static_cast<int64_t>(sg.c) * scale_page, scale_page,
                        full_bar(stage));
              break;
            default:
              bulk_load(st + p.off_vs + pg * scale_page,
                        p.v_sc + (bad ? 0 : phys0) * p.v_sc_page + static_cast<int64_t>(sg.c) * scale_page, scale_page,
                        full_bar(stage));
          }
        }
        if (++stage == nstage) {
          stage = 0;
          ++round;
        }
      }
    }
    return;
  }

  // ============================== consumers ================================
  const int cw = warp - 1;
  if (cw >= ncw) return;
  const int team = cw % (HC * MT), kw = cw / (HC * MT);
  const int hh = team / MT, wt = team - hh * MT;
  const int gq = lane >> 2, tig = lane & 3;
  const int G = p.G, row0 = 8 * NT * wt;
  StateQ4<D, NT> cs;
  bool first = true;
  uint32_t seg_no = 0;
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
            cs.m[n][e] = p.sinks[hq_base + r2 % G] * 1.4426950408889634f;
            cs.l[n][e] = gq == 0 ? 1.f : 0.f;
          }
        }
      }
    }
    for (int jb = sg.j0; jb < sg.j1; jb += BP) {
      if (!mbar_wait(full_bar(stage), round & 1u, p.wait_ns)) {
        if (lane == 0) atomicOr(p.err, kErrTimeout);
        return;
      }
      if (active) {
        const uint32_t st = base + p.off_stage + static_cast<uint32_t>(stage) * p.stage_bytes;
        const int np = min(BP, sg.j1 - jb);
        for (int pg = kw; pg < np; pg += KW) {
          const uint32_t co = st + pg * code_page + static_cast<uint32_t>(hh * GG::TILE);
          const uint32_t so = st + pg * scale_page + static_cast<uint32_t>(hh * GG::STILE);
          cs.page(co, co + p.off_v, so + p.off_ks, so + p.off_vs, kPage * (si.js + jb + pg), si.L, min_lim, window,
                  lane);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty_bar(stage));
      if (++stage == nstage) {
        stage = 0;
        ++round;
      }
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
    if (KW == 1) {
      if (!active) continue;
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
            if (gq == 0) p.ws_ml[ws_row + rl] = make_float2(lt != lt && mm == -INFINITY ? 0.f : mm, lt);
          }
        }
      continue;
    }
    // KW warps of a team meet: each leaves its rows in shared memory, then
    // combines its share of the features of all of them.
    constexpr int PITCH = D + 4;                                  // floats between rows
    constexpr int WROWS = 8 * NT;
    constexpr uint32_t WARP_BYTES = WROWS * PITCH * 4 + WROWS * 8;
    float* const xo = reinterpret_cast<float*>(gbase + p.off_xchg + cw * WARP_BYTES);
    float2* const xml = reinterpret_cast<float2*>(gbase + p.off_xchg + cw * WARP_BYTES + WROWS * PITCH * 4);
    if (seg_no > 0 && !mbar_wait(got_bar(team), (seg_no - 1) & 1u, p.wait_ns)) {
      if (lane == 0) atomicOr(p.err, kErrTimeout);
      return;
    }
    if (active) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rl = 8 * n + 2 * tig + e;
          float* o = xo + rl * PITCH + FPL * gq;
#pragma unroll
          for (int i = 0; i < GG::KS; i += 2)
            *reinterpret_cast<float4*>(o + 2 * i) =
                make_float4(cs.O[i][n][e], cs.O[i][n][2 + e], cs.O[i + 1][n][e], cs.O[i + 1][n][2 + e]);
          if (gq == 0) xml[rl] = make_float2(cs.m[n][e], cs.l[n][e]);
        }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(put_bar(team));
    if (!mbar_wait(put_bar(team), seg_no & 1u, p.wait_ns)) {
      if (lane == 0) atomicOr(p.err, kErrTimeout);
      return;
    }
    if (active) {
      const int per = D / 4 / KW;                                 // float4 columns of this warp's share
      for (int x = lane; x < WROWS * per; x += 32) {
        const int rl = x / per, col = kw * per + x - rl * per, rho = row0 + rl;
        if (rho >= R) continue;
        float mx = -INFINITY, lt = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < KW; ++k)
          mx = fmaxf(mx, reinterpret_cast<const float2*>(gbase + p.off_xchg + (team + k * HC * MT) * WARP_BYTES +
                                                         WROWS * PITCH * 4)[rl].x);
        const float b0 = mx == -INFINITY ? 0.f : mx;
        for (int k = 0; k < KW; ++k) {
          const uint8_t* from = gbase + p.off_xchg + (team + k * HC * MT) * WARP_BYTES;
          const float2 ml = reinterpret_cast<const float2*>(from + WROWS * PITCH * 4)[rl];
          const float4 v = reinterpret_cast<const float4*>(from + rl * PITCH * 4)[col];
          const float a = ml.x == mx && mx != -INFINITY ? 1.f : fast_exp2(ml.x - b0);
          lt += a * ml.y;
          acc.x += a * v.x;
          acc.y += a * v.y;
          acc.z += a * v.z;
          acc.w += a * v.w;
        }
        if (complete) {
          const int t = si.t0 + rho / G, hq = hq_base + rho % G;
          const float inv = lt == 0.f ? 0.f : p.v_scale / lt;
          *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(t) * p.out_stride_t +
                                    static_cast<int64_t>(hq) * p.out_stride_h + 4 * col) =
              make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
          if (p.lse != nullptr && col == 0)
            p.lse[static_cast<int64_t>(t) * p.lse_stride_t + static_cast<int64_t>(hq) * p.lse_stride_h] =
                lt == 0.f ? -INFINITY : (mx + fast_log2(lt)) * 0.69314718055994530942f;
        } else {
          *reinterpret_cast<float4*>(p.ws_o + (ws_row + rl) * D + 4 * col) = acc;
          if (col == 0) p.ws_ml[ws_row + rl] = make_float2(lt != lt && mx == -INFINITY ? 0.f : mx, lt);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(got_bar(team));
    ++seg_no;
  }
}

namespace {

template <int D, int NT, int MINB>
cudaError_t launch_nt(cudaLaunchConfig_t* cfg, const CUtensorMap& tk, const CUtensorMap& tv, const SplitQ4Params& p) {
  return p.window > 0 ? cudaLaunchKernelEx(cfg, pa_split_q4_kernel<D, NT, true, MINB>, tk, tv, p)
                      : cudaLaunchKernelEx(cfg, pa_split_q4_kernel<D, NT, false, MINB>, tk, tv, p);
}

template <int D>
cudaError_t launch_d(cudaLaunchConfig_t* cfg, int nt, const CUtensorMap& tk, const CUtensorMap& tv,
                     const SplitQ4Params& p) {
  if (nt == 1) return launch_nt<D, 1, 2>(cfg, tk, tv, p);
  if (nt == 2) return launch_nt<D, 2, 1>(cfg, tk, tv, p);
  if (nt == 4) return launch_nt<D, 4, 1>(cfg, tk, tv, p);
  return cudaErrorInvalidValue;
}

template <int D, int NT, int MINB>
cudaError_t limit_nt(int smem) {
  cudaError_t e = cudaFuncSetAttribute(pa_split_q4_kernel<D, NT, false, MINB>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(pa_split_q4_kernel<D, NT, true, MINB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              smem);
}

}  // namespace

cudaError_t launch_split_q4(int head_dim, int nt, const CUtensorMap& tk, const CUtensorMap& tv, const SplitQ4Params& p,
                            int grid, int threads, int smem, bool pdl, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
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
  if ((e = limit_nt<128, 1, 2>(smem)) || (e = limit_nt<128, 2, 1>(smem)) || (e = limit_nt<128, 4, 1>(smem)) ||
      (e = limit_nt<64, 1, 2>(smem)) || (e = limit_nt<64, 2, 1>(smem)) || (e = limit_nt<64, 4, 1>(smem)))
    return e;
  return cudaSuccess;
}

}  // namespace pa
