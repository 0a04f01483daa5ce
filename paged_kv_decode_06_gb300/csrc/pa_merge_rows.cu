// Log-sum-exp merge of the walks with a hole (windows with first tokens, sequences behind
// a shared prefix).  A row's pieces are those that the split kernel left, as in
// pa_merge.cu, and, for a shared prefix, those of its tile in the prefix kernel:
//   out = v_scale * sum_s 2^(m_s - M) O_s / sum_s 2^(m_s - M) l_s
//   lse = ln 2 * (M + log2 sum_s 2^(m_s - M) l_s),   M = max_s m_s.
// A NaN in a piece stays in the row.  Bound by the latency of a row's few loads: a lane
// group of D / 4 lanes takes a piece, and the loads of four pieces are in flight.
#include "pa_device.cuh"
#include "pa_kernels.h"
#include "pa_shared.h"
#include "pa_split.cuh"

namespace pa {
namespace {

constexpr int kRowThreads = 256;

__device__ __forceinline__ void acc_piece(float& mx, float& l, float4& acc, float2 ml, const float4& o) {
  // a piece without a visible key has weight 0; one whose scores are all NaN has m = -inf too
  if (ml.x == -INFINITY && ml.y == 0.f) return;
  const float nm = fmaxf(mx, ml.x);
  const float base = nm == -INFINITY ? 0.f : nm;
  const float a = fast_exp2(mx - base);
  const float b = fast_exp2(ml.x - base);
  acc.x = acc.x * a + o.x * b;
  acc.y = acc.y * a + o.y * b;
  acc.z = acc.z * a + o.z * b;
  acc.w = acc.w * a + o.w * b;
  l = l * a + ml.y * b;
  mx = nm;
}

// A row's pieces of a shared prefix: its tile's in every CTA that has some (both slots' of a
// single tile).
struct PrePieces {
  int64_t row0;             // padded rows before the tile in the first CTA
  int count, single, second;
  int rho, rows;            // the row in its tile, the tile's rows
  __device__ __forceinline__ void start(const SharedGroup& sg, const SharedTotals& all, int h, int rg) {
    const int pair = rg / kSharedPair;
    single = shared_single(sg, pair);
    const int slot = single ? 0 : rg % kSharedPair / kSharedTile;
    second = single ? sg.last_rows : slot * kSharedTile;      // (rows of the first slot's tile)
    rho = rg % kSharedTile;
    rows = shared_tile_rows(sg, pair, slot);
    const int64_t a = sg.step0 + static_cast<int64_t>(h) * sg.steps_head + static_cast<int64_t>(pair) * sg.blocks;
    const int c0 = shared_cta_of(a, all.steps, all.ctas);
    const int c1 = shared_cta_of(a + shared_steps(sg, pair) - 1, all.steps, all.ctas);
    count = (c1 - c0 + 1) << single;
    row0 = sg.row0 + static_cast<int64_t>(h) * sg.rows_head + static_cast<int64_t>(pair + c0) * kSharedPair;
  }
  // The tile of partial rows of piece k.
  __device__ __forceinline__ int64_t tile(int k) const {
    return row0 + static_cast<int64_t>(k >> single) * kSharedPair + (!single || (k & 1) ? second : 0);
  }
};

// TPR threads a row (32: a warp; else the block).
template <int D, Walk WALK, int TPR>
__global__ void __launch_bounds__(kRowThreads) pa_merge_rows_kernel(const MergeRowsParams p) {
  constexpr int LPD = D / 4;             // lanes of a piece
  constexpr int PG = TPR / LPD;          // pieces side by side
  constexpr bool kShared = WALK == Walk::kOwn;
  grid_dependency_wait();
  grid_launch_dependents();
  if (kShared && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *p.ready = 0;   // (a graph's next replay has the same number)
  const int lane = threadIdx.x % TPR;
  const int row = TPR == 32 ? blockIdx.y * (kRowThreads / 32) + threadIdx.x / 32 : blockIdx.y;
  const int u = blockIdx.x;
  const int i = u / p.NC, c = u - i * p.NC;
  const int hh = row / p.R_max, rho = row - hh * p.R_max;
  if (row >= p.HC * p.R_max) return;
  // (row-uniform branches: a row is a group of warps or the block)
  // what does not depend on another load, in one go
  const int t0 = p.qsl != nullptr ? p.qsl[i] : i, qn = p.qsl != nullptr ? p.qsl[i + 1] - t0 : 1;
  const int L = p.seq_lens[i], skip = kShared ? p.skip[i] : 0, g = kShared ? p.seq_group[i] : -1;
  const int4 d = p.ws_unit[u];
  SharedTotals totals = {};
  if constexpr (kShared) totals = *p.totals;
  if (qn < 1 || qn > p.max_qlen || t0 < 0 || t0 > p.num_tokens - qn || rho >= p.G * qn) return;
  const int t = t0 + rho / p.G, h = c * p.HC + hh, hq = h * p.G + rho % p.G;
  const View view = view_of<WALK>(p, L, qn, skip);
  int gf = 0, nparts = 0, tail = 0;
  if (view.n > 0) {
    gf = d.x;
    nparts = d.y & 0x3fffffff;
    tail = (d.y >> 30) & 1;
    // a descriptor that this call's split kernel did not write (its CTA gave up on a
    // timed-out wait) may hold anything
    if (gf < 0 || nparts < 1 || nparts > p.split_grid - gf) return;
    if (!kShared && nparts == 1) return;             // finished by its CTA
  }
  const int dq = lane % LPD, pg = lane / LPD;
  PrePieces pre = {};
  if constexpr (kShared) {
    if (g >= 0) {
      const SharedGroup sg = p.groups[g];
      pre.start(sg, totals, h, (t - sg.t0) * p.G + rho % p.G);
    }
  }
  float mx = -INFINITY, l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  const int total = nparts + (kShared ? pre.count : 0);
  for (int s0 = pg; s0 < total; s0 += 4 * PG) {
    float2 ml[4];
    float4 o[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int s = s0 + k * PG;
      ml[k] = make_float2(-INFINITY, 0.f);
      o[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (s >= total) continue;
      if (s < nparts) {
        int64_t at = (static_cast<int64_t>(2 * (gf + s) + (s == 0 && tail ? 1 : 0)) * p.HC + hh) * p.R_max + rho;
        if (kShared && nparts == 1) at = p.whole_row0 + static_cast<int64_t>(t) * p.Hq + hq;
        ml[k] = p.ws_ml[at];
        o[k] = *reinterpret_cast<const float4*>(p.ws_o + at * D + 4 * dq);
      } else {
        // (a tile of partial rows holds chunk dq of all its rows side by side)
        const int64_t tile = pre.tile(s - nparts);
        ml[k] = p.pre_ml[tile + pre.rho];
        o[k] = *reinterpret_cast<const float4*>(p.pre_o + tile * D + 4 * (static_cast<int64_t>(dq) * pre.rows + pre.rho));
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) acc_piece(mx, l, acc, ml[k], o[k]);
  }
  if constexpr (TPR == 32) {
#pragma unroll
    for (int d = LPD; d < 32; d <<= 1) {
      float2 m2;
      float4 o2;
      m2.x = __shfl_xor_sync(0xffffffffu, mx, d);
      m2.y = __shfl_xor_sync(0xffffffffu, l, d);
      o2.x = __shfl_xor_sync(0xffffffffu, acc.x, d);
      o2.y = __shfl_xor_sync(0xffffffffu, acc.y, d);
      o2.z = __shfl_xor_sync(0xffffffffu, acc.z, d);
      o2.w = __shfl_xor_sync(0xffffffffu, acc.w, d);
      acc_piece(mx, l, acc, m2, o2);
    }
  } else {
    __shared__ float4 s_o[PG][LPD];
    __shared__ float2 s_ml[PG][LPD];
#pragma unroll
    for (int half = PG / 2; half >= 1; half >>= 1) {
      if (pg >= half && pg < 2 * half) {
        s_o[pg][dq] = acc;
        s_ml[pg][dq] = make_float2(mx, l);
      }
      __syncthreads();
      if (pg < half) acc_piece(mx, l, acc, s_ml[pg + half][dq], s_o[pg + half][dq]);
    }
  }
  if (pg != 0) return;
  float lse;
  float inv = 0.f;
  if (total == 0) {
    // no page to read: an empty context; the sink alone is left
    const float sink = p.sinks != nullptr ? p.sinks[hq] : -INFINITY;
    lse = sink;
    acc.x = acc.y = acc.z = acc.w = inv = sink != sink ? sink : 0.f;
    if (lane == 0) atomicOr(p.err, kErrSeqLen);
  } else {
    inv = l > 0.f ? p.v_scale / l : (l != l ? l : 0.f);
    lse = l > 0.f || l != l ? (mx + fast_log2(l)) * 0.69314718055994530942f : -INFINITY;
  }
  uint2 pk;
  pk.x = pack_bf16(acc.x * inv, acc.y * inv);
  pk.y = pack_bf16(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(t) * p.out_stride_t +
                            static_cast<int64_t>(hq) * p.out_stride_h + 4 * dq) = pk;
  if (lane == 0 && p.lse != nullptr)
    p.lse[static_cast<int64_t>(t) * p.lse_stride_t + static_cast<int64_t>(hq) * p.lse_stride_h] = lse;
}

template <int D, Walk WALK>
cudaError_t launch_form(const cudaLaunchConfig_t& cfg, const MergeRowsParams& p, bool wide) {
  return wide ? cudaLaunchKernelEx(&cfg, pa_merge_rows_kernel<D, WALK, kRowThreads>, p)
              : cudaLaunchKernelEx(&cfg, pa_merge_rows_kernel<D, WALK, 32>, p);
}

}  // namespace

cudaError_t launch_merge_rows(int head_dim, bool shared, const MergeRowsParams& p, int units, int rows, bool wide,
                              bool pdl, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units), static_cast<unsigned>(wide ? rows : (rows + 7) / 8), 1);
  cfg.blockDim = dim3(kRowThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  if (head_dim == 128)
    return shared ? launch_form<128, Walk::kOwn>(cfg, p, wide) : launch_form<128, Walk::kFirst>(cfg, p, wide);
  if (head_dim == 64)
    return shared ? launch_form<64, Walk::kOwn>(cfg, p, wide) : launch_form<64, Walk::kFirst>(cfg, p, wide);
  return cudaErrorInvalidValue;
}

}  // namespace pa
