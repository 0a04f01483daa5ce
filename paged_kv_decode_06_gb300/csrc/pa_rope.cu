// Rotary positions with several axes, fused with the KV-cache write (ATOM
// model-operations guide, "KV cache operations": fused_qk_rope_reshape_and_cache;
// the multi-axis form of vision-language models).  Pair i of a row's rotated
// features (x, y) has an axis a_i; with c, s the cosine and sine of row
// positions[a_i][t] of the caller's table,
//
//     x' = x c - y s        y' = y c + x s
//
// every product, difference and sum rounded to fp32 (no FMA, so the codes of an fp8
// cache do not depend on how a compiler contracts), one rounding to bf16 or e4m3 at
// the end.  The query's rows are written out, the key's to their cache slots (and
// out, where the caller asks), the value's to theirs.
//
// A thread takes one chunk of 2 W features of a head (W pairs, or 2 W features that
// do not rotate) for one or more heads of a token: the angles are loaded once for
// all of them.  Bound by memory: 16384 tokens of 32 / 8 heads of 128, fp8 cache, 378 MB,
// take 64 us in a graph, 87 % of the rate of a copy (bf16 cache, 411 MB, 62 us, 98 %).
#include <algorithm>
#include <cmath>

#include "pa_host.h"
#include "pa_kernels.h"
#include "pa_pack.cuh"
#include "pa_quant.cuh"

namespace pa {
namespace {

constexpr int kMaxAxes = 3;
constexpr int kThreads = 256;
constexpr int kMaxHeadDim = 512;
// Heads of a thread on the way.  With four CTAs an SM three are enough (16384 tokens, fp8: 64.2
// us, 64.4 with four; with three CTAs 67.2 for three, 66.7 for four).
constexpr int kDepth = 3;

struct RopeParams {
  const uint16_t *query, *key, *value;
  int64_t q_t, q_h, k_t, k_h, v_t, v_h;        // strides, elements
  uint16_t *query_out, *key_out;               // key_out may be nullptr
  int64_t qo_t, qo_h, ko_t, ko_h;
  const int32_t* positions;                    // [axes][T]
  int64_t pos_stride;
  const float* table;                          // [rows][rot]: cosines, then sines
  int64_t table_stride;
  const int32_t* slots;
  uint8_t *k_cache, *v_cache;
  int64_t kc_page, kc_slot, kc_head, vc_page, vc_slot, vc_head;   // elements
  int32_t tokens, axes, rows, rot, hq, hkv, chunks, groups;       // chunks a head, head groups a token
  int32_t neighbours;
  int64_t num_slots;
  float k_scale, v_scale;
  uint32_t* err;
  uint32_t axis[kMaxHeadDim / 2 / 16];         // two bits a pair
};

__device__ __forceinline__ int axis_of(const RopeParams& p, int pair) {
  return (p.axis[pair >> 4] >> (2 * (pair & 15))) & 3;
}

// N = 8 or 2 consecutive bf16 values, 16 or 4 bytes.
template <int N>
struct Raw;
template <>
struct Raw<8> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = bf16_lo(w[e]);
      f[2 * e + 1] = bf16_hi(w[e]);
    }
  }
};
template <>
struct Raw<2> {
  uint32_t v;
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ void get(float (&f)[2]) const {
    f[0] = bf16_lo(v);
    f[1] = bf16_hi(v);
  }
};

// N bytes (16 or 4) of global memory on their way to shared memory.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int N>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float (&f)[N]) {
  if constexpr (N == 8)
    *reinterpret_cast<uint4*>(p) =
        make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  else
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(f[0], f[1]);
}

template <int N>
__device__ __forceinline__ void store_fp8(uint8_t* p, const float (&f)[N], const ScaleDiv& d) {
  uint32_t c[N / 2];
#pragma unroll
  for (int e = 0; e < N / 2; ++e) {
    float lo, hi;
    if (d.fast) {
      div_by2(d, f[2 * e], f[2 * e + 1], lo, hi);
    } else {
      lo = __fdiv_rn(f[2 * e], d.s);
      hi = __fdiv_rn(f[2 * e + 1], d.s);
    }
    c[e] = e4m3x2_from_f32(lo, hi);
  }
  if constexpr (N == 8)
    *reinterpret_cast<uint2*>(p) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
  else
    *reinterpret_cast<uint16_t*>(p) = static_cast<uint16_t>(c[0]);
}

// W pairs a chunk (two runs of W features: 16-byte accesses for W = 8, 4-byte ones for
// W = 2).  RING: a thread takes several heads of its token and keeps kDepth of them on the
// way, in shared memory of its own (asynchronous copies need no registers); else one.
template <int W, bool RING, bool FP8>
__global__ void __launch_bounds__(kThreads, RING ? 4 : 1) pa_rope_write_kernel(const RopeParams p) {
  const uint64_t per_token = static_cast<uint64_t>(p.chunks) * p.groups;
  const uint64_t x = static_cast<uint64_t>(blockIdx.x) * kThreads + threadIdx.x;
  grid_dependency_wait();
  grid_launch_dependents();
  if (x >= per_token * static_cast<uint64_t>(p.tokens)) return;
  const int t = static_cast<int>(x >> 32 ? x / per_token : static_cast<uint32_t>(x) / static_cast<uint32_t>(per_token));
  const uint32_t rem = static_cast<uint32_t>(x - static_cast<uint64_t>(t) * per_token);
  const int hg = static_cast<int>(rem / static_cast<uint32_t>(p.chunks));
  const int c = static_cast<int>(rem) - hg * p.chunks;
  const int half = p.rot / 2, turning = half / W;          // chunks that rotate
  const bool turn = c < turning;
  // the two runs of W features
  const int f0 = turn ? (p.neighbours ? 2 * W * c : W * c) : p.rot + 2 * W * (c - turning);
  const int f1 = turn && !p.neighbours ? half + W * c : f0 + W;
  const int heads = p.hq + 2 * p.hkv;

  // the two runs of a head
  auto runs_of = [&](int h, const uint16_t*& r0, const uint16_t*& r1) {
    const uint16_t* row;
    if (h < p.hq) row = p.query + t * p.q_t + h * p.q_h;
    else if (h < p.hq + p.hkv) row = p.key + t * p.k_t + (h - p.hq) * p.k_h;
    else row = p.value + t * p.v_t + (h - p.hq - p.hkv) * p.v_h;
    const bool plain = h >= p.hq + p.hkv;                 // a value's chunk: 2 W features in a row
    r0 = row + (plain ? 2 * W * c : f0);
    r1 = row + (plain ? 2 * W * c + W : f1);
  };
  __shared__ Raw<W> ring[RING ? 2 * kDepth : 1][RING ? kThreads : 1];
  Raw<W> a, b;
  const uint16_t *r0, *r1;
  auto start = [&](int h, int stage) {
    if (h < heads) {
      runs_of(h, r0, r1);
      cp_async<2 * W>(smem_addr(&ring[2 * stage][threadIdx.x]), r0);
      cp_async<2 * W>(smem_addr(&ring[2 * stage + 1][threadIdx.x]), r1);
    }
    cp_async_commit();
  };
  if constexpr (RING) {
#pragma unroll
    for (int s = 0; s < kDepth; ++s) start(hg + s * p.groups, s);
  } else {
    runs_of(hg, r0, r1);
    a.load(r0);
    b.load(r1);
  }
  const int slot = p.slots[t];
  int pos[kMaxAxes];
  bool fine = true;
#pragma unroll
  for (int k = 0; k < kMaxAxes; ++k) {
    pos[k] = k < p.axes ? p.positions[k * p.pos_stride + t] : 0;
    fine &= pos[k] >= 0 && pos[k] < p.rows;
  }
  if (!fine) {
    if (rem == 0) atomicOr(p.err, kErrPosition);
    if (RING) cp_async_wait<0>();
    return;
  }
  const bool bad_slot = slot >= p.num_slots;
  if (bad_slot && rem == 0) atomicOr(p.err, kErrPageRange);
  const bool live = slot >= 0 && !bad_slot;
  float co[W], si[W];
  if (turn) {
    const int ax = axis_of(p, W * c);
    bool same = true;
#pragma unroll
    for (int i = 1; i < W; ++i) same &= axis_of(p, W * c + i) == ax;
    if (same && W == 8) {
      const float* r = p.table + static_cast<int64_t>(ax == 0 ? pos[0] : ax == 1 ? pos[1] : pos[2]) * p.table_stride + W * c;
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(r + i), w = *reinterpret_cast<const float4*>(r + half + i);
        co[i] = v.x; co[i + 1] = v.y; co[i + 2] = v.z; co[i + 3] = v.w;
        si[i] = w.x; si[i + 1] = w.y; si[i + 2] = w.z; si[i + 3] = w.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const int k = axis_of(p, W * c + i);
        const float* r = p.table + static_cast<int64_t>(k == 0 ? pos[0] : k == 1 ? pos[1] : pos[2]) * p.table_stride + W * c + i;
        co[i] = r[0];
        si[i] = r[half];
      }
    }
  }
  const ScaleDiv dk = scale_div(p.k_scale), dv = scale_div(p.v_scale);
  const int64_t page = live ? slot / kPage : 0, off = live ? slot % kPage : 0;
  auto finish = [&](int h, const Raw<W>& ra, const Raw<W>& rb) {
    float va[W], vb[W];
    ra.get(va);
    rb.get(vb);
    const bool is_value = h >= p.hq + p.hkv;
    if (turn && !is_value) {
      if (p.neighbours) {
        // features 2 i, 2 i + 1 of the chunk's 2 W are pair i
#pragma unroll
        for (int i = 0; i < W / 2; ++i) {
          const float x0 = va[2 * i], y0 = va[2 * i + 1], x1 = vb[2 * i], y1 = vb[2 * i + 1];
          const float c0 = co[i], s0 = si[i], c1 = co[W / 2 + i], s1 = si[W / 2 + i];
          va[2 * i] = __fsub_rn(__fmul_rn(x0, c0), __fmul_rn(y0, s0));
          va[2 * i + 1] = __fadd_rn(__fmul_rn(y0, c0), __fmul_rn(x0, s0));
          vb[2 * i] = __fsub_rn(__fmul_rn(x1, c1), __fmul_rn(y1, s1));
          vb[2 * i + 1] = __fadd_rn(__fmul_rn(y1, c1), __fmul_rn(x1, s1));
        }
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) {
          const float x0 = va[i], y0 = vb[i];
          va[i] = __fsub_rn(__fmul_rn(x0, co[i]), __fmul_rn(y0, si[i]));
          vb[i] = __fadd_rn(__fmul_rn(y0, co[i]), __fmul_rn(x0, si[i]));
        }
      }
    }
    const int g0 = is_value ? 2 * W * c : f0, g1 = is_value ? 2 * W * c + W : f1;
    if (h < p.hq) {
      uint16_t* row = p.query_out + t * p.qo_t + h * p.qo_h;
      store_bf16<W>(row + g0, va);
      store_bf16<W>(row + g1, vb);
      return;
    }
    const int kh = is_value ? h - p.hq - p.hkv : h - p.hq;
    if (!is_value && p.key_out != nullptr) {
      uint16_t* row = p.key_out + t * p.ko_t + kh * p.ko_h;
      store_bf16<W>(row + g0, va);
      store_bf16<W>(row + g1, vb);
    }
    if (!live) return;
    const int64_t at = is_value ? page * p.vc_page + off * p.vc_slot + kh * p.vc_head
                                : page * p.kc_page + off * p.kc_slot + kh * p.kc_head;
    uint8_t* cache = is_value ? p.v_cache : p.k_cache;
    if constexpr (FP8) {
      const ScaleDiv& d = is_value ? dv : dk;
      store_fp8<W>(cache + at + g0, va, d);
      store_fp8<W>(cache + at + g1, vb, d);
    } else {
      uint16_t* row = reinterpret_cast<uint16_t*>(cache) + at;
      store_bf16<W>(row + g0, va);
      store_bf16<W>(row + g1, vb);
    }
  };
  if constexpr (RING) {
    int stage = 0;
    for (int h = hg; h < heads; h += p.groups) {
      cp_async_wait<kDepth - 1>();
      a = ring[2 * stage][threadIdx.x];
      b = ring[2 * stage + 1][threadIdx.x];
      start(h + kDepth * p.groups, stage);
      finish(h, a, b);
      stage = stage + 1 == kDepth ? 0 : stage + 1;
    }
  } else {
    finish(hg, a, b);
  }
}

template <int W, bool RING>
cudaError_t launch_form(const RopeParams& p, bool fp8, int64_t blocks, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return fp8 ? cudaLaunchKernelEx(&cfg, pa_rope_write_kernel<W, RING, true>, p)
             : cudaLaunchKernelEx(&cfg, pa_rope_write_kernel<W, RING, false>, p);
}

int rope_cache_write(const pa_tensor_t* query, const pa_tensor_t* key, const pa_tensor_t* value,
                     const pa_tensor_t* pos, const pa_tensor_t* table, const uint8_t* pair_axis, int32_t neighbours,
                     const pa_tensor_t* slots, const pa_tensor_t* kc, const pa_tensor_t* vc, float k_scale,
                     float v_scale, const pa_tensor_t* query_out, const pa_tensor_t* key_out, cudaStream_t stream) {
  int st;
  const bool none = query != nullptr && query->ndim == 3 && query->shape[0] == 0;   // no tokens: nothing to do
  if ((st = host_check_tensor(query, "query", 3, none)) || (st = host_check_tensor(key, "key", 3, none)) ||
      (st = host_check_tensor(value, "value", 3, none)) ||
      (st = host_check_tensor(pos, "positions", pos != nullptr && pos->ndim == 1 ? 1 : 2, none)) ||
      (st = host_check_tensor(table, "cos_sin", 2, false)) || (st = host_check_tensor(slots, "slot_mapping", 1, none)) ||
      (st = host_check_tensor(kc, "k_cache", 4, false)) || (st = host_check_tensor(vc, "v_cache", 4, false)) ||
      (st = host_check_tensor(query_out, "query_out", 3, none)) || (st = host_check_tensor(key_out, "key_out", 3, true)))
    return st;
  if (none) return PA_OK;
  if (query->dtype != PA_BF16 || key->dtype != PA_BF16 || value->dtype != PA_BF16 || query_out->dtype != PA_BF16 ||
      (key_out->data && key_out->dtype != PA_BF16))
    return host_fail(PA_ERR_INVALID_ARG, "query, key, value, query_out and key_out must be bf16");
  if (pos->dtype != PA_I32 || slots->dtype != PA_I32)
    return host_fail(PA_ERR_INVALID_ARG, "positions and slot_mapping must be int32");
  if (table->dtype != PA_F32) return host_fail(PA_ERR_INVALID_ARG, "cos_sin must be float32");
  if (kc->dtype != PA_BF16 && kc->dtype != PA_FP8_E4M3)
    return host_fail(PA_ERR_INVALID_ARG, "k_cache must be bf16 or fp8 e4m3");
  if (vc->dtype != kc->dtype) return host_fail(PA_ERR_INVALID_ARG, "v_cache dtype differs from k_cache");
  const int64_t T = query->shape[0], Hq = query->shape[1], D = query->shape[2], Hkv = key->shape[1];
  const int64_t axes = pos->ndim == 1 ? 1 : pos->shape[0], P = table->shape[0], R = table->shape[1];
  const int64_t NB = kc->shape[0];
  if (key->shape[0] != T || key->shape[2] != D)
    return host_fail(PA_ERR_INVALID_ARG, "key must be [T, Hkv, D] with query's T and D");
  for (int d = 0; d < 3; ++d)
    if (value->shape[d] != key->shape[d]) return host_fail(PA_ERR_INVALID_ARG, "value shape differs from key");
  for (int d = 0; d < 3; ++d)
    if (query_out->shape[d] != query->shape[d])
      return host_fail(PA_ERR_INVALID_ARG, "query_out shape differs from query");
  for (int d = 0; d < 3 && key_out->data; ++d)
    if (key_out->shape[d] != key->shape[d]) return host_fail(PA_ERR_INVALID_ARG, "key_out shape differs from key");
  if (axes < 1 || axes > kMaxAxes)
    return host_fail(PA_ERR_UNSUPPORTED, "positions with %lld axes, 1 to %d are supported",
                     static_cast<long long>(axes), kMaxAxes);
  if (pos->shape[pos->ndim - 1] != T || slots->shape[0] != T)
    return host_fail(PA_ERR_INVALID_ARG, "positions and slot_mapping need one entry per token (and axis)");
  if (T > 1 && (pos->stride[pos->ndim - 1] != 1 || slots->stride[0] != 1))
    return host_fail(PA_ERR_INVALID_ARG, "positions rows and slot_mapping must be contiguous");
  if (D % 8 != 0 || D > kMaxHeadDim || D < 8)
    return host_fail(PA_ERR_UNSUPPORTED, "head_dim must be a multiple of 8 up to %d", kMaxHeadDim);
  if (R % 4 != 0 || R < 4) return host_fail(PA_ERR_UNSUPPORTED, "cos_sin needs a multiple of 4 columns");
  if (R > D)
    return host_fail(PA_ERR_INVALID_ARG, "cos_sin has %lld columns, more than head_dim %lld",
                     static_cast<long long>(R), static_cast<long long>(D));
  if (Hq < 1 || Hkv < 1) return host_fail(PA_ERR_INVALID_ARG, "query and key need at least one head");
  if (T > (int64_t(1) << 30) || Hq > 4096 || Hkv > 4096 || NB > (int64_t(1) << 31) - 1 || P > (int64_t(1) << 31) - 1)
    return host_fail(PA_ERR_UNSUPPORTED, "tensor extents too large");
  if (P > 1 && (table->stride[0] % 4 || table->stride[0] == 0))
    return host_fail(PA_ERR_INVALID_ARG, "cos_sin rows must lie a positive multiple of 4 elements apart");
  if (table->stride[1] != 1 || !host_aligned(table->data, 16))
    return host_fail(PA_ERR_INVALID_ARG, "cos_sin needs contiguous rows and 16-byte alignment");
  if (kc->shape[1] != kPage) return host_fail(PA_ERR_UNSUPPORTED, "page size must be 16");
  if (kc->shape[2] != Hkv || kc->shape[3] != D)
    return host_fail(PA_ERR_INVALID_ARG, "cache [NB, 16, Hkv, D] does not match key [T, Hkv, D]");
  for (int d = 0; d < 4; ++d)
    if (vc->shape[d] != kc->shape[d]) return host_fail(PA_ERR_INVALID_ARG, "v_cache shape differs from k_cache");
  const pa_tensor_t* rows[5] = {query, key, value, query_out, key_out};
  const char* names[5] = {"query", "key", "value", "query_out", "key_out"};
  for (int k = 0; k < 5; ++k) {
    const pa_tensor_t* r = rows[k];
    if (r->data == nullptr) continue;
    if (r->stride[2] != 1 || (r->shape[1] > 1 && r->stride[1] % 8) || (T > 1 && r->stride[0] % 8) ||
        !host_aligned(r->data, 16))
      return host_fail(PA_ERR_INVALID_ARG, "%s rows must be contiguous and 16-byte aligned (strides multiple of 8)",
                       names[k]);
    if (k >= 3 && ((r->shape[1] > 1 && r->stride[1] == 0) || (T > 1 && r->stride[0] == 0)))
      return host_fail(PA_ERR_INVALID_ARG, "%s is written: its strides must not be 0", names[k]);
  }
  const int esz = kc->dtype == PA_FP8_E4M3 ? 1 : 2;
  for (const pa_tensor_t* c : {kc, vc}) {
    if (c->stride[3] != 1) return host_fail(PA_ERR_INVALID_ARG, "KV cache last dim must be contiguous");
    for (int d = 0; d < 3; ++d)
      if (c->shape[d] > 1 && ((c->stride[d] * esz) % 16 != 0 || c->stride[d] == 0))
        return host_fail(PA_ERR_INVALID_ARG, "KV cache strides must be positive multiples of 16 bytes");
    if (!host_aligned(c->data, 16)) return host_fail(PA_ERR_INVALID_ARG, "KV cache data must be 16-byte aligned");
  }
  if (esz == 1 && (!std::isfinite(k_scale) || !std::isfinite(v_scale) || k_scale == 0.f || v_scale == 0.f))
    return host_fail(PA_ERR_INVALID_ARG, "fp8 caches need finite, non-zero k_scale and v_scale");
  RopeParams p = {};
  for (int64_t i = 0; i < R / 2 && pair_axis != nullptr; ++i) {
    if (pair_axis[i] >= axes)
      return host_fail(PA_ERR_INVALID_ARG, "pair_axis[%lld] = %d, positions has %lld axes", static_cast<long long>(i),
                       pair_axis[i], static_cast<long long>(axes));
    p.axis[i >> 4] |= static_cast<uint32_t>(pair_axis[i]) << (2 * (i & 15));
  }
  p.query = static_cast<const uint16_t*>(query->data);
  p.key = static_cast<const uint16_t*>(key->data);
  p.value = static_cast<const uint16_t*>(value->data);
  p.q_t = query->stride[0];
  p.q_h = query->stride[1];
  p.k_t = key->stride[0];
  p.k_h = key->stride[1];
  p.v_t = value->stride[0];
  p.v_h = value->stride[1];
  p.query_out = static_cast<uint16_t*>(query_out->data);
  p.qo_t = query_out->stride[0];
  p.qo_h = query_out->stride[1];
  p.key_out = static_cast<uint16_t*>(key_out->data);
  p.ko_t = key_out->data ? key_out->stride[0] : 0;
  p.ko_h = key_out->data ? key_out->stride[1] : 0;
  p.positions = static_cast<const int32_t*>(pos->data);
  p.pos_stride = pos->ndim == 1 ? 0 : pos->stride[0];
  p.table = static_cast<const float*>(table->data);
  p.table_stride = table->stride[0];
  p.slots = static_cast<const int32_t*>(slots->data);
  p.k_cache = static_cast<uint8_t*>(kc->data);
  p.v_cache = static_cast<uint8_t*>(vc->data);
  p.kc_page = kc->stride[0];
  p.kc_slot = kc->stride[1];
  p.kc_head = kc->stride[2];
  p.vc_page = vc->stride[0];
  p.vc_slot = vc->stride[1];
  p.vc_head = vc->stride[2];
  p.tokens = static_cast<int32_t>(T);
  p.axes = static_cast<int32_t>(axes);
  p.rows = static_cast<int32_t>(P);
  p.rot = static_cast<int32_t>(R);
  p.hq = static_cast<int32_t>(Hq);
  p.hkv = static_cast<int32_t>(Hkv);
  p.neighbours = neighbours != 0;
  p.num_slots = NB * kPage;
  p.k_scale = esz == 1 ? k_scale : 1.f;
  p.v_scale = esz == 1 ? v_scale : 1.f;

  auto lock = host_lock();
  HostDevice dev;
  if ((st = host_device(&dev)) != PA_OK) return st;
  p.err = dev.status;
  // 16-byte accesses where the head's halves and what does not rotate keep their
  // alignment, else 4-byte ones.
  const bool wide = R % 16 == 0 && D % 16 == 0;
  p.chunks = static_cast<int32_t>(wide ? D / 16 : D / 4);
  const int64_t heads = Hq + 2 * Hkv;
  // Heads a thread: enough threads for an SM's 512 or so, then more heads for each, so that
  // what waits in turn (positions, then angles) is paid once for them, up to 12 (16384 tokens
  // of 48 heads, fp8: 64 us for 12, 66 for 8, 68 for 24, 149 for one; 500 tokens: 6.5 us for
  // 2, 7.0 for one).  With 4-byte accesses (24 features rotate) 24 heads would take 105 us,
  // 12 take 114 (bf16 85 and 94).
  const int64_t threads = T * heads * p.chunks;
  const int64_t turns = std::min<int64_t>(std::min<int64_t>(heads, 12), threads / (dev.num_sms * int64_t(512)));
  const bool many = turns > 1;
  p.groups = static_cast<int32_t>(many ? (heads + turns - 1) / turns : heads);
  const int64_t blocks = (T * p.chunks * p.groups + kThreads - 1) / kThreads;
  if (blocks > (int64_t(1) << 31) - 1) return host_fail(PA_ERR_UNSUPPORTED, "tensor extents too large");
  const cudaError_t e = wide ? (many ? launch_form<8, true>(p, esz == 1, blocks, stream) : launch_form<8, false>(p, esz == 1, blocks, stream))
                             : (many ? launch_form<2, true>(p, esz == 1, blocks, stream) : launch_form<2, false>(p, esz == 1, blocks, stream));
  if (e != cudaSuccess) return host_cuda_fail(e, "rotary cache write kernel launch");
  return PA_OK;
}

}  // namespace
}  // namespace pa

extern "C" int paged_attn_rope_cache_write(const pa_tensor_t* query, const pa_tensor_t* key, const pa_tensor_t* value,
                                           const pa_tensor_t* positions, const pa_tensor_t* cos_sin,
                                           const uint8_t* pair_axis, int32_t neighbours,
                                           const pa_tensor_t* slot_mapping, const pa_tensor_t* k_cache,
                                           const pa_tensor_t* v_cache, float k_scale, float v_scale,
                                           const pa_tensor_t* query_out, const pa_tensor_t* key_out,
                                           pa_stream_t stream) {
  return pa::host_entry([&] {
    return pa::rope_cache_write(query, key, value, positions, cos_sin, pair_axis, neighbours, slot_mapping, k_cache,
                                v_cache, k_scale, v_scale, query_out, key_out, reinterpret_cast<cudaStream_t>(stream));
  });
}
