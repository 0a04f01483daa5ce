// Rows of the 4-bit paged cache: write (quantise) and read back (dequantise).
//
// Write, for every token t with slot s >= 0, KV head h and group of 16
// consecutive features x of its key (or value) row, with ts the tensor's scale:
//     S     = e4m3fn(amax / (6 ts)),  amax = max |x|        (6 = the largest e2m1)
//     code  = e2m1(x / (S ts))
// Products are rounded to fp32, quotients are IEEE fp32 quotients, both
// encodings round to nearest even and saturate.  S = 0 (or a group that holds
// a NaN, whose S is the e4m3fn NaN) stores codes 0.  Read is the inverse:
// code * S (exact) times ts rounded to fp32, then to bf16.
//
// Both are bound by memory: 4 bytes of bf16 a (key, value) feature pair against
// 9/8 bytes of codes and scales.  A (token, head) row belongs to L lanes, so that the
// index arithmetic of a row serves several pieces of it.  Writing, a lane takes whole
// groups (every L-th, two in flight): a group's maximum, scale and reciprocal are
// computed once and its codes leave as 8 bytes.  Reading, a lane takes 8-feature chunks
// (every L-th, four in flight), so that a store instruction fills whole sectors.
// 16384 tokens x 8 heads x 128: 21 us to write (86 MB, 4.0 TB/s; in chunks 26 us, a
// thread a group 27) and 15 to read (86 MB, 5.6 TB/s; in groups 19, a thread a group 19).
// Neither memory nor issue is full while writing (DRAM 37%, issue slots 58%, 44% of the
// warps resident): a lane waits for its loads, then computes (40 instructions a chunk for
// the quotients), with nothing of its next row in flight.
#include "pa_device.cuh"
#include "pa_host.h"
#include "pa_q4.cuh"
#include "pa_quant.cuh"

#include <algorithm>
#include <cmath>

namespace pa {

struct RowsQ4Params {
  uint16_t* rows[2];           // key, value: bf16 [T, Hkv, D]
  int64_t row_t[2], row_h[2];  // their token and head strides (elements)
  const int32_t* slots;
  uint8_t* codes[2];           // K, V codes [NB, 16, Hkv, D / 2]
  int64_t code_page[2], code_slot[2], code_head[2];
  uint8_t* scales[2];          // K, V group scales [NB, Hkv, 16, D / 16]
  int64_t sc_page[2], sc_head[2], sc_slot[2], sc_group[2];
  int32_t num_tokens, num_kv_heads, groups, num_pages;   // groups of a row
  int32_t lg;                  // 2^lg lanes a row
  float ts[2];                 // tensor scales
  float six_ts[2];             // fp32(6 ts)
  uint32_t* err;
};

constexpr int kRowGroups = 2;      // groups of a lane at a time (write)
constexpr int kRowChunks = 4;      // 8-feature chunks of a lane at a time (read)
constexpr int kRowWaves = 8;       // CTAs an SM and tensor (4 or 16: 1 us more)

// Where a row's codes and scales lie.
__device__ __forceinline__ uint8_t* codes_at(const RowsQ4Params& p, int y, int slot, int h) {
  const int64_t page = slot / kPage;
  return p.codes[y] + page * p.code_page[y] + (slot % kPage) * p.code_slot[y] + h * p.code_head[y];
}
__device__ __forceinline__ uint8_t* scales_at(const RowsQ4Params& p, int y, int slot, int h) {
  const int64_t page = slot / kPage;
  return p.scales[y] + page * p.sc_page[y] + (slot % kPage) * p.sc_slot[y] + h * p.sc_head[y];
}

// e2m1 codes of eight features over the group's scale sd.s > 0 (amax: the group's
// largest magnitude).
__device__ __forceinline__ uint32_t quantise8(const uint4 v, const ScaleDiv& sd, float amax) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const float d = sd.s;
  float q[8];
  // Quotients below 1024 need none of div_by2's exceptions but the sign of a zero,
  // which every quotient takes from its feature here.
  if (sd.fast && amax < 1000.f * d) {
    const uint64_t r2 = f2_pack(sd.r, sd.r), ns2 = f2_pack(-d, -d);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float a = bf16_lo(w[e]), b = bf16_hi(w[e]);
      const uint64_t x = f2_pack(a, b), q0 = fmul2(x, r2);
      float qa, qb;
      f2_unpack(ffma2(ffma2(q0, ns2, x), r2, q0), qa, qb);
      q[2 * e] = copysignf(qa, a);
      q[2 * e + 1] = copysignf(qb, b);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      q[2 * e] = __fdiv_rn(bf16_lo(w[e]), d);
      q[2 * e + 1] = __fdiv_rn(bf16_hi(w[e]), d);
    }
  }
  return e2m1x8_from_f32(q);
}

// One row a group of L = 2^lg lanes at a time, of one tensor (blockIdx.y: 0 = K, 1 = V).
__global__ void __launch_bounds__(256) pa_cache_write_q4_kernel(const RowsQ4Params p) {
  const int y = blockIdx.y, q = threadIdx.x & ((1 << p.lg) - 1);
  const int64_t rows = static_cast<int64_t>(p.num_tokens) * p.num_kv_heads;
  const bool narrow = rows <= 0xFFFFFFFFll;
  const int64_t num_slots = static_cast<int64_t>(p.num_pages) * kPage;
  const float ts = p.ts[y], six = p.six_ts[y];
  const int64_t step = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> p.lg;
  for (int64_t r = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> p.lg; r < rows; r += step) {
    const int64_t t = cw_div(r, p.num_kv_heads, narrow);
    const int h = static_cast<int>(r - t * p.num_kv_heads);
    const uint16_t* src = p.rows[y] + t * p.row_t[y] + h * p.row_h[y];
    const int slot = p.slots[t];
    if (slot < 0) continue;                        // padding token
    if (slot >= num_slots) {
      if (h == 0 && q == 0) atomicOr(p.err, kErrPageRange);
      continue;
    }
    uint8_t* codes = codes_at(p, y, slot, h);
    uint8_t* scales = scales_at(p, y, slot, h);
    for (int g0 = 0; g0 < p.groups; g0 += kRowGroups << p.lg) {
      uint4 v[kRowGroups][2];
#pragma unroll
      for (int u = 0; u < kRowGroups; ++u) {
        const int g = g0 + (u << p.lg) + q;
        if (g >= p.groups) break;
        const uint4* x = reinterpret_cast<const uint4*>(src + g * kQ4Group);
        v[u][0] = x[0];
        v[u][1] = x[1];
      }
#pragma unroll
      for (int u = 0; u < kRowGroups; ++u) {
        const int g = g0 + (u << p.lg) + q;
        if (g >= p.groups) break;
        // magnitudes in bf16 order as their bits
        uint32_t m2 = 0u;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          m2 = max_u16x2(m2, max_u16x2(max_u16x2(v[u][k].x & 0x7FFF7FFFu, v[u][k].y & 0x7FFF7FFFu),
                                       max_u16x2(v[u][k].z & 0x7FFF7FFFu, v[u][k].w & 0x7FFF7FFFu)));
        const float amax = __uint_as_float(max(m2 << 16, m2 & 0xFFFF0000u));
        const uint32_t s8 = e4m3x2_from_f32(__fdiv_rn(amax, six), 0.f) & 0xFFu;
        const float d = __fmul_rn(f16_lo(e4m3x2_to_f16x2(s8)), ts);
        uint2 c = make_uint2(0u, 0u);
        if (d > 0.f) {                             // else 0 or NaN
          const ScaleDiv sd = scale_div(d);
          c = make_uint2(quantise8(v[u][0], sd, amax), quantise8(v[u][1], sd, amax));
        }
        *reinterpret_cast<uint2*>(codes + g * (kQ4Group / 2)) = c;
        scales[g * p.sc_group[y]] = static_cast<uint8_t>(s8);
      }
    }
  }
}

// One row a group of L lanes at a time, read back.
__global__ void __launch_bounds__(256) pa_cache_read_q4_kernel(const RowsQ4Params p) {
  const int y = blockIdx.y, q = threadIdx.x & ((1 << p.lg) - 1);
  const int64_t rows = static_cast<int64_t>(p.num_tokens) * p.num_kv_heads;
  const bool narrow = rows <= 0xFFFFFFFFll;
  const int64_t num_slots = static_cast<int64_t>(p.num_pages) * kPage;
  const float ts = p.ts[y];
  const int chunks = 2 * p.groups;                 // of 8 features
  const int64_t step = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> p.lg;
  for (int64_t r = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> p.lg; r < rows; r += step) {
    const int64_t t = cw_div(r, p.num_kv_heads, narrow);
    const int h = static_cast<int>(r - t * p.num_kv_heads);
    const int slot = p.slots[t];
    if (slot < 0) continue;                        // padding token: its row stays as it was
    if (slot >= num_slots) {
      if (h == 0 && q == 0) atomicOr(p.err, kErrPageRange);
      continue;
    }
    const uint8_t* codes = codes_at(p, y, slot, h);
    const uint8_t* scales = scales_at(p, y, slot, h);
    uint16_t* dst = p.rows[y] + t * p.row_t[y] + h * p.row_h[y];
    for (int c0 = 0; c0 < chunks; c0 += kRowChunks << p.lg) {
      uint32_t w[kRowChunks], s8[kRowChunks];
#pragma unroll
      for (int u = 0; u < kRowChunks; ++u) {
        const int c = c0 + (u << p.lg) + q;
        w[u] = s8[u] = 0u;
        if (c < chunks) {
          w[u] = *reinterpret_cast<const uint32_t*>(codes + c * 4);
          s8[u] = scales[(c >> 1) * p.sc_group[y]];
        }
      }
#pragma unroll
      for (int u = 0; u < kRowChunks; ++u) {
        const int c = c0 + (u << p.lg) + q;
        if (c >= chunks) break;
        const uint32_t s2 = e4m3x2_to_f16x2(s8[u] * 0x0101u);
        uint32_t x[4], o[4];
        e2m1x8_to_f16(w[u], x);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t f = hmul2(x[e], s2);
          o[e] = pack_bf16(__fmul_rn(f16_lo(f), ts), __fmul_rn(f16_hi(f), ts));
        }
        *reinterpret_cast<uint4*>(dst + c * 8) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

namespace {

// Codes [NB, 16, Hkv, D / 2] and group scales [NB, Hkv, 16, D / 16] of K and V.
int check_q4_cache(const pa_tensor_t* const* code, const pa_tensor_t* const* scale, int64_t Hkv, int64_t D,
                   bool written) {
  const char* cn[2] = {"k_cache", "v_cache"};
  const char* sn[2] = {"k_group_scales", "v_group_scales"};
  for (int y = 0; y < 2; ++y) {
    int st;
    if ((st = host_check_tensor(code[y], cn[y], 4, false)) != PA_OK) return st;
    if ((st = host_check_tensor(scale[y], sn[y], 4, false)) != PA_OK) return st;
    if (code[y]->dtype != PA_FP4_E2M1X2) return host_fail(PA_ERR_INVALID_ARG, "%s must hold packed e2m1 codes", cn[y]);
    if (scale[y]->dtype != PA_FP8_E4M3) return host_fail(PA_ERR_INVALID_ARG, "%s must be fp8 e4m3", sn[y]);
    if (code[y]->shape[1] != kPage) return host_fail(PA_ERR_UNSUPPORTED, "page size must be 16");
    if (code[y]->shape[0] != code[0]->shape[0] || code[y]->shape[2] != Hkv || code[y]->shape[3] * 2 != D)
      return host_fail(PA_ERR_INVALID_ARG, "%s must be [NB, 16, Hkv, D / 2] with D = %lld, Hkv = %lld", cn[y],
                       static_cast<long long>(D), static_cast<long long>(Hkv));
    if (scale[y]->shape[0] != code[0]->shape[0] || scale[y]->shape[1] != Hkv || scale[y]->shape[2] != kPage ||
        scale[y]->shape[3] * kQ4Group != D)
      return host_fail(PA_ERR_INVALID_ARG, "%s must be [NB, Hkv, 16, D / 16]", sn[y]);
    if (code[y]->stride[3] != 1) return host_fail(PA_ERR_INVALID_ARG, "%s last dim must be contiguous", cn[y]);
    for (int d = 0; d < 3; ++d)
      if (code[y]->stride[d] % 8 != 0)
        return host_fail(PA_ERR_INVALID_ARG, "%s strides must be multiples of 8 bytes", cn[y]);
    if (!host_aligned(code[y]->data, 8)) return host_fail(PA_ERR_INVALID_ARG, "%s must be 8-byte aligned", cn[y]);
    if (written)
      for (int d = 0; d < 4; ++d)
        if ((code[y]->stride[d] == 0 && code[y]->shape[d] > 1) || (scale[y]->stride[d] == 0 && scale[y]->shape[d] > 1))
          return host_fail(PA_ERR_INVALID_ARG, "%s and %s are written: their strides must not be 0", cn[y], sn[y]);
  }
  return PA_OK;
}

int rows_q4(bool write, const pa_tensor_t* key, const pa_tensor_t* value, const pa_tensor_t* slots,
            const pa_tensor_t* kc, const pa_tensor_t* vc, const pa_tensor_t* ks, const pa_tensor_t* vs, float k_scale,
            float v_scale, cudaStream_t stream) {
  int st;
  const bool none = key != nullptr && key->ndim == 3 && key->shape[0] == 0;   // no tokens: empty tensors have no memory
  if ((st = host_check_tensor(key, "key", 3, none)) || (st = host_check_tensor(value, "value", 3, none)) ||
      (st = host_check_tensor(slots, "slot_mapping", 1, none)))
    return st;
  if (key->dtype != PA_BF16 || value->dtype != PA_BF16)
    return host_fail(PA_ERR_INVALID_ARG, "key and value must be bf16");
  if (slots->dtype != PA_I32) return host_fail(PA_ERR_INVALID_ARG, "slot_mapping must be int32");
  const int64_t T = key->shape[0], Hkv = key->shape[1], D = key->shape[2];
  for (int d = 0; d < 3; ++d)
    if (value->shape[d] != key->shape[d]) return host_fail(PA_ERR_INVALID_ARG, "value shape differs from key");
  if (slots->shape[0] != T) return host_fail(PA_ERR_INVALID_ARG, "slot_mapping needs one entry per token");
  if (T > 1 && slots->stride[0] != 1) return host_fail(PA_ERR_INVALID_ARG, "slot_mapping must be contiguous");
  if (D < 16 || D % kQ4Group != 0 || D > 512)
    return host_fail(PA_ERR_UNSUPPORTED, "head_dim must be a multiple of 16 up to 512");
  if (Hkv < 1) return host_fail(PA_ERR_INVALID_ARG, "num_kv_heads %lld < 1", static_cast<long long>(Hkv));
  const pa_tensor_t *code[2] = {kc, vc}, *scale[2] = {ks, vs}, *rows[2] = {key, value};
  if ((st = check_q4_cache(code, scale, Hkv, D, write)) != PA_OK) return st;
  if (T > (int64_t(1) << 30) || Hkv > 4096 || kc->shape[0] > (int64_t(1) << 31) - 1)
    return host_fail(PA_ERR_UNSUPPORTED, "tensor extents too large");
  for (const pa_tensor_t* t : rows) {
    if (t->stride[2] != 1 || t->stride[1] % 8 != 0 || t->stride[0] % 8 != 0 || !host_aligned(t->data, 16))
      return host_fail(PA_ERR_INVALID_ARG,
                       "key/value rows must be contiguous and 16-byte aligned (strides multiple of 8)");
    if (!write && ((t->stride[0] == 0 && T > 1) || (t->stride[1] == 0 && Hkv > 1)))
      return host_fail(PA_ERR_INVALID_ARG, "key and value are written: their strides must not be 0");
  }
  if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || !(k_scale > 0.f) || !(v_scale > 0.f))
    return host_fail(PA_ERR_INVALID_ARG, "k_scale and v_scale must be finite and positive");
  if (T == 0) return PA_OK;
  auto lock = host_lock();
  HostDevice dev;
  if ((st = host_device(&dev)) != PA_OK) return st;
  RowsQ4Params p = {};
  for (int y = 0; y < 2; ++y) {
    p.rows[y] = static_cast<uint16_t*>(rows[y]->data);
    p.row_t[y] = rows[y]->stride[0];
    p.row_h[y] = rows[y]->stride[1];
    p.codes[y] = static_cast<uint8_t*>(code[y]->data);
    p.code_page[y] = code[y]->stride[0];
    p.code_slot[y] = code[y]->stride[1];
    p.code_head[y] = code[y]->stride[2];
    p.scales[y] = static_cast<uint8_t*>(scale[y]->data);
    p.sc_page[y] = scale[y]->stride[0];
    p.sc_head[y] = scale[y]->stride[1];
    p.sc_slot[y] = scale[y]->stride[2];
    p.sc_group[y] = scale[y]->stride[3];
    p.ts[y] = y ? v_scale : k_scale;
    p.six_ts[y] = 6.f * p.ts[y];
  }
  p.slots = static_cast<const int32_t*>(slots->data);
  p.num_tokens = static_cast<int32_t>(T);
  p.num_kv_heads = static_cast<int32_t>(Hkv);
  p.groups = static_cast<int32_t>(D / kQ4Group);
  const int pieces = write ? p.groups : 2 * p.groups, at_once = write ? kRowGroups : kRowChunks;
  // A lane's pieces at a time; where the rows leave most of the device idle, they lie side
  // by side instead (write and read of 64 tokens x 8 heads x 128: 4.1 us against 4.9; from
  // half a CTA an SM on the several in flight win: 1000 tokens 6.4 us against 8.7).
  for (p.lg = 0; p.lg < 5 && (at_once << p.lg) < pieces;) ++p.lg;
  while (p.lg < 5 && (1 << p.lg) < pieces && ((T * Hkv) << p.lg) < int64_t(dev.num_sms) * 128) ++p.lg;
  p.num_pages = static_cast<int32_t>(kc->shape[0]);
  p.err = dev.status;
  const int64_t blocks = (((T * Hkv) << p.lg) + 255) / 256;
  const dim3 grid(static_cast<unsigned>(std::min<int64_t>(blocks, int64_t(dev.num_sms) * kRowWaves)), 2, 1);
  if (write)
    pa_cache_write_q4_kernel<<<grid, 256, 0, stream>>>(p);
  else
    pa_cache_read_q4_kernel<<<grid, 256, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? PA_OK : host_cuda_fail(e, write ? "4-bit cache write launch" : "4-bit cache read launch");
}

}  // namespace
}  // namespace pa

extern "C" int paged_attn_cache_write_q4(const pa_tensor_t* key, const pa_tensor_t* value,
                                         const pa_tensor_t* slot_mapping, const pa_tensor_t* k_cache,
                                         const pa_tensor_t* v_cache, const pa_tensor_t* k_group_scales,
                                         const pa_tensor_t* v_group_scales, float k_scale, float v_scale,
                                         pa_stream_t stream) {
  return pa::host_entry([&] {
    return pa::rows_q4(true, key, value, slot_mapping, k_cache, v_cache, k_group_scales, v_group_scales, k_scale,
                       v_scale, reinterpret_cast<cudaStream_t>(stream));
  });
}

extern "C" int paged_attn_cache_read_q4(const pa_tensor_t* slot_mapping, const pa_tensor_t* k_cache,
                                        const pa_tensor_t* v_cache, const pa_tensor_t* k_group_scales,
                                        const pa_tensor_t* v_group_scales, float k_scale, float v_scale,
                                        const pa_tensor_t* key, const pa_tensor_t* value, pa_stream_t stream) {
  return pa::host_entry([&] {
    return pa::rows_q4(false, key, value, slot_mapping, k_cache, v_cache, k_group_scales, v_group_scales, k_scale,
                       v_scale, reinterpret_cast<cudaStream_t>(stream));
  });
}
