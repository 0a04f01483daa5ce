// Host side of decode attention over a 4-bit paged cache: validation, launch
// plan, the split and merge launches.
#include <algorithm>
#include <cmath>

#include "pa_host.h"
#include "pa_kernels.h"

namespace pa {
namespace {

constexpr int kPageTokens = 16;
constexpr int kGroup = 16;             // features that share a scale code
constexpr int kMaxRows = 64;           // query rows per KV head
constexpr int kMaxCtas = 1 << 14;

struct PlanQ4 {
  int G, R_max, NT, MT, HC, NC, KW, nstage, threads, grid, min_pages;
  uint32_t off_q, off_xchg, off_state, off_prefix, smem;
  size_t ws_unit, ws_ml, ws_o, ws_bytes;
};

size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }

int check_shape(int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t max_qlen, const pa_options_t* o) {
  if (B < 1 || B > kMaxSeqsHost)
    return host_fail(PA_ERR_UNSUPPORTED, "num_seqs %lld outside [1, %d]", static_cast<long long>(B), kMaxSeqsHost);
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0)
    return host_fail(PA_ERR_INVALID_ARG, "num_q_heads %lld must be a positive multiple of num_kv_heads %lld",
                     static_cast<long long>(Hq), static_cast<long long>(Hkv));
  if (Hq > (1 << 20)) return host_fail(PA_ERR_UNSUPPORTED, "tensor extents too large");
  if (D != 64 && D != 128)
    return host_fail(PA_ERR_UNSUPPORTED, "head_dim %lld not in {64, 128}", static_cast<long long>(D));
  if (max_qlen < 1)
    return host_fail(PA_ERR_INVALID_ARG, "max_query_len %lld < 1", static_cast<long long>(max_qlen));
  if (Hq / Hkv * max_qlen > kMaxRows)
    return host_fail(PA_ERR_UNSUPPORTED, "group size %lld x max_query_len %lld exceeds %d query rows per KV head",
                     static_cast<long long>(Hq / Hkv), static_cast<long long>(max_qlen), kMaxRows);
  if (o == nullptr) return PA_OK;
  const bool tok = (o->k_token_scales && o->k_token_scales->data) || (o->v_token_scales && o->v_token_scales->data);
  if (o->use_tcgen05 != 0 || o->page_pairing != 0 || tok || o->test_starve_cta != 0 || o->segment_cost_pages != 0)
    return host_fail(PA_ERR_UNSUPPORTED, "4-bit decode takes none of use_tcgen05, page_pairing, token scales, "
                     "test_starve_cta, segment_cost_pages");
  if (o->num_ctas < 0 || o->num_ctas > kMaxCtas || o->min_pages_per_cta < 0)
    return host_fail(PA_ERR_INVALID_ARG, "num_ctas must be in [0, %d] and min_pages_per_cta not negative", kMaxCtas);
  if (o->heads_per_cta < 0 || (o->heads_per_cta > 0 && Hkv % o->heads_per_cta != 0))
    return host_fail(PA_ERR_INVALID_ARG, "heads_per_cta %d must divide num_kv_heads %lld", o->heads_per_cta,
                     static_cast<long long>(Hkv));
  if (o->wait_limit_us < 0) return host_fail(PA_ERR_INVALID_ARG, "wait_limit_us must not be negative");
  if (o->sinks && !host_aligned(o->sinks, 4)) return host_fail(PA_ERR_INVALID_ARG, "sinks must be 4-byte aligned");
  return PA_OK;
}

int make_plan(int B, int Hq, int Hkv, int D, int max_qlen, const pa_options_t* o, const HostDevice& dev, PlanQ4* out) {
  PlanQ4 p = {};
  p.G = Hq / Hkv;
  p.R_max = p.G * max_qlen;
  // Tiles of 8 NT query rows, a warp each.  Two warps that both convert a page beat one
  // with 32 rows of 128 features, whose outputs leave no registers for two pages at once
  // (32 sequences of 4 tokens, 8 heads, 32 rows: 70 us against 81; one head: 28 against
  // 43).  With 64 features the 32 rows fit, and win where the heads fill the CTA and the
  // batch the device (32 sequences: 45 us against 51, 64 rows 72 against 90; 16 short
  // sequences: 21 against 17; one head: 31 against 22).
  const bool wide = D == 64 && p.R_max > 16 && Hkv * ((p.R_max + 31) / 32) >= 8 && B >= 32;
  p.NT = p.R_max <= 8 ? 1 : (wide ? 4 : 2);
  p.MT = (p.R_max + 8 * p.NT - 1) / (8 * p.NT);
  const int warps = split_q4_warps();
  // As many heads as the CTA has warps for: a head's rows of a page lie beside the next
  // head's, and fewer heads a CTA make more and shorter segments (8, 4, 2 and 1 heads:
  // batch of 256, 133, 149, 166 and 371 us; 16 sequences of 2000 tokens 20.2, 20.2, 20.3,
  // 23.1; one of 32768, 64 features, 14.8, 15.7, 15.9, 20.2; of 4000 11.8, 11.4, 11.6,
  // 12.6; one of 32768, 128 features, 21.1, 20.7, 20.6, 26.6; caches in L2 but the batch's).
  const int forced = o ? o->heads_per_cta : 0;
  if (forced > warps / p.MT)
    return host_fail(PA_ERR_UNSUPPORTED, "heads_per_cta %d x %d row tiles exceeds %d warps", forced, p.MT, warps);
  for (p.HC = forced > 0 ? forced : std::min(Hkv, warps / p.MT); Hkv % p.HC != 0; --p.HC) {
  }
  p.NC = Hkv / p.HC;
  p.threads = 32 * warps;
  const uint32_t state = static_cast<uint32_t>(up(split_q4_state_bytes(), 16));
  const uint32_t prefix = static_cast<uint32_t>(up(4u * (3 * static_cast<size_t>(B) + 2), 16));
  const uint32_t query = p.HC * p.MT * split_q4_query_bytes(D, p.NT);
  // The shared memory of the CTAs that an SM's registers hold, and as many warps a head
  // as the CTA has; where the sequences' metadata (12 bytes each) leaves too little: one
  // CTA an SM, then half as many warps a head until it fits.  (8192 sequences, 16 rows of
  // one head of 128, four warps a head against one: up to 3000 tokens 959 us against 2431,
  // up to 400 527 against 565, up to 40, whose three pages leave warps idle, 403 against
  // 291.)  Where all eight warps take one head's pages in turn, one CTA an SM as well: its
  // segments are twice as long against the cost of their ends (64 sequences, one KV head:
  // 21.5 us against 25.6; with two heads and four warps each, two CTAs: 18.7 against 20.7).
  p.nstage = split_q4_stages(D);
  const uint32_t ring = static_cast<uint32_t>(warps * p.nstage * 2 * kPageTokens * (D / 2 + D / kGroup));
  uint32_t xchg = 0;
  int per_sm = split_q4_ctas_per_sm(p.NT) == 2 && p.HC * p.MT > 1 ? 2 : 1;
  for (p.KW = 1; p.KW < 8 && 2 * p.KW * p.HC * p.MT <= warps;) p.KW *= 2;
  for (;;) {
    // partial rows the KW warps of a head exchange (pa_split_q4.cu): the features a
    // warp does not gather, and each row's maximum and sum
    const int cols = D - D / p.KW + 4;
    xchg = p.KW == 1 ? 0u
                     : static_cast<uint32_t>(up(static_cast<size_t>(p.HC * p.MT * p.KW) * 8 * p.NT * (cols * 4 + 8), 128));
    const int64_t budget = per_sm == 2 ? (dev.smem_optin + 2048) / 2 - 1024 - 512 : dev.smem_optin;
    if (static_cast<int64_t>(ring) + query + xchg + state + prefix <= budget) break;
    if (per_sm == 2) per_sm = 1;
    else if (p.KW > 1) p.KW /= 2;
    else return host_fail(PA_ERR_UNSUPPORTED, "no launch configuration fits %d bytes of shared memory", dev.smem_optin);
  }
  p.grid = (o && o->num_ctas > 0) ? o->num_ctas : per_sm * dev.num_sms;
  // Short calls gain more from a second CTA than its partials cost the merge (2 pages a
  // CTA against 4: 3 sequences of up to 100 tokens 8.5 us against 11.5, 64 of up to 300
  // 15.0 against 17.1, one of 4000 13.1 against 12.5), but for eight warps on one head's
  // pages (4 sequences of 2000 tokens: 14.4 against 12.5).
  p.min_pages = (o && o->min_pages_per_cta > 0) ? o->min_pages_per_cta : std::max(2, p.KW / 2);
  p.off_q = ring;
  p.off_xchg = p.off_q + query;
  p.off_state = p.off_xchg + xchg;
  p.off_prefix = p.off_state + state;
  p.smem = p.off_prefix + prefix;
  const size_t rows = static_cast<size_t>(2) * p.grid * p.HC * p.R_max;
  p.ws_ml = up(static_cast<size_t>(16) * B * p.NC, 256);
  p.ws_o = up(p.ws_ml + rows * 8, 256);
  p.ws_bytes = up(p.ws_o + rows * D * 4, 256);
  *out = p;
  return PA_OK;
}

int decode_q4(const pa_tensor_t* q, const pa_tensor_t* kc, const pa_tensor_t* vc, const pa_tensor_t* ks,
              const pa_tensor_t* vs, const pa_tensor_t* bt, const pa_tensor_t* sl, const pa_tensor_t* qsl,
              int32_t max_qlen, float scale, float k_scale, float v_scale, const pa_tensor_t* out,
              const pa_tensor_t* lse, const pa_options_t* opts, cudaStream_t stream) {
  int st;
  const bool none = (q != nullptr && q->ndim == 3 && q->shape[0] == 0);   // no query tokens: nothing to do
  if ((st = host_check_tensor(q, "q", 3, none)) || (st = host_check_tensor(kc, "k_cache", 4, false)) ||
      (st = host_check_tensor(vc, "v_cache", 4, false)) || (st = host_check_tensor(ks, "k_group_scales", 4, false)) ||
      (st = host_check_tensor(vs, "v_group_scales", 4, false)) ||
      (st = host_check_tensor(bt, "block_tables", 2, none)) || (st = host_check_tensor(sl, "seq_lens", 1, none)) ||
      (st = host_check_tensor(qsl, "query_start_loc", 1, true)) || (st = host_check_tensor(out, "out", 3, none)) ||
      (st = host_check_tensor(lse, "lse", 2, true)))
    return st;
  if (none) return PA_OK;
  if (q->dtype != PA_BF16 || out->dtype != PA_BF16) return host_fail(PA_ERR_INVALID_ARG, "q and out must be bf16");
  if (kc->dtype != PA_FP4_E2M1X2 || vc->dtype != PA_FP4_E2M1X2)
    return host_fail(PA_ERR_INVALID_ARG, "k_cache and v_cache must hold packed e2m1 codes");
  if (ks->dtype != PA_FP8_E4M3 || vs->dtype != PA_FP8_E4M3)
    return host_fail(PA_ERR_INVALID_ARG, "group scales must be fp8 e4m3");
  if (bt->dtype != PA_I32 || sl->dtype != PA_I32 || (qsl->data && qsl->dtype != PA_I32))
    return host_fail(PA_ERR_INVALID_ARG, "block_tables, seq_lens and query_start_loc must be int32");
  if (lse->data && lse->dtype != PA_F32) return host_fail(PA_ERR_INVALID_ARG, "lse must be float32");
  const int64_t T = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const int64_t NB = kc->shape[0], Hkv = kc->shape[2], B = bt->shape[0], MB = bt->shape[1];
  if ((st = check_shape(B, Hq, Hkv, D, max_qlen, opts)) != PA_OK) return st;
  if (kc->shape[1] != kPageTokens)
    return host_fail(PA_ERR_UNSUPPORTED, "page size %lld, only 16 is supported", static_cast<long long>(kc->shape[1]));
  if (NB < 1 || NB > (int64_t(1) << 31) - 1 || T > (int64_t(1) << 30) || MB > (1 << 27) - 64 || B * MB >= (int64_t(1) << 31))
    return host_fail(PA_ERR_UNSUPPORTED, "tensor extents too large");
  const pa_tensor_t *code[2] = {kc, vc}, *sc[2] = {ks, vs};
  const char *cn[2] = {"k_cache", "v_cache"}, *sn[2] = {"k_group_scales", "v_group_scales"};
  for (int y = 0; y < 2; ++y) {
    const pa_tensor_t *c = code[y], *s = sc[y];
    if (c->shape[0] != NB || c->shape[1] != kPageTokens || c->shape[2] != Hkv || c->shape[3] * 2 != D)
      return host_fail(PA_ERR_INVALID_ARG, "%s must be [NB, 16, Hkv, D / 2]", cn[y]);
    if (c->stride[3] != 1 || c->stride[0] % 16 || c->stride[1] % 16 || c->stride[2] % 16 || !host_aligned(c->data, 16))
      return host_fail(PA_ERR_INVALID_ARG,
                       "%s needs a contiguous last dim, strides that are multiples of 16 bytes and 16-byte alignment",
                       cn[y]);
    if (c->stride[0] >= (int64_t(1) << 32) || s->stride[0] >= (int64_t(1) << 32))
      return host_fail(PA_ERR_UNSUPPORTED, "%s and %s: pages 4 GiB or more apart", cn[y], sn[y]);
    if (s->shape[0] != NB || s->shape[1] != Hkv || s->shape[2] != kPageTokens || s->shape[3] * kGroup != D)
      return host_fail(PA_ERR_INVALID_ARG, "%s must be [NB, Hkv, 16, D / 16]", sn[y]);
    if (s->stride[3] != 1 || s->stride[2] != D / kGroup || (Hkv > 1 && s->stride[1] != D) ||
        (NB > 1 && s->stride[0] % 16) || !host_aligned(s->data, 16))
      return host_fail(PA_ERR_INVALID_ARG, "%s: each page's [Hkv, 16, D / 16] block must be contiguous and 16-byte "
                       "aligned", sn[y]);
  }
  if (sl->shape[0] != B)
    return host_fail(PA_ERR_INVALID_ARG, "seq_lens has %lld entries, block_tables %lld rows",
                     static_cast<long long>(sl->shape[0]), static_cast<long long>(B));
  if (out->shape[0] != T || out->shape[1] != Hq || out->shape[2] != D)
    return host_fail(PA_ERR_INVALID_ARG, "out shape differs from q");
  if (lse->data && (lse->shape[0] != T || lse->shape[1] != Hq))
    return host_fail(PA_ERR_INVALID_ARG, "lse shape must be [T, Hq]");
  if (qsl->data) {
    if (qsl->shape[0] != B + 1 || qsl->stride[0] != 1)
      return host_fail(PA_ERR_INVALID_ARG, "query_start_loc must be contiguous with B+1 entries");
  } else if (T < B || max_qlen != 1) {
    return host_fail(PA_ERR_INVALID_ARG, "without query_start_loc q needs a token for every sequence and "
                     "max_query_len must be 1");
  }
  if (B > 1 && sl->stride[0] != 1) return host_fail(PA_ERR_INVALID_ARG, "seq_lens must be contiguous");
  if (MB > 1 && bt->stride[1] != 1) return host_fail(PA_ERR_INVALID_ARG, "block_tables rows must be contiguous");
  if (q->stride[2] != 1 || (Hq > 1 && q->stride[1] != D) || (T > 1 && q->stride[0] % 4) || !host_aligned(q->data, 8))
    return host_fail(PA_ERR_INVALID_ARG, "q must have contiguous heads and 8-byte aligned rows");
  if (out->stride[2] != 1 || out->stride[1] % 4 || out->stride[0] % 4 || !host_aligned(out->data, 8))
    return host_fail(PA_ERR_INVALID_ARG,
                     "out must have a contiguous last dim, strides multiple of 4 elements, 8-byte alignment");
  if ((out->stride[0] == 0 && T > 1) || (out->stride[1] == 0 && Hq > 1) ||
      (lse->data && ((lse->stride[0] == 0 && T > 1) || (lse->stride[1] == 0 && Hq > 1))))
    return host_fail(PA_ERR_INVALID_ARG, "out and lse are written: their strides must not be 0");
  if (!std::isfinite(scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
    return host_fail(PA_ERR_INVALID_ARG, "scale, k_scale and v_scale must be finite");

  auto lock = host_lock();
  HostDevice dev;
  if ((st = host_device(&dev)) != PA_OK) return st;
  PlanQ4 pl;
  if ((st = make_plan(static_cast<int>(B), static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(D), max_qlen,
                      opts, dev, &pl)) != PA_OK)
    return st;
  void* ws = nullptr;
  if ((st = host_workspace(opts, pl.ws_bytes, stream, "paged_attn_q4_reserve", &ws)) != PA_OK) return st;
  SplitQ4Params sp = {};
  sp.q = static_cast<const uint16_t*>(q->data);
  sp.q_stride_t = q->stride[0];
  sp.out = static_cast<uint16_t*>(out->data);
  sp.out_stride_t = out->stride[0];
  sp.out_stride_h = out->stride[1];
  sp.lse = static_cast<float*>(lse->data);
  sp.lse_stride_t = lse->data ? lse->stride[0] : 0;
  sp.lse_stride_h = lse->data ? lse->stride[1] : 0;
  sp.block_tables = static_cast<const int32_t*>(bt->data);
  sp.bt_stride = bt->stride[0];
  sp.seq_lens = static_cast<const int32_t*>(sl->data);
  sp.qsl = static_cast<const int32_t*>(qsl->data);
  sp.num_seqs = static_cast<int32_t>(B);
  sp.num_tokens = static_cast<int32_t>(T);
  sp.Hq = static_cast<int32_t>(Hq);
  sp.Hkv = static_cast<int32_t>(Hkv);
  sp.G = pl.G;
  sp.max_qlen = max_qlen;
  sp.num_pages = static_cast<int32_t>(NB);
  sp.max_blocks = static_cast<int32_t>(MB);
  sp.HC = pl.HC;
  sp.NC = pl.NC;
  sp.MT = pl.MT;
  sp.R_max = pl.R_max;
  sp.min_pages = pl.min_pages;
  // A window as wide as the longest sequence hides nothing; the kernels' differences of
  // positions and windows stay within 32 bits below that.
  constexpr int32_t kWidest = kPageTokens * ((1 << 27) - 64);
  sp.window = (opts && opts->sliding_window > 0 && opts->sliding_window < kWidest) ? opts->sliding_window : 0;
  sp.sinks = opts ? static_cast<const float*>(opts->sinks) : nullptr;
  sp.scale_log2 = scale * k_scale * 1.4426950408889634f;
  sp.v_scale = v_scale;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  sp.ws_unit = reinterpret_cast<int4*>(wsb + pl.ws_unit);
  sp.ws_ml = reinterpret_cast<float2*>(wsb + pl.ws_ml);
  sp.ws_o = reinterpret_cast<float*>(wsb + pl.ws_o);
  sp.err = dev.status;
  sp.off_prefix = pl.off_prefix;
  sp.off_q = pl.off_q;
  sp.off_xchg = pl.off_xchg;
  sp.off_state = pl.off_state;
  sp.k_codes = static_cast<const uint8_t*>(kc->data);
  sp.v_codes = static_cast<const uint8_t*>(vc->data);
  sp.kc_stride_page = static_cast<uint32_t>(kc->stride[0]);
  sp.kc_stride_slot = kc->stride[1];
  sp.kc_stride_head = kc->stride[2];
  sp.vc_stride_page = static_cast<uint32_t>(vc->stride[0]);
  sp.vc_stride_slot = vc->stride[1];
  sp.vc_stride_head = vc->stride[2];
  sp.k_sc = static_cast<const uint8_t*>(ks->data);
  sp.v_sc = static_cast<const uint8_t*>(vs->data);
  sp.k_sc_page = static_cast<uint32_t>(ks->stride[0]);
  sp.v_sc_page = static_cast<uint32_t>(vs->stride[0]);
  sp.KW = pl.KW;

  MergeParams mp = {};
  mp.out = sp.out;
  mp.out_stride_t = sp.out_stride_t;
  mp.out_stride_h = sp.out_stride_h;
  mp.lse = sp.lse;
  mp.lse_stride_t = sp.lse_stride_t;
  mp.lse_stride_h = sp.lse_stride_h;
  mp.seq_lens = sp.seq_lens;
  mp.qsl = sp.qsl;
  mp.num_seqs = sp.num_seqs;
  mp.num_tokens = sp.num_tokens;
  mp.max_blocks = sp.max_blocks;
  mp.window = sp.window;
  mp.G = pl.G;
  mp.HC = pl.HC;
  mp.NC = pl.NC;
  mp.R_max = pl.R_max;
  mp.max_qlen = max_qlen;
  mp.split_grid = pl.grid;
  mp.v_scale = v_scale;
  mp.ws_unit = sp.ws_unit;
  mp.ws_ml = sp.ws_ml;
  mp.ws_o = sp.ws_o;
  mp.err = sp.err;
  mp.sinks = sp.sinks;
  mp.keep_nan = true;

  cudaEvent_t ev0 = opts ? static_cast<cudaEvent_t>(opts->split_start_event) : nullptr;
  cudaEvent_t ev1 = opts ? static_cast<cudaEvent_t>(opts->split_stop_event) : nullptr;
  const bool pdl = !(opts && opts->disable_pdl);
  cudaError_t e;
  unsigned int rec = cudaEventRecordDefault;
  if (ev0 || ev1) {
    cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
    if ((e = cudaStreamIsCapturing(stream, &cs)) != cudaSuccess) return host_cuda_fail(e, "cudaStreamIsCapturing");
    if (cs == cudaStreamCaptureStatusActive) rec = cudaEventRecordExternal;
  }
  if (ev0 && (e = cudaEventRecordWithFlags(ev0, stream, rec)) != cudaSuccess)
    return host_cuda_fail(e, "cudaEventRecord(start)");
  if ((e = launch_split_q4(static_cast<int>(D), pl.NT, sp, pl.grid, static_cast<int>(pl.smem), pdl && !ev0, stream)) != cudaSuccess)
    return host_cuda_fail(e, "4-bit split kernel launch");
  if (ev1 && (e = cudaEventRecordWithFlags(ev1, stream, rec)) != cudaSuccess)
    return host_cuda_fail(e, "cudaEventRecord(stop)");
  const int units = static_cast<int>(B) * pl.NC;
  // The merge that reads a row's partials with a whole block is for few rows cut
  // into many pieces: up to two blocks an SM (one sequence of 32768 tokens: 15 us a
  // call against 33 with a warp a row; 512 rows of 19 pieces: 25 us against 21).
  const bool wide = pl.grid >= 4 * units && static_cast<int64_t>(units) * pl.HC * pl.R_max <= 2 * dev.num_sms;
  if ((e = launch_merge(static_cast<int>(D), mp, units, pl.HC * pl.R_max, wide, pdl && !ev1, stream,
                        true)) != cudaSuccess)
    return host_cuda_fail(e, "merge kernel launch");
  return PA_OK;
}

int plan_for(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t max_qlen, const pa_options_t* o, PlanQ4* pl) {
  int st = check_shape(B, Hq, Hkv, D, max_qlen, o);
  if (st != PA_OK) return st;
  HostDevice dev;
  if ((st = host_device(&dev)) != PA_OK) return st;
  return make_plan(B, Hq, Hkv, D, max_qlen, o, dev, pl);
}

}  // namespace
}  // namespace pa

extern "C" int paged_attn_decode_q4(const pa_tensor_t* q, const pa_tensor_t* k_cache, const pa_tensor_t* v_cache,
                                    const pa_tensor_t* k_group_scales, const pa_tensor_t* v_group_scales,
                                    const pa_tensor_t* block_tables, const pa_tensor_t* seq_lens,
                                    const pa_tensor_t* query_start_loc, int32_t max_query_len, float scale,
                                    float k_scale, float v_scale, const pa_tensor_t* out, const pa_tensor_t* lse,
                                    const pa_options_t* opts, pa_stream_t stream) {
  return pa::host_entry([&] {
    return pa::decode_q4(q, k_cache, v_cache, k_group_scales, v_group_scales, block_tables, seq_lens, query_start_loc,
                         max_query_len, scale, k_scale, v_scale, out, lse, opts,
                         reinterpret_cast<cudaStream_t>(stream));
  });
}

extern "C" int paged_attn_q4_plan(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                  int32_t max_query_len, const pa_options_t* opts, pa_plan_t* plan) {
  return pa::host_entry([&] {
    if (plan == nullptr) return pa::host_fail(PA_ERR_INVALID_ARG, "plan pointer is NULL");
    auto lock = pa::host_lock();
    pa::PlanQ4 pl;
    const int st = pa::plan_for(num_seqs, num_q_heads, num_kv_heads, head_dim, max_query_len, opts, &pl);
    if (st != PA_OK) return st;
    plan->num_ctas = pl.grid;
    plan->heads_per_cta = pl.HC;
    plan->row_tiles = pl.MT;
    plan->num_stages = pl.nstage;
    plan->threads_per_cta = pl.threads;
    plan->smem_bytes = static_cast<int32_t>(pl.smem);
    plan->min_pages_per_cta = pl.min_pages;
    plan->merge_rows = pl.HC * pl.R_max;
    plan->page_pairing = 1;
    plan->warps_per_head = pl.KW;
    plan->workspace_bytes = static_cast<int64_t>(pl.ws_bytes);
    plan->variant = 4;
    plan->block_pages = 2;
    return static_cast<int>(PA_OK);
  });
}

extern "C" int paged_attn_q4_workspace_size(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads,
                                            int32_t head_dim, int32_t max_query_len, size_t* bytes) {
  return pa::host_entry([&] {
    if (bytes == nullptr) return pa::host_fail(PA_ERR_INVALID_ARG, "bytes pointer is NULL");
    auto lock = pa::host_lock();
    pa::PlanQ4 pl;
    const int st = pa::plan_for(num_seqs, num_q_heads, num_kv_heads, head_dim, max_query_len, nullptr, &pl);
    if (st == PA_OK) *bytes = pl.ws_bytes;
    return st;
  });
}

extern "C" int paged_attn_q4_reserve(int32_t num_seqs, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
                                     int32_t max_query_len) {
  return pa::host_entry([&] {
    auto lock = pa::host_lock();
    pa::PlanQ4 pl;
    const int st = pa::plan_for(num_seqs, num_q_heads, num_kv_heads, head_dim, max_query_len, nullptr, &pl);
    return st != PA_OK ? st : pa::host_reserve(pl.ws_bytes);
  });
}
