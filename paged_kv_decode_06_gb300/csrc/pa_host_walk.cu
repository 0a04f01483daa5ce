// Host side of the decode calls whose walk over a sequence has a hole: sliding windows
// with first tokens that stay visible, and batches that share prefixes.  Validation, the
// workspace and the launches.
#include <algorithm>
#include <cmath>
#include <initializer_list>

#include "pa_host.h"
#include "pa_kernels.h"
#include "pa_shared.h"

namespace pa {
namespace {

constexpr int kPageTokens = 16;
constexpr int kMaxRows = 64;                       // query rows per KV head
constexpr int kMaxCtas = 1 << 14;
static_assert(kMaxCtas < 1 << kReadyBits, "the split kernel's CTAs stand below a call's number");
constexpr int64_t kMaxBlocks = (int64_t(1) << 27) - 64;   // positions stay below 2^31 - 1024

size_t up(size_t x, size_t a) { return (x + a - 1) / a * a; }
long long ll(int64_t x) { return static_cast<long long>(x); }

struct Shape {
  int64_t T, Hq, Hkv, D, NB, B, MB;
  int esz;
};

int check_options(const pa_options_t* o, int64_t Hkv, bool tokens_too) {
  if (o == nullptr) return PA_OK;
  const bool tok = (o->k_token_scales && o->k_token_scales->data) || (o->v_token_scales && o->v_token_scales->data);
  if (o->sliding_window > 0 || o->use_tcgen05 != 0 || o->segment_cost_pages != 0 || (tok && !tokens_too) ||
      (o->test_starve_cta != 0 && !tokens_too))
    return host_fail(PA_ERR_UNSUPPORTED, "this call takes none of sliding_window, use_tcgen05, segment_cost_pages%s",
                     tokens_too ? "" : ", token scales, test_starve_cta");
  if (o->num_ctas < 0 || o->num_ctas > kMaxCtas || o->min_pages_per_cta < 0)
    return host_fail(PA_ERR_INVALID_ARG, "num_ctas must be in [0, %d] and min_pages_per_cta not negative", kMaxCtas);
  if (o->heads_per_cta < 0 || (o->heads_per_cta > 0 && Hkv % o->heads_per_cta != 0))
    return host_fail(PA_ERR_INVALID_ARG, "heads_per_cta %d must divide num_kv_heads %lld", o->heads_per_cta, ll(Hkv));
  if (o->wait_limit_us < 0 || o->test_starve_cta < 0 || o->test_give_up_cta < 0)
    return host_fail(PA_ERR_INVALID_ARG, "wait_limit_us, test_starve_cta and test_give_up_cta must not be negative");
  if (o->sinks && !host_aligned(o->sinks, 4)) return host_fail(PA_ERR_INVALID_ARG, "sinks must be 4-byte aligned");
  return PA_OK;
}

int check_rows(int64_t Hq, int64_t Hkv, int64_t max_qlen) {
  if (max_qlen < 1) return host_fail(PA_ERR_INVALID_ARG, "max_query_len %lld < 1", ll(max_qlen));
  if (Hq < 1 || Hkv < 1 || Hq % Hkv != 0)
    return host_fail(PA_ERR_INVALID_ARG, "num_q_heads %lld must be a positive multiple of num_kv_heads %lld", ll(Hq),
                     ll(Hkv));
  if (Hq / Hkv * max_qlen > kMaxRows)
    return host_fail(PA_ERR_UNSUPPORTED, "group size %lld x max_query_len %lld exceeds %d query rows per KV head",
                     ll(Hq / Hkv), ll(max_qlen), kMaxRows);
  return PA_OK;
}

// The tensors that both calls take.  *none: no query tokens, nothing to do.
int check_call(const pa_tensor_t* q, const pa_tensor_t* kc, const pa_tensor_t* vc, const pa_tensor_t* bt,
               const pa_tensor_t* sl, const pa_tensor_t* qsl, int32_t max_qlen, float scale, float k_scale,
               float v_scale, const pa_tensor_t* out, const pa_tensor_t* lse, Shape* shape, bool* none) {
  int st;
  *none = q != nullptr && q->ndim == 3 && q->shape[0] == 0;
  if ((st = host_check_tensor(q, "q", 3, *none)) || (st = host_check_tensor(kc, "k_cache", 4, false)) ||
      (st = host_check_tensor(vc, "v_cache", 4, false)) || (st = host_check_tensor(bt, "block_tables", 2, *none)) ||
      (st = host_check_tensor(sl, "seq_lens", 1, *none)) || (st = host_check_tensor(qsl, "query_start_loc", 1, true)) ||
      (st = host_check_tensor(out, "out", 3, *none)) || (st = host_check_tensor(lse, "lse", 2, true)))
    return st;
  if (*none) return PA_OK;
  if (q->dtype != PA_BF16 || out->dtype != PA_BF16) return host_fail(PA_ERR_INVALID_ARG, "q and out must be bf16");
  if (kc->dtype != PA_BF16 && kc->dtype != PA_FP8_E4M3)
    return host_fail(PA_ERR_INVALID_ARG, "k_cache must be bf16 or fp8 e4m3");
  if (vc->dtype != kc->dtype) return host_fail(PA_ERR_INVALID_ARG, "v_cache dtype differs from k_cache");
  if (bt->dtype != PA_I32 || sl->dtype != PA_I32 || (qsl->data && qsl->dtype != PA_I32))
    return host_fail(PA_ERR_INVALID_ARG, "block_tables, seq_lens and query_start_loc must be int32");
  if (lse->data && lse->dtype != PA_F32) return host_fail(PA_ERR_INVALID_ARG, "lse must be float32");
  const int64_t T = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const int64_t NB = kc->shape[0], Hkv = kc->shape[2], B = bt->shape[0], MB = bt->shape[1];
  if (B < 1 || B > kMaxSeqsHost)
    return host_fail(PA_ERR_UNSUPPORTED, "num_seqs %lld outside [1, %d]", ll(B), kMaxSeqsHost);
  if ((st = check_rows(Hq, Hkv, max_qlen)) != PA_OK) return st;
  if (D != 64 && D != 128) return host_fail(PA_ERR_UNSUPPORTED, "head_dim %lld not in {64, 128}", ll(D));
  if (kc->shape[1] != kPageTokens)
    return host_fail(PA_ERR_UNSUPPORTED, "page size %lld, only 16 is supported", ll(kc->shape[1]));
  if (kc->shape[3] != D)
    return host_fail(PA_ERR_INVALID_ARG, "k_cache head_dim %lld != q head_dim %lld", ll(kc->shape[3]), ll(D));
  for (int d = 0; d < 4; ++d)
    if (vc->shape[d] != kc->shape[d]) return host_fail(PA_ERR_INVALID_ARG, "v_cache shape differs from k_cache");
  if (Hq > (1 << 20) || T > (int64_t(1) << 30) || NB < 1 || NB > (int64_t(1) << 31) - 1 || MB > kMaxBlocks ||
      B * MB >= (int64_t(1) << 31))
    return host_fail(PA_ERR_UNSUPPORTED, "tensor extents too large");
  if (MB < 1) return host_fail(PA_ERR_INVALID_ARG, "block_tables needs a column");
  if (sl->shape[0] != B)
    return host_fail(PA_ERR_INVALID_ARG, "seq_lens has %lld entries, block_tables %lld rows", ll(sl->shape[0]), ll(B));
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
  if (q->stride[2] != 1 || (Hq > 1 && q->stride[1] != D) || (T > 1 && q->stride[0] % 8) || !host_aligned(q->data, 16))
    return host_fail(PA_ERR_INVALID_ARG, "q must have contiguous heads and 16-byte aligned rows");
  if (out->stride[2] != 1 || out->stride[1] % 4 || out->stride[0] % 4 || !host_aligned(out->data, 8))
    return host_fail(PA_ERR_INVALID_ARG,
                     "out must have a contiguous last dim, strides multiple of 4 elements, 8-byte alignment");
  if ((out->stride[0] == 0 && T > 1) || (out->stride[1] == 0 && Hq > 1) ||
      (lse->data && ((lse->stride[0] == 0 && T > 1) || (lse->stride[1] == 0 && Hq > 1))))
    return host_fail(PA_ERR_INVALID_ARG, "out and lse are written: their strides must not be 0");
  const int esz = kc->dtype == PA_FP8_E4M3 ? 1 : 2;
  for (const pa_tensor_t* c : {kc, vc}) {
    if (c->stride[3] != 1) return host_fail(PA_ERR_INVALID_ARG, "KV cache last dim must be contiguous");
    for (int d = 0; d < 3; ++d)
      if ((c->stride[d] * esz) % 16 != 0)
        return host_fail(PA_ERR_INVALID_ARG, "KV cache strides must be multiples of 16 bytes");
    if (!host_aligned(c->data, 16)) return host_fail(PA_ERR_INVALID_ARG, "KV cache data must be 16-byte aligned");
  }
  if (!std::isfinite(scale) || !std::isfinite(k_scale) || !std::isfinite(v_scale))
    return host_fail(PA_ERR_INVALID_ARG, "scale, k_scale and v_scale must be finite");
  *shape = Shape{T, Hq, Hkv, D, NB, B, MB, esz};
  return PA_OK;
}

// The call's own fields of the split kernel's parameters, and the merge's from them.
void fill_split(SplitParams* sp, const Shape& s, const pa_tensor_t* q, const pa_tensor_t* bt, const pa_tensor_t* sl,
                const pa_tensor_t* qsl, float scale, float k_scale, float v_scale, const pa_tensor_t* out,
                const pa_tensor_t* lse, const pa_options_t* opts, uint32_t* err) {
  sp->q = static_cast<const uint16_t*>(q->data);
  sp->q_stride_t = q->stride[0];
  sp->out = static_cast<uint16_t*>(out->data);
  sp->out_stride_t = out->stride[0];
  sp->out_stride_h = out->stride[1];
  sp->lse = static_cast<float*>(lse->data);
  sp->lse_stride_t = lse->data ? lse->stride[0] : 0;
  sp->lse_stride_h = lse->data ? lse->stride[1] : 0;
  sp->block_tables = static_cast<const int32_t*>(bt->data);
  sp->bt_stride = bt->stride[0];
  sp->seq_lens = static_cast<const int32_t*>(sl->data);
  sp->qsl = static_cast<const int32_t*>(qsl->data);
  sp->num_tokens = static_cast<int32_t>(s.T);
  sp->num_pages = static_cast<int32_t>(s.NB);
  sp->max_blocks = static_cast<int32_t>(s.MB);
  sp->sinks = opts ? static_cast<const float*>(opts->sinks) : nullptr;
  sp->scale_log2 = scale * (s.esz == 1 ? k_scale : 1.0f) * 1.4426950408889634f;
  sp->v_scale = s.esz == 1 ? v_scale : 1.0f;
  sp->err = err;
}

void fill_merge(MergeRowsParams* mp, const SplitParams& sp, int grid) {
  mp->out = sp.out;
  mp->out_stride_t = sp.out_stride_t;
  mp->out_stride_h = sp.out_stride_h;
  mp->lse = sp.lse;
  mp->lse_stride_t = sp.lse_stride_t;
  mp->lse_stride_h = sp.lse_stride_h;
  mp->seq_lens = sp.seq_lens;
  mp->qsl = sp.qsl;
  mp->num_seqs = sp.num_seqs;
  mp->num_tokens = sp.num_tokens;
  mp->max_blocks = sp.max_blocks;
  mp->window = sp.window;
  mp->first_tokens = sp.first_tokens;
  mp->G = sp.G;
  mp->HC = sp.HC;
  mp->NC = sp.NC;
  mp->R_max = sp.R_max;
  mp->max_qlen = sp.max_qlen;
  mp->Hq = sp.Hq;
  mp->split_grid = grid;
  mp->v_scale = sp.v_scale;
  mp->ws_unit = sp.ws_unit;
  mp->ws_ml = sp.ws_ml;
  mp->ws_o = sp.ws_o;
  mp->err = sp.err;
  mp->sinks = sp.sinks;
  mp->skip = sp.skip;
  mp->whole_row0 = sp.whole_row0;
}

// Pages a CTA takes at least: two, where a few sequences do not fill the CTAs (in a graph, 5
// short ones: 8.5 us, 10.4 with four; 3 of 200 tokens, 64 / 8 heads, fp8: 11.8 and 13.3).  One
// would take 7.2 and 9.3 there.
int min_pages_of(const pa_options_t* opts) {
  return opts && opts->min_pages_per_cta > 0 ? opts->min_pages_per_cta : 2;
}

// The options' split events (external nodes under capture).
struct Events {
  cudaEvent_t start, stop;
  unsigned int flags;
};
int events_of(const pa_options_t* opts, cudaStream_t stream, Events* ev) {
  ev->start = opts ? static_cast<cudaEvent_t>(opts->split_start_event) : nullptr;
  ev->stop = opts ? static_cast<cudaEvent_t>(opts->split_stop_event) : nullptr;
  ev->flags = cudaEventRecordDefault;
  if (ev->start == nullptr && ev->stop == nullptr) return PA_OK;
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  const cudaError_t e = cudaStreamIsCapturing(stream, &cs);
  if (e != cudaSuccess) return host_cuda_fail(e, "cudaStreamIsCapturing");
  if (cs == cudaStreamCaptureStatusActive) ev->flags = cudaEventRecordExternal;
  return PA_OK;
}
int record(cudaEvent_t ev, const Events& evs, cudaStream_t stream) {
  if (ev == nullptr) return PA_OK;
  const cudaError_t e = cudaEventRecordWithFlags(ev, stream, evs.flags);
  return e == cudaSuccess ? static_cast<int>(PA_OK) : host_cuda_fail(e, "cudaEventRecord");
}

int decode_window(const pa_tensor_t* q, const pa_tensor_t* kc, const pa_tensor_t* vc, const pa_tensor_t* bt,
                  const pa_tensor_t* sl, const pa_tensor_t* qsl, int32_t max_qlen, int32_t window, int32_t first,
                  float scale, float k_scale, float v_scale, const pa_tensor_t* out, const pa_tensor_t* lse,
                  const pa_options_t* opts, cudaStream_t stream) {
  Shape s;
  bool none;
  int st = check_call(q, kc, vc, bt, sl, qsl, max_qlen, scale, k_scale, v_scale, out, lse, &s, &none);
  if (st != PA_OK) return st;
  if (window < 1 || first < 0)
    return host_fail(PA_ERR_INVALID_ARG, "window %d must be positive and first_tokens %d not negative", window, first);
  if (none) return PA_OK;
  if ((st = check_options(opts, s.Hkv, true)) != PA_OK) return st;
  const pa_tensor_t* ts[2] = {opts ? opts->k_token_scales : nullptr, opts ? opts->v_token_scales : nullptr};
  const bool tok = (ts[0] && ts[0]->data) || (ts[1] && ts[1]->data);
  for (int x = 0; x < 2 && tok; ++x) {
    const char* nm = x ? "v_token_scales" : "k_token_scales";
    if (s.esz != 1) return host_fail(PA_ERR_INVALID_ARG, "per-token scales need an fp8 cache");
    if ((st = host_check_tensor(ts[x], nm, 3, false)) != PA_OK) return st;
    if (ts[x]->dtype != PA_F32 || ts[x]->shape[0] != s.NB || ts[x]->shape[1] != s.Hkv || ts[x]->shape[2] != kPageTokens)
      return host_fail(PA_ERR_INVALID_ARG, "%s must be float32 [NB, Hkv, 16]", nm);
    if (ts[x]->stride[2] != 1 || ts[x]->stride[1] != kPageTokens || ts[x]->stride[0] % 4 != 0 ||
        !host_aligned(ts[x]->data, 16))
      return host_fail(PA_ERR_INVALID_ARG, "%s: each page's [Hkv, 16] block must be contiguous and 16-byte aligned", nm);
    if (ts[0]->stride[0] != ts[x]->stride[0])
      return host_fail(PA_ERR_INVALID_ARG, "k_token_scales and v_token_scales need the same page stride");
  }

  auto lock = host_lock();
  HostDevice dev;
  if ((st = host_device(&dev)) != PA_OK) return st;
  HostSplitPlan pl;
  if ((st = host_split_plan(static_cast<int>(s.B), static_cast<int>(s.Hq), static_cast<int>(s.Hkv),
                            static_cast<int>(s.D), kc->dtype, max_qlen, opts, 3, dev, &pl)) != PA_OK)
    return st;
  // the layout and size of paged_attn_decode's workspace
  const size_t ws_ml = up(static_cast<size_t>(16) * s.B * pl.sp.NC, 256), ws_o = up(ws_ml + pl.rows * 8, 256);
  void* ws = nullptr;
  if ((st = host_workspace(opts, up(ws_o + pl.rows * s.D * 4, 256), stream, "paged_attn_reserve", &ws)) != PA_OK)
    return st;
  CUtensorMap tk, tv;
  const int D = static_cast<int>(s.D), Hkv = static_cast<int>(s.Hkv);
  if ((st = host_cache_map(&tk, kc, s.esz, D, Hkv, pl.sp.HC, s.NB)) != PA_OK) return st;
  if ((st = host_cache_map(&tv, vc, s.esz, D, Hkv, pl.sp.HC, s.NB)) != PA_OK) return st;
  SplitParams& sp = pl.sp;
  sp.min_pages = min_pages_of(opts);
  fill_split(&sp, s, q, bt, sl, qsl, scale, k_scale, v_scale, out, lse, opts, dev.status);
  // Nothing changes once a window or the first tokens hold every position a row of the
  // block table has; the kernels' sums of positions and windows stay within 32 bits.
  const int64_t most = kPageTokens * s.MB;
  sp.window = static_cast<int32_t>(std::min<int64_t>(window, most));
  sp.first_tokens = static_cast<int32_t>(std::min<int64_t>(first, most));
  if (tok) {
    sp.k_tok = static_cast<const float*>(ts[0]->data);
    sp.v_tok = static_cast<const float*>(ts[1]->data);
    sp.tok_stride_page = ts[0]->stride[0];
  }
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  sp.ws_unit = reinterpret_cast<int4*>(wsb);
  sp.ws_ml = reinterpret_cast<float2*>(wsb + ws_ml);
  sp.ws_o = reinterpret_cast<float*>(wsb + ws_o);
  MergeRowsParams mp = {};
  fill_merge(&mp, sp, pl.grid);

  Events ev;
  if ((st = events_of(opts, stream, &ev)) != PA_OK) return st;
  const bool pdl = !(opts && opts->disable_pdl);
  if ((st = record(ev.start, ev, stream)) != PA_OK) return st;
  cudaError_t e = launch_split_first(D, s.esz == 1, tk, tv, sp, pl.grid, pl.threads, pl.smem, pdl && !ev.start, stream);
  if (e != cudaSuccess) return host_cuda_fail(e, "split kernel launch");
  if ((st = record(ev.stop, ev, stream)) != PA_OK) return st;
  const int units = static_cast<int>(s.B) * sp.NC;
  const bool wide = pl.grid >= 4 * units;
  if ((e = launch_merge_rows(D, false, mp, units, sp.HC * sp.R_max, wide, pdl && !ev.stop, stream)) != cudaSuccess)
    return host_cuda_fail(e, "merge kernel launch");
  return PA_OK;
}

// ------------------------------------------------------------ shared prefixes
// Prefixes that are left to the sequences, where both parts run side by side (elsewhere every
// prefix is shared): of fewer than 16 pages (200 sequences of 32 / 8 heads of 128 behind 100
// tokens, in a graph: 99 us shared, 52 not; behind 300, 62 and 73), and all of a call that
// would cost an SM less than 2 us (4 sequences behind 1000 tokens: 15.8 and 16.7 us, of 2 heads
// of 64, 14.3 and 14.6; of those behind 100, 14.2 and 13.2).
constexpr int kMinSharedPages = 16;
constexpr int kAloneCost = 2000;          // ns, as below
// What the plan cuts the SMs by (nanoseconds on one SM).  Measured with 4 and 128 of 152 SMs
// for one part: a step (pa_shared.h) takes 1.6 us (fp8 codes 2.3, of 64 features 1.75), a
// page for one head and 16 query rows 0.165 us (64 features 0.06, fp8 0.064; 128, fp8,
// 0.094), and a sequence about what three of its pages do.
struct Costs {
  int step, page;
};
Costs costs_of(int64_t D, bool fp8) {
  if (D == 128) return fp8 ? Costs{2300, 94} : Costs{1600, 165};
  return fp8 ? Costs{1750, 64} : Costs{1600, 59};
}

struct SharedPlan {
  HostSplitPlan split;
  int grid;                      // of the prefix kernel
  size_t skip, ready, group_of, groups, totals, pre_ml, pre_o, unit, ml, o, bytes;
};

// Grids and the workspace of a call.
int plan_shared(int64_t T, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int kv_dtype, int max_qlen,
                const pa_options_t* opts, const HostDevice& dev, SharedPlan* out) {
  if (dev.shared_prefix != cudaSuccess) return host_cuda_fail(dev.shared_prefix, "set-up of the shared prefix kernel");
  SharedPlan p = {};
  const int st = host_split_plan(static_cast<int>(B), static_cast<int>(Hq), static_cast<int>(Hkv), static_cast<int>(D),
                                 kv_dtype, max_qlen, opts, 4, dev, &p.split);
  if (st != PA_OK) return st;
  p.grid = opts && opts->num_ctas > 0 ? opts->num_ctas : dev.num_sms;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = up(at + bytes, 256);
    return here;
  };
  p.skip = take(4 * static_cast<size_t>(B));
  p.ready = take(sizeof(uint64_t));
  p.group_of = take(4 * static_cast<size_t>(B));
  p.groups = take(sizeof(SharedGroup) * static_cast<size_t>(B));
  p.totals = take(sizeof(SharedTotals));
  p.unit = take(static_cast<size_t>(16) * B * p.split.sp.NC);
  // cut units' rows, then a row for every (token, query head)
  const size_t rows = p.split.rows + static_cast<size_t>(T) * Hq;
  p.ml = take(rows * 8);
  p.o = take(rows * D * 4);
  // a pair's rows at most twice (a single tile's two slots), and 256 a CTA
  const size_t pre = 2 * static_cast<size_t>(T) * Hq + static_cast<size_t>(kSharedPair) * p.grid;
  p.pre_ml = take(pre * 8);
  p.pre_o = take(pre * D * 4);
  p.bytes = at;
  *out = p;
  return PA_OK;
}

int decode_shared(const pa_tensor_t* q, const pa_tensor_t* kc, const pa_tensor_t* vc, const pa_tensor_t* bt,
                  const pa_tensor_t* sl, const pa_tensor_t* qsl, int32_t max_qlen, const pa_tensor_t* gsl,
                  const pa_tensor_t* lens, float scale, float k_scale, float v_scale, const pa_tensor_t* out,
                  const pa_tensor_t* lse, const pa_options_t* opts, cudaStream_t stream) {
  Shape s;
  bool none;
  int st = check_call(q, kc, vc, bt, sl, qsl, max_qlen, scale, k_scale, v_scale, out, lse, &s, &none);
  if (st != PA_OK) return st;
  const bool no_groups = lens != nullptr && lens->ndim == 1 && lens->shape[0] == 0;
  if ((st = host_check_tensor(gsl, "group_start_loc", 1, none || no_groups)) ||
      (st = host_check_tensor(lens, "shared_lens", 1, none || no_groups)))
    return st;
  if (none) return PA_OK;
  const int64_t NG = lens->shape[0];
  if (!no_groups) {
    if (gsl->dtype != PA_I32 || lens->dtype != PA_I32)
      return host_fail(PA_ERR_INVALID_ARG, "group_start_loc and shared_lens must be int32");
    if (gsl->shape[0] != NG + 1 || gsl->stride[0] != 1 || (NG > 1 && lens->stride[0] != 1))
      return host_fail(PA_ERR_INVALID_ARG, "group_start_loc needs one entry more than shared_lens, both contiguous");
  }
  if (NG > s.B)
    return host_fail(PA_ERR_UNSUPPORTED, "%lld groups for %lld sequences", ll(NG), ll(s.B));
  if (s.T * s.Hq >= (int64_t(1) << 30)) return host_fail(PA_ERR_UNSUPPORTED, "tensor extents too large");
  if ((st = check_options(opts, s.Hkv, false)) != PA_OK) return st;

  auto lock = host_lock();
  HostDevice dev;
  if ((st = host_device(&dev)) != PA_OK) return st;
  SharedPlan pl;
  if ((st = plan_shared(s.T, s.B, s.Hq, s.Hkv, s.D, kc->dtype, max_qlen, opts, dev, &pl)) != PA_OK) return st;
  void* ws = nullptr;
  if ((st = host_workspace(opts, pl.bytes, stream, "paged_attn_shared_reserve", &ws)) != PA_OK) return st;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  CUtensorMap tk, tv, pk, pv;
  const int D = static_cast<int>(s.D), Hkv = static_cast<int>(s.Hkv);
  SplitParams& sp = pl.split.sp;
  sp.min_pages = min_pages_of(opts);
  if ((st = host_cache_map(&tk, kc, s.esz, D, Hkv, sp.HC, s.NB)) != PA_OK) return st;
  if ((st = host_cache_map(&tv, vc, s.esz, D, Hkv, sp.HC, s.NB)) != PA_OK) return st;
  bool split_k = false, split_v = false;
  if ((st = host_prefix_map(&pk, kc, s.esz, D, Hkv, s.NB, &split_k)) != PA_OK) return st;
  if ((st = host_prefix_map(&pv, vc, s.esz, D, Hkv, s.NB, &split_v)) != PA_OK) return st;
  fill_split(&sp, s, q, bt, sl, qsl, scale, k_scale, v_scale, out, lse, opts, dev.status);
  sp.ws_unit = reinterpret_cast<int4*>(wsb + pl.unit);
  sp.ws_ml = reinterpret_cast<float2*>(wsb + pl.ml);
  sp.ws_o = reinterpret_cast<float*>(wsb + pl.o);
  sp.skip = reinterpret_cast<const int32_t*>(wsb + pl.skip);
  sp.whole_row0 = static_cast<int64_t>(pl.split.rows);

  const bool pdl = !(opts && opts->disable_pdl);
  SharedParams hp = {};
  hp.q = sp.q;
  hp.q_stride_t = sp.q_stride_t;
  hp.block_tables = sp.block_tables;
  hp.bt_stride = sp.bt_stride;
  hp.seq_lens = sp.seq_lens;
  hp.qsl = sp.qsl;
  hp.group_start = static_cast<const int32_t*>(gsl->data);
  hp.shared_lens = static_cast<const int32_t*>(lens->data);
  hp.num_seqs = sp.num_seqs;
  hp.num_tokens = sp.num_tokens;
  hp.num_groups = static_cast<int32_t>(NG);
  hp.max_qlen = max_qlen;
  hp.max_blocks = sp.max_blocks;
  hp.num_pages = sp.num_pages;
  hp.G = sp.G;
  hp.Hkv = sp.Hkv;
  hp.split_boxes = (split_k ? 1 : 0) | (split_v ? 2 : 0);
  hp.ctas = pl.grid;
  hp.own_ctas = pl.split.grid;
  // Both grids are then one CTA an SM at most, the plan's shares add up to the SMs, and the
  // split kernel may start when the plan is made.
  hp.beside = pdl && pl.grid == dev.num_sms && pl.split.grid == dev.num_sms;
  hp.min_pages = hp.beside ? kMinSharedPages : 1;
  const Costs cost = costs_of(s.D, s.esz == 1);
  hp.step_cost = cost.step;
  hp.page_cost = cost.page * ((sp.R_max + 15) / 16);
  hp.unit_cost = 3 * hp.page_cost;
  hp.alone_cost = kAloneCost;
  hp.scale_log2 = sp.scale_log2;
  hp.wait_ns = sp.wait_ns;
  hp.give_up_cta = sp.give_up_cta;
  hp.err = dev.status;
  hp.skip = reinterpret_cast<int32_t*>(wsb + pl.skip);
  hp.seq_group = reinterpret_cast<int32_t*>(wsb + pl.group_of);
  hp.groups = reinterpret_cast<SharedGroup*>(wsb + pl.groups);
  hp.totals = reinterpret_cast<SharedTotals*>(wsb + pl.totals);
  hp.ready = reinterpret_cast<uint64_t*>(wsb + pl.ready);
  // (odd multiples: no two calls have the same 48 bits, and few look like what a workspace holds)
  static uint64_t calls = 0;
  hp.call = (++calls * 0x9E3779B97F4A7C15ull) & ((uint64_t(1) << (64 - kReadyBits)) - 1);
  hp.ws_ml = reinterpret_cast<float2*>(wsb + pl.pre_ml);
  hp.ws_o = reinterpret_cast<float*>(wsb + pl.pre_o);

  MergeRowsParams mp = {};
  fill_merge(&mp, sp, pl.split.grid);
  mp.seq_group = hp.seq_group;
  mp.groups = hp.groups;
  mp.totals = hp.totals;
  mp.pre_ml = hp.ws_ml;
  mp.pre_o = hp.ws_o;
  mp.ready = hp.ready;
  sp.ready = hp.ready;
  sp.call = hp.call;

  Events ev;
  if ((st = events_of(opts, stream, &ev)) != PA_OK) return st;
  cudaError_t e;
  if ((st = record(ev.start, ev, stream)) != PA_OK) return st;
  if ((e = launch_shared_plan(hp, pdl && !ev.start, stream)) != cudaSuccess)
    return host_cuda_fail(e, "shared prefix plan kernel launch");
  if ((e = launch_shared_prefix(D, s.esz == 1, pk, pv, hp, pl.grid, pdl, stream)) != cudaSuccess)
    return host_cuda_fail(e, "shared prefix kernel launch");
  if ((e = launch_split_own(D, s.esz == 1, tk, tv, sp, pl.split.grid, pl.split.threads, pl.split.smem, pdl, stream)) !=
      cudaSuccess)
    return host_cuda_fail(e, "split kernel launch");
  if ((st = record(ev.stop, ev, stream)) != PA_OK) return st;
  const int units = static_cast<int>(s.B) * sp.NC;
  const bool wide = pl.split.grid >= 4 * units;
  if ((e = launch_merge_rows(D, true, mp, units, sp.HC * sp.R_max, wide, pdl && !ev.stop, stream)) != cudaSuccess)
    return host_cuda_fail(e, "merge kernel launch");
  return PA_OK;
}

int shared_plan_for(int32_t T, int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t kv_dtype, int32_t max_qlen,
                    const pa_options_t* o, SharedPlan* pl) {
  int st;
  if (B < 1 || B > kMaxSeqsHost)
    return host_fail(PA_ERR_UNSUPPORTED, "num_seqs %d outside [1, %d]", B, kMaxSeqsHost);
  if (T < 0 || static_cast<int64_t>(T) * std::max(Hq, 0) >= (int64_t(1) << 30))
    return host_fail(PA_ERR_UNSUPPORTED, "num_tokens %d x num_q_heads %d outside [0, 2^30)", T, Hq);
  if ((st = check_rows(Hq, Hkv, max_qlen)) != PA_OK || (st = check_options(o, Hkv, false)) != PA_OK) return st;
  HostDevice dev;
  if ((st = host_device(&dev)) != PA_OK) return st;
  return plan_shared(T, B, Hq, Hkv, D, kv_dtype, max_qlen, o, dev, pl);
}

}  // namespace
}  // namespace pa

extern "C" int paged_attn_decode_shared(const pa_tensor_t* q, const pa_tensor_t* k_cache, const pa_tensor_t* v_cache,
                                        const pa_tensor_t* block_tables, const pa_tensor_t* seq_lens,
                                        const pa_tensor_t* query_start_loc, int32_t max_query_len,
                                        const pa_tensor_t* group_start_loc, const pa_tensor_t* shared_lens, float scale,
                                        float k_scale, float v_scale, const pa_tensor_t* out, const pa_tensor_t* lse,
                                        const pa_options_t* opts, pa_stream_t stream) {
  return pa::host_entry([&] {
    return pa::decode_shared(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, max_query_len,
                             group_start_loc, shared_lens, scale, k_scale, v_scale, out, lse, opts,
                             reinterpret_cast<cudaStream_t>(stream));
  });
}

extern "C" int paged_attn_shared_workspace_size(int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                                                int32_t num_kv_heads, int32_t head_dim, int32_t kv_dtype,
                                                int32_t max_query_len, const pa_options_t* opts, size_t* bytes) {
  return pa::host_entry([&] {
    if (bytes == nullptr) return pa::host_fail(PA_ERR_INVALID_ARG, "bytes pointer is NULL");
    auto lock = pa::host_lock();
    pa::SharedPlan pl;
    const int st = pa::shared_plan_for(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, kv_dtype,
                                       max_query_len, opts, &pl);
    if (st == PA_OK) *bytes = pl.bytes;
    return st;
  });
}

extern "C" int paged_attn_shared_reserve(int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                                         int32_t num_kv_heads, int32_t head_dim, int32_t kv_dtype,
                                         int32_t max_query_len) {
  return pa::host_entry([&] {
    auto lock = pa::host_lock();
    pa::SharedPlan pl;
    const int st = pa::shared_plan_for(num_tokens, num_seqs, num_q_heads, num_kv_heads, head_dim, kv_dtype,
                                       max_query_len, nullptr, &pl);
    return st != PA_OK ? st : pa::host_reserve(pl.bytes);
  });
}

extern "C" int paged_attn_decode_window(const pa_tensor_t* q, const pa_tensor_t* k_cache, const pa_tensor_t* v_cache,
                                        const pa_tensor_t* block_tables, const pa_tensor_t* seq_lens,
                                        const pa_tensor_t* query_start_loc, int32_t max_query_len, int32_t window,
                                        int32_t first_tokens, float scale, float k_scale, float v_scale,
                                        const pa_tensor_t* out, const pa_tensor_t* lse, const pa_options_t* opts,
                                        pa_stream_t stream) {
  return pa::host_entry([&] {
    return pa::decode_window(q, k_cache, v_cache, block_tables, seq_lens, query_start_loc, max_query_len, window,
                             first_tokens, scale, k_scale, v_scale, out, lse, opts,
                             reinterpret_cast<cudaStream_t>(stream));
  });
}
