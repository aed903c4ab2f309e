// block_api.cpp -- the C ABI of the operators around a block's products (include/muon_block.h): argument
// checks, workspaces and launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/muon_block.h"
#include "api_common.h"
#include "gate.h"
#include "mx.h"
#include "norm.h"

namespace {

using muon::aligned;
using muon::bad;
using muon::elem;
using muon::hip_result;
using muon::set_error;

constexpr int64_t kMaxRows = (int64_t(1) << 31) - 1024;  // as a layer's
constexpr int64_t kMaxCols = int64_t(1) << 24;           // a norm's: its kernels count columns in 32 bits
constexpr int64_t kMaxMx = int64_t(1) << 23;             // k and n of a weight
constexpr int kCus = 256;

int check_dtype(int32_t dtype) {
  return dtype == MUON_F32 || dtype == MUON_BF16 ? MUON_OK : bad("dtype must be MUON_F32 or MUON_BF16");
}
// A pointer that has to be there (`count` elements of `size` bytes behind it), or may be null (count 0).
int check_at(const void* p, int64_t count, int size, const char* name) {
  if (count > 0 && !p) return set_error(MUON_ERR_INVALID_ARGUMENT, "%s is null", name);
  if (!aligned(p, size)) return set_error(MUON_ERR_INVALID_ARGUMENT, "%s is not %d-byte aligned", name, size);
  return MUON_OK;
}
int check_space(uint64_t need, const void* ws, uint64_t bytes) {
  if (bytes < need || (need && !ws)) return bad("the workspace is smaller than the operator's workspace call says");
  return aligned(ws, 16) ? MUON_OK : bad("the workspace is not 16-byte aligned");
}

// ---- norms

int check_norm(const muon_norm_desc_t* d) {
  if (!d) return bad("desc is null");
  MUON_TRY(check_dtype(d->dtype));
  if (d->kind != MUON_NORM_LAYER && d->kind != MUON_NORM_RMS) return bad("unknown norm");
  if (d->rows < 0 || d->rows > kMaxRows) return bad("rows outside [0, 2^31 - 1024]");
  if (d->cols < 0 || d->cols > kMaxCols) return bad("cols outside [0, 2^24]");
  if (d->ldx < 0 || d->ldr < 0 || d->ldg < 0 || d->ldd < 0) return bad("a stride is negative");
  if (!(d->eps >= 0.0 && d->eps < 1e30)) return bad("eps is negative or not finite");
  return MUON_OK;
}
uint64_t norm_bytes(const muon_norm_desc_t* d) { return (uint64_t)muon::norm_parts(d->rows, d->cols) * 2 * d->cols * 4; }

// ---- gate and balance

int check_gate(const muon_gate_desc_t* d) {
  if (!d) return bad("desc is null");
  MUON_TRY(check_dtype(d->dtype));
  if (d->experts < 1 || d->experts > muon::kGateMaxExperts) return bad("experts outside [1, 1024]");
  if (d->top < 1 || d->top > d->experts) return bad("top outside [1, experts]");
  if (d->tokens < 0 || d->tokens > kMaxRows) return bad("tokens outside [0, 2^31 - 1024]");
  if (d->ldz < 0) return bad("a stride is negative");
  return MUON_OK;
}
// Counts are held in 32 bits, so the balance loss ends where they would.
int check_balance(const muon_gate_desc_t* d) {
  if (d && d->top >= 1 && d->tokens > kMaxRows / d->top) return bad("tokens * top is over 2^31 - 1024");
  // An id list may be longer than there are experts (a token's choices need not differ here).
  muon_gate_desc_t one = d ? *d : muon_gate_desc_t{};
  if (d && one.top > one.experts) one.top = one.experts;
  return check_gate(d ? &one : nullptr);
}
uint64_t balance_bytes(const muon_gate_desc_t* d) {
  return (uint64_t)muon::balance_blocks(d->tokens, d->experts) * (2 * d->experts + 1) * 4;
}
muon::GateArgs gate_args(const muon_gate_desc_t* d, const void* logits, const uint8_t* mask) {
  muon::GateArgs a{};
  a.logits = logits;
  a.mask = mask;
  a.tokens = d->tokens;
  a.ldz = d->ldz;
  a.experts = d->experts;
  a.top = d->top;
  a.normalize = d->normalize;
  return a;
}
muon::BalanceArgs balance_args(const muon_gate_desc_t* d, const void* logits, const uint8_t* mask) {
  muon::BalanceArgs a{};
  a.logits = logits;
  a.mask = mask;
  a.tokens = d->tokens;
  a.ldz = d->ldz;
  a.experts = d->experts;
  a.top = d->top;
  return a;
}

// ---- four bits

int check_mx(const muon_mx_desc_t* d) {
  if (!d) return bad("desc is null");
  MUON_TRY(check_dtype(d->dtype));
  if (d->act < MUON_ACT_NONE || d->act > MUON_ACT_GELU_TANH) return bad("unknown activation");
  if (d->groups < 0 || d->groups > 65535) return bad("groups outside [0, 65535]");
  if (d->w_layout != 0 && d->w_layout != 1) return bad("w_layout must be 0 or 1");
  if (d->rows < 0 || d->rows > kMaxRows) return bad("rows outside [0, 2^31 - 1024]");
  if (d->k < 0 || d->n < 0 || d->k > kMaxMx || d->n > kMaxMx) return bad("k or n outside [0, 2^23]");
  if (d->ldx < 0 || d->ldw < 0 || d->w_stride < 0 || d->ldr < 0) return bad("a stride is negative");
  return MUON_OK;
}
int64_t mx_weights(const muon_mx_desc_t* d) { return std::max(d->groups, 1); }
int check_mx_weight(const muon_mx_desc_t* d, const uint8_t* values, const uint8_t* scales) {
  MUON_TRY(check_at(values, d->k * d->n, 16, "values"));
  return check_at(scales, d->k * d->n, 16, "scales");
}
muon::MxArgs mx_args(const muon_mx_desc_t* d) {
  muon::MxArgs a{};
  a.rows = d->n;
  a.k = d->k;
  a.ld = d->ldw;
  a.step = d->w_stride;
  a.groups = (int32_t)mx_weights(d);
  a.t = d->w_layout == 0;
  return a;
}
// A layer's product: its tile and split, and what it takes of the workspace.  Times in us, bf16, of a whole
// call without bias, activation or residual, the weights from HBM; each pair is the kernel named first and the other:
//  - Up to 4 rows (on average, of experts) the product takes x to four bits itself, where a launch ahead of it costs
//    more than doing so in every workgroup.  x [4096, 16384]: 1 row 9.4 and 11.9, 4 rows 10.7 and 11.7, 5 rows 11.2 and 11.9,
//    8 rows 13.3 and 11.7, 16 rows 18.7 and 12.1.
//  - Up to 32 rows, or 16 an expert, the weight goes straight to registers (32 x 4096 x 16384: 12.8 and 13.4); from 64 on
//    64 x 64 tiles are faster (64 x 4096 x 16384: 13.8 and 17.7; 64 experts [2048, 1408] with 32 rows each: 31 and 35, with 16
//    each 28 either way).
//  - 64 x 64 below 256 tiles of 128 x 128 (128 x 4096 x 16384: 16.8 and 30.6), and for up to 32 rows an expert.
//  - 128 x 128 below 256 rows (64 experts with 128 each: 44 and 53) or 256 tiles of 256 x 128 (256 x 4096 x 16384: 19 and 43;
//    1024 x 4096 x 4096: 19 and 41).
//  - 256 x 128 above (8192 x 4096 x 16384: 327, with 128 x 128 389, with 64 x 64 511; with gelu, bias and residual 391 and 446;
//    2048 x 4096 x 4096: 31.5 and 31).
//    256 x 256 with one workgroup a unit was 4 - 7% faster without an activation or a residual and 4 - 8% slower with
//    both, whose work nothing hides then.
// Tiles that do not fill the card are split along the contraction, two chunks of 512 each at least.
constexpr int64_t kMxOwnRows = 4;
struct MxPlan {
  muon::MxProduct p{};
  int tile = 0, cols = 0;
  uint64_t x_values = 0, x_scales = 0, partials = 0;  // bytes
  bool own() const { return tile == muon::kMxRowsOwn; }
  uint64_t bytes() const { return x_values + x_scales + partials; }
};

MxPlan mx_plan(const muon_mx_desc_t* d) {
  MxPlan q;
  muon::GemmArgs& g = q.p.g;
  const bool grouped = d->groups > 0;
  g.m = d->rows;
  g.n = d->n;
  g.k = muon::mx_slices(d->k);
  g.groups = std::max(d->groups, 1);
  g.sb = muon::mx_value_bytes(d->n, d->k);
  g.splits = 1;
  g.k_per = g.k;
  auto blocks_m = [&](int tile) { return muon::group_blocks(d->rows, d->groups, grouped, muon::mx_tile_m(tile)); };
  auto tiles = [&](int tile) { return blocks_m(tile) * ((d->n + muon::mx_tile_n(tile, 0, 0) - 1) / muon::mx_tile_n(tile, 0, 0)); };
  const int64_t m_each = grouped ? d->rows / d->groups : d->rows;
  if (m_each <= (grouped ? 16 : 32))
    q.tile = m_each <= kMxOwnRows ? muon::kMxRowsOwn : m_each <= 16 ? muon::kMxRows16 : muon::kMxRows32;
  else if (m_each >= 256 && tiles(muon::kMx256x128) >= kCus) q.tile = muon::kMx256x128;
  else if (m_each > 32 && tiles(muon::kMx128) >= kCus) q.tile = muon::kMx128;
  else q.tile = muon::kMx64;
  q.cols = muon::mx_tile_n(q.tile, blocks_m(q.tile), d->n);
  g.tiles_m = (int32_t)blocks_m(q.tile);
  g.tiles_n = (int32_t)((d->n + q.cols - 1) / q.cols);
  if (q.own()) return q;
  q.x_values = (uint64_t)muon::mx_value_bytes(d->rows, d->k);
  q.x_scales = (uint64_t)muon::mx_scale_bytes(d->rows, d->k);
  const int64_t t = (int64_t)g.tiles_m * g.tiles_n, chunks = muon::mx_chunks(d->k);
  if (q.tile <= muon::kMx64 && !grouped && t > 0 && t < kCus && chunks >= 4) {
    const int64_t s = std::min<int64_t>((2 * kCus + t - 1) / t, chunks / 2), per = (chunks + s - 1) / s;
    if (per < chunks) {
      g.k_per = 4 * per;
      g.splits = (int32_t)((chunks + per - 1) / per);
      q.partials = (uint64_t)g.splits * g.m * g.n * 4;
    }
  }
  return q;
}

}  // namespace

extern "C" {

int muon_norm_workspace(const muon_norm_desc_t* d, uint64_t* bytes) {
  if (!bytes) return bad("bytes is null");
  *bytes = 0;
  MUON_TRY(check_norm(d));
  *bytes = norm_bytes(d);
  return set_error(MUON_OK, "%s", "");
}

int muon_norm_forward(const muon_norm_desc_t* d, const void* x, const void* residual, const void* w, const void* b,
                      void* y, void* s, float* stats, void* stream) {
  MUON_TRY(check_norm(d));
  const int es = elem(d->dtype);
  const int64_t count = d->rows * d->cols;
  MUON_TRY(check_at(x, count, es, "x"));
  MUON_TRY(check_at(residual, 0, es, "residual"));
  MUON_TRY(check_at(w, 0, es, "w"));
  MUON_TRY(check_at(b, 0, es, "b"));
  MUON_TRY(check_at(y, count, es, "y"));
  MUON_TRY(check_at(s, residual ? count : 0, es, "s"));
  MUON_TRY(check_at(stats, 0, 4, "stats"));
  if (s && !residual) return bad("s is given without a residual");
  const muon::NormArgs a{x,       residual, w,      b,      y, s, stats, d->rows, d->cols, d->ldx, d->ldr, (float)d->eps,
                         d->kind == MUON_NORM_LAYER};
  return hip_result(muon::launch_norm(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_norm_forward");
}

int muon_norm_backward(const muon_norm_desc_t* d, const void* dy, const void* x, const void* residual, const void* w,
                       const float* stats, const void* ds, void* dx, void* dw, void* db, void* ws, uint64_t ws_bytes,
                       void* stream) {
  MUON_TRY(check_norm(d));
  if (!dx && !dw && !db) return set_error(MUON_OK, "%s", "");
  const int es = elem(d->dtype);
  const int64_t count = d->rows * d->cols;
  MUON_TRY(check_at(dy, count, es, "dy"));
  MUON_TRY(check_at(x, count, es, "x"));
  MUON_TRY(check_at(residual, 0, es, "residual"));
  MUON_TRY(check_at(w, 0, es, "w"));
  MUON_TRY(check_at(stats, count, 4, "stats"));
  MUON_TRY(check_at(ds, 0, es, "ds"));
  MUON_TRY(check_at(dx, 0, es, "dx"));
  MUON_TRY(check_at(dw, 0, es, "dw"));
  MUON_TRY(check_at(db, 0, es, "db"));
  if (dw || db) MUON_TRY(check_space(norm_bytes(d), ws, ws_bytes));
  const muon::NormGradArgs a{dy, x, residual, w, ds, stats, dx, dw, db, dw || db ? static_cast<float*>(ws) : nullptr,
                             d->rows, d->cols, d->ldg, d->ldx, d->ldr, d->ldd, d->kind == MUON_NORM_LAYER};
  return hip_result(muon::launch_norm_grad(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_norm_backward");
}

int muon_gate_forward(const muon_gate_desc_t* d, const void* logits, const uint8_t* mask, float* weights, int32_t* ids,
                      void* stream) {
  MUON_TRY(check_gate(d));
  MUON_TRY(check_at(logits, d->tokens, elem(d->dtype), "logits"));
  MUON_TRY(check_at(weights, d->tokens, 4, "weights"));
  MUON_TRY(check_at(ids, d->tokens, 4, "ids"));
  muon::GateArgs a = gate_args(d, logits, mask);
  a.weights = weights;
  a.ids = ids;
  return hip_result(muon::launch_gate(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_gate_forward");
}

int muon_gate_backward(const muon_gate_desc_t* d, const void* logits, const uint8_t* mask, const float* weights,
                       const int32_t* ids, const float* dweights, void* dlogits, void* stream) {
  MUON_TRY(check_gate(d));
  MUON_TRY(check_at(logits, d->normalize ? 0 : d->tokens, elem(d->dtype), "logits"));
  MUON_TRY(check_at(weights, d->tokens, 4, "weights"));
  MUON_TRY(check_at(ids, d->tokens, 4, "ids"));
  MUON_TRY(check_at(dweights, d->tokens, 4, "dweights"));
  MUON_TRY(check_at(dlogits, d->tokens, elem(d->dtype), "dlogits"));
  muon::GateArgs a = gate_args(d, logits, mask);
  a.weights = const_cast<float*>(weights);
  a.ids = const_cast<int32_t*>(ids);
  a.dweights = dweights;
  a.dlogits = dlogits;
  return hip_result(muon::launch_gate_grad(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_gate_backward");
}

int muon_balance_workspace(const muon_gate_desc_t* d, uint64_t* bytes) {
  if (!bytes) return bad("bytes is null");
  *bytes = 0;
  MUON_TRY(check_balance(d));
  *bytes = balance_bytes(d);
  return set_error(MUON_OK, "%s", "");
}

int muon_balance_forward(const muon_gate_desc_t* d, const void* logits, const void* ids, int32_t ids_bytes,
                         const uint8_t* mask, float* loss, int32_t* counts, float* shares, void* ws, uint64_t ws_bytes,
                         void* stream) {
  MUON_TRY(check_balance(d));
  if (ids_bytes != 4 && ids_bytes != 8) return bad("ids_bytes must be 4 or 8");
  MUON_TRY(check_at(logits, d->tokens, elem(d->dtype), "logits"));
  MUON_TRY(check_at(ids, d->tokens, ids_bytes, "ids"));
  MUON_TRY(check_at(loss, 1, 4, "loss"));
  MUON_TRY(check_at(counts, 1, 4, "counts"));
  MUON_TRY(check_at(shares, 1, 4, "shares"));
  MUON_TRY(check_space(balance_bytes(d), ws, ws_bytes));
  muon::BalanceArgs a = balance_args(d, logits, mask);
  a.ids = ids;
  a.ids64 = ids_bytes == 8;
  a.loss = loss;
  a.counts = counts;
  a.shares = shares;
  a.part = static_cast<float*>(ws);
  a.part_counts = reinterpret_cast<int32_t*>(a.part + (int64_t)muon::balance_blocks(d->tokens, d->experts) * d->experts);
  return hip_result(muon::launch_balance(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_balance_forward");
}

int muon_balance_backward(const muon_gate_desc_t* d, const void* logits, const uint8_t* mask, const float* shares,
                          const float* dloss, void* dlogits, void* stream) {
  MUON_TRY(check_balance(d));
  MUON_TRY(check_at(logits, d->tokens, elem(d->dtype), "logits"));
  MUON_TRY(check_at(shares, 1, 4, "shares"));
  MUON_TRY(check_at(dloss, 1, 4, "dloss"));
  MUON_TRY(check_at(dlogits, d->tokens, elem(d->dtype), "dlogits"));
  muon::BalanceArgs a = balance_args(d, logits, mask);
  a.shares = const_cast<float*>(shares);
  a.dloss = dloss;
  a.dlogits = dlogits;
  return hip_result(muon::launch_balance_grad(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_balance_backward");
}

int muon_mx_sizes(const muon_mx_desc_t* d, uint64_t* values_bytes, uint64_t* scales_bytes) {
  if (!values_bytes || !scales_bytes) return bad("values_bytes or scales_bytes is null");
  *values_bytes = *scales_bytes = 0;
  MUON_TRY(check_mx(d));
  *values_bytes = (uint64_t)mx_weights(d) * muon::mx_value_bytes(d->n, d->k);
  *scales_bytes = (uint64_t)mx_weights(d) * muon::mx_scale_bytes(d->n, d->k);
  return set_error(MUON_OK, "%s", "");
}

int muon_mx_quantize(const muon_mx_desc_t* d, const void* w, uint8_t* values, uint8_t* scales, void* stream) {
  MUON_TRY(check_mx(d));
  MUON_TRY(check_at(w, d->k * d->n, elem(d->dtype), "w"));
  MUON_TRY(check_mx_weight(d, values, scales));
  if (!muon::mx_weight_fits(mx_weights(d), d->n, d->k)) return bad("groups * n * k (n at least 4, k in steps of 512) is 2^35 or more");
  muon::MxArgs a = mx_args(d);
  a.src = w;
  a.values = values;
  a.scales = scales;
  return hip_result(muon::launch_mx_quantize(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_mx_quantize");
}

int muon_mx_dequantize(const muon_mx_desc_t* d, const uint8_t* values, const uint8_t* scales, void* w, void* stream) {
  MUON_TRY(check_mx(d));
  MUON_TRY(check_mx_weight(d, values, scales));
  MUON_TRY(check_at(w, d->k * d->n, elem(d->dtype), "w"));
  if (!muon::mx_weight_fits(mx_weights(d), d->n, d->k)) return bad("groups * n * k (n at least 4, k in steps of 512) is 2^35 or more");
  muon::MxArgs a = mx_args(d);
  a.values = const_cast<uint8_t*>(values);
  a.scales = const_cast<uint8_t*>(scales);
  a.dst = w;
  return hip_result(muon::launch_mx_dequantize(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_mx_dequantize");
}

int muon_mx_linear_workspace(const muon_mx_desc_t* d, uint64_t* bytes) {
  if (!bytes) return bad("bytes is null");
  *bytes = 0;
  MUON_TRY(check_mx(d));
  if (d->rows > 0 && d->n > 0) *bytes = mx_plan(d).bytes();
  return set_error(MUON_OK, "%s", "");
}

int muon_mx_linear(const muon_mx_desc_t* d, const int32_t* offsets, const void* x, const uint8_t* values,
                   const uint8_t* scales, const void* bias, const void* residual, void* y, void* ws, uint64_t ws_bytes,
                   void* stream) {
  const char* what = "muon_mx_linear";
  MUON_TRY(check_mx(d));
  const int es = elem(d->dtype);
  if (d->groups > 0 && !offsets) return bad("offsets is null");
  if (d->groups == 0 && offsets) return bad("offsets given, but groups is 0");
  MUON_TRY(check_at(offsets, 0, 4, "offsets"));
  MUON_TRY(check_at(x, d->rows * d->k, es, "x"));
  MUON_TRY(check_mx_weight(d, values, scales));
  MUON_TRY(check_at(bias, 0, es, "bias"));
  MUON_TRY(check_at(residual, 0, es, "residual"));
  MUON_TRY(check_at(y, d->rows * d->n, es, "y"));
  if (d->groups > 0 && residual) return bad("a grouped layer takes no residual");
  if (d->rows == 0 || d->n == 0) return set_error(MUON_OK, "%s", "");
  if (!muon::mx_rows_fit(d->rows, d->k)) return bad("rows * k (k in steps of 512) is 2^35 or more");
  MxPlan p = mx_plan(d);
  if ((int64_t)p.p.g.tiles_m * p.p.g.tiles_n * p.p.g.splits > 0x7fffff) return bad("rows * n has too many tiles for a launch");
  MUON_TRY(check_space(p.bytes(), ws, ws_bytes));
  hipStream_t s = static_cast<hipStream_t>(stream);
  muon::GemmArgs& g = p.p.g;
  if (!p.own()) {
    muon::MxArgs q{};
    q.src = x;
    q.values = static_cast<uint8_t*>(ws);
    q.scales = q.values + p.x_values;
    q.rows = d->rows;
    q.k = d->k;
    q.ld = d->ldx;
    q.groups = 1;
    MUON_TRY(hip_result(muon::launch_mx_quantize(q, d->dtype, s), what));
    g.a = q.values;
    p.p.sca = q.scales;
    if (g.splits > 1) g.part = reinterpret_cast<float*>(q.scales + p.x_scales);
  }
  p.p.x = x;
  p.p.ldx = d->ldx;
  p.p.kx = d->k;
  p.p.scb = scales;
  g.b = values;
  g.offsets = offsets;
  g.c = y;
  g.bias = bias;
  g.res = residual;
  g.ldc = d->n;
  g.ldr = d->ldr;
  g.sbias = d->n;
  g.act = d->act;
  hipError_t e = muon::launch_mx_product(p.p, d->dtype, p.tile, p.cols, s);
  if (e == hipSuccess && g.splits > 1) e = muon::launch_gemm_join(g, d->dtype, s);
  return hip_result(e, what);
}

}  // extern "C"
