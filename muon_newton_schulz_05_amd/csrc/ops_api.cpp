// ops_api.cpp -- the C ABI of the layer operators (include/muon_ops.h): argument
// checks, the choice of tile and split, and the launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>

#include "../../include/muon_ops.h"
#include "api_common.h"
#include "ops.h"

namespace {

using muon::aligned;
using muon::bad;
using muon::elem;
using muon::hip_result;
using muon::set_error;

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;
// A layer's kernels count rows in 32 bits and step up to one block (256 rows) past their end.
constexpr int64_t kMaxLayer = (int64_t(1) << 31) - 1024;
constexpr int kCus = 256;

int check_desc(const muon_linear_desc_t* d) {
  if (!d) return bad("desc is null");
  if (d->dtype != MUON_F32 && d->dtype != MUON_BF16) return bad("dtype must be MUON_F32 or MUON_BF16");
  if (d->act < MUON_ACT_NONE || d->act > MUON_ACT_GELU_TANH) return bad("unknown activation");
  if (d->groups < 0 || d->groups > 65535) return bad("groups outside [0, 65535]");
  if (d->w_layout != 0 && d->w_layout != 1) return bad("w_layout must be 0 or 1");
  if (d->rows < 0 || d->k < 0 || d->n < 0 || d->rows > kMaxLayer || d->k > kMaxLayer || d->n > kMaxLayer)
    return bad("a size is negative or over 2^31 - 1024");
  if (d->ldx < 0 || d->ldw < 0 || d->w_stride < 0 || d->ldr < 0 || d->ldg < 0) return bad("a stride is negative");
  return MUON_OK;
}

// How an operand may be loaded: directly to LDS by aligned pieces of 16 or of 4
// bytes with 32-bit offsets inside a tile, or through registers.  rows
// contiguous along k: whole pieces along k; contiguous along its rows (t): whole
// pieces along them.
int loads_of(const void* p, int64_t ld, int64_t group_stride, bool t, int64_t rows, int64_t k, int es) {
  if (ld * es * (t ? 128 / es : 256) >= (int64_t(1) << 31) - 4096) return muon::kStaged;
  for (int bytes : {16, 4}) {
    const int64_t piece = std::max(1, bytes / es);
    if (aligned(p, bytes) && ld % piece == 0 && group_stride % piece == 0 && (t ? rows : k) % piece == 0)
      return bytes == 16 ? muon::kDirect16 : muon::kDirect4;
  }
  return muon::kStaged;
}
// Both operands of a product take the same kind.
int both_loads(int a, int b) {
  if (a == muon::kStaged || b == muon::kStaged) return muon::kStaged;
  return a == muon::kDirect16 && b == muon::kDirect16 ? muon::kDirect16 : muon::kDirect4;
}

struct Product {
  muon::GemmArgs g{};
  int tile = muon::kTile128;
  int loads = muon::kStaged;
  uint64_t ws = 0;            // partials of a split contraction
  muon::AlignArgs copy[2]{};  // of A and B, where copy_bytes > 0
  uint64_t copy_bytes[2] = {0, 0};
  bool pairs = false;         // rows 2r and 2r + 1 are added to one row of C
  uint64_t total() const { return ws + copy_bytes[0] + copy_bytes[1]; }
  uint64_t need() const { return g.m == 0 || g.n == 0 ? 0 : total(); }  // nothing to compute: nothing is used
};

// A larger bf16 product whose operands no 16-byte loads reach first copies them
// into rows that they do, padded with zeros, which add nothing.  Without and with
// the copies, in us (forward / dx / dW, weight [K, N]):
//    4001 x 2001 x 4003   204 / 182 / 333    77 / 85 / 85
//    2001 x 1001 x 2003    43 /  35 /  72    30 / 36 / 34
//    1031 x 1001 x 1003    29 /  20 /  32    21 / 20 / 19
//  - From 2 GFLOP on that pays, or costs nothing (513 x 2001 x 1003: 28 / 21 / 20,
//    27 / 22 / 19), except where both operands lie along the contraction (dx here):
//    the other loads serve those better, and it takes 8 GFLOP.
//  - A copy has to be used often enough: 100001 x 101 x 101 (100 FLOP per byte
//    copied) 33 and 38 forward, 64 experts of 1001 x 999 over 2000 rows (30) 84 and
//    98, 129 x 4001 x 4003 (124) 52 and 42.  dW, whose other loads are the slowest,
//    gains at any rate (100001 x 101 x 101: 142 and 87).
//  - Float32 is bound by its matrix instructions either way: forward 583 without and 556
//    with copies at the first of these, 79 and 89 at the second.
bool align_operands(Product* p, int dtype, bool ta, bool tb, const int (&have)[2], int groups) {
  muon::GemmArgs& g = p->g;
  const double flop = 2.0 * g.m * g.n * g.k;
  if (dtype != MUON_BF16 || std::min({g.m, g.n, g.k}) < 64 || flop < (tb ? 2e9 : 8e9)) return false;
  const bool t[2] = {ta, tb};
  const int64_t rows[2] = {ta ? g.k : g.m, tb ? g.k : g.n}, cols[2] = {ta ? g.m : g.k, tb ? g.n : g.k};
  const int64_t from[2] = {g.lda, g.ldb};
  muon::AlignArgs c[2]{};
  uint64_t bytes[2] = {0, 0};
  for (int i = 0; i < 2; ++i) {
    if (have[i] == muon::kDirect16) continue;
    const bool each = i == 1 && !ta && groups > 0;  // a weight for each group
    c[i] = muon::AlignArgs{nullptr, nullptr, rows[i], cols[i], from[i], each ? g.sb : 0, (cols[i] + 7) / 8 * 8,
                           each ? groups : 1, 0};
    bytes[i] = (uint64_t)c[i].ld * c[i].rows * c[i].groups * 2;
    if (loads_of(nullptr, c[i].ld, 0, t[i], c[i].ld, c[i].ld, 2) != muon::kDirect16) return false;
  }
  if (!ta && flop < 120.0 * (double)(bytes[0] + bytes[1])) return false;
  for (int i = 0; i < 2; ++i) {
    if (bytes[i] == 0) continue;
    p->copy[i] = c[i];
    p->copy_bytes[i] = bytes[i];
    (i ? g.ldb : g.lda) = c[i].ld;
    if (c[i].groups > 1) g.sb = c[i].rows * c[i].ld;
  }
  return true;
}

// The tile and the split of a product, by how many tiles there are for the
// card's 256 compute units (times in us, bf16, forward / dx / dW):
//  - 256 x 256 has the best rate (about 1400 TFLOP/s at 8192^3) once every unit has
//    a tile: 4096^3 takes 113 / 109 / 110, with 256 x 128 130 / 127 / 134, with
//    128 x 128 134 / 134 / 129.
//  - 256 x 256 split in two for more than 64 such tiles (64 are 256 of 128 x 128, one a
//    unit) and up to 128, from 12288 deep: below, the join costs what the split
//    gives.  Time against the rules below, forward / dx / dW:
//       tiles      8192 deep            10240               12288               16384
//        64   1.20 / 1.23 / 1.17            -         1.05 / 1.02 / 1.11   1.05 / 1.04 / 1.09
//        66    .90 /  .89 / 1.03   .87 / .88 / .99     .87 /  .85 /  .97    .85 /  .84 /  .93
//        80    .93 /  .93 / 1.10   .93 / .93 / 1.08    .91 /  .90 / 1.03    .89 /  .89 /  .98
//       100    .95 /  .92 / 1.03   .93 / .88 / .97     .89 /  .86 /  .95    .87 /  .85 /  .88
//       120    .97 /  .95 / 1.02   .94 / .93 / 1.02    .91 /  .90 / 1.00    .87 /  .84 /  .99
//       128   1.05 / 1.02 /  .99  1.00 / 1.00 / .93    .96 /  .97 /  .92    .99 /  .96 /  .87
//  - 256 x 128 where only it fills the card (2048 x 8192 x 4096: 117).
//  - 128 x 128 down to half a card of tiles (2048^3: 29 / 28 / 30, with 256 x 128
//    51, with 64 x 64 31) and for groups of fewer than 256 rows (64 experts over
//    8192 rows: 116 / 113, with 256 x 256 137 / 132), then 64 x 64 (1024^3: 12, with
//    128 x 128 18).
//  - 32 x 128 for at most 32 rows (a group), where time goes to reading B, and for
//    grouped products whose 64-tiles leave units idle.  At least 1024 deep,
//    for dense ones and for at most 64 columns of grouped ones: 32 x 64, the
//    contraction shared by four sets of waves (16 x 4096 x 16384: 25 / 27, with
//    32 x 128 and a join 27 / 30; [24, 10240] experts over 8192 rows, dx from
//    memory: 71, with 32 x 128 84).
//  - Operands that no 16-byte loads reach and that are not copied: 64 x 64, whose staging
//    hides better behind other workgroups (4001 x 2001 x 4003, before such sizes were
//    copied: 184 / 226 / 324 against 204 / 272 / 472 with 128 x 128).
//  - float32 products are bound by their lower matrix rate, not by operand
//    traffic: 64 x 64, or 32 x 64 while 64 x 64 fills the card at most twice
//    (777 x 1001 x 1343: 38 / 37 / 35 against 45 / 37 / 37).
// A product whose tiles do not fill the card is split along the contraction, at
// least 512 of it each, and joined; one over grouped rows is not, its tiles
// number at least the groups with rows.  A grouped contraction has groups of
// unlike length, and is split until the card is filled four times (three
// experts' [678, 520] over 31936 rows, float32 dW: 345 against 383).
void plan_product(Product* p, int dtype, bool ta, bool tb, int loads, int groups) {
  muon::GemmArgs& g = p->g;
  const bool gk = ta && tb, grouped = groups > 0;
  auto tiles = [&](int t) {
    const int64_t bm = muon::gemm_tile_m(t), bn = muon::gemm_tile_n(t);
    const int64_t tm = gk ? (g.m + bm - 1) / bm : muon::group_blocks(g.m, groups, grouped, bm);
    return tm * ((g.n + bn - 1) / bn) * (gk && grouped ? groups : 1);
  };
  const int64_t m_each = gk || !grouped ? g.m : g.m / groups;
  const bool f32 = dtype == MUON_F32;
  const int64_t t256 = tiles(muon::kTile256);
  const bool halves = !f32 && !grouped && m_each >= 256 && g.n >= 256 && 4 * t256 > kCus && 2 * t256 <= kCus &&
                      g.k >= 12288;
  p->loads = loads;
  if (loads != muon::kDirect16) {
    p->tile = muon::kTile64;
  } else if (m_each <= 32) {
    p->tile = !grouped && !gk && g.k >= 1024 ? muon::kTileRows32K : muon::kTileRows32;
  } else if (!f32 && m_each >= 256 && g.n >= 256 && tiles(muon::kTile256) >= kCus) {
    p->tile = muon::kTile256;
  } else if (halves) {
    p->tile = muon::kTile256;
  } else if (!f32 && m_each >= 256 && tiles(muon::kTile256x128) >= kCus) {
    p->tile = muon::kTile256x128;
  } else if (!f32 && tiles(muon::kTile128) >= kCus / 2) {
    p->tile = muon::kTile128;
  } else {
    p->tile = !(grouped && !gk && tiles(muon::kTile64) < kCus) ? muon::kTile64
              : g.n <= 64 && g.k >= 1024                        ? muon::kTileRows32K
                                                                : muon::kTileRows32;
  }
  if (f32 && p->tile == muon::kTile64 && tiles(muon::kTile64) <= 2 * kCus) p->tile = muon::kTile32x64;
  const int64_t bm = muon::gemm_tile_m(p->tile), bn = muon::gemm_tile_n(p->tile);
  g.tiles_m = (int32_t)(gk ? (g.m + bm - 1) / bm : muon::group_blocks(g.m, groups, grouped, bm));
  g.tiles_n = (int32_t)((g.n + bn - 1) / bn);
  g.groups = grouped ? groups : 1;
  g.splits = 1;
  g.k_per = g.k;
  const int64_t t = tiles(p->tile);
  const bool sets = p->tile == muon::kTileRows32K;
  const int64_t k_each = grouped && gk ? g.k / groups : g.k;
  const int64_t below = sets ? kCus / 2 : grouped ? 2 * kCus : kCus, want = sets ? kCus : grouped ? 4 * kCus : 2 * kCus;
  if ((gk || !grouped) && t > 0 && t < below && k_each >= 1024) {
    int64_t s = std::min<int64_t>((want + t - 1) / t, k_each / 512);
    s = p->tile == muon::kTile256 ? 2 : std::min<int64_t>(s, 64);
    if (s > 1) {
      g.k_per = ((g.k + s - 1) / s + 63) / 64 * 64;
      g.splits = (int32_t)(grouped ? s : (g.k + g.k_per - 1) / g.k_per);
      p->ws = (uint64_t)g.splits * g.groups * g.m * g.n * 4;
    }
  }
}

void plan_aligned(Product* p, int dtype, bool ta, bool tb, int la, int lb, int groups) {
  int loads = both_loads(la, lb);
  if (loads != muon::kDirect16 && align_operands(p, dtype, ta, tb, {la, lb}, groups)) loads = muon::kDirect16;
  plan_product(p, dtype, ta, tb, loads, groups);
}

int check_workspace(uint64_t need, const void* ws, uint64_t ws_bytes) {
  if (ws_bytes < need || (need && !ws)) return bad("the workspace is smaller than muon_linear_workspace says");
  if (!aligned(ws, 16)) return bad("the workspace is not 16-byte aligned");
  return MUON_OK;
}

// A product whose pointers and workspace have been checked.
int run_product(Product* p, int dtype, bool ta, bool tb, void* ws, void* stream, const char* what) {
  muon::GemmArgs& g = p->g;
  if (g.m == 0 || g.n == 0) return set_error(MUON_OK, "%s", "");
  hipStream_t s = static_cast<hipStream_t>(stream);
  char* at = static_cast<char*>(ws);
  hipError_t e = hipSuccess;
  const void** operand[2] = {&g.a, &g.b};
  for (int i = 0; i < 2; ++i) {
    if (p->copy_bytes[i] == 0) continue;
    p->copy[i].src = *operand[i];
    p->copy[i].dst = at;
    *operand[i] = at;
    at += p->copy_bytes[i];
    if (e == hipSuccess) e = muon::launch_align(p->copy[i], s);
  }
  if (e != hipSuccess) return hip_result(e, what);
  if (g.splits > 1 || p->pairs) g.part = reinterpret_cast<float*>(at);
  e = muon::launch_gemm(g, dtype, ta, tb, p->loads, p->tile, s);
  if (p->pairs) {
    g.m /= 2;
    g.groups = 1;
    g.splits *= 2;
    g.pairs = 1;
  }
  if (e == hipSuccess && g.splits > 1) e = muon::launch_gemm_join(g, dtype, s);
  return hip_result(e, what);
}

// The three products of a layer as C = A B^T; with what their operands' alignment allows.
Product forward_product(const muon_linear_desc_t* d, const void* x, const void* w, bool* tb) {
  Product p;
  p.g.a = x;
  p.g.b = w;
  p.g.lda = d->ldx;
  p.g.ldb = d->ldw;
  p.g.sb = d->groups > 0 ? d->w_stride : 0;
  p.g.m = d->rows;
  p.g.n = d->n;
  p.g.k = d->k;
  *tb = d->w_layout == 0;
  const int es = elem(d->dtype);
  plan_aligned(&p, d->dtype, false, *tb, loads_of(x, d->ldx, 0, false, d->rows, d->k, es),
               loads_of(w, d->ldw, p.g.sb, *tb, d->n, d->k, es), d->groups);
  return p;
}
Product input_product(const muon_linear_desc_t* d, const void* dz, const void* w, bool* tb) {
  Product p;
  p.g.a = dz;
  p.g.b = w;
  p.g.lda = d->ldg;
  p.g.ldb = d->ldw;
  p.g.sb = d->groups > 0 ? d->w_stride : 0;
  p.g.m = d->rows;
  p.g.n = d->k;
  p.g.k = d->n;
  *tb = d->w_layout == 1;
  const int es = elem(d->dtype);
  plan_aligned(&p, d->dtype, false, *tb, loads_of(dz, d->ldg, 0, false, d->rows, d->n, es),
               loads_of(w, d->ldw, p.g.sb, *tb, d->k, d->n, es), d->groups);
  return p;
}
Product weight_product(const muon_linear_desc_t* d, const void* x, const void* dz) {
  Product p;
  const bool t = d->w_layout == 1;  // dW^T = dz^T x
  p.g.a = t ? dz : x;
  p.g.b = t ? x : dz;
  p.g.lda = t ? d->ldg : d->ldx;
  p.g.ldb = t ? d->ldx : d->ldg;
  p.g.m = t ? d->n : d->k;
  p.g.n = t ? d->k : d->n;
  p.g.k = d->rows;
  p.g.sc = p.g.m * p.g.n;
  const int es = elem(d->dtype);
  plan_aligned(&p, d->dtype, true, true, loads_of(p.g.a, p.g.lda, 0, true, p.g.m, p.g.k, es),
               loads_of(p.g.b, p.g.ldb, 0, true, p.g.n, p.g.k, es), d->groups);
  return p;
}

int check_offsets(const muon_linear_desc_t* d, const int32_t* offsets) {
  if (d->groups > 0 && !offsets) return bad("offsets is null");
  if (d->groups == 0 && offsets) return bad("offsets given, but groups is 0");
  if (!aligned(offsets, 4)) return bad("offsets is not 4-byte aligned");
  return MUON_OK;
}
int check_ptr(const muon_linear_desc_t* d, const void* p, int64_t count, const char* name) {
  if (count > 0 && !p) return set_error(MUON_ERR_INVALID_ARGUMENT, "%s is null", name);
  if (!aligned(p, elem(d->dtype))) return set_error(MUON_ERR_INVALID_ARGUMENT, "%s is not aligned to its elements", name);
  return MUON_OK;
}
// A bf16 layer's dz is rounded to bf16 for the products that follow, like every
// operand of the matrix instructions: dx and dW are then about 1.4 times as far
// off in the norm as their own rounding, which for a few rows may be 1.9 times
// (an error that few values share is not averaged).  Where a weight meets few rows,
// and the products wait for the weight, what the rounding lost is kept too: dz has
// two rows for each, the rounded one and the rest, dx adds the pairs of its rows in
// float32, and dW multiplies each row of x twice.  An infinite operand meets the
// rounded row alone: dx drops the rest of a sum that is not finite, and the row of x
// for the rest has zeros there.  (relu's slope is 0 or 1: its dz loses nothing.)
// The whole backward pass without and with, in us:
//  - one weight, up to 64 rows: 1 x 4096 x 16384 73 and 78, 16 x 4096 x 4096 37 and 43,
//    64 x 1024 x 4096 30 and 39; 128 x 4096 x 16384 would take 116 and 161.
//  - experts, up to 16 rows each on average (the host knows no more): 64 x [2048,
//    1408] with 2 rows each 217 and 226, with 16 245 and 262; with 32 it would be 251
//    and 302, with 64 288 and 358.  16 x [1024, 1024] with 16: 36 and 42, with 32 36 and 51.
//    An expert with few rows among experts with many has its dz rounded like theirs.
constexpr int64_t kPairRows = 64, kPairRowsEach = 16;
struct Pairs {
  bool on = false;
  muon_linear_desc_t d{};            // the layer of twice the rows
  muon::AlignArgs x{};               // each row of x twice
  uint64_t dz = 0, x2 = 0, offsets = 0;  // bytes, multiples of 16
  uint64_t bytes() const { return dz + x2 + offsets; }
};
Pairs pairs_of(const muon_linear_desc_t* d) {
  Pairs q;
  q.on = d->dtype == MUON_BF16 && d->act > MUON_ACT_RELU && d->rows > 0 && d->k > 0 && d->n > 0 &&
         d->rows <= std::max(kPairRows, kPairRowsEach * d->groups);
  if (!q.on) return q;
  q.x = muon::AlignArgs{nullptr, nullptr, 2, d->k, 0, d->ldx, (d->k + 7) / 8 * 8, (int32_t)d->rows, 1};
  q.d = *d;
  q.d.rows = 2 * d->rows;
  q.d.ldg = d->n;
  q.d.ldx = q.x.ld;
  q.dz = ((uint64_t)q.d.rows * d->n * 2 + 15) / 16 * 16;
  q.x2 = (uint64_t)q.d.rows * q.x.ld * 2;
  q.offsets = d->groups > 0 ? ((uint64_t)d->groups * 4 + 4 + 15) / 16 * 16 : 0;
  return q;
}
// The input gradient of a layer of pairs.
Product pairs_input(const Pairs& q, const void* dz, const void* w, bool* tb) {
  Product p = input_product(&q.d, dz, w, tb);
  p.pairs = true;
  p.ws = (uint64_t)p.g.splits * p.g.m * p.g.n * 4;
  return p;
}

// dz of a layer with an activation, as part of a workspace.
uint64_t dz_bytes(const muon_linear_desc_t* d) {
  return d->act == MUON_ACT_NONE ? 0 : ((uint64_t)d->rows * d->n * elem(d->dtype) + 15) / 16 * 16;
}// The column sums of the activation's gradient, by blocks of rows.
uint64_t col_sum_bytes(const muon_linear_desc_t* d) {
  return (uint64_t)muon::act_grad_blocks(d->rows, d->n, std::max(d->groups, 1), d->groups > 0) * d->n * 4;
}

int check_move(const muon_move_desc_t* d) {
  if (!d) return bad("desc is null");
  if (d->dtype != MUON_F32 && d->dtype != MUON_BF16) return bad("dtype must be MUON_F32 or MUON_BF16");
  if (d->top < 1 || d->tokens < 0 || d->h < 0 || d->h > kMaxDim) return bad("top, tokens or h out of range");
  if (d->tokens > kMaxDim / d->top) return bad("tokens * top is over 2^31 - 1");
  if (d->experts < 1 || d->experts > MUON_ROUTE_MAX_EXPERTS) return bad("experts outside [1, 1024]");
  if (d->ldx < 0 || d->ldg < 0 || d->ldr < 0) return bad("a stride is negative");
  return MUON_OK;
}
int check_rows(const muon_move_desc_t* d, const void* p, const char* name) {
  if (d->tokens > 0 && d->h > 0 && !p) return set_error(MUON_ERR_INVALID_ARGUMENT, "%s is null", name);
  if (!aligned(p, elem(d->dtype))) return set_error(MUON_ERR_INVALID_ARGUMENT, "%s is not aligned to its elements", name);
  return MUON_OK;
}
int check_ints(const muon_move_desc_t* d, const void* p, const char* name) {
  if (d->tokens > 0 && !p) return set_error(MUON_ERR_INVALID_ARGUMENT, "%s is null", name);
  if (!aligned(p, 4)) return set_error(MUON_ERR_INVALID_ARGUMENT, "%s is not 4-byte aligned", name);
  return MUON_OK;
}
muon::MoveArgs move_args(const muon_move_desc_t* d) {
  muon::MoveArgs a{};
  a.experts = d->experts;
  a.top = d->top;
  a.tokens = d->tokens;
  a.h = d->h;
  a.ldx = d->ldx;
  a.ldg = d->ldg;
  a.ldr = d->ldr;
  return a;
}

}  // namespace

extern "C" {

int muon_linear_workspace(const muon_linear_desc_t* d, int32_t op, uint64_t* bytes) {
  if (!bytes) return bad("bytes is null");
  *bytes = 0;
  MUON_TRY(check_desc(d));
  if (op == MUON_LINEAR_GRAD_ACT) {
    *bytes = col_sum_bytes(d);
    return set_error(MUON_OK, "%s", "");
  }
  if (op == MUON_LINEAR_BACKWARD) {
    // dz, then one area that the three steps use in turn.
    uint64_t most = 0, b = 0;
    muon_linear_desc_t dd = *d;
    const Pairs q = pairs_of(d);
    if (q.on) {
      MUON_TRY(muon_linear_workspace(d, MUON_LINEAR_GRAD_ACT, &most));
      MUON_TRY(muon_linear_workspace(&q.d, MUON_LINEAR_GRAD_WEIGHT, &b));
      most = std::max(most, b);
      for (uintptr_t w : {0, 4, 2}) {
        bool tb;
        most = std::max(most, pairs_input(q, nullptr, reinterpret_cast<const void*>(w), &tb).total());
      }
      *bytes = q.bytes() + most;
      return set_error(MUON_OK, "%s", "");
    }
    for (int32_t step : {MUON_LINEAR_GRAD_ACT, MUON_LINEAR_GRAD_INPUT, MUON_LINEAR_GRAD_WEIGHT}) {
      for (int64_t ld : {d->ldg, d->n}) {
        dd.ldg = ld;
        MUON_TRY(muon_linear_workspace(&dd, step, &b));
        most = std::max(most, b);
      }
    }
    *bytes = dz_bytes(d) + most;
    return set_error(MUON_OK, "%s", "");
  }
  if (op < 0 || op > MUON_LINEAR_GRAD_WEIGHT) return bad("unknown operation");
  // The plan depends on the pointers' alignment: the largest of the answers.
  const void* probes[3] = {nullptr, reinterpret_cast<const void*>(uintptr_t(4)),
                           reinterpret_cast<const void*>(uintptr_t(2))};
  for (const void* q : probes)
    for (const void* r : probes) {
      bool tb;
      const Product p = op == MUON_LINEAR_FORWARD      ? forward_product(d, q, r, &tb)
                        : op == MUON_LINEAR_GRAD_INPUT ? input_product(d, q, r, &tb)
                                                       : weight_product(d, q, r);
      *bytes = std::max(*bytes, p.total());
    }
  return set_error(MUON_OK, "%s", "");
}

int muon_linear_forward(const muon_linear_desc_t* d, const int32_t* offsets, const void* x, const void* w,
                        const void* bias, const void* residual, void* y, void* z, void* ws, uint64_t ws_bytes,
                        void* stream) {
  MUON_TRY(check_desc(d));
  MUON_TRY(check_offsets(d, offsets));
  MUON_TRY(check_ptr(d, x, d->rows * d->k, "x"));
  MUON_TRY(check_ptr(d, w, d->k * d->n, "w"));
  MUON_TRY(check_ptr(d, bias, 0, "bias"));
  MUON_TRY(check_ptr(d, residual, 0, "residual"));
  MUON_TRY(check_ptr(d, y, d->rows * d->n, "y"));
  MUON_TRY(check_ptr(d, z, 0, "z"));
  if (d->groups > 0 && residual) return bad("a grouped layer takes no residual");
  bool tb;
  Product p = forward_product(d, x, w, &tb);
  p.g.offsets = offsets;
  p.g.c = y;
  p.g.z = z;
  p.g.bias = bias;
  p.g.res = residual;
  p.g.ldc = d->n;
  p.g.ldr = d->ldr;
  p.g.sbias = d->n;
  p.g.act = d->act;
  MUON_TRY(check_workspace(p.need(), ws, ws_bytes));
  return run_product(&p, d->dtype, false, tb, ws, stream, "muon_linear_forward");
}

// The activation's gradient: its checks, and its launch.
static int check_grad_act(const muon_linear_desc_t* d, const void* dy, const void* z, const void* dz, const void* db) {
  MUON_TRY(check_ptr(d, dy, d->rows * d->n, "dy"));
  MUON_TRY(check_ptr(d, z, d->act != MUON_ACT_NONE ? d->rows * d->n : 0, "z"));
  MUON_TRY(check_ptr(d, dz, 0, "dz"));
  return check_ptr(d, db, 0, "db");
}
static int run_grad_act(const muon_linear_desc_t* d, const int32_t* offsets, const void* dy, const void* z, void* dz,
                        int32_t* offsets2, bool pairs, void* db, void* ws, void* stream, const char* what) {
  muon::ActGradArgs a{};
  a.dy = dy;
  a.z = d->act != MUON_ACT_NONE ? z : nullptr;
  a.dz = dz;
  a.db = db;
  a.part = static_cast<float*>(ws);
  a.rows = d->rows;
  a.n = d->n;
  a.lddy = d->ldg;
  a.ldz = d->n;
  a.lddz = d->n;
  a.offsets = offsets;
  a.groups = std::max(d->groups, 1);
  a.act = d->act;
  a.pairs = pairs;
  a.offsets2 = offsets2;
  return hip_result(muon::launch_act_grad(a, d->dtype, static_cast<hipStream_t>(stream)), what);
}

int muon_linear_grad_act(const muon_linear_desc_t* d, const int32_t* offsets, const void* dy, const void* z, void* dz,
                         void* db, void* ws, uint64_t ws_bytes, void* stream) {
  MUON_TRY(check_desc(d));
  MUON_TRY(check_offsets(d, offsets));
  MUON_TRY(check_grad_act(d, dy, z, dz, db));
  if (!dz && !db) return set_error(MUON_OK, "%s", "");
  if (db) MUON_TRY(check_workspace(col_sum_bytes(d), ws, ws_bytes));
  return run_grad_act(d, offsets, dy, z, dz, nullptr, false, db, ws, stream, "muon_linear_grad_act");
}

int muon_linear_grad_input(const muon_linear_desc_t* d, const int32_t* offsets, const void* dz, const void* w, void* dx,
                           void* ws, uint64_t ws_bytes, void* stream) {
  MUON_TRY(check_desc(d));
  MUON_TRY(check_offsets(d, offsets));
  MUON_TRY(check_ptr(d, dz, d->rows * d->n, "dz"));
  MUON_TRY(check_ptr(d, w, d->k * d->n, "w"));
  MUON_TRY(check_ptr(d, dx, d->rows * d->k, "dx"));
  bool tb;
  Product p = input_product(d, dz, w, &tb);
  MUON_TRY(check_workspace(p.need(), ws, ws_bytes));
  p.g.offsets = offsets;
  p.g.c = dx;
  p.g.ldc = d->k;
  return run_product(&p, d->dtype, false, tb, ws, stream, "muon_linear_grad_input");
}

int muon_linear_grad_weight(const muon_linear_desc_t* d, const int32_t* offsets, const void* x, const void* dz, void* dw,
                            void* ws, uint64_t ws_bytes, void* stream) {
  MUON_TRY(check_desc(d));
  MUON_TRY(check_offsets(d, offsets));
  MUON_TRY(check_ptr(d, x, d->rows * d->k, "x"));
  MUON_TRY(check_ptr(d, dz, d->rows * d->n, "dz"));
  MUON_TRY(check_ptr(d, dw, d->k * d->n, "dw"));
  Product p = weight_product(d, x, dz);
  MUON_TRY(check_workspace(p.need(), ws, ws_bytes));
  p.g.offsets = offsets;
  p.g.c = dw;
  p.g.ldc = p.g.n;
  return run_product(&p, d->dtype, true, true, ws, stream, "muon_linear_grad_weight");
}

int muon_linear_backward(const muon_linear_desc_t* d, const int32_t* offsets, const void* x, const void* w,
                         const void* z, const void* dy, void* dx, void* dw, void* db, void* ws, uint64_t ws_bytes,
                         void* stream) {
  const char* what = "muon_linear_backward";
  MUON_TRY(check_desc(d));
  if (!dx && !dw && !db) return set_error(MUON_OK, "%s", "");
  MUON_TRY(check_offsets(d, offsets));
  MUON_TRY(check_grad_act(d, dy, z, nullptr, db));
  MUON_TRY(check_ptr(d, dx, 0, "dx"));
  MUON_TRY(check_ptr(d, dw, 0, "dw"));
  if (dx) MUON_TRY(check_ptr(d, w, d->k * d->n, "w"));
  if (dw) MUON_TRY(check_ptr(d, x, d->rows * d->k, "x"));
  const bool products = dx || dw;
  const Pairs q = products ? pairs_of(d) : Pairs{};
  const uint64_t head = !products ? 0 : q.on ? q.bytes() : dz_bytes(d);

  // The workspace: dz, with pairs of rows x twice and the offsets of the pairs, then an area that the steps use in turn.
  char* const at = static_cast<char*>(ws);
  char* const x2 = q.on ? at + q.dz : nullptr;
  int32_t* const offsets2 = q.on && offsets ? reinterpret_cast<int32_t*>(x2 + q.x2) : nullptr;
  char* const rest = ws ? at + head : nullptr;
  const void* dz = head ? ws : dy;
  muon_linear_desc_t dd = q.on ? q.d : *d;
  if (head) dd.ldg = d->n;
  const int32_t* const off = q.on ? offsets2 : offsets;
  Product pi, pw;
  bool tb = false;
  if (dx) pi = q.on ? pairs_input(q, dz, w, &tb) : input_product(&dd, dz, w, &tb);
  if (dw) pw = weight_product(&dd, q.on ? x2 : x, dz);
  const uint64_t most = std::max({db ? col_sum_bytes(d) : 0, dx ? pi.need() : 0, dw ? pw.need() : 0});
  MUON_TRY(check_workspace(head + most, ws, ws_bytes));

  if (head || db) MUON_TRY(run_grad_act(d, offsets, dy, z, head ? ws : nullptr, offsets2, q.on, db, rest, stream, what));
  if (dx) {
    pi.g.offsets = off;
    pi.g.c = dx;
    pi.g.ldc = d->k;
    MUON_TRY(run_product(&pi, d->dtype, false, tb, rest, stream, what));
  }
  if (dw) {
    if (q.on) {
      muon::AlignArgs twice = q.x;
      twice.src = x;
      twice.dst = x2;
      MUON_TRY(hip_result(muon::launch_align(twice, static_cast<hipStream_t>(stream)), what));
    }
    pw.g.offsets = off;
    pw.g.c = dw;
    pw.g.ldc = pw.g.n;
    MUON_TRY(run_product(&pw, d->dtype, true, true, rest, stream, what));
  }
  return set_error(MUON_OK, "%s", "");
}

int muon_route_workspace(int64_t entries, int32_t experts, uint64_t* bytes) {
  if (!bytes) return bad("bytes is null");
  *bytes = 0;
  if (entries < 0 || entries > kMaxDim) return bad("entries out of range");
  if (experts < 1 || experts > MUON_ROUTE_MAX_EXPERTS) return bad("experts outside [1, 1024]");
  *bytes = (uint64_t)((entries + muon::kRouteBlock - 1) / muon::kRouteBlock) * experts * 4;
  return set_error(MUON_OK, "%s", "");
}

int muon_route(const void* ids, int32_t ids_bytes, int64_t tokens, int32_t top, int32_t experts, int32_t* offsets,
               int32_t* order, int32_t* position, void* ws, uint64_t ws_bytes, void* stream) {
  if (ids_bytes != 4 && ids_bytes != 8) return bad("ids_bytes must be 4 or 8");
  if (tokens < 0 || top < 1 || tokens > kMaxDim / top) return bad("tokens or top out of range");
  const int64_t entries = tokens * top;
  uint64_t need = 0;
  MUON_TRY(muon_route_workspace(entries, experts, &need));
  if (!offsets) return bad("offsets is null");
  if (entries > 0 && (!ids || !order || !position)) return bad("ids, order or position is null");
  if (!aligned(ids, ids_bytes) || !aligned(offsets, 4) || !aligned(order, 4) || !aligned(position, 4))
    return bad("a pointer is not aligned to its elements");
  if (need > ws_bytes || (need && !ws)) return bad("the workspace is smaller than muon_route_workspace says");
  if (!aligned(ws, 16)) return bad("the workspace is not 16-byte aligned");
  muon::RouteArgs a{ids, ids_bytes == 8, experts, top, entries, order, position, offsets, static_cast<int32_t*>(ws)};
  return hip_result(muon::launch_route(a, static_cast<hipStream_t>(stream)), "muon_route");
}

int muon_dispatch(const muon_move_desc_t* d, const int32_t* offsets, const int32_t* position, const void* x, void* xs,
                  void* stream) {
  MUON_TRY(check_move(d));
  MUON_TRY(check_ints(d, offsets, "offsets"));
  MUON_TRY(check_ints(d, position, "position"));
  MUON_TRY(check_rows(d, x, "x"));
  MUON_TRY(check_rows(d, xs, "xs"));
  muon::MoveArgs a = move_args(d);
  a.offsets = offsets;
  a.position = position;
  a.x = x;
  a.out = xs;
  return hip_result(muon::launch_dispatch(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_dispatch");
}

int muon_dispatch_grad(const muon_move_desc_t* d, const int32_t* position, const void* dxs, void* dx, void* stream) {
  MUON_TRY(check_move(d));
  MUON_TRY(check_ints(d, position, "position"));
  MUON_TRY(check_rows(d, dxs, "dxs"));
  MUON_TRY(check_rows(d, dx, "dx"));
  muon::MoveArgs a = move_args(d);
  a.position = position;
  a.x = dxs;
  a.out = dx;
  return hip_result(muon::launch_gather_sum(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_dispatch_grad");
}

int muon_combine(const muon_move_desc_t* d, const int32_t* position, const float* weights, const void* ys,
                 const void* residual, void* y, void* stream) {
  MUON_TRY(check_move(d));
  MUON_TRY(check_ints(d, position, "position"));
  MUON_TRY(check_ints(d, weights, "weights"));
  MUON_TRY(check_rows(d, ys, "ys"));
  MUON_TRY(check_rows(d, y, "y"));
  if (!aligned(residual, elem(d->dtype))) return bad("residual is not aligned to its elements");
  muon::MoveArgs a = move_args(d);
  a.position = position;
  a.w = weights;
  a.x = ys;
  a.res = residual;
  a.out = y;
  return hip_result(muon::launch_gather_sum(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_combine");
}

int muon_combine_grad(const muon_move_desc_t* d, const int32_t* offsets, const int32_t* position, const float* weights,
                      const void* ys, const void* dy, void* dys, float* dweights, void* stream) {
  MUON_TRY(check_move(d));
  MUON_TRY(check_ints(d, offsets, "offsets"));
  MUON_TRY(check_ints(d, position, "position"));
  MUON_TRY(check_ints(d, weights, "weights"));
  MUON_TRY(check_rows(d, dy, "dy"));
  if (dweights) MUON_TRY(check_rows(d, ys, "ys"));
  if (!aligned(dys, elem(d->dtype)) || !aligned(dweights, 4)) return bad("a pointer is not aligned to its elements");
  if (!dys && !dweights) return set_error(MUON_OK, "%s", "");
  muon::MoveArgs a = move_args(d);
  a.offsets = offsets;
  a.position = position;
  a.w = weights;
  a.x = dweights ? ys : nullptr;
  a.g = dy;
  a.out = dys;
  a.dw = dweights;
  return hip_result(muon::launch_combine_grad(a, d->dtype, static_cast<hipStream_t>(stream)), "muon_combine_grad");
}

int muon_dropout(int32_t dtype, int64_t n, const void* x, const void* residual, void* y, double p, uint64_t seed,
                 uint64_t offset, const uint64_t* state, void* stream) {
  if (dtype != MUON_F32 && dtype != MUON_BF16) return bad("dtype must be MUON_F32 or MUON_BF16");
  if (n < 0 || n > (int64_t(1) << 40)) return bad("n out of range");
  if (!(p >= 0.0 && p < 1.0)) return bad("p outside [0, 1)");
  const uint32_t drop = (uint32_t)std::nearbyint(p * 65536.0);
  if (drop >= 65536u) return bad("p rounds to 1 (of 65536 steps)");
  if (n > 0 && (!x || !y)) return bad("x or y is null");
  const uintptr_t es = (uintptr_t)elem(dtype);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(y, es) || !aligned(state, 8))
    return bad("a pointer is not aligned to its elements");
  const muon::DropoutArgs a{x, residual, y, n, seed, offset, state, drop};
  return hip_result(muon::launch_dropout(a, dtype, static_cast<hipStream_t>(stream)), "muon_dropout");
}

}  // extern "C"
