// C ABI of the operators around the step: the gradient norm and clip, the
// block-scaled e4m3 operands and their product.  A call enqueues kernel launches
// only (place_table), so that it can be captured into a graph.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <vector>

#include "abi_common.hpp"
#include "grad_plan.hpp"
#include "muon_internal.hpp"
#include "muon_mi355x.h"

namespace muon {
namespace {

// ---------------------------------------------------------------------------
// Gradient norm and clip
// ---------------------------------------------------------------------------
int32_t check_norm_params(const muon_grad_norm_params* p) {
  if (p == nullptr) return fail(MUON_ERR_INVALID_ARG, "params pointer is null");
  if (p->kind != MUON_NORM_L2 && p->kind != MUON_NORM_MAX)
    return fail(MUON_ERR_INVALID_ARG, "unknown norm kind %d", p->kind);
  if (p->clip != 0 && p->clip != 1) return fail(MUON_ERR_INVALID_ARG, "clip must be 0 or 1");
  if (p->clip && (!(p->max_norm >= 0.f) || !std::isfinite(p->max_norm)))
    return fail(MUON_ERR_INVALID_ARG, "max_norm must be finite and >= 0");
  if (!std::isfinite(p->eps) || p->eps < 0.f)
    return fail(MUON_ERR_INVALID_ARG, "eps must be finite and >= 0");
  return MUON_OK;
}

int32_t check_float_ptr(const void* p, const char* what) {
  if (p == nullptr) return fail(MUON_ERR_INVALID_ARG, "%s pointer is null", what);
  if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0)
    return fail(MUON_ERR_INVALID_ARG, "%s pointer not 4-byte aligned", what);
  return MUON_OK;
}

GradNormArgs norm_args(const GradPlan& pl, const muon_grad_norm_params& p, float* result,
                       char* ws) {
  GradNormArgs a{};
  a.result = result;
  a.partials = ws + pl.partials_off;
  a.chunks = pl.chunks;
  a.clip = p.clip;
  a.max_norm = p.max_norm;
  a.eps = p.eps;
  return a;
}

int32_t run_norm(const GradPlan& pl, const ArgTable& t, const GradCtx& c, const GradNormArgs& a,
                 int32_t kind) {
  TimedLaunch tl(MUON_K_GRAD_NORM, c.stream);
  const hipError_t e = launch_grad_norm(t, c, a, kind, pl.in_bytes);
  if (e != hipSuccess) return hip_fail(e, "launch gradient norm");
  tl.done();
  return MUON_OK;
}

int32_t run_scale(const GradPlan& pl, const ArgTable& t, const GradCtx& c, const float* scale,
                  const GradNormArgs* joined = nullptr, int32_t kind = 0) {
  TimedLaunch tl(MUON_K_GRAD_SCALE, c.stream);
  const hipError_t e =
      launch_grad_scale(t, c, pl.chunks, scale, joined, kind, pl.in_bytes + pl.out_bytes);
  if (e != hipSuccess) return hip_fail(e, "launch gradient scale");
  tl.done();
  return MUON_OK;
}

// ---------------------------------------------------------------------------
// Block-scaled e4m3
// ---------------------------------------------------------------------------
int32_t check_f8_dim(int64_t v, const char* what, int32_t i) {
  if (v < 0)
    return fail(MUON_ERR_INVALID_ARG, "matrix %d: %s = %lld is negative", i, what,
                static_cast<long long>(v));
  if (v > MUON_F8_MAX_DIM)
    return fail(MUON_ERR_UNSUPPORTED, "matrix %d: %s = %lld; the maximum is %d", i, what,
                static_cast<long long>(v), MUON_F8_MAX_DIM);
  return MUON_OK;
}

size_t f8_desc_bytes(int32_t batch) {
  return align_up(std::max(sizeof(F8QuantDesc), sizeof(F8ProdDesc)) * static_cast<size_t>(batch),
                  kAlign);
}
size_t f8_ws_bytes(int32_t batch) {
  return f8_desc_bytes(batch) + align_up(4 * sizeof(int32_t) * (static_cast<size_t>(batch) + 1), kAlign);
}

int32_t check_ptr(const void* p, const char* what, int32_t i) {
  if (p == nullptr) return fail(MUON_ERR_INVALID_ARG, "matrix %d: %s is null", i, what);
  if (!aligned16(p))
    return fail(MUON_ERR_INVALID_ARG, "matrix %d: %s not 16-byte aligned", i, what);
  return MUON_OK;
}

// A launch holds fewer than 2^32 threads.
constexpr int64_t kMaxBlocks = (1ll << 24) - 1;
int32_t add_blocks(int64_t a, int64_t b, int64_t& total) {
  total += a * b;  // at most 2^32 blocks of one matrix
  if (total > kMaxBlocks) return fail(MUON_ERR_UNSUPPORTED, "batch needs 2^24 blocks or more");
  return MUON_OK;
}

int64_t cdiv(int64_t x, int64_t a) { return (x + a - 1) / a; }

constexpr int32_t kFewRows = 64;  // most rows of one block of the kernel of few rows
// Bytes of operands and outputs from which the outputs pass the caches by, which
// leaves the operands there (8 products 4096 x 6144 x 2048, bf16: 367 us against
// 403; 8 of 2048 x 6144 x 4096 added to fp32: 752 against 770).  Smaller calls gain
// nothing, and the next one finds the outputs in the caches (8192 x 4096 x 2048,
// fp32, and its norm: 143 us against 148 with the hint).
constexpr int64_t kNtBytes = 256'000'000;
constexpr double kFixedSlices = 12;  // a tile's fixed cost in K slices of 64
constexpr double kUneven = 1.05;
constexpr int64_t kSpreadTiles = 16;
constexpr int64_t kCus = 256;

struct SmallPlan {
  int32_t mt = 1, nt = 4;
};

// Prefixes over the products (batch + 1 each): their full, half and quarter tiles
// and their blocks in the kernel of few rows.
struct BlockCounts {
  static constexpr int kKinds = 4;
  size_t batch;
  std::vector<int32_t> prefix;
  explicit BlockCounts(size_t n) : batch(n), prefix(kKinds * (n + 1), 0) {}
  int32_t* at(int kind) { return prefix.data() + kind * (batch + 1); }
  const int32_t* at(int kind) const { return prefix.data() + kind * (batch + 1); }
  int32_t total(int kind) const { return at(kind)[batch]; }
};

// Times of a full, a half and a quarter tile, us, by the K slices of 64 (fitted
// to launches of two whole rounds at K = 2048 and 6144; bf16, K = 6144: 87, 52 and
// 33 us), and what a launch takes besides.
struct TileTimes {
  double t[3];
  TileTimes(bool bf16, double slices)
      : t{bf16 ? 6.4 + 0.84 * slices : 9.8 + 1.54 * slices,
          bf16 ? 5.3 + 0.48 * slices : 9.9 + 0.77 * slices,
          bf16 ? 5.2 + 0.29 * slices : 6.5 + 0.53 * slices} {}
};
constexpr double kLaunch = 4;

// When the launch's last CU ends: its full tiles, then the half ones, then the
// quarter ones, each on the CU that is free first.
double launch_end(const TileTimes& c, const int64_t (&n)[3]) {
  // CUs by the time at which they are free, earliest first: one group, and one
  // more for each kind that ends within a group
  struct Group {
    double at;
    int64_t cus;
  } g[5] = {{0.0, kCus}};
  int groups = 1;
  double end = 0;
  for (int k = 0; k < 3; ++k) {
    int64_t left = n[k];
    if (left == 0) continue;
    if (left >= 4 * kCus) {  // whole rounds of one kind
      const int64_t r = left / kCus - 2;
      for (int i = 0; i < groups; ++i) g[i].at += static_cast<double>(r) * c.t[k];
      left -= r * kCus;
    }
    while (left > 0) {
      const double at = g[0].at + c.t[k];
      const int64_t take = std::min(left, g[0].cus);
      left -= take;
      if ((g[0].cus -= take) == 0) {
        for (int i = 1; i < groups; ++i) g[i - 1] = g[i];
        --groups;
      }
      int to = groups;
      for (; to > 0 && g[to - 1].at > at; --to) g[to] = g[to - 1];
      g[to] = {at, take};
      ++groups;
    }
    end = g[groups - 1].at;
  }
  return end;
}

// Rows of full, half and quarter tiles of the products that the large-tile
// kernel takes: a product's rest of up to 64, 128 or 192 rows is a quarter tile, a
// half one, or one of each (or quarter ones only), and where it ends the launch
// earlier, full tiles of its last round become two half or four quarter ones
// each.  (2048^3, 64 full tiles: 15.7 us in quarter tiles, 18.3 in half ones; with an
// fp32 result 26 and 37; 16 products 1089 x 2048 x 6144: 196 us, with half tiles only
// 201.)  Returns when the launch ends.
double cut_rows(std::vector<F8ProdDesc>& desc, const std::vector<char>& large, const TileTimes& c) {
  int64_t f = 0, base[2][3] = {};  // by whether the rests take half tiles
  for (size_t i = 0; i < desc.size(); ++i) {
    F8ProdDesc& d = desc[i];
    if (!large[i]) continue;
    const int64_t tn = cdiv(d.n, kF8Tile), q = cdiv(d.m % kF8Tile, kF8Tile / 4);
    d.full = static_cast<uint16_t>(d.m / kF8Tile + (q == 4 ? 1 : 0));
    f += d.full * tn;
    if (q < 4) {
      base[0][2] += q * tn;
      base[1][1] += q / 2 * tn;
      base[1][2] += q % 2 * tn;
    }
  }
  // one row of tiles at a time, from the end, as long as a whole last round's
  // worth has not been cut
  const int64_t most = f % kCus, step = most / 16;
  int64_t best_take = 0;
  int best_kind = 1, best_rest = 1;
  const double uncut = launch_end(c, {f, base[1][1], base[1][2]});
  // more and smaller tiles have to gain 5%: they load more, and this knows
  // nothing of the clock (16 products 300 x 2048 x 6144, bf16: one round with whole
  // tiles 76 us, two without 86)
  double best = 0.95 * uncut;
  auto consider = [&](int64_t taken) {
    for (int rest = base[1][1] > 0 ? 0 : 1; rest < 2; ++rest)
      for (int kind = 1; kind < (taken > 0 ? 3 : 2); ++kind) {
        int64_t n[3] = {f - taken, base[rest][1], base[rest][2]};
        n[kind] += taken * 2 * kind;
        const double r = launch_end(c, n);
        if (r < best) {
          best = r;
          best_take = taken;
          best_kind = kind;
          best_rest = rest;
        }
      }
  };
  consider(0);
  int64_t taken = 0, next = 0;
  for (size_t i = desc.size(); i-- > 0 && taken < most;) {
    if (!large[i]) continue;
    const int64_t tn = cdiv(desc[i].n, kF8Tile);
    for (int32_t k = 0; k < desc[i].full && taken < most; ++k) {
      taken += tn;
      if (taken < next && taken < most) continue;
      consider(taken);
      next = taken + step;
    }
  }
  if (best_take == 0 && best_rest == 1) best = uncut;
  taken = best_take;
  for (size_t i = desc.size(); i-- > 0;) {
    if (!large[i]) continue;
    F8ProdDesc& d = desc[i];
    const int64_t tn = cdiv(d.n, kF8Tile);
    const int64_t q = cdiv(d.m % kF8Tile, kF8Tile / 4);
    int64_t half = best_rest == 1 && q < 4 ? q / 2 : 0;
    for (; d.full > 0 && taken > 0; taken -= tn) {
      --d.full;
      half += best_kind == 1 ? 2 : 0;
    }
    d.half = static_cast<uint16_t>(half);
  }
  return best;
}

// What the estimates take from a set of products.
struct Load {
  double tiles = 0, slices = 0;  // full tiles, and the K slices of 64 in them
  double blocks = 0, steps = 0;  // 64 x 64 blocks, and the steps of 512 in them
  double bytes = 0;              // of the operands
  int32_t rows = 0;              // most rows of a product
  int32_t kp = 0;                // longest sum
  void add(const F8ProdDesc& d) {
    const double t = static_cast<double>(cdiv(d.m, kF8Tile)) * static_cast<double>(cdiv(d.n, kF8Tile));
    tiles += t;
    slices += t * (d.kp / 64);
    const double b = static_cast<double>(cdiv(d.m, 64)) * static_cast<double>(cdiv(d.n, 64));
    blocks += b;
    steps += b * static_cast<double>(cdiv(d.kp, 4 * kF8Block));
    bytes += (static_cast<double>(d.m) + d.n) * d.kp;
    rows = std::max(rows, d.m);
    kp = std::max(kp, d.kp);
  }
};

int32_t few_rows_mt(int32_t rows) { return rows <= 16 ? 1 : rows <= 32 ? 2 : 4; }

// When a call of the kernel of few rows ends, us: per block on one of the 256 CUs
// a fixed part and one per 512 of K, which its four waves share, one block of the
// longest sum, or the operands' bytes at the rates measured with 16, 32 and 64 rows (5.4, 4.9, 4.5 TB/s).
double blocks_end(const Load& l) {
  if (l.blocks == 0) return 0;
  const int32_t mt = few_rows_mt(l.rows);
  return std::max({std::ceil(l.blocks / kCus) * (3.0 + 1.25 * l.steps / l.blocks),
                   3.0 + 1.25 * static_cast<double>(cdiv(l.kp, 4 * kF8Block)),
                   l.bytes / (mt == 1 ? 5.4e6 : mt == 2 ? 4.95e6 : 4.5e6)});
}

// When a launch of tiles ends: TileTimes at the mean length of the sums, a
// quarter tile of the longest one, or the operands' bytes at 5.5 TB/s (fp32
// results: 4.75).
double tiles_end(std::vector<F8ProdDesc>& desc, const std::vector<char>& large, const Load& l,
                 bool bf16) {
  if (l.tiles == 0) return 0;
  return std::max({kLaunch + cut_rows(desc, large, TileTimes(bf16, l.slices / l.tiles)),
                   kLaunch + TileTimes(bf16, l.kp / 64).t[2], l.bytes / (bf16 ? 5.5e6 : 4.75e6)});
}

// Which kernel takes which product, the rows of its tiles, and the block shape
// of the kernel of few rows: all of the products in tiles, all in blocks, or those
// of up to kFewRows rows in blocks and the others in tiles, as the estimates say.
// (bf16, 1024^3: 14 us in tiles, 6.5 in blocks; 2048^3: 15.7 and 28; 4096^3: 58 and
// 189; 8 products 8 x 2048 x 6144: 31 and 18; 32 of 48 rows 75 and 87, with fp32
// results 87 and 97, of 8 rows 84 and 76.)
int32_t plan_products(std::vector<F8ProdDesc>& desc, bool bf16, BlockCounts& out,
                      SmallPlan& sp) {
  Load few, many, all;
  std::vector<char> large(desc.size(), 0);
  auto take = [&](int32_t above) {  // products of more rows than this in tiles
    for (size_t i = 0; i < desc.size(); ++i) large[i] = desc[i].m > above;
  };
  for (const F8ProdDesc& d : desc) {
    if (d.m == 0) continue;
    (d.m <= kFewRows ? few : many).add(d);
    all.add(d);
  }
  const bool mixed = few.tiles > 0 && many.tiles > 0;
  double best = 0.97 * blocks_end(all);  // near the same: blocks (16 of 4 rows: 32 us, tiles 34)
  int32_t above = INT32_MAX;
  for (int32_t a : {0, kFewRows}) {
    if (a > 0 && !mixed) continue;
    take(a);
    const double us = tiles_end(desc, large, a > 0 ? many : all, bf16) + (a > 0 ? blocks_end(few) : 0);
    if (us < best) {
      best = us;
      above = a;
    }
  }
  take(above);
  if (above == 0) tiles_end(desc, large, all, bf16);  // the rows of its tiles
  if (above == kFewRows) tiles_end(desc, large, many, bf16);
  sp.mt = few_rows_mt(above == INT32_MAX ? all.rows : few.rows);
  // narrower blocks while there are too few to occupy the chip (one product 4 x
  // 2048 x 6144: 9.3 us in 32 blocks, 7.6 in 64, 7.2 in 128)
  double n64 = 0;
  for (size_t i = 0; i < desc.size(); ++i)
    if (const F8ProdDesc& d = desc[i]; d.m > 0 && !large[i])
      n64 += static_cast<double>(cdiv(d.m, 16 * sp.mt)) * static_cast<double>(cdiv(d.n, 64));
  sp.nt = n64 >= 96 ? 4 : n64 >= 48 ? 2 : 1;
  int64_t n[BlockCounts::kKinds] = {};
  int32_t st;
  for (size_t i = 0; i < desc.size(); ++i) {
    const F8ProdDesc& d = desc[i];
    if (large[i]) {
      const int64_t tn = cdiv(d.n, kF8Tile);
      const int64_t left = d.m - static_cast<int64_t>(d.full) * kF8Tile - d.half * (kF8Tile / 2);
      const int64_t rows[3] = {d.full, d.half, left > 0 ? cdiv(left, kF8Tile / 4) : 0};
      for (int k = 0; k < 3; ++k)
        if ((st = add_blocks(rows[k], tn, n[k])) != MUON_OK) return st;
      if (n[0] + n[1] + n[2] > kMaxBlocks)
        return fail(MUON_ERR_UNSUPPORTED, "batch needs 2^24 blocks or more");
    } else if (d.m > 0) {
      if ((st = add_blocks(cdiv(d.m, 16 * sp.mt), cdiv(d.n, 16 * sp.nt), n[3])) != MUON_OK) return st;
    }
    for (int k = 0; k < BlockCounts::kKinds; ++k) out.at(k)[i + 1] = static_cast<int32_t>(n[k]);
  }
  return MUON_OK;
}

// Whether eighths of the launch in table order (equal numbers of blocks, one
// eighth per XCD) differ in their work by more than kUneven.  Every XCD then
// takes an eighth of every product, and the longest products come first: 16
// products 2048 x 2048, K 1618 to 4328: 200 us against 223 (fp32: 351 against
// 420); 32 of 16 x 2048, K 2118 to 5863: 50 against 57.  Neighbouring tiles
// share operands in an XCD's L2, and eighths of few tiles lose that: equal K, 16
// products 1024 x 2048 x 6144: 195 us against 184; 8 tiles a product, 32 products
// 512 x 1024, K 1059 to 2931: 52 against 43.  Products of fewer than
// kSpreadTiles tiles on average stay whole.
bool uneven(const std::vector<F8ProdDesc>& desc, const int32_t* prefix) {
  const int64_t n = prefix[desc.size()];
  double all = 0, most = 0, sum = 0;
  int64_t at = 0;
  int32_t x = 0;
  for (size_t i = 0; i < desc.size(); ++i) {
    const double cost = desc[i].kp / 64 + kFixedSlices;
    while (at < prefix[i + 1]) {
      const int64_t end = n / 8 * (x + 1) + std::min<int64_t>(n % 8, x + 1);  // of the eighth
      const int64_t to = std::min<int64_t>(prefix[i + 1], end);
      sum += cost * static_cast<double>(to - at);
      at = to;
      if (at == end) {
        all += sum;
        most = std::max(most, sum);
        sum = 0;
        ++x;
      }
    }
  }
  return most * 8 > all * kUneven;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" size_t muon_grad_workspace_bytes(int32_t batch, const int64_t* numel) {
  try {
    clear_detail();
    GradPlan pl;
    if (make_grad_plan(batch, numel, pl) != MUON_OK) return SIZE_MAX;
    return pl.total_bytes;
  } catch (...) {
    fail(MUON_ERR_HIP, "unexpected host exception");
    return SIZE_MAX;
  }
}

extern "C" int32_t muon_grad_norm_batched(int32_t batch, const int64_t* numel,
                                          const void* const* g, const int32_t* dtype,
                                          const muon_grad_norm_params* p, float* result,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  try {
    clear_detail();
    GradPlan pl;
    int32_t st = make_grad_plan(batch, numel, pl);
    if (st != MUON_OK) return st;
    if ((st = check_norm_params(p)) != MUON_OK) return st;
    if ((st = check_float_ptr(result, "result")) != MUON_OK) return st;
    if ((st = bind_grads(batch, numel, g, dtype, nullptr, nullptr, pl)) != MUON_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, pl.total_bytes)) != MUON_OK) return st;
    char* ws = static_cast<char*>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    ArgTable t;
    GradCtx c{};
    if ((st = grad_table(pl, ws, s, t, c)) != MUON_OK) return st;
    return run_norm(pl, t, c, norm_args(pl, *p, result, ws), p->kind);
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}

extern "C" int32_t muon_grad_scale_batched(int32_t batch, const int64_t* numel,
                                           const void* const* g, const int32_t* dtype,
                                           void* const* out, const int32_t* out_dtype,
                                           const float* scale, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  try {
    clear_detail();
    GradPlan pl;
    int32_t st = make_grad_plan(batch, numel, pl);
    if (st != MUON_OK) return st;
    if ((st = check_float_ptr(scale, "scale")) != MUON_OK) return st;
    if (batch == 0) return MUON_OK;
    if (out == nullptr) return fail(MUON_ERR_INVALID_ARG, "out array is null");
    if ((st = bind_grads(batch, numel, g, dtype, out, out_dtype, pl)) != MUON_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, pl.total_bytes)) != MUON_OK) return st;
    hipStream_t s = static_cast<hipStream_t>(stream);
    ArgTable t;
    GradCtx c{};
    if ((st = grad_table(pl, static_cast<char*>(workspace), s, t, c)) != MUON_OK) return st;
    return run_scale(pl, t, c, scale);
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}

extern "C" int32_t muon_grad_clip_batched(int32_t batch, const int64_t* numel,
                                          const void* const* g, const int32_t* dtype,
                                          void* const* out, const int32_t* out_dtype,
                                          const muon_grad_norm_params* p, float* result,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  try {
    clear_detail();
    GradPlan pl;
    int32_t st = make_grad_plan(batch, numel, pl);
    if (st != MUON_OK) return st;
    if ((st = check_norm_params(p)) != MUON_OK) return st;
    if (!p->clip) return fail(MUON_ERR_INVALID_ARG, "clip must be 1");
    if ((st = check_float_ptr(result, "result")) != MUON_OK) return st;
    if (batch > 0 && out == nullptr) return fail(MUON_ERR_INVALID_ARG, "out array is null");
    if ((st = bind_grads(batch, numel, g, dtype, out, out_dtype, pl)) != MUON_OK) return st;
    if ((st = check_workspace(workspace, workspace_bytes, pl.total_bytes)) != MUON_OK) return st;
    char* ws = static_cast<char*>(workspace);
    hipStream_t s = static_cast<hipStream_t>(stream);
    ArgTable t;
    GradCtx c{};
    if ((st = grad_table(pl, ws, s, t, c)) != MUON_OK) return st;
    GradNormArgs a = norm_args(pl, *p, result, ws);
    a.keep_partials = grad_few_blocks(pl.chunks) ? 1 : 0;
    if ((st = run_norm(pl, t, c, a, p->kind)) != MUON_OK) return st;
    return run_scale(pl, t, c, result + 1, a.keep_partials ? &a : nullptr, p->kind);
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}

extern "C" size_t muon_f8_workspace_bytes(int32_t batch) {
  clear_detail();
  if (batch < 0) {
    fail(MUON_ERR_INVALID_ARG, "batch = %d is negative", batch);
    return SIZE_MAX;
  }
  return f8_ws_bytes(batch);
}

extern "C" int32_t muon_f8_quantize_batched(int32_t batch, const int64_t* rows,
                                            const int64_t* cols, const void* const* x,
                                            int32_t dtype, int32_t block_rows, void* const* q,
                                            void* const* s, void* const* qt, void* const* st_,
                                            void* workspace, size_t workspace_bytes,
                                            void* stream) {
  try {
    clear_detail();
    if (batch < 0) return fail(MUON_ERR_INVALID_ARG, "batch = %d is negative", batch);
    if (dtype != MUON_BF16 && dtype != MUON_FP32)
      return fail(MUON_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (block_rows != 1 && block_rows != kF8Block)
      return fail(MUON_ERR_INVALID_ARG, "block_rows = %d: must be 1 or %d", block_rows, kF8Block);
    if ((q == nullptr) != (s == nullptr) || (qt == nullptr) != (st_ == nullptr))
      return fail(MUON_ERR_INVALID_ARG, "values and scales of an operand go together");
    if (batch == 0) return MUON_OK;
    if (q == nullptr && qt == nullptr)
      return fail(MUON_ERR_INVALID_ARG, "neither the operand nor its transpose is asked for");
    if (rows == nullptr || cols == nullptr || x == nullptr)
      return fail(MUON_ERR_INVALID_ARG, "rows/cols/x array is null");
    std::vector<F8QuantDesc> desc(batch);
    std::vector<int32_t> prefix(static_cast<size_t>(batch) + 1, 0);
    int64_t total = 0, bytes = 0;
    int32_t st;
    for (int32_t i = 0; i < batch; ++i) {
      if ((st = check_f8_dim(rows[i], "rows", i)) != MUON_OK) return st;
      if ((st = check_f8_dim(cols[i], "cols", i)) != MUON_OK) return st;
      F8QuantDesc& d = desc[i];
      d = F8QuantDesc{};
      d.rows = static_cast<int32_t>(rows[i]);
      d.cols = static_cast<int32_t>(cols[i]);
      if (d.rows > 0 && d.cols > 0) {
        if ((st = check_ptr(x[i], "x", i)) != MUON_OK) return st;
        d.x = x[i];
        if (q != nullptr) {
          if ((st = check_ptr(q[i], "q", i)) != MUON_OK) return st;
          if ((st = check_ptr(s[i], "s", i)) != MUON_OK) return st;
          d.q = static_cast<uint8_t*>(q[i]);
          d.s = static_cast<uint8_t*>(s[i]);
        }
        if (qt != nullptr) {
          if ((st = check_ptr(qt[i], "qt", i)) != MUON_OK) return st;
          if ((st = check_ptr(st_[i], "st", i)) != MUON_OK) return st;
          d.qt = static_cast<uint8_t*>(qt[i]);
          d.st = static_cast<uint8_t*>(st_[i]);
        }
      }
      if ((st = add_blocks(cdiv(rows[i], kF8Block), cdiv(cols[i], kF8Block), total)) != MUON_OK)
        return st;
      prefix[i + 1] = static_cast<int32_t>(total);
      bytes += rows[i] * cols[i] * (dtype == MUON_BF16 ? 2 : 4);
    }
    if ((st = check_workspace(workspace, workspace_bytes, f8_ws_bytes(batch))) != MUON_OK) return st;
    char* ws = static_cast<char*>(workspace);
    hipStream_t stm = static_cast<hipStream_t>(stream);
    ArgTable t;
    F8QuantCtx c{};
    if ((st = place_table(desc.data(), sizeof(F8QuantDesc) * batch, prefix.data(),
                          sizeof(int32_t) * prefix.size(), ws, stm, t, &c.table)) != MUON_OK)
      return st;
    c.prefix_off = static_cast<int32_t>(align_up(sizeof(F8QuantDesc) * batch, kAlign));
    c.batch = batch;
    c.stream = stm;
    TimedLaunch tl(MUON_K_F8_QUANTIZE, stm);
    const hipError_t e = launch_f8_quantize(t, c, prefix[batch], dtype == MUON_BF16, block_rows, bytes);
    if (e != hipSuccess) return hip_fail(e, "launch e4m3 quantization");
    tl.done();
    return MUON_OK;
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}

extern "C" int32_t muon_f8_matmul_batched(int32_t batch, const int64_t* m, const int64_t* n,
                                          const int64_t* k, const void* const* a,
                                          const void* const* sa, const void* const* b,
                                          const void* const* sb, void* const* c, int32_t dtype,
                                          int32_t accumulate, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  try {
    clear_detail();
    if (batch < 0) return fail(MUON_ERR_INVALID_ARG, "batch = %d is negative", batch);
    if (dtype != MUON_BF16 && dtype != MUON_FP32)
      return fail(MUON_ERR_INVALID_ARG, "unknown dtype %d", dtype);
    if (accumulate != 0 && accumulate != 1)
      return fail(MUON_ERR_INVALID_ARG, "accumulate must be 0 or 1");
    if (batch == 0) return MUON_OK;
    if (m == nullptr || n == nullptr || k == nullptr || a == nullptr || sa == nullptr ||
        b == nullptr || sb == nullptr || c == nullptr)
      return fail(MUON_ERR_INVALID_ARG, "an argument array is null");
    std::vector<F8ProdDesc> desc(batch);
    int32_t st;
    int64_t bytes = 0;
    for (int32_t i = 0; i < batch; ++i) {
      if ((st = check_f8_dim(m[i], "m", i)) != MUON_OK) return st;
      if ((st = check_f8_dim(n[i], "n", i)) != MUON_OK) return st;
      if ((st = check_f8_dim(k[i], "k", i)) != MUON_OK) return st;
      F8ProdDesc& d = desc[i];
      d = F8ProdDesc{};
      d.m = static_cast<int32_t>(m[i]);
      d.n = static_cast<int32_t>(n[i]);
      d.kp = static_cast<int32_t>(cdiv(k[i], kF8Block) * kF8Block);
      bytes += m[i] * n[i] * (dtype == MUON_BF16 ? 2 : 4) + (m[i] + n[i]) * k[i];
      // nothing to store, or nothing to add
      const bool none = d.m == 0 || d.n == 0 || (d.kp == 0 && accumulate);
      if (!none) {
        if ((st = check_ptr(c[i], "c", i)) != MUON_OK) return st;
        d.c = c[i];
        if (d.kp > 0) {
          if ((st = check_ptr(a[i], "a", i)) != MUON_OK) return st;
          if ((st = check_ptr(sa[i], "sa", i)) != MUON_OK) return st;
          if ((st = check_ptr(b[i], "b", i)) != MUON_OK) return st;
          if ((st = check_ptr(sb[i], "sb", i)) != MUON_OK) return st;
          d.a = static_cast<const uint8_t*>(a[i]);
          d.sa = static_cast<const uint8_t*>(sa[i]);
          d.b = static_cast<const uint8_t*>(b[i]);
          d.sb = static_cast<const uint8_t*>(sb[i]);
        }
      } else {
        d.m = 0;
      }
    }
    BlockCounts blocks(batch);
    SmallPlan sp;
    if ((st = plan_products(desc, dtype == MUON_BF16, blocks, sp)) != MUON_OK) return st;
    const bool spread_tiles =
        blocks.total(0) >= kSpreadTiles * batch && uneven(desc, blocks.at(0));
    const bool spread_small = uneven(desc, blocks.at(3));
    if (spread_tiles || spread_small) {
      std::stable_sort(desc.begin(), desc.end(),
                       [](const F8ProdDesc& x, const F8ProdDesc& y) { return x.kp > y.kp; });
      if ((st = plan_products(desc, dtype == MUON_BF16, blocks, sp)) != MUON_OK) return st;
    }
    if ((st = check_workspace(workspace, workspace_bytes, f8_ws_bytes(batch))) != MUON_OK) return st;
    char* ws = static_cast<char*>(workspace);
    hipStream_t stm = static_cast<hipStream_t>(stream);
    ArgTable t;
    F8ProdCtx x{};
    if ((st = place_table(desc.data(), sizeof(F8ProdDesc) * batch, blocks.prefix.data(),
                          sizeof(int32_t) * blocks.prefix.size(), ws, stm, t, &x.table)) != MUON_OK)
      return st;
    x.prefix_off = static_cast<int32_t>(align_up(sizeof(F8ProdDesc) * batch, kAlign));
    x.batch = batch;
    x.accumulate = accumulate;
    x.spread = spread_tiles ? 1 : 0;
    x.nt = bytes > kNtBytes ? 1 : 0;
    x.stream = stm;
    TimedLaunch tl(MUON_K_F8_PROD, stm);
    hipError_t e = launch_f8_prod(t, x, blocks.total(0), blocks.total(1), blocks.total(2),
                                  dtype == MUON_BF16);
    x.spread = spread_small ? 1 : 0;
    x.prefix_off += 3 * static_cast<int32_t>(sizeof(int32_t)) * (batch + 1);
    if (e == hipSuccess) e = launch_f8_small(t, x, blocks.total(3), dtype == MUON_BF16, sp.mt, sp.nt);
    if (e != hipSuccess) return hip_fail(e, "launch e4m3 product");
    tl.done();
    return MUON_OK;
  } catch (...) {
    return fail(MUON_ERR_HIP, "unexpected host exception");
  }
}
