// C-ABI of the gated feed-forward block (include/ge_block.h): validate / create / forward /
// backward / destroy.  Host code only; the handle holds host memory only.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <new>

#include "../../include/ge_block.h"
#include "block_host.h"
#include "ge_block_internal.h"

struct ge_ffn_plan {
  ge_ffn_desc_t desc;
  int device;
  struct Choice { int tile, splits; } pair, down, grad, dx, dw;   // ge::FfnTile and splits per product
};

namespace {

using ge::block::aligned;
using ge::block::ceil_div;
using ge::block::Matrix;

static_assert((int)GE_FFN_TILE_256 == ge::FFN_T256 && (int)GE_FFN_TILE_128 == ge::FFN_T128 &&
                  (int)GE_FFN_TILE_64 == ge::FFN_T64 && (int)GE_FFN_TILE_COUNT == ge::FFN_TILES,
              "public tile ids mirror the kernel instances");

// Sizes are 32-bit in the kernels, which add at most two tiles to them.
constexpr int64_t kMaxSize = 0x7FFFFFFF - 512;
// A row operand's buffer spans up to 256 rows of one leading dimension in 31-bit byte offsets.
constexpr int64_t kMaxLd = int64_t(1) << 22;

// Up to 16 rows the forward products of large weights stream them through registers instead of tiles
// (4096 x 11008, one row: 53 us against 68 in tiles, 16 rows 58 against 70; 2048 x 5632: 23 against 29;
// 1024 x 2816: equal; 256 x 512: 10-14 against 10, and with 24 rows the tiles win or are even).
constexpr int64_t kFewWeights = int64_t(8) << 20;
// A tile's contraction is split over at most this many workgroups.
constexpr int kMaxSplits = 16;

// Whether a launch's threads can be counted in 32 bits, which the runtime asks for.
bool grid_fits(int tile, int64_t M, int64_t N, bool pair, int products) {
  const ge::FfnTileInfo ti = ge::ffn_tile_info(tile);
  const double tiles = (double)ceil_div(M, ti.bm) * (double)ceil_div(N, pair ? ti.bn_pair : ti.bn) * products;
  return tiles * (tile == ge::FFN_T64 ? 256 : 512) <= 4294967295.0;
}

// Tile and splits of one launch: the least estimated time in microseconds.  A tile costs `fixed` and
// `slot` for every 64 values of the contraction, `crowd` instead where workgroups share a compute
// unit or come in rounds; a split adds the partial sums' way through memory and back.  The figures
// were measured over grids of 64 to 768 workgroups; they need only rank the choices.
using Choice = ge_ffn_plan::Choice;
Choice pick(int mode, int64_t M, int64_t N, int64_t K, int products, int32_t asked) {
  if (asked) return Choice{asked - 1, 1};
  const bool pair = mode == ge::FFN_PAIR, dw = mode == ge::FFN_WGRAD;
  const int64_t slots = ceil_div(K, 64) * (mode == ge::FFN_DUAL ? 2 : 1);
  struct Cost { double fixed, slot, crowd; };
  const Cost cost[ge::FFN_TILES] = {{7.0, 1.3, 1.4},
                                    {3.0, pair ? 1.0 : 0.5, pair ? 1.0 : dw ? 0.65 : 0.57},
                                    {1.5, pair ? 0.45 : 0.26, pair ? 0.43 : dw ? 0.27 : 0.21}};
  Choice best{ge::FFN_T256, 1};
  double least = 1e300;
  for (int t = 0; t < ge::FFN_TILES; ++t) {
    if (!grid_fits(t, M, N, pair, products)) continue;
    const ge::FfnTileInfo ti = ge::ffn_tile_info(t);
    const int bn = pair ? ti.bn_pair : ti.bn;
    const double tiles = (double)ceil_div(M, ti.bm) * (double)ceil_div(N, bn) * products;
    for (int s = 1; s <= (t == ge::FFN_T256 ? 1 : kMaxSplits); s *= 2) {
      if (s > 1 && (slots < 4 * s || tiles * s > ge::kFfnMaxSplitGroups)) break;
      // (workgroups of many rounds no longer end together)
      const double ratio = tiles * s / 256.0, rounds = ratio < 4.0 ? std::ceil(ratio) : ratio;
      const double mine = (double)ceil_div(slots, s);
      double us = rounds > 1.0 ? rounds * (cost[t].fixed + mine * cost[t].crowd) : cost[t].fixed + mine * cost[t].slot;
      if (s > 1) us += 2.5 + tiles * s * ti.bm * bn * (pair ? 8.0 : 4.0) * 2 / 3e6;
      if (us < least) {
        least = us;
        best = Choice{t, s};
      }
    }
  }
  return best;
}

// Adds a product to a launch; returns false if the grid would pass 31 bits.
bool add(ge::FfnLaunch& l, ge::FfnProduct p, const Choice& c, bool pair) {
  const int tile = c.tile;
  l.splits = c.splits;
  const ge::FfnTileInfo ti = ge::ffn_tile_info(tile);
  const int64_t tm = ceil_div(p.M, ti.bm), tn = ceil_div(p.N, pair ? ti.bn_pair : ti.bn);
  if ((l.tiles + tm * tn) * c.splits > 0x7FFFFFFF) return false;
  p.tiles_m = (int32_t)tm;
  p.tiles_n = (int32_t)tn;
  p.tile0 = l.tiles;
  if (tm * tn > 0) l.prod[l.n++] = p;
  l.tiles += (int32_t)(tm * tn);
  return true;
}

// Few rows: how a product is split.  One workgroup of eight waves on every compute unit at most (so a
// split launch has no more than 256), and no more splits than the longest wave's share needs.
struct FewPlan { int tiles, splits; };
FewPlan few_plan(int64_t N, int64_t K) {
  FewPlan f;
  f.tiles = (int)ceil_div(N, ge::kFfnFewCols);
  const int64_t units = ceil_div(K, ge::kFfnFewUnit), waves = 8;
  const int64_t most = std::max<int64_t>(1, 256 / std::max<int64_t>(f.tiles, 1));
  const int64_t share = std::max<int64_t>(1, ceil_div(units, waves * most));     // units of the longest wave
  f.splits = (int)std::max<int64_t>(1, ceil_div(units, waves * share));
  return f;
}
size_t few_part_bytes(const FewPlan& f, int operands) {
  return f.splits > 1 ? (size_t)f.tiles * f.splits * operands * ge::kFfnFewRows * ge::kFfnFewCols * 4 : 0;
}

size_t hidden_bytes(const ge_ffn_desc_t& d) { return (size_t)d.M * (size_t)d.h * 2; }
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

// Workspace of both calls: [tickets][partial sums][H], or [tickets][partial sums][dG][dU][H].  The
// tickets come first and take the same room in every workspace; the launches of a call follow each
// other and use the tickets and the partial sums in turn.
struct Layout { size_t part, hidden, total; };
bool few_rows(const ge_ffn_desc_t& d) { return d.tile == 0 && d.M <= ge::kFfnFewRows && d.d * d.h >= kFewWeights; }
FewPlan few_up(const ge_ffn_desc_t& d) { return few_plan(d.h, d.d); }
FewPlan few_down(const ge_ffn_desc_t& d) { return few_plan(d.d, d.h); }
size_t part_bytes(const Choice& c, int64_t M, int64_t N, bool pair, int products = 1) {
  if (c.splits < 2) return 0;
  const ge::FfnTileInfo ti = ge::ffn_tile_info(c.tile);
  const int bn = pair ? ti.bn_pair : ti.bn;
  return (size_t)(ceil_div(M, ti.bm) * ceil_div(N, bn) * products) * c.splits * ti.bm * bn * (pair ? 8 : 4);
}
Layout forward_layout(const ge_ffn_plan* p) {
  const ge_ffn_desc_t& d = p->desc;
  Layout l{};
  l.part = ge::kTicketBytes;
  const size_t sums = few_rows(d) ? std::max(few_part_bytes(few_up(d), 2), few_part_bytes(few_down(d), 1))
                                  : std::max(part_bytes(p->pair, d.M, d.h, true), part_bytes(p->down, d.M, d.d, false));
  l.hidden = l.part + round256(sums);
  l.total = l.hidden + round256(hidden_bytes(d));
  return l;
}
Layout backward_layout(const ge_ffn_plan* p) {
  const ge_ffn_desc_t& d = p->desc;
  Layout l{};
  l.part = ge::kTicketBytes;
  l.hidden = l.part + round256(std::max({part_bytes(p->grad, d.M, d.h, false), part_bytes(p->dx, d.M, d.d, false),
                                         part_bytes(p->dw, d.d, d.h, false, 3)}));
  l.total = l.hidden + 3 * round256(hidden_bytes(d));
  return l;
}
size_t forward_bytes(const ge_ffn_plan* p) { return forward_layout(p).total; }
size_t backward_bytes(const ge_ffn_plan* p) { return backward_layout(p).total; }
// Points a launch at the workspace's tickets and partial sums.
void share(ge::FfnLaunch& l, unsigned char* ws, const Layout& lay) {
  l.ctr = reinterpret_cast<uint32_t*>(ws);
  l.part = reinterpret_cast<float*>(ws + lay.part);
}

Matrix weight_in(const ge_ffn_desc_t& d, const void* p, int64_t ld) {      // Wg, Wu and their gradients
  return d.w_layout == GE_LAYOUT_KN ? Matrix{p, d.d, d.h, ld} : Matrix{p, d.h, d.d, ld};
}
Matrix weight_out(const ge_ffn_desc_t& d, const void* p, int64_t ld) {     // Wd and its gradient
  return d.w_layout == GE_LAYOUT_KN ? Matrix{p, d.h, d.d, ld} : Matrix{p, d.d, d.h, ld};
}

const uint16_t* in(const void* p) { return static_cast<const uint16_t*>(p); }
uint16_t* out(void* p) { return static_cast<uint16_t*>(p); }

}  // namespace

extern "C" {

ge_status_t ge_ffn_validate(const ge_ffn_desc_t* d) {
  if (!d) return GE_ERR_INVALID_ARG;
  if (d->M < 0 || d->d < 0 || d->h < 0) return GE_ERR_INVALID_ARG;
  if (d->act < GE_ACT_NONE || d->act > GE_ACT_SILU) return GE_ERR_INVALID_ARG;
  if (d->w_layout != GE_LAYOUT_KN && d->w_layout != GE_LAYOUT_NK) return GE_ERR_INVALID_ARG;
  if ((d->residual | 1) != 1 || (d->save | 1) != 1) return GE_ERR_INVALID_ARG;
  if (d->tile < 0 || d->tile > GE_FFN_TILE_COUNT) return GE_ERR_INVALID_ARG;
  const int64_t wi = d->w_layout == GE_LAYOUT_KN ? d->h : d->d, wo = d->w_layout == GE_LAYOUT_KN ? d->d : d->h;
  const int64_t lds[][2] = {{d->ldx, d->d}, {d->ldy, d->d}, {d->ldr, d->d}, {d->ldg, d->h}, {d->lddy, d->d},
                            {d->lddx, d->d}, {d->ldw, wi}, {d->ldwd, wo}, {d->lddw, wi}, {d->lddwd, wo}};
  for (auto& l : lds)
    if (l[0] < l[1]) return GE_ERR_INVALID_ARG;
  if (d->d % 8 || d->h % 8) return GE_ERR_UNSUPPORTED;
  for (auto& l : lds)
    if (l[0] % 8 || l[0] >= kMaxLd) return GE_ERR_UNSUPPORTED;
  if (d->M > kMaxSize || d->d > kMaxSize || d->h > kMaxSize) return GE_ERR_UNSUPPORTED;
  const int tile = d->tile ? d->tile - 1 : ge::FFN_T256;
  if (!grid_fits(tile, d->M, d->h, true, 1) || !grid_fits(tile, d->M, d->h, false, 1) ||
      !grid_fits(tile, d->M, d->d, false, 1) || !grid_fits(tile, std::max(d->d, d->h), std::min(d->d, d->h), false, 3))
    return GE_ERR_UNSUPPORTED;
  return GE_OK;
}

ge_status_t ge_ffn_create(const ge_ffn_desc_t* d, ge_ffn_handle_t* handle) {
  if (!handle) return GE_ERR_INVALID_ARG;
  *handle = nullptr;
  const ge_status_t st = ge_ffn_validate(d);
  if (st != GE_OK) return st;
  int device = 0;
  if (!ge::block::current_gfx950(&device)) return GE_ERR_DEVICE;
  ge_ffn_plan* p = new (std::nothrow) ge_ffn_plan();
  if (!p) return GE_ERR_HIP;
  p->desc = *d;
  p->device = device;
  p->pair = pick(ge::FFN_PAIR, d->M, d->h, d->d, 1, d->tile);
  p->down = pick(ge::FFN_DOWN, d->M, d->d, d->h, 1, d->tile);
  p->grad = pick(ge::FFN_GRAD, d->M, d->h, d->d, 1, d->tile);
  p->dx = pick(ge::FFN_DUAL, d->M, d->d, d->h, 1, d->tile);
  p->dw = pick(ge::FFN_WGRAD, d->d, d->h, d->M, 3, d->tile);
  *handle = p;
  return GE_OK;
}

void ge_ffn_destroy(ge_ffn_handle_t h) { delete h; }

ge_status_t ge_ffn_workspace_size(ge_ffn_handle_t h, int32_t backward, size_t* bytes) {
  if (!h || !bytes || (backward | 1) != 1) return GE_ERR_INVALID_ARG;
  *bytes = backward ? backward_bytes(h) : forward_bytes(h);
  return GE_OK;
}

ge_status_t ge_ffn_describe(ge_ffn_handle_t h, char* buf, size_t len) {
  if (!h || !buf || len == 0) return GE_ERR_INVALID_ARG;
  const int rows[] = {256, 128, 64};
  char up[32];
  if (few_rows(h->desc)) std::snprintf(up, sizeof up, "few rows");
  else std::snprintf(up, sizeof up, "pair=%d/%d down=%d/%d", rows[h->pair.tile], h->pair.splits, rows[h->down.tile], h->down.splits);
  std::snprintf(buf, len, "%s grad=%d/%d dx=%d/%d dw=%d/%d b=%s act=%d", up, rows[h->grad.tile], h->grad.splits,
                rows[h->dx.tile], h->dx.splits, rows[h->dw.tile], h->dw.splits,
                h->desc.w_layout == GE_LAYOUT_NK ? "NK" : "KN", (int)h->desc.act);
  return GE_OK;
}

ge_status_t ge_ffn_forward(ge_ffn_handle_t h, const ge_ffn_args_t* a, void* stream) {
  if (!h || !a) return GE_ERR_INVALID_ARG;
  const ge_ffn_desc_t& d = h->desc;
  if (d.M == 0 || (d.d == 0 && !(d.save && d.h > 0))) return GE_OK;   // nothing to write
  const Matrix inputs[] = {{a->X, d.M, d.d, d.ldx}, weight_in(d, a->Wg, d.ldw), weight_in(d, a->Wu, d.ldw),
                           weight_out(d, a->Wd, d.ldwd), {d.residual ? a->residual : nullptr, d.residual ? d.M : 0, d.d, d.ldr}};
  const Matrix outputs[] = {{a->Y, d.M, d.d, d.ldy}, {d.save ? a->G : nullptr, d.save ? d.M : 0, d.h, d.ldg},
                            {d.save ? a->U : nullptr, d.save ? d.M : 0, d.h, d.ldg},
                            {a->workspace, 1, (int64_t)(forward_bytes(h) / 2), (int64_t)(forward_bytes(h) / 2)}};
  const bool in_place = d.residual && a->residual == a->Y && d.ldr == d.ldy;    // Y over R: allowed
  if (!ge::block::usable(inputs, 5, outputs, 4, in_place ? 4 : -1, in_place ? 0 : -1)) return GE_ERR_INVALID_ARG;
  if (a->workspace_bytes < forward_bytes(h)) return GE_ERR_INVALID_ARG;
  if (!ge::block::is_current(h->device)) return GE_ERR_DEVICE;

  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool nk = d.w_layout == GE_LAYOUT_NK;
  const Layout lay = forward_layout(h);
  unsigned char* ws = static_cast<unsigned char*>(a->workspace);
  uint16_t* H = out(ws + lay.hidden);
  if (few_rows(d)) {
    FewPlan f = few_up(d);
    ge::FfnFew q{};
    q.A = in(a->X); q.B = in(a->Wg); q.B2 = in(a->Wu);
    q.Y = H; q.Y2 = d.save ? out(a->G) : nullptr; q.Y3 = d.save ? out(a->U) : nullptr;
    q.part = reinterpret_cast<float*>(ws + lay.part); q.ctr = reinterpret_cast<uint32_t*>(ws);
    q.lda = d.ldx; q.ldb = d.ldw; q.ldy = d.h; q.ldy2 = d.ldg;
    q.M = (int32_t)d.M; q.N = (int32_t)d.h; q.K = (int32_t)d.d;
    q.tiles = f.tiles; q.splits = f.splits;
    if (ge::launch_ffn_few(true, d.act, nk, q, s) != hipSuccess) return GE_ERR_HIP;
    f = few_down(d);
    q = ge::FfnFew{};
    q.A = H; q.B = in(a->Wd); q.E1 = d.residual ? in(a->residual) : nullptr; q.Y = out(a->Y);
    q.part = reinterpret_cast<float*>(ws + lay.part); q.ctr = reinterpret_cast<uint32_t*>(ws);
    q.lda = d.h; q.ldb = d.ldwd; q.lde = d.ldr; q.ldy = d.ldy;
    q.M = (int32_t)d.M; q.N = (int32_t)d.d; q.K = (int32_t)d.h;
    q.tiles = f.tiles; q.splits = f.splits;
    return ge::launch_ffn_few(false, ge::ACT_NONE, nk, q, s) == hipSuccess ? GE_OK : GE_ERR_HIP;
  }
  ge::FfnLaunch pair{}, down{};
  ge::FfnProduct p{};
  p.A = in(a->X); p.B = in(a->Wg); p.B2 = in(a->Wu);
  p.Y = H; p.Y2 = d.save ? out(a->G) : nullptr; p.Y3 = d.save ? out(a->U) : nullptr;
  p.lda = d.ldx; p.ldb = d.ldw; p.ldy = d.h; p.ldy2 = d.ldg;
  p.M = (int32_t)d.M; p.N = (int32_t)d.h; p.K = (int32_t)d.d;
  if (!add(pair, p, h->pair, true)) return GE_ERR_UNSUPPORTED;
  p = ge::FfnProduct{};
  p.A = H; p.B = in(a->Wd); p.E1 = d.residual ? in(a->residual) : nullptr;
  p.Y = out(a->Y);
  p.lda = d.h; p.ldb = d.ldwd; p.lde = d.ldr; p.ldy = d.ldy;
  p.M = (int32_t)d.M; p.N = (int32_t)d.d; p.K = (int32_t)d.h;
  if (!add(down, p, h->down, false)) return GE_ERR_UNSUPPORTED;
  share(pair, ws, lay);
  share(down, ws, lay);
  if (ge::launch_ffn_pair(h->pair.tile, d.act, nk, pair, s) != hipSuccess) return GE_ERR_HIP;
  if (ge::launch_ffn_plain(ge::FFN_DOWN, h->down.tile, nk, down, s) != hipSuccess) return GE_ERR_HIP;
  return GE_OK;
}

ge_status_t ge_ffn_backward(ge_ffn_handle_t h, const ge_ffn_args_t* a, void* stream) {
  if (!h || !a) return GE_ERR_INVALID_ARG;
  const ge_ffn_desc_t& d = h->desc;
  const bool want_dx = a->dX != nullptr, want_dw = a->dWg || a->dWu || a->dWd;
  const int64_t rows_dx = want_dx ? d.M : 0;
  const size_t hb = round256(hidden_bytes(d));
  const Matrix none{nullptr, 0, 0, 0};
  const Matrix inputs[] = {want_dw ? Matrix{a->X, d.M, d.d, d.ldx} : none,
                           want_dx ? weight_in(d, a->Wg, d.ldw) : none,
                           want_dx ? weight_in(d, a->Wu, d.ldw) : none,
                           weight_out(d, a->Wd, d.ldwd),
                           {a->G, d.M, d.h, d.ldg}, {a->U, d.M, d.h, d.ldg}, {a->dY, d.M, d.d, d.lddy}};
  const Matrix outputs[] = {{a->dX, rows_dx, d.d, d.lddx},
                            want_dw ? weight_in(d, a->dWg, d.lddw) : none, want_dw ? weight_in(d, a->dWu, d.lddw) : none,
                            want_dw ? weight_out(d, a->dWd, d.lddwd) : none,
                            {a->workspace, 1, (int64_t)(backward_bytes(h) / 2), (int64_t)(backward_bytes(h) / 2)}};
  if (!ge::block::usable(inputs, 7, outputs, 5, -1, -1)) return GE_ERR_INVALID_ARG;
  if (a->workspace_bytes < backward_bytes(h)) return GE_ERR_INVALID_ARG;
  if (!ge::block::is_current(h->device)) return GE_ERR_DEVICE;

  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool nk = d.w_layout == GE_LAYOUT_NK;
  const Layout lay = backward_layout(h);
  unsigned char* ws = static_cast<unsigned char*>(a->workspace);
  uint16_t* dG = out(ws + lay.hidden);
  uint16_t* dU = dG + hb / 2;
  uint16_t* H = dU + hb / 2;
  ge::FfnLaunch grad{}, dx{}, dw{};
  ge::FfnProduct p{};
  // dH = dY Wd^T: Wd [h][d] is B [N][K], Wd [d][h] is B [K][N]
  p.A = in(a->dY); p.B = in(a->Wd); p.E1 = in(a->G); p.E2 = in(a->U);
  p.Y = dG; p.Y2 = dU; p.Y3 = H;
  p.lda = d.lddy; p.ldb = d.ldwd; p.lde = d.ldg; p.ldy = d.h; p.ldy2 = d.h;
  p.M = (int32_t)d.M; p.N = (int32_t)d.h; p.K = (int32_t)d.d;
  if (!add(grad, p, h->grad, false)) return GE_ERR_UNSUPPORTED;
  if (want_dx) {
    p = ge::FfnProduct{};
    p.A = dG; p.A2 = dU; p.B = in(a->Wg); p.B2 = in(a->Wu); p.Y = out(a->dX);
    p.lda = d.h; p.ldb = d.ldw; p.ldy = d.lddx;
    p.M = (int32_t)d.M; p.N = (int32_t)d.d; p.K = (int32_t)d.h;
    if (!add(dx, p, h->dx, false)) return GE_ERR_UNSUPPORTED;
  }
  if (want_dw) {
    // contraction over the rows; [in][out] weights: X^T dG, X^T dU, H^T dY; [out][in]: swapped
    const struct { const uint16_t *l, *r; int64_t ldl, ldr, m, n; void* y; int64_t ldy; } w[3] = {
        {in(a->X), dG, d.ldx, d.h, d.d, d.h, a->dWg, d.lddw},
        {in(a->X), dU, d.ldx, d.h, d.d, d.h, a->dWu, d.lddw},
        {H, in(a->dY), d.h, d.lddy, d.h, d.d, a->dWd, d.lddwd}};
    for (auto& t : w) {
      p = ge::FfnProduct{};
      p.A = nk ? t.r : t.l; p.B = nk ? t.l : t.r;
      p.lda = nk ? t.ldr : t.ldl; p.ldb = nk ? t.ldl : t.ldr;
      p.M = (int32_t)(nk ? t.n : t.m); p.N = (int32_t)(nk ? t.m : t.n); p.K = (int32_t)d.M;
      p.Y = out(t.y); p.ldy = t.ldy;
      if (!add(dw, p, h->dw, false)) return GE_ERR_UNSUPPORTED;
    }
  }
  for (ge::FfnLaunch* l : {&grad, &dx, &dw}) share(*l, ws, lay);
  if (ge::launch_ffn_grad(h->grad.tile, d.act, !nk, grad, s) != hipSuccess) return GE_ERR_HIP;
  if (ge::launch_ffn_plain(ge::FFN_DUAL, h->dx.tile, !nk, dx, s) != hipSuccess) return GE_ERR_HIP;
  if (ge::launch_ffn_plain(ge::FFN_WGRAD, h->dw.tile, false, dw, s) != hipSuccess) return GE_ERR_HIP;
  return GE_OK;
}

}  // extern "C"
