// C-ABI of the gated feed-forward block (include/ge_block.h): validate / create / forward /
// backward / destroy.  Host code only; the handle holds host memory only.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <new>

#include "../../include/ge_block.h"
#include "block_host.h"
#include "ge_block_internal.h"

struct ge_ffn_plan {
  ge_ffn_desc_t desc;
  int device;
  int tile_pair, tile_down, tile_grad, tile_dx, tile_dw;   // ge::FfnTile per product
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

// Tile of one product by its grid: the largest tile that still gives `want` workgroups, so that
// all 256 compute units have work (the 64-row tiles run several workgroups per unit).
int pick_tile(int64_t M, int64_t N, bool pair, int32_t asked) {
  if (asked) return asked - 1;
  for (int t : {ge::FFN_T256, ge::FFN_T128}) {
    const ge::FfnTileInfo ti = ge::ffn_tile_info(t);
    if (ceil_div(M, ti.bm) * ceil_div(N, pair ? ti.bn_pair : ti.bn) >= 192) return t;
  }
  return ge::FFN_T64;
}

// Adds a product to a launch; returns false if the grid would pass 31 bits.
bool add(ge::FfnLaunch& l, ge::FfnProduct p, int tile, bool pair) {
  const ge::FfnTileInfo ti = ge::ffn_tile_info(tile);
  const int64_t tm = ceil_div(p.M, ti.bm), tn = ceil_div(p.N, pair ? ti.bn_pair : ti.bn);
  if (l.tiles + tm * tn > 0x7FFFFFFF) return false;
  p.tiles_m = (int32_t)tm;
  p.tiles_n = (int32_t)tn;
  p.tile0 = l.tiles;
  if (tm * tn > 0) l.prod[l.n++] = p;
  l.tiles += (int32_t)(tm * tn);
  return true;
}

size_t hidden_bytes(const ge_ffn_desc_t& d) { return (size_t)d.M * (size_t)d.h * 2; }
size_t round256(size_t b) { return (b + 255) / 256 * 256; }

size_t forward_bytes(const ge_ffn_plan* p) { return round256(hidden_bytes(p->desc)); }
size_t backward_bytes(const ge_ffn_plan* p) { return 3 * round256(hidden_bytes(p->desc)); }

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
  // every launch's grid in 31 bits even with the smallest tile, three products at once
  const int64_t bm = 64;
  if (ceil_div(d->M, bm) * ceil_div(d->h, bm) > 0x3FFFFFFF || ceil_div(d->M, bm) * ceil_div(d->d, bm) > 0x3FFFFFFF ||
      ceil_div(d->d, bm) * ceil_div(d->h, bm) > 0x1FFFFFFF)
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
  p->tile_pair = pick_tile(d->M, d->h, true, d->tile);
  p->tile_down = pick_tile(d->M, d->d, false, d->tile);
  p->tile_grad = pick_tile(d->M, d->h, false, d->tile);
  p->tile_dx = pick_tile(d->M, d->d, false, d->tile);
  p->tile_dw = pick_tile(d->d, 3 * d->h, false, d->tile);
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
  std::snprintf(buf, len, "pair=%d down=%d grad=%d dx=%d dw=%d b=%s act=%d", rows[h->tile_pair], rows[h->tile_down],
                rows[h->tile_grad], rows[h->tile_dx], rows[h->tile_dw], h->desc.w_layout == GE_LAYOUT_NK ? "NK" : "KN",
                (int)h->desc.act);
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
  uint16_t* H = out(a->workspace);
  ge::FfnLaunch pair{}, down{};
  ge::FfnProduct p{};
  p.A = in(a->X); p.B = in(a->Wg); p.B2 = in(a->Wu);
  p.Y = H; p.Y2 = d.save ? out(a->G) : nullptr; p.Y3 = d.save ? out(a->U) : nullptr;
  p.lda = d.ldx; p.ldb = d.ldw; p.ldy = d.h; p.ldy2 = d.ldg;
  p.M = (int32_t)d.M; p.N = (int32_t)d.h; p.K = (int32_t)d.d;
  if (!add(pair, p, h->tile_pair, true)) return GE_ERR_UNSUPPORTED;
  p = ge::FfnProduct{};
  p.A = H; p.B = in(a->Wd); p.E1 = d.residual ? in(a->residual) : nullptr;
  p.Y = out(a->Y);
  p.lda = d.h; p.ldb = d.ldwd; p.lde = d.ldr; p.ldy = d.ldy;
  p.M = (int32_t)d.M; p.N = (int32_t)d.d; p.K = (int32_t)d.h;
  if (!add(down, p, h->tile_down, false)) return GE_ERR_UNSUPPORTED;
  if (ge::launch_ffn_pair(h->tile_pair, d.act, nk, pair, s) != hipSuccess) return GE_ERR_HIP;
  if (ge::launch_ffn_plain(ge::FFN_DOWN, h->tile_down, nk, down, s) != hipSuccess) return GE_ERR_HIP;
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
                            {a->workspace, 1, (int64_t)(3 * hb / 2), (int64_t)(3 * hb / 2)}};
  if (!ge::block::usable(inputs, 7, outputs, 5, -1, -1)) return GE_ERR_INVALID_ARG;
  if (a->workspace_bytes < backward_bytes(h)) return GE_ERR_INVALID_ARG;
  if (!ge::block::is_current(h->device)) return GE_ERR_DEVICE;

  hipStream_t s = static_cast<hipStream_t>(stream);
  const bool nk = d.w_layout == GE_LAYOUT_NK;
  uint16_t* dG = out(a->workspace);
  uint16_t* dU = dG + hb / 2;
  uint16_t* H = dU + hb / 2;
  ge::FfnLaunch grad{}, dx{}, dw{};
  ge::FfnProduct p{};
  // dH = dY Wd^T: Wd [h][d] is B [N][K], Wd [d][h] is B [K][N]
  p.A = in(a->dY); p.B = in(a->Wd); p.E1 = in(a->G); p.E2 = in(a->U);
  p.Y = dG; p.Y2 = dU; p.Y3 = H;
  p.lda = d.lddy; p.ldb = d.ldwd; p.lde = d.ldg; p.ldy = d.h; p.ldy2 = d.h;
  p.M = (int32_t)d.M; p.N = (int32_t)d.h; p.K = (int32_t)d.d;
  if (!add(grad, p, h->tile_grad, false)) return GE_ERR_UNSUPPORTED;
  if (want_dx) {
    p = ge::FfnProduct{};
    p.A = dG; p.A2 = dU; p.B = in(a->Wg); p.B2 = in(a->Wu); p.Y = out(a->dX);
    p.lda = d.h; p.ldb = d.ldw; p.ldy = d.lddx;
    p.M = (int32_t)d.M; p.N = (int32_t)d.d; p.K = (int32_t)d.h;
    if (!add(dx, p, h->tile_dx, false)) return GE_ERR_UNSUPPORTED;
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
      if (!add(dw, p, h->tile_dw, false)) return GE_ERR_UNSUPPORTED;
    }
  }
  if (ge::launch_ffn_grad(h->tile_grad, d.act, !nk, grad, s) != hipSuccess) return GE_ERR_HIP;
  if (ge::launch_ffn_plain(ge::FFN_DUAL, h->tile_dx, !nk, dx, s) != hipSuccess) return GE_ERR_HIP;
  if (ge::launch_ffn_plain(ge::FFN_WGRAD, h->tile_dw, false, dw, s) != hipSuccess) return GE_ERR_HIP;
  return GE_OK;
}

}  // extern "C"
