// C-ABI of the row operators (include/ge_rows.h): layer norm with dropout and residual, dropout, int8
// codes, and the product of codes.  Host code only; the handles hold host memory only.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <new>

#include "../../include/ge_rows.h"
#include "block_host.h"
#include "ge_rows_internal.h"

using ge::block::aligned;
using ge::block::ceil_div;
using ge::block::Matrix;

struct ge_norm_plan {
  ge_norm_desc_t desc;
  int device;
  int grid_forward, grid_backward;
};
struct ge_dropout_plan {
  ge_dropout_desc_t desc;
  int device;
};
struct ge_quant_plan {
  ge_quant_desc_t desc;
  int device, grid;
};
struct ge_i8_plan {
  ge_i8_desc_t desc;
  int device;
  int tile, splits;           // ge::FfnTile
  bool few;                   // the few-row kernel instead of a tile
  int32_t cols;               // its columns a workgroup
};

namespace {

constexpr int64_t kMaxRows = int64_t(1) << 40, kMaxPitch = int64_t(1) << 40;
constexpr uint32_t kDropSteps = 65536;

int64_t size_of(int32_t dtype) { return dtype == GE_DT_BF16 ? 2 : 4; }

ge_status_t check_type(int32_t dtype) {
  if (dtype == GE_DT_FP8_E4M3) return GE_ERR_UNSUPPORTED;
  return dtype == GE_DT_BF16 || dtype == GE_DT_FP32 ? GE_OK : GE_ERR_INVALID_ARG;
}

// Half-words below this are dropped (p was checked).
uint32_t drop_below(float p) { return (uint32_t)std::lround((double)p * kDropSteps); }
bool drop_in_range(float p) { return p >= 0.0f && (double)p <= (double)(kDropSteps - 1) / kDropSteps; }
ge::DropParams drop_params(float p, uint32_t site, const int64_t* rng) {
  const uint32_t below = drop_below(p);
  return ge::DropParams{rng, site, below, (float)((double)kDropSteps / (double)(kDropSteps - below))};
}
// Every block has a counter of its own in 32 bits.
bool blocks_fit(int64_t rows, int64_t d) { return (double)rows * (double)ceil_div(d, 8) <= 4294967296.0; }

// Sizes and pitches whose byte offsets stay below 2^62.
ge_status_t check_rows(int64_t rows, int64_t d, const int64_t* pitches, int n) {
  if (rows < 0 || d < 0) return GE_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (pitches[i] < d) return GE_ERR_INVALID_ARG;
  if (rows > kMaxRows) return GE_ERR_UNSUPPORTED;
  for (int i = 0; i < n; ++i)
    if (pitches[i] > kMaxPitch || (double)rows * (double)pitches[i] > 1e18) return GE_ERR_UNSUPPORTED;
  return GE_OK;
}

// What a call reads and writes: pointers are checked when they are added, overlaps at the end.
struct Buffers {
  Matrix in[8], out[8];
  int n_in = 0, n_out = 0;
  bool ok = true;

  bool fits(const Matrix& m, int64_t align, bool optional) {
    if (m.empty()) return false;
    if (!m.p && optional) return false;
    if (!m.p || !aligned(m.p, (size_t)align)) ok = false;
    return ok;
  }
  void read(const Matrix& m, int64_t align, bool optional = false) {
    if (fits(m, align, optional)) in[n_in++] = m;
  }
  void write(const Matrix& m, int64_t align, bool optional = false) {
    if (fits(m, align, optional)) out[n_out++] = m;
  }
  // An output may be one of the inputs [0, same), element for element.
  bool apart(int same) const {
    if (!ok) return false;
    for (int o = 0; o < n_out; ++o) {
      for (int i = 0; i < n_in; ++i) {
        const bool is = i < same && in[i].p == out[o].p && in[i].rows == out[o].rows && in[i].cols == out[o].cols &&
                        in[i].size == out[o].size && (in[i].ld == out[o].ld || in[i].rows == 1);
        if (!is && ge::block::overlap(in[i], out[o])) return false;
      }
      for (int q = 0; q < o; ++q)
        if (ge::block::overlap(out[o], out[q])) return false;
    }
    return true;
  }
};

// At most `most` workgroups, fewer where that gives each the same number of turns.
int even_grid(int64_t turns, int64_t most) {
  return turns > 0 ? (int)ceil_div(turns, ceil_div(turns, most)) : 0;
}
// Workgroups that fit `waves` waves on every compute unit.
int64_t resident(const ge::RowShape& s, int64_t waves) {
  return 256 * std::max<int64_t>(1, waves * 64 / std::max(s.threads, 256));
}

// Whether a call's outputs pass what the caches would keep of them for the next one.
bool large(int64_t rows, int64_t d, int64_t size, int outputs) { return rows * d * size * outputs > ge::kRowsLarge; }

hipStream_t stream_of(void* s) { return static_cast<hipStream_t>(s); }
ge_status_t status_of(hipError_t e) { return e == hipSuccess ? GE_OK : GE_ERR_HIP; }

template <class P>
ge_status_t make(P** out, P** handle) {
  *handle = nullptr;
  int device = 0;
  if (!ge::block::current_gfx950(&device)) return GE_ERR_DEVICE;
  P* p = new (std::nothrow) P();
  if (!p) return GE_ERR_HIP;
  p->device = device;
  *out = *handle = p;
  return GE_OK;
}

size_t norm_bytes(const ge_norm_plan* h) {
  return ge::kTicketBytes + (size_t)h->grid_backward * 2 * (size_t)h->desc.d * 4;
}

}  // namespace

extern "C" {

// ---------------------------------------------------------------------------------------------
// layer norm
// ---------------------------------------------------------------------------------------------
ge_status_t ge_norm_validate(const ge_norm_desc_t* d) {
  if (!d) return GE_ERR_INVALID_ARG;
  if (d->d < 1 || (d->residual | 1) != 1 || !drop_in_range(d->dropout)) return GE_ERR_INVALID_ARG;
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return GE_ERR_INVALID_ARG;
  const ge_status_t type = check_type(d->dtype);
  if (type == GE_ERR_INVALID_ARG) return type;
  const int64_t pitches[] = {d->ldx, d->ldr, d->lds, d->ldy, d->lddy, d->ldds, d->lddx, d->lddr};
  const ge_status_t st = check_rows(d->rows, d->d, pitches, 8);
  if (st != GE_OK || type != GE_OK) return st == GE_ERR_INVALID_ARG ? st : type != GE_OK ? type : st;
  if (d->d > ge::kRowMax) return GE_ERR_UNSUPPORTED;
  if (drop_below(d->dropout) && !blocks_fit(d->rows, d->d)) return GE_ERR_UNSUPPORTED;
  return GE_OK;
}

ge_status_t ge_norm_create(const ge_norm_desc_t* d, ge_norm_handle_t* handle) {
  if (!handle) return GE_ERR_INVALID_ARG;
  *handle = nullptr;
  ge_status_t st = ge_norm_validate(d);
  if (st != GE_OK) return st;
  ge_norm_plan* p = nullptr;
  st = make(&p, handle);
  if (st != GE_OK) return st;
  p->desc = *d;
  const int shape = ge::row_shape(d->d);
  const ge::RowShape &fwd = ge::kRowShape[shape], &bwd = ge::kGradShape[shape];
  p->grid_forward = (int)std::min<int64_t>(ceil_div(d->rows, ge::rows_at_once(fwd)), 1 << 20);
  // Eight waves on a compute unit, though more would fit: a workgroup leaves 8 d bytes of partial sums, and each row's
  // loads are ahead of it anyhow (16384 x 4096 bf16 112.8 us against 125.9 with 16 waves, x 2048 63.4 against 71.0; 4
  // waves 83).
  p->grid_backward = even_grid(ceil_div(d->rows, ge::rows_at_once(bwd)), resident(bwd, 8));
  return GE_OK;
}

void ge_norm_destroy(ge_norm_handle_t h) { delete h; }

ge_status_t ge_norm_workspace_size(ge_norm_handle_t h, size_t* bytes) {
  if (!h || !bytes) return GE_ERR_INVALID_ARG;
  *bytes = norm_bytes(h);
  return GE_OK;
}

ge_status_t ge_norm_forward(ge_norm_handle_t h, const ge_norm_args_t* a, void* stream) {
  if (!h || !a) return GE_ERR_INVALID_ARG;
  const ge_norm_desc_t& d = h->desc;
  if (d.rows == 0) return GE_OK;
  const int64_t size = size_of(d.dtype);
  const bool drop = drop_below(d.dropout) != 0;
  Buffers b;
  b.read({a->X, d.rows, d.d, d.ldx, size}, size);
  if (d.residual) b.read({a->residual, d.rows, d.d, d.ldr, size}, size);
  const int same = b.n_in;
  b.read({a->gain, 1, d.d, d.d, size}, size, true);
  b.read({a->bias, 1, d.d, d.d, size}, size, true);
  if (drop) b.read({a->rng, 1, 2, 2, 8}, 8);
  b.write({a->S, d.rows, d.d, d.lds, size}, size, true);
  b.write({a->Y, d.rows, d.d, d.ldy, size}, size);
  b.write({a->mean, 1, d.rows, d.rows, 4}, 4, true);
  b.write({a->rstd, 1, d.rows, d.rows, 4}, 4, true);
  if (!b.apart(same)) return GE_ERR_INVALID_ARG;
  if (!ge::block::is_current(h->device)) return GE_ERR_DEVICE;
  ge::NormParams p{};
  p.x = a->X; p.r = d.residual ? a->residual : nullptr; p.s = a->S; p.y = a->Y;
  p.gain = a->gain; p.bias = a->bias; p.mean = a->mean; p.rstd = a->rstd;
  p.drop = drop_params(d.dropout, d.site, a->rng);
  p.rows = d.rows; p.ldx = d.ldx; p.ldr = d.ldr; p.lds = d.lds; p.ldy = d.ldy;
  p.d = (int32_t)d.d;
  p.eps = d.eps;
  return status_of(ge::launch_norm_forward(d.dtype == GE_DT_BF16, large(d.rows, d.d, size, a->S ? 2 : 1), p, h->grid_forward, stream_of(stream)));
}

ge_status_t ge_norm_backward(ge_norm_handle_t h, const ge_norm_args_t* a, void* stream) {
  if (!h || !a) return GE_ERR_INVALID_ARG;
  const ge_norm_desc_t& d = h->desc;
  const int64_t size = size_of(d.dtype);
  const bool drop = drop_below(d.dropout) != 0 && a->dX, sums = a->dgain || a->dbias;
  Buffers b;
  b.read({a->dY, d.rows, d.d, d.lddy, size}, size);
  b.read({a->S, d.rows, d.d, d.lds, size}, size);
  b.read({a->dS, d.rows, d.d, d.ldds, size}, size, true);
  const int same = b.n_in;
  b.read({a->mean, 1, d.rows, d.rows, 4}, 4);
  b.read({a->rstd, 1, d.rows, d.rows, 4}, 4);
  if (d.rows > 0) {
    b.read({a->gain, 1, d.d, d.d, size}, size, true);
    if (drop) b.read({a->rng, 1, 2, 2, 8}, 8);
  }
  b.write({a->dX, d.rows, d.d, d.lddx, size}, size, true);
  b.write({a->dR, d.rows, d.d, d.lddr, size}, size, true);
  b.write({a->dgain, 1, d.d, d.d, 4}, 4, true);
  b.write({a->dbias, 1, d.d, d.d, 4}, 4, true);
  if (sums) {
    const int64_t bytes = (int64_t)norm_bytes(h);
    b.write({a->workspace, 1, bytes, bytes, 1}, 16);
    if (a->workspace_bytes < norm_bytes(h)) return GE_ERR_INVALID_ARG;
  }
  if (!b.apart(same)) return GE_ERR_INVALID_ARG;
  if (!ge::block::is_current(h->device)) return GE_ERR_DEVICE;
  if (!a->dX && !a->dR && !sums) return GE_OK;
  float* const part = sums ? reinterpret_cast<float*>(static_cast<unsigned char*>(a->workspace) + ge::kTicketBytes) : nullptr;
  hipStream_t s = stream_of(stream);
  ge::NormGradParams p{};
  p.dy = a->dY; p.s = a->S; p.ds = a->dS; p.gain = a->gain; p.mean = a->mean; p.rstd = a->rstd;
  p.dx = a->dX; p.dr = a->dR; p.part = part;
  p.drop = drop_params(d.dropout, d.site, a->rng);
  if (!drop) p.drop.below = 0;
  p.rows = d.rows; p.lddy = d.lddy; p.lds = d.lds; p.ldds = d.ldds; p.lddx = d.lddx; p.lddr = d.lddr;
  p.d = (int32_t)d.d;
  const int outputs = (a->dX != nullptr) + (a->dR != nullptr);
  if (ge::launch_norm_backward(d.dtype == GE_DT_BF16, large(d.rows, d.d, size, outputs), p, h->grid_backward, s) != hipSuccess) return GE_ERR_HIP;
  if (!sums) return GE_OK;
  return status_of(ge::launch_norm_sums(part, h->grid_backward, p.d, a->dgain, a->dbias, s));
}

// ---------------------------------------------------------------------------------------------
// dropout
// ---------------------------------------------------------------------------------------------
ge_status_t ge_dropout_validate(const ge_dropout_desc_t* d) {
  if (!d) return GE_ERR_INVALID_ARG;
  if ((d->residual | 1) != 1 || !drop_in_range(d->p)) return GE_ERR_INVALID_ARG;
  const ge_status_t type = check_type(d->dtype);
  if (type == GE_ERR_INVALID_ARG) return type;
  const int64_t pitches[] = {d->ldx, d->ldr, d->ldy, d->lddy, d->lddx};
  const ge_status_t st = check_rows(d->rows, d->d, pitches, 5);
  if (st != GE_OK || type != GE_OK) return st == GE_ERR_INVALID_ARG ? st : type != GE_OK ? type : st;
  if (d->d > 0x7FFFFFF0 || !blocks_fit(d->rows, d->d)) return GE_ERR_UNSUPPORTED;
  return GE_OK;
}

ge_status_t ge_dropout_create(const ge_dropout_desc_t* d, ge_dropout_handle_t* handle) {
  if (!handle) return GE_ERR_INVALID_ARG;
  *handle = nullptr;
  ge_status_t st = ge_dropout_validate(d);
  if (st != GE_OK) return st;
  ge_dropout_plan* p = nullptr;
  st = make(&p, handle);
  if (st == GE_OK) p->desc = *d;
  return st;
}

void ge_dropout_destroy(ge_dropout_handle_t h) { delete h; }

namespace {
ge_status_t run_dropout(const ge_dropout_plan* h, const void* x, int64_t ldx, const void* r, int64_t ldr, void* y, int64_t ldy,
                        const int64_t* rng, void* stream) {
  const ge_dropout_desc_t& d = h->desc;
  if (d.rows == 0 || d.d == 0) return GE_OK;
  const int64_t size = size_of(d.dtype);
  Buffers b;
  b.read({x, d.rows, d.d, ldx, size}, size);
  b.read({r, d.rows, d.d, ldr, size}, size, true);
  const int same = b.n_in;
  b.read({rng, 1, 2, 2, 8}, 8);
  b.write({y, d.rows, d.d, ldy, size}, size);
  if (!b.apart(same)) return GE_ERR_INVALID_ARG;
  if (!ge::block::is_current(h->device)) return GE_ERR_DEVICE;
  ge::DropoutParams p{};
  p.x = x; p.r = r; p.y = y;
  p.drop = drop_params(d.p, d.site, rng);
  p.rows = d.rows; p.ldx = ldx; p.ldr = ldr; p.ldy = ldy;
  p.d = (int32_t)d.d;
  return status_of(ge::launch_dropout(d.dtype == GE_DT_BF16, large(d.rows, d.d, size, 1), p, stream_of(stream)));
}
}  // namespace

ge_status_t ge_dropout_forward(ge_dropout_handle_t h, const ge_dropout_args_t* a, void* stream) {
  if (!h || !a) return GE_ERR_INVALID_ARG;
  const ge_dropout_desc_t& d = h->desc;
  if (d.residual && !a->residual && d.rows > 0 && d.d > 0) return GE_ERR_INVALID_ARG;
  return run_dropout(h, a->X, d.ldx, d.residual ? a->residual : nullptr, d.ldr, a->Y, d.ldy, a->rng, stream);
}

ge_status_t ge_dropout_backward(ge_dropout_handle_t h, const ge_dropout_args_t* a, void* stream) {
  if (!h || !a) return GE_ERR_INVALID_ARG;
  return run_dropout(h, a->dY, h->desc.lddy, nullptr, 0, a->dX, h->desc.lddx, a->rng, stream);
}

// ---------------------------------------------------------------------------------------------
// int8 codes
// ---------------------------------------------------------------------------------------------
ge_status_t ge_quant_validate(const ge_quant_desc_t* d) {
  if (!d) return GE_ERR_INVALID_ARG;
  const ge_status_t type = check_type(d->dtype);
  if (type == GE_ERR_INVALID_ARG) return type;
  const int64_t pitches[] = {d->ldx, d->ldq};
  const ge_status_t st = check_rows(d->rows, d->d, pitches, 2);
  if (st != GE_OK || type != GE_OK) return st == GE_ERR_INVALID_ARG ? st : type != GE_OK ? type : st;
  return d->d > ge::kRowMax ? GE_ERR_UNSUPPORTED : GE_OK;
}

ge_status_t ge_quant_create(const ge_quant_desc_t* d, ge_quant_handle_t* handle) {
  if (!handle) return GE_ERR_INVALID_ARG;
  *handle = nullptr;
  ge_status_t st = ge_quant_validate(d);
  if (st != GE_OK) return st;
  ge_quant_plan* p = nullptr;
  st = make(&p, handle);
  if (st != GE_OK) return st;
  p->desc = *d;
  const ge::RowShape& shape = ge::kRowShape[ge::row_shape(d->d)];
  p->grid = even_grid(ceil_div(d->rows, ge::rows_at_once(shape)), resident(shape, 32));
  return GE_OK;
}

void ge_quant_destroy(ge_quant_handle_t h) { delete h; }

ge_status_t ge_quant_run(ge_quant_handle_t h, const ge_quant_args_t* a, void* stream) {
  if (!h || !a) return GE_ERR_INVALID_ARG;
  const ge_quant_desc_t& d = h->desc;
  if (d.rows == 0) return GE_OK;
  const int64_t size = size_of(d.dtype);
  Buffers b;
  b.read({a->X, d.rows, d.d, d.ldx, size}, size);
  b.write({a->codes, d.rows, d.d, d.ldq, 1}, 1);
  b.write({a->scale, 1, d.rows, d.rows, 4}, 4);
  if (!b.apart(0)) return GE_ERR_INVALID_ARG;
  if (!ge::block::is_current(h->device)) return GE_ERR_DEVICE;
  ge::QuantParams p{};
  p.x = a->X; p.codes = a->codes; p.scale = a->scale;
  p.rows = d.rows; p.ldx = d.ldx; p.ldq = d.ldq;
  p.d = (int32_t)d.d;
  return status_of(ge::launch_quant(d.dtype == GE_DT_BF16, large(d.rows, d.d, 1, 1), p, h->grid, stream_of(stream)));
}

}  // extern "C"

// ---------------------------------------------------------------------------------------------
// product of codes
// ---------------------------------------------------------------------------------------------
namespace {

static_assert((int)GE_I8_TILE_256 == ge::FFN_T256 && (int)GE_I8_TILE_128 == ge::FFN_T128 &&
                  (int)GE_I8_TILE_64 == ge::FFN_T64 && (int)GE_I8_TILE_COUNT == ge::FFN_TILES,
              "public tile ids mirror the kernel instances");
// Sizes are 32-bit in the kernels, which add at most two tiles to them.
constexpr int64_t kMaxSize = 0x7FFFFFFF - 512;
// A tile's buffers span up to 256 rows of one pitch in 31-bit byte offsets.
constexpr int64_t kMaxLd = int64_t(1) << 22;
constexpr int64_t kMaxK = int64_t(1) << 17;
constexpr int kMaxSplits = 16;

// Whether a launch's threads can be counted in 32 bits, which the runtime asks for.
bool grid_fits(int tile, int64_t M, int64_t N) {
  const ge::FfnTileInfo ti = ge::ffn_tile_info(tile);
  return (double)ceil_div(M, ti.bm) * (double)ceil_div(N, ti.bn) * (tile == ge::FFN_T64 ? 256 : 512) <= 4294967295.0;
}

// Whether the few-row kernel takes the product (N x K, everything from memory, against the tiles, us).  Where each workgroup
// has a compute unit to itself, the tokens' codes only have to fit its LDS (4096 x 4096: one token 6.5 against 8.2, 16 tokens
// 8.4 against 8.2, 32 tokens 9.6 against 9.4; 2856 x 1040, 27 tokens 4.6 against 5.0).  Where several share one, two have to
// fit (11008 x 4096, 27 tokens in 109 KiB: 21.9 against 14.2), and the tokens' way to LDS counts: up to 12 tokens (one token:
// 6144 x 4096 7.5 against 10.2, 11008 x 4096 12.2 against 13.3; 12 tokens: 6144 x 2048 6.7 against 7.8, 8192 x 5120
// 11.7 against 12.5), 8 where K is long (8192 x 8192 16.6 against 19.1), and none where they come in rounds of little
// work each (one token: 32000 x 1024 12.5 against 10.0, but x 2064 15.0 against 18.3, x 4096 27 against 33).  The borders are
// not exact: past 4 tokens K = 4096 would be faster in tiles (8 tokens: 11008 x 4096 14.5 against 13.5), and with all weights
// in the caches tiles are faster at many sizes from 11008 columns on (one token: 11008 x 4096 9.9 against 9.4).
// (Fewer than 2^22 outputs a token, the most that a pitch allows: the launch's threads fit 32 bits.)
bool few_rows(const ge_i8_desc_t& d) {
  if (d.tile || d.M > ge::kI8FewRows) return false;
  const int64_t lds = ge::i8_few_lds(d.M, d.K), groups = ceil_div(d.N, ge::kI8FewCols);
  if (groups <= 256) return lds <= ge::kI8FewLds;
  return d.M <= (d.K <= 4096 ? 12 : 8) && lds <= ge::kI8FewLds / 2 && (groups <= 768 || d.K > 2048);
}

// Columns of its workgroups: half as many where each workgroup then still has a compute unit to itself (one token: 264 x 11008
// 7.6 -> 5.9 us, 2048 x 8192 6.6 -> 6.1; 3000 x 4000, past it, would take 5.1 against 4.7), and for few tokens where some
// compute units would have two workgroups of whole width and the others one (4608 x 4096 7.8 -> 6.9, 6144 x 4096 8.7 -> 8.2;
// with 16 tokens 5120 x 5120 would take 15 us against 13, and from 512 workgroups on, 8192 x 8192, one token 16.5 against 15.2).
int few_cols(const ge_i8_desc_t& d) {
  const int64_t groups = ceil_div(d.N, ge::kI8FewCols);
  return groups <= 128 || (d.M <= 4 && groups > 256 && groups <= 384) ? ge::kI8FewCols / 2 : ge::kI8FewCols;
}

// Tile and splits: the least estimated time in microseconds.  A tile costs `fixed` and `slot` for every 128
// codes of the contraction, `crowd` instead where workgroups share a compute unit or come in rounds; a
// split adds a ticket, the last workgroup's reads and the partial sums' way through memory and back.  The
// figures were measured over 27 to 8192 tokens and 4 to 86 slots; they need only rank the choices.
void pick(ge_i8_plan* p) {
  const ge_i8_desc_t& d = p->desc;
  p->tile = d.tile ? d.tile - 1 : (int)ge::FFN_T256;
  p->splits = 1;
  p->few = few_rows(d);
  p->cols = few_cols(d);
  if (d.tile || p->few) return;
  const int64_t slots = ceil_div(d.K, 128);
  struct Cost { double fixed, slot, crowd; };
  const Cost cost[ge::FFN_TILES] = {{7.0, 1.0, 1.35}, {3.5, 0.4, 0.57}, {3.0, 0.25, 0.21}};
  double least = 1e300;
  for (int t = 0; t < ge::FFN_TILES; ++t) {
    if (!grid_fits(t, d.M, d.N)) continue;
    const ge::FfnTileInfo ti = ge::ffn_tile_info(t);
    const int64_t tiles_m = ceil_div(d.M, ti.bm);
    const double tiles = (double)tiles_m * (double)ceil_div(d.N, ti.bn);
    for (int s = 1; s <= (t == ge::FFN_T256 ? 1 : kMaxSplits); ++s) {
      if (s > 1 && (slots < 2 * s || tiles * s > ge::kFfnMaxSplitGroups)) break;
      const double ratio = tiles * s / 256.0, rounds = ratio < 4.0 ? std::ceil(ratio) : ratio;
      const double mine = (double)ceil_div(slots, s);
      double us = rounds > 1.0 ? rounds * (cost[t].fixed + mine * cost[t].crowd) : cost[t].fixed + mine * cost[t].slot;
      const double rows = (double)std::min<int64_t>(ceil_div(d.M, 16) * 16, tiles_m * ti.bm);
      if (s > 1) us += 1.5 + 0.3 * s + rows * (double)ceil_div(d.N, ti.bn) * ti.bn * s * 4.0 * 0.9e-6;
      if (us < least) {
        least = us;
        p->tile = t;
        p->splits = s;
      }
    }
  }
}

size_t i8_bytes(const ge_i8_plan* p) {
  if (p->splits < 2) return 0;
  const ge::FfnTileInfo ti = ge::ffn_tile_info(p->tile);
  return ge::kTicketBytes + (size_t)(ceil_div(p->desc.M, ti.bm) * ceil_div(p->desc.N, ti.bn)) * p->splits * ti.bm * ti.bn * 4;
}

}  // namespace

extern "C" {

ge_status_t ge_i8_validate(const ge_i8_desc_t* d) {
  if (!d) return GE_ERR_INVALID_ARG;
  if (d->M < 0 || d->N < 0 || d->K < 0) return GE_ERR_INVALID_ARG;
  if (d->act < GE_ACT_NONE || d->act > GE_ACT_SILU) return GE_ERR_INVALID_ARG;
  if ((d->bias | 1) != 1 || (d->residual | 1) != 1) return GE_ERR_INVALID_ARG;
  if (d->tile < 0 || d->tile > GE_I8_TILE_COUNT) return GE_ERR_INVALID_ARG;
  if (d->ldx < d->K || d->ldw < d->K || d->ldy < d->N || d->ldr < d->N) return GE_ERR_INVALID_ARG;
  const ge_status_t type = check_type(d->dtype);
  if (type != GE_OK) return type;
  if (d->N % 8 || d->K % 16 || d->K >= kMaxK) return GE_ERR_UNSUPPORTED;
  if (d->ldx % 16 || d->ldw % 16 || d->ldy % 8 || d->ldr % 8) return GE_ERR_UNSUPPORTED;
  const int64_t most = d->dtype == GE_DT_BF16 ? kMaxLd : kMaxLd / 2;
  if (d->ldx >= kMaxLd || d->ldw >= kMaxLd || d->ldy >= most || d->ldr >= most) return GE_ERR_UNSUPPORTED;
  if (d->M > kMaxSize || d->N > kMaxSize) return GE_ERR_UNSUPPORTED;
  if (!grid_fits(d->tile ? d->tile - 1 : (int)ge::FFN_T256, d->M, d->N)) return GE_ERR_UNSUPPORTED;
  return GE_OK;
}

ge_status_t ge_i8_create(const ge_i8_desc_t* d, ge_i8_handle_t* handle) {
  if (!handle) return GE_ERR_INVALID_ARG;
  *handle = nullptr;
  ge_status_t st = ge_i8_validate(d);
  if (st != GE_OK) return st;
  ge_i8_plan* p = nullptr;
  st = make(&p, handle);
  if (st != GE_OK) return st;
  p->desc = *d;
  pick(p);
  return GE_OK;
}

void ge_i8_destroy(ge_i8_handle_t h) { delete h; }

ge_status_t ge_i8_workspace_size(ge_i8_handle_t h, size_t* bytes) {
  if (!h || !bytes) return GE_ERR_INVALID_ARG;
  *bytes = i8_bytes(h);
  return GE_OK;
}

ge_status_t ge_i8_describe(ge_i8_handle_t h, char* buf, size_t len) {
  if (!h || !buf || len == 0) return GE_ERR_INVALID_ARG;
  const int rows[] = {256, 128, 64};
  if (h->few) std::snprintf(buf, len, "few rows act=%d", (int)h->desc.act);
  else std::snprintf(buf, len, "tile=%d splits=%d act=%d", rows[h->tile], h->splits, (int)h->desc.act);
  return GE_OK;
}

ge_status_t ge_i8_run(ge_i8_handle_t h, const ge_i8_args_t* a, void* stream) {
  if (!h || !a) return GE_ERR_INVALID_ARG;
  const ge_i8_desc_t& d = h->desc;
  if (d.M == 0 || d.N == 0) return GE_OK;
  const int64_t size = size_of(d.dtype), bytes = (int64_t)i8_bytes(h);
  Buffers b;
  if (d.residual) b.read({a->residual, d.M, d.N, d.ldr, size}, 16);
  const int same = b.n_in;
  b.read({a->X, d.M, d.K, d.ldx, 1}, 16);
  b.read({a->W, d.N, d.K, d.ldw, 1}, 16);
  b.read({a->x_scale, 1, d.M, d.M, 4}, 4);
  b.read({a->w_scale, 1, d.N, d.N, 4}, 4);
  if (d.bias) b.read({a->bias, 1, d.N, d.N, size}, 16);
  b.write({a->Y, d.M, d.N, d.ldy, size}, 16);
  b.write({a->workspace, 1, bytes, bytes, 1}, 16);
  if (!b.apart(same) || (bytes > 0 && a->workspace_bytes < (size_t)bytes)) return GE_ERR_INVALID_ARG;
  if (!ge::block::is_current(h->device)) return GE_ERR_DEVICE;
  const ge::I8Epilogue ep{a->x_scale, a->w_scale, d.bias ? a->bias : nullptr, d.act, d.dtype == GE_DT_FP32};
  if (h->few) {
    const ge::I8Few f{a->X, a->W, d.residual ? a->residual : nullptr, a->Y, ep, d.ldx, d.ldw, d.ldy, d.ldr,
                      (int32_t)d.M, (int32_t)d.N, (int32_t)d.K, (int32_t)ge::i8_few_pitch(d.K), h->cols};
    return status_of(ge::launch_i8_few(f, stream_of(stream)));
  }
  const ge::FfnTileInfo ti = ge::ffn_tile_info(h->tile);
  ge::I8Launch l{};
  ge::FfnProduct& p = l.prod[0];
  p.A = reinterpret_cast<const uint16_t*>(a->X);
  p.B = reinterpret_cast<const uint16_t*>(a->W);
  p.E1 = d.residual ? static_cast<const uint16_t*>(a->residual) : nullptr;
  p.Y = static_cast<uint16_t*>(a->Y);
  p.lda = d.ldx / 2; p.ldb = d.ldw / 2; p.lde = d.ldr; p.ldy = d.ldy;
  p.M = (int32_t)d.M; p.N = (int32_t)d.N; p.K = (int32_t)(d.K / 2);
  p.tiles_m = (int32_t)ceil_div(d.M, ti.bm);
  p.tiles_n = (int32_t)ceil_div(d.N, ti.bn);
  l.n = 1;
  l.tiles = p.tiles_m * p.tiles_n;
  l.splits = h->splits;
  if (bytes > 0) {
    l.ctr = static_cast<uint32_t*>(a->workspace);
    l.part = reinterpret_cast<float*>(static_cast<unsigned char*>(a->workspace) + ge::kTicketBytes);
  }
  l.ep = ep;
  return status_of(ge::launch_i8(h->tile, l, stream_of(stream)));
}

}  // extern "C"
