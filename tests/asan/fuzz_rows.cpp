// Drives the C-ABI of the row operators on the host, under the sanitizers: random and mutated descriptors
// through validate, create, workspace_size and the calls, with stand-ins for the HIP runtime (one gfx950 that
// is current) and for the launches, which check what the kernels rely on: grids the runtime can count, tickets
// and partial sums inside their part of the workspace, LDS that a workgroup has, offsets and counters in
// their bits.  Then single calls that have to be refused or taken.  Nothing is dereferenced.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>

#include "../../gemm_epilogue_transformer_tiled_amd/csrc/ge_rows_internal.h"
#include "../../include/ge_rows.h"

static int g_device = 0;
extern "C" hipError_t hipGetDevice(int* d) { *d = g_device; return hipSuccess; }
#undef hipGetDeviceProperties
extern "C" hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {
  std::memset(p, 0, sizeof *p);
  std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
  return hipSuccess;
}
extern "C" hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_t* p, int d) { return hipGetDeviceProperties(p, d); }
extern "C" hipError_t hipGetLastError(void) { return hipSuccess; }

namespace {
uintptr_t g_ws = 0;
size_t g_ws_bytes = 0;
long g_launches = 0;
#define CHECK(c)                                                           \
  do {                                                                     \
    if (!(c)) {                                                            \
      std::fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__);  \
      std::abort();                                                        \
    }                                                                      \
  } while (0)

bool in_ws(const void* p, size_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return a >= g_ws && a + bytes <= g_ws + g_ws_bytes;
}
// data lies behind the room of the most tickets, which every workspace begins with
bool behind_tickets(const void* p) { return reinterpret_cast<uintptr_t>(p) >= g_ws + ge::kTicketBytes; }

void check_drop(const ge::DropParams& p, int64_t rows, int64_t d) {
  CHECK(p.below <= 65535u);
  if (p.below) CHECK(p.rng && reinterpret_cast<uintptr_t>(p.rng) % 8 == 0 && (double)rows * ((d + 7) / 8) <= 4294967296.0);
  CHECK(std::isfinite(p.factor) && p.factor >= 1.0f);
}
void check_shape(int64_t d, const ge::RowShape* shapes) {
  const ge::RowShape& s = shapes[ge::row_shape(d)];
  CHECK(8 * (int64_t)s.threads * s.vecs >= d);
}
}  // namespace

namespace ge {
hipError_t launch_norm_forward(bool bf16, bool, const NormParams& p, int grid, hipStream_t) {
  ++g_launches;
  const uintptr_t size = bf16 ? 2 : 4;
  CHECK(p.rows > 0 && grid > 0 && grid <= (1 << 20) && p.d >= 1 && p.d <= kRowMax);
  check_shape(p.d, kRowShape);
  check_drop(p.drop, p.rows, p.d);
  for (const void* q : {p.x, (const void*)p.y}) CHECK(q && reinterpret_cast<uintptr_t>(q) % size == 0);
  CHECK(p.ldx >= p.d && p.ldy >= p.d && p.lds >= p.d && p.ldr >= p.d);
  return hipSuccess;
}
hipError_t launch_norm_backward(bool bf16, bool, const NormGradParams& p, int grid, hipStream_t) {
  CHECK((grid == 0) == (p.rows == 0));
  if (grid == 0) return hipSuccess;
  ++g_launches;
  const uintptr_t size = bf16 ? 2 : 4;
  CHECK(p.rows > 0 && grid <= 4096 && grid * (int64_t)rows_at_once(kGradShape[row_shape(p.d)]) < p.rows + 4);
  check_shape(p.d, kGradShape);
  check_drop(p.drop, p.rows, p.d);
  CHECK(p.mean && p.rstd && p.dy && p.s && (p.dx || p.dr || p.part));
  for (const void* q : {p.dy, p.s, p.ds, (const void*)p.dx, (const void*)p.dr}) CHECK(reinterpret_cast<uintptr_t>(q) % size == 0);
  if (p.part) CHECK(in_ws(p.part, (size_t)grid * 2 * p.d * 4) && behind_tickets(p.part));
  return hipSuccess;
}
hipError_t launch_norm_sums(const float* part, int parts, int d, float* dgain, float* dbias, hipStream_t) {
  ++g_launches;
  CHECK(in_ws(part, (size_t)parts * 2 * d * 4) && (dgain || dbias));
  return hipSuccess;
}
hipError_t launch_dropout(bool, bool, const DropoutParams& p, hipStream_t) {
  ++g_launches;
  CHECK(p.rows > 0 && p.d > 0 && p.x && p.y && p.ldx >= p.d && p.ldy >= p.d && (!p.r || p.ldr >= p.d));
  CHECK((double)p.rows * ((p.d + 7) / 8) <= 4294967296.0);
  check_drop(p.drop, p.rows, p.d);
  return hipSuccess;
}
hipError_t launch_quant(bool, bool, const QuantParams& p, int grid, hipStream_t) {
  ++g_launches;
  CHECK(p.rows > 0 && grid > 0 && grid <= 8192 && p.d >= 0 && p.d <= kRowMax && p.scale);
  check_shape(p.d, kRowShape);
  return hipSuccess;
}
hipError_t launch_i8(int tile, const I8Launch& l, hipStream_t) {
  ++g_launches;
  const FfnTileInfo ti = ffn_tile_info(tile);
  const FfnProduct& p = l.prod[0];
  CHECK(l.n == 1 && p.tile0 == 0 && l.splits >= 1 && (tile != FFN_T256 || l.splits == 1));
  CHECK((int64_t)p.tiles_m * p.tiles_n == l.tiles && l.tiles > 0);
  CHECK((int64_t)p.tiles_m * ti.bm >= p.M && (int64_t)p.tiles_n * ti.bn >= p.N);
  CHECK((double)l.tiles * l.splits * (tile == FFN_T64 ? 256 : 512) < 4294967296.0);
  CHECK(p.N % 8 == 0 && p.K % 8 == 0 && p.K < (1 << 16));
  CHECK(256.0 * p.lda * 2 < 2147483648.0 && 256.0 * p.ldb * 2 < 2147483648.0 && 256.0 * p.ldy * (l.ep.wide ? 4 : 2) < 2147483648.0);
  CHECK(p.K == 0 || (p.A && p.B));
  CHECK(l.ep.x_scale && l.ep.w_scale && p.Y);
  if (l.splits > 1) {
    CHECK(l.tiles * l.splits <= kFfnMaxSplitGroups);
    CHECK(in_ws(l.ctr, (size_t)l.tiles * kFfnCtrStride * 4) && in_ws(l.part, (size_t)l.tiles * l.splits * ti.bm * ti.bn * 4));
    CHECK(reinterpret_cast<uintptr_t>(l.ctr) == g_ws && behind_tickets(l.part));
  }
  return hipSuccess;
}
hipError_t launch_i8_few(const I8Few& p, hipStream_t) {
  ++g_launches;
  CHECK(p.M >= 1 && p.M <= kI8FewRows && p.N >= 8 && p.N % 8 == 0 && p.K % 16 == 0);
  CHECK(i8_few_lds(p.M, p.K) <= kI8FewLds && p.x_pitch == i8_few_pitch(p.K) && p.x_pitch % 256 == 32);
  CHECK(p.cols == kI8FewCols || p.cols == kI8FewCols / 2);
  // whole steps of the tokens' codes lie before the next token's
  CHECK((p.K + kI8FewStep - 1) / kI8FewStep * (int64_t)kI8FewStep <= p.x_pitch);
  CHECK((double)((p.N + kI8FewCols - 1) / kI8FewCols) * 512 < 4294967296.0);
  return hipSuccess;
}
}  // namespace ge

static void* at(int i) { return reinterpret_cast<void*>((uintptr_t)(i + 1) << 40); }

// ---- single calls ----
static void arguments() {
  const auto f = [](int i) { return static_cast<float*>(at(i)); };
  const auto rng = static_cast<const int64_t*>(at(20));
  g_ws = reinterpret_cast<uintptr_t>(at(30));
  {
    ge_norm_desc_t d{};
    d.rows = 100; d.d = 64;
    for (int64_t* p : {&d.ldx, &d.ldr, &d.lds, &d.ldy, &d.lddy, &d.ldds, &d.lddx, &d.lddr}) *p = 64;
    d.residual = 1; d.dropout = 0.5f; d.eps = 1e-5f;
    ge_norm_handle_t h = nullptr;
    CHECK(ge_norm_create(&d, &h) == GE_OK);
    size_t bytes = 0;
    CHECK(ge_norm_workspace_size(h, &bytes) == GE_OK);
    g_ws_bytes = bytes;
    ge_norm_args_t a{};
    a.X = at(0); a.residual = at(1); a.S = at(2); a.Y = at(3); a.gain = at(4); a.bias = at(5); a.mean = f(6); a.rstd = f(7); a.rng = rng;
    CHECK(ge_norm_forward(h, &a, nullptr) == GE_OK);
    auto b = a;
#define REFUSED(call, change) b = a; change; CHECK(call(h, &b, nullptr) == GE_ERR_INVALID_ARG)
#define TAKEN(call, change) b = a; change; CHECK(call(h, &b, nullptr) == GE_OK)
    REFUSED(ge_norm_forward, b.X = nullptr);
    REFUSED(ge_norm_forward, b.residual = nullptr);
    REFUSED(ge_norm_forward, b.Y = nullptr);
    REFUSED(ge_norm_forward, b.rng = nullptr);
    REFUSED(ge_norm_forward, b.rng = reinterpret_cast<const int64_t*>((uintptr_t)at(20) + 4));
    REFUSED(ge_norm_forward, b.X = (char*)at(0) + 1);
    REFUSED(ge_norm_forward, b.Y = a.S);
    REFUSED(ge_norm_forward, b.Y = (char*)a.X + 2);           // overlaps, not the same
    REFUSED(ge_norm_forward, b.Y = const_cast<void*>(a.gain));
    REFUSED(ge_norm_forward, b.mean = reinterpret_cast<float*>(at(3)));
    REFUSED(ge_norm_forward, b.rstd = a.mean + 99);
    REFUSED(ge_norm_forward, b.mean = reinterpret_cast<float*>((uintptr_t)at(6) + 2));
    TAKEN(ge_norm_forward, b.S = nullptr; b.mean = b.rstd = nullptr; b.gain = b.bias = nullptr);
    TAKEN(ge_norm_forward, b.S = const_cast<void*>(a.residual); b.Y = const_cast<void*>(a.X));
    a = ge_norm_args_t{};
    a.S = at(0); a.dY = at(1); a.dS = at(2); a.gain = at(4); a.mean = f(6); a.rstd = f(7); a.rng = rng;
    a.dX = at(8); a.dR = at(9); a.dgain = f(10); a.dbias = f(11); a.workspace = at(30); a.workspace_bytes = bytes;
    TAKEN(ge_norm_backward, (void)0);
    REFUSED(ge_norm_backward, b.workspace_bytes = bytes - 1);
    REFUSED(ge_norm_backward, b.workspace = nullptr);
    REFUSED(ge_norm_backward, b.workspace = (char*)at(30) + 8);
    REFUSED(ge_norm_backward, b.workspace = at(8));
    REFUSED(ge_norm_backward, b.mean = nullptr);
    REFUSED(ge_norm_backward, b.dY = nullptr);
    REFUSED(ge_norm_backward, b.S = nullptr);
    REFUSED(ge_norm_backward, b.rng = nullptr);
    REFUSED(ge_norm_backward, b.dX = b.dR);
    REFUSED(ge_norm_backward, b.dX = (char*)b.dR + 64 * 100);
    REFUSED(ge_norm_backward, b.dgain = f(4));
    TAKEN(ge_norm_backward, b.dgain = b.dbias = nullptr; b.workspace = nullptr; b.workspace_bytes = 0);
    TAKEN(ge_norm_backward, b.dX = nullptr; b.rng = nullptr);   // no mask is drawn
    TAKEN(ge_norm_backward, b.dX = const_cast<void*>(a.dY); b.dR = const_cast<void*>(a.dS); b.gain = nullptr);
    const long before = g_launches;
    TAKEN(ge_norm_backward, b.dX = b.dR = nullptr; b.dgain = b.dbias = nullptr);
    CHECK(g_launches == before);                                // nothing to compute
    g_device = 1;
    b = a;
    CHECK(ge_norm_backward(h, &b, nullptr) == GE_ERR_DEVICE);
    g_device = 0;
    ge_norm_destroy(h);
  }
  {
    ge_dropout_desc_t d{};
    d.rows = 100; d.d = 64;
    for (int64_t* p : {&d.ldx, &d.ldr, &d.ldy, &d.lddy, &d.lddx}) *p = 64;
    d.residual = 1; d.p = 0.1f; d.dtype = GE_DT_FP32;
    ge_dropout_handle_t h = nullptr;
    CHECK(ge_dropout_create(&d, &h) == GE_OK);
    ge_dropout_args_t a{}, b;
    a.X = at(0); a.residual = at(1); a.Y = at(2); a.dY = at(3); a.dX = at(4); a.rng = rng;
    TAKEN(ge_dropout_forward, (void)0);
    TAKEN(ge_dropout_forward, b.Y = const_cast<void*>(a.residual));
    TAKEN(ge_dropout_forward, b.Y = const_cast<void*>(a.X));
    TAKEN(ge_dropout_backward, b.dX = const_cast<void*>(a.dY); b.X = b.residual = nullptr; b.Y = nullptr);
    REFUSED(ge_dropout_forward, b.residual = nullptr);
    REFUSED(ge_dropout_forward, b.X = nullptr);
    REFUSED(ge_dropout_forward, b.Y = nullptr);
    REFUSED(ge_dropout_forward, b.rng = nullptr);
    REFUSED(ge_dropout_forward, b.Y = (char*)a.X + 4);
    REFUSED(ge_dropout_forward, b.X = (char*)at(0) + 2);
    REFUSED(ge_dropout_backward, b.dY = nullptr);
    REFUSED(ge_dropout_backward, b.dX = nullptr);
    ge_dropout_destroy(h);
  }
  {
    ge_quant_desc_t d{100, 64, 64, 64, GE_DT_BF16};
    ge_quant_handle_t h = nullptr;
    CHECK(ge_quant_create(&d, &h) == GE_OK);
    ge_quant_args_t a{at(0), static_cast<int8_t*>(at(1)), f(2)}, b;
    TAKEN(ge_quant_run, b.codes += 3);
    REFUSED(ge_quant_run, b.X = nullptr);
    REFUSED(ge_quant_run, b.codes = nullptr);
    REFUSED(ge_quant_run, b.scale = nullptr);
    REFUSED(ge_quant_run, b.scale = reinterpret_cast<float*>((uintptr_t)at(2) + 2));
    REFUSED(ge_quant_run, b.codes = static_cast<int8_t*>(at(0)));
    REFUSED(ge_quant_run, b.scale = reinterpret_cast<float*>(at(1)));
    ge_quant_destroy(h);
  }
  for (int tile : {0, 1, 2, 3}) {
    ge_i8_desc_t d{};
    d.M = 40; d.N = 64; d.K = 4096; d.ldx = d.ldw = 4096; d.ldy = d.ldr = 64; d.bias = d.residual = 1; d.tile = tile;
    ge_i8_handle_t h = nullptr;
    CHECK(ge_i8_create(&d, &h) == GE_OK);
    size_t bytes = 0;
    CHECK(ge_i8_workspace_size(h, &bytes) == GE_OK && (bytes > 0) == (tile == 0));     // (40 rows of one tile: split)
    g_ws_bytes = bytes;
    ge_i8_args_t a{}, b;
    a.X = static_cast<int8_t*>(at(0)); a.W = static_cast<int8_t*>(at(1)); a.x_scale = f(2); a.w_scale = f(3); a.bias = at(4);
    a.residual = at(5); a.Y = at(6); a.workspace = at(30); a.workspace_bytes = bytes;
    TAKEN(ge_i8_run, (void)0);
    TAKEN(ge_i8_run, b.Y = const_cast<void*>(a.residual));
    TAKEN(ge_i8_run, b.x_scale = f(2) + 1; b.w_scale = f(3) + 3);
    REFUSED(ge_i8_run, b.X = nullptr);
    REFUSED(ge_i8_run, b.W += 8);
    REFUSED(ge_i8_run, b.x_scale = nullptr);
    REFUSED(ge_i8_run, b.w_scale = reinterpret_cast<float*>((uintptr_t)at(3) + 1));
    REFUSED(ge_i8_run, b.bias = nullptr);
    REFUSED(ge_i8_run, b.bias = (char*)at(4) + 8);
    REFUSED(ge_i8_run, b.residual = nullptr);
    REFUSED(ge_i8_run, b.Y = nullptr);
    REFUSED(ge_i8_run, b.Y = (char*)at(6) + 8);
    REFUSED(ge_i8_run, b.Y = (char*)at(5) + 16);
    REFUSED(ge_i8_run, b.Y = at(0));
    if (bytes > 0) {
      REFUSED(ge_i8_run, b.workspace = nullptr);
      REFUSED(ge_i8_run, b.workspace_bytes = bytes - 1);
      REFUSED(ge_i8_run, b.workspace = at(6));
    }
    ge_i8_destroy(h);
  }
}

int main(int argc, char** argv) {
  arguments();
  std::mt19937_64 rng(argc > 1 ? std::strtoull(argv[1], nullptr, 10) : 1);
  const long turns = argc > 2 ? std::strtol(argv[2], nullptr, 10) : 10000;
  auto pick = [&](std::initializer_list<int64_t> v) { return *(v.begin() + rng() % v.size()); };
  auto size = [&]() -> int64_t {
    return rng() % 4 == 0 ? pick({-1, 0, 1, 7, 8, 16, 17, 64, 256, 32768, 32769, int64_t(1) << 20, (int64_t(1) << 31) - 1024, int64_t(1) << 40,
                                  (int64_t(1) << 62) + 5, INT64_MAX})
                          : (int64_t)(rng() % (rng() % 2 ? 300 : 20000));
  };
  auto many = [&](int64_t v, int64_t of) { return rng() % 8 ? (v > 0 ? v / of * of : v) : v; };
  auto ld = [&](int64_t n) { return n > (int64_t(1) << 61) ? n : n + pick({0, 0, 0, 0, 16, 64, 8, -8, 5, int64_t(1) << 22}); };
  auto p_of = [&]() -> float {
    const float v[] = {0.0f, 0.1f, 0.5f, 1e-6f, 0.99999f, 1.0f, -0.1f, NAN};
    return v[rng() % 8];
  };
  long ok = 0;
  for (long it = 0; it < turns; ++it) {
    uintptr_t next = uintptr_t(1) << 40;
    auto fake = [&]() -> void* { next += uintptr_t(1) << 45; return rng() % 64 ? reinterpret_cast<void*>(next) : nullptr; };
    auto workspace = [&](size_t bytes) {
      next += uintptr_t(1) << 45;
      g_ws = next;
      g_ws_bytes = bytes;
      return reinterpret_cast<void*>(next);
    };
    auto good = [&](ge_status_t st) {
      CHECK(st == GE_OK || st == GE_ERR_INVALID_ARG || st == GE_ERR_UNSUPPORTED || st == GE_ERR_DEVICE);
      ok += st == GE_OK;
    };
    g_device = 0;
    {
      ge_norm_desc_t d{};
      d.rows = size(); d.d = size(); d.dtype = (int32_t)pick({0, 2, 0, 2, 1, 5}); d.residual = (int32_t)pick({0, 1, 1, 2});
      d.site = (uint32_t)rng(); d.dropout = p_of(); d.eps = rng() % 16 ? 1e-5f : -1.0f;
      for (int64_t* p : {&d.ldx, &d.ldr, &d.lds, &d.ldy, &d.lddy, &d.ldds, &d.lddx, &d.lddr}) *p = rng() % 16 ? d.d : ld(d.d);
      ge_norm_handle_t h = nullptr;
      const ge_status_t st = ge_norm_validate(&d);
      CHECK(ge_norm_create(&d, &h) == st && (h != nullptr) == (st == GE_OK));
      if (h) {
        size_t bytes = 0;
        CHECK(ge_norm_workspace_size(h, &bytes) == GE_OK);
        ge_norm_args_t a{};
        a.X = fake(); a.residual = fake(); a.S = fake(); a.Y = fake(); a.gain = fake(); a.bias = fake(); a.mean = (float*)fake();
        a.rstd = (float*)fake(); a.rng = (const int64_t*)fake(); a.dY = fake(); a.dS = fake(); a.dX = fake(); a.dR = fake();
        a.dgain = (float*)fake(); a.dbias = (float*)fake(); a.workspace = workspace(bytes);
        a.workspace_bytes = rng() % 16 ? bytes : bytes / 2;
        if (rng() % 16 == 0) a.Y = const_cast<void*>(a.X);
        g_device = rng() % 32 ? 0 : 1;
        good(ge_norm_forward(h, &a, nullptr));
        good(ge_norm_backward(h, &a, nullptr));
        g_device = 0;
        ge_norm_destroy(h);
      }
    }
    {
      ge_dropout_desc_t d{};
      d.rows = size(); d.d = size(); d.dtype = (int32_t)pick({0, 2, 0, 2, 1, 5}); d.residual = (int32_t)pick({0, 1, 1, 2}); d.p = p_of();
      for (int64_t* p : {&d.ldx, &d.ldr, &d.ldy, &d.lddy, &d.lddx}) *p = rng() % 16 ? d.d : ld(d.d);
      ge_dropout_handle_t h = nullptr;
      const ge_status_t st = ge_dropout_validate(&d);
      CHECK(ge_dropout_create(&d, &h) == st && (h != nullptr) == (st == GE_OK));
      if (h) {
        ge_dropout_args_t a{};
        a.X = fake(); a.residual = fake(); a.Y = fake(); a.dY = fake(); a.dX = fake(); a.rng = (const int64_t*)fake();
        good(ge_dropout_forward(h, &a, nullptr));
        good(ge_dropout_backward(h, &a, nullptr));
        ge_dropout_destroy(h);
      }
    }
    {
      ge_quant_desc_t d{};
      d.rows = size(); d.d = size(); d.dtype = (int32_t)pick({0, 2, 0, 2, 1, 5}); d.ldx = ld(d.d); d.ldq = ld(d.d);
      ge_quant_handle_t h = nullptr;
      const ge_status_t st = ge_quant_validate(&d);
      CHECK(ge_quant_create(&d, &h) == st && (h != nullptr) == (st == GE_OK));
      if (h) {
        ge_quant_args_t a{fake(), (int8_t*)fake(), (float*)fake()};
        good(ge_quant_run(h, &a, nullptr));
        ge_quant_destroy(h);
      }
    }
    {
      ge_i8_desc_t d{};
      d.M = size(); d.N = many(size(), 8); d.K = many(size(), 16); d.act = (int32_t)pick({0, 1, 2, 3, 3, 3, 4, -1});
      d.bias = (int32_t)(rng() % 2); d.residual = (int32_t)(rng() % 2); d.dtype = (int32_t)pick({0, 2, 0, 2, 1, 5});
      d.tile = (int32_t)pick({0, 0, 0, 0, 1, 2, 3, 4});
      d.ldx = ld(d.K); d.ldw = ld(d.K); d.ldy = ld(d.N); d.ldr = ld(d.N);
      ge_i8_handle_t h = nullptr;
      const ge_status_t st = ge_i8_validate(&d);
      CHECK(ge_i8_create(&d, &h) == st && (h != nullptr) == (st == GE_OK));
      if (h) {
        char line[256];
        CHECK(ge_i8_describe(h, line, sizeof line) == GE_OK && ge_i8_describe(h, line, 5) == GE_OK);
        size_t bytes = 0;
        CHECK(ge_i8_workspace_size(h, &bytes) == GE_OK);
        ge_i8_args_t a{};
        a.X = (int8_t*)fake(); a.W = (int8_t*)fake(); a.x_scale = (float*)fake(); a.w_scale = (float*)fake(); a.bias = fake();
        a.residual = fake(); a.Y = fake(); a.workspace = workspace(bytes); a.workspace_bytes = rng() % 16 ? bytes : bytes / 2;
        g_device = rng() % 32 ? 0 : 1;
        good(ge_i8_run(h, &a, nullptr));
        g_device = 0;
        ge_i8_destroy(h);
      }
    }
  }
  std::printf("fuzz ok: %ld calls, %ld launches\n", ok, g_launches);
  return ok > 0 ? 0 : 1;
}
