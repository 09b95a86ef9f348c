// Drives the C-ABI of the transformer-block operators on the host, under the sanitizers: random and
// mutated descriptors through validate, create, workspace_size and the calls, with stand-ins for the HIP
// runtime (one gfx950 that is current) and for the launches.  The launch stand-ins check what the kernels
// rely on: grids the runtime can count, tickets and partial sums inside their part of the workspace,
// intermediate values inside the workspace, chunk tables in order.  Nothing is dereferenced but host arrays.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <random>
#include <vector>

#include "../../gemm_epilogue_transformer_tiled_amd/csrc/ge_block_internal.h"
#include "../../include/ge_block.h"

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

hipError_t check_launch(int tile, const ge::FfnLaunch& l, bool pair) {
  ++g_launches;
  if (l.tiles == 0) return hipSuccess;
  const ge::FfnTileInfo ti = ge::ffn_tile_info(tile);
  const int bn = pair ? ti.bn_pair : ti.bn;
  CHECK(l.splits >= 1 && (tile != ge::FFN_T256 || l.splits == 1));
  CHECK((double)l.tiles * l.splits * (tile == ge::FFN_T64 ? 256 : 512) < 4294967296.0);
  int64_t tiles = 0;
  for (int i = 0; i < l.n; ++i) {
    const ge::FfnProduct& p = l.prod[i];
    CHECK(p.tile0 == tiles && p.tiles_m > 0 && p.tiles_n > 0);
    CHECK((int64_t)p.tiles_m * ti.bm >= p.M && (int64_t)p.tiles_n * bn >= p.N);
    CHECK(p.lda < (1 << 22) && p.ldb < (1 << 22) && p.ldy < (1 << 22));
    tiles += (int64_t)p.tiles_m * p.tiles_n;
  }
  CHECK(tiles == l.tiles);
  if (l.splits > 1) {
    CHECK(in_ws(l.ctr, (size_t)l.tiles * ge::kFfnCtrStride * 4));
    CHECK(reinterpret_cast<uintptr_t>(l.ctr) + (size_t)l.tiles * ge::kFfnCtrStride * 4 <= reinterpret_cast<uintptr_t>(l.part));
    const size_t sums = (size_t)l.tiles * l.splits * ti.bm * bn * (pair ? 8 : 4);
    CHECK(in_ws(l.part, sums));
    for (int i = 0; i < l.n; ++i)         // what lies behind them in the workspace is not reached
      for (const void* q : {(const void*)l.prod[i].A, (const void*)l.prod[i].A2, (const void*)l.prod[i].B,
                            (const void*)l.prod[i].Y, (const void*)l.prod[i].Y2, (const void*)l.prod[i].Y3})
        if (in_ws(q, 0)) CHECK(reinterpret_cast<uintptr_t>(l.part) + sums <= reinterpret_cast<uintptr_t>(q));
  }
  return hipSuccess;
}
}  // namespace

namespace ge {
hipError_t launch_ffn_pair(int tile, int, bool, const FfnLaunch& l, hipStream_t) {
  for (int i = 0; i < l.n; ++i) CHECK(in_ws(l.prod[i].Y, (size_t)l.prod[i].M * l.prod[i].N * 2));
  return check_launch(tile, l, true);
}
hipError_t launch_ffn_grad(int tile, int, bool, const FfnLaunch& l, hipStream_t) {
  for (int i = 0; i < l.n; ++i)
    for (const void* y : {l.prod[i].Y, l.prod[i].Y2, l.prod[i].Y3}) CHECK(in_ws(y, (size_t)l.prod[i].M * l.prod[i].N * 2));
  return check_launch(tile, l, false);
}
hipError_t launch_ffn_plain(int, int tile, bool, const FfnLaunch& l, hipStream_t) { return check_launch(tile, l, false); }
hipError_t launch_ffn_few(bool pair, int, bool, const FfnFew& p, hipStream_t) {
  ++g_launches;
  CHECK(p.M <= kFfnFewRows && (int64_t)p.tiles * kFfnFewCols >= p.N && p.splits >= 1);
  CHECK((double)p.tiles * p.splits * 512 < 4294967296.0);
  if (p.splits > 1) {
    const size_t sums = (size_t)p.tiles * p.splits * (pair ? 2 : 1) * kFfnFewRows * kFfnFewCols * 4;
    CHECK(in_ws(p.ctr, (size_t)p.tiles * kFfnCtrStride * 4) && in_ws(p.part, sums));
    CHECK(reinterpret_cast<uintptr_t>(p.ctr) + (size_t)p.tiles * kFfnCtrStride * 4 <= reinterpret_cast<uintptr_t>(p.part));
    const void* h = pair ? (const void*)p.Y : (const void*)p.A;
    CHECK(reinterpret_cast<uintptr_t>(p.part) + sums <= reinterpret_cast<uintptr_t>(h));
  }
  return hipSuccess;
}
hipError_t launch_qk(const QkKind& k, const QkParams& p, hipStream_t) {
  ++g_launches;
  CHECK(p.group >= 1 && p.group <= 64 && p.group * 8 >= p.head_dim && (p.group & (p.group - 1)) == 0);
  CHECK(p.tokens_per_wg >= 1 && p.tokens_per_wg * (p.rot_dim / 2) <= kQkMaxAngles);
  CHECK(p.workgroups >= 0 && p.workgroups <= (1 << 22));
  CHECK(p.workgroups > 0 || p.tokens == 0 || p.heads[0] + p.heads[1] == 0);
  CHECK(p.head_splits == 1 || (p.tokens_per_wg == 1 && p.turns < (int64_t(1) << 31)));
  if (k.wide)
    for (int w = 0; w < 2; ++w) CHECK(p.xt[w] >= 0 && p.head_dim % 8 == 0 && p.rot_dim % 8 == 0);
  if (k.backward && k.norm) CHECK(in_ws(p.part, (size_t)p.workgroups * 2 * p.head_dim * 4));
  return hipSuccess;
}
hipError_t launch_qk_gains(const float* part, int rows, int head_dim, float*, float*, hipStream_t) {
  CHECK(in_ws(part, (size_t)rows * 2 * head_dim * 4));
  return hipSuccess;
}
static hipError_t check_table(const ClipTable& t, int grid) {
  ++g_launches;
  CHECK(t.n >= 1 && t.n <= kClipTensors && t.chunk0[0] == 0 && grid >= 1 && grid <= kClipPartials);
  for (int i = 0; i < t.n; ++i) {
    CHECK(t.numel[i] > 0 && t.chunk0[i + 1] - t.chunk0[i] == (uint32_t)((t.numel[i] + kClipChunk - 1) / kClipChunk));
    CHECK(t.in[i] != nullptr);
  }
  return hipSuccess;
}
hipError_t launch_clip_norm(const ClipTable& t, int grid, int, double* part, hipStream_t) {
  CHECK(in_ws(part, (size_t)grid * 8));
  return check_table(t, grid);
}
hipError_t launch_clip_finish(const double* part, int n, float*, hipStream_t) {
  CHECK(in_ws(part, (size_t)n * 8));
  return hipSuccess;
}
hipError_t launch_clip_scale(const ClipTable& t, int grid, int, const double* part, int n, float, float, float*, hipStream_t) {
  CHECK(in_ws(part, (size_t)n * 8));
  return check_table(t, grid);
}
}  // namespace ge

int main(int argc, char** argv) {
  std::mt19937_64 rng(argc > 1 ? std::strtoull(argv[1], nullptr, 10) : 1);
  const long turns = argc > 2 ? std::strtol(argv[2], nullptr, 10) : 10000;
  auto pick = [&](std::initializer_list<int64_t> v) { return *(v.begin() + rng() % v.size()); };
  auto size = [&]() -> int64_t {
    return rng() % 4 == 0 ? pick({-1, 0, 1, 7, 8, 16, 17, 64, 256, int64_t(1) << 20, (int64_t(1) << 31) - 1024, int64_t(1) << 40})
                          : (int64_t)(rng() % (rng() % 2 ? 300 : 20000));
  };
  auto eight = [&](int64_t v) { return rng() % 8 ? (v > 0 ? v / 8 * 8 : v) : v; };
  long ok = 0;
  for (long it = 0; it < turns; ++it) {
    // distinct fake allocations, far apart
    uintptr_t next = uintptr_t(1) << 40;
    auto fake = [&]() -> void* { next += uintptr_t(1) << 44; return rng() % 64 ? reinterpret_cast<void*>(next) : nullptr; };
    {
      ge_ffn_desc_t d{};
      d.M = size(); d.d = eight(size()); d.h = eight(size());
      d.act = (int32_t)pick({0, 1, 2, 3, 3, 3, 4, -1}); d.w_layout = (int32_t)pick({0, 1, 0, 1, 2});
      d.residual = (int32_t)(rng() % 2); d.save = (int32_t)(rng() % 2); d.tile = (int32_t)pick({0, 0, 0, 0, 1, 2, 3, 4});
      const int64_t wi = d.w_layout == 0 ? d.h : d.d, wo = d.w_layout == 0 ? d.d : d.h;
      auto ld = [&](int64_t n) { return n + pick({0, 0, 0, 8, 64, -8, 4}); };
      d.ldx = ld(d.d); d.ldy = ld(d.d); d.ldr = ld(d.d); d.ldg = ld(d.h); d.lddy = ld(d.d); d.lddx = ld(d.d);
      d.ldw = ld(wi); d.ldwd = ld(wo); d.lddw = ld(wi); d.lddwd = ld(wo);
      ge_ffn_handle_t h = nullptr;
      const ge_status_t st = ge_ffn_validate(&d);
      CHECK(st == GE_OK || st == GE_ERR_INVALID_ARG || st == GE_ERR_UNSUPPORTED);
      CHECK(ge_ffn_create(&d, &h) == st && (h != nullptr) == (st == GE_OK));
      if (h) {
        char line[256];
        CHECK(ge_ffn_describe(h, line, sizeof line) == GE_OK && ge_ffn_describe(h, line, 5) == GE_OK);
        for (int backward = 0; backward < 2; ++backward) {
          size_t bytes = 0;
          CHECK(ge_ffn_workspace_size(h, backward, &bytes) == GE_OK);
          ge_ffn_args_t a{};
          a.X = fake(); a.Wg = fake(); a.Wu = fake(); a.Wd = fake(); a.residual = fake(); a.Y = fake(); a.G = fake(); a.U = fake();
          a.dY = fake(); a.dX = fake(); a.dWg = fake(); a.dWu = fake(); a.dWd = fake();
          next += uintptr_t(1) << 44;
          g_ws = next; g_ws_bytes = bytes;
          next += uintptr_t(1) << 46;
          a.workspace = reinterpret_cast<void*>(g_ws);
          a.workspace_bytes = rng() % 16 ? bytes : bytes / 2;
          if (rng() % 16 == 0) a.Y = const_cast<void*>(a.X);
          g_device = rng() % 32 ? 0 : 1;
          const ge_status_t run = backward ? ge_ffn_backward(h, &a, nullptr) : ge_ffn_forward(h, &a, nullptr);
          CHECK(run == GE_OK || run == GE_ERR_INVALID_ARG || run == GE_ERR_DEVICE || run == GE_ERR_UNSUPPORTED);
          ok += run == GE_OK;
          g_device = 0;
        }
        ge_ffn_destroy(h);
      }
    }
    {
      ge_qk_desc_t d{};
      d.tokens = size(); d.heads_q = size() % 70; d.heads_k = size() % 20;
      d.head_dim = (int32_t)pick({2, 8, 20, 64, 80, 128, 256, 512, 514, 7, 0});
      d.rot_dim = (int32_t)(rng() % 3 ? d.head_dim : rng() % (d.head_dim + 2));
      d.pairs = (int32_t)(rng() % 2); d.norm = (int32_t)(rng() % 2); d.dtype = (int32_t)pick({0, 2, 0, 2, 1, 5});
      d.pos64 = (int32_t)(rng() % 2); d.eps = 1e-6f;
      int64_t* s[] = {&d.q_token, &d.k_token, &d.oq_token, &d.ok_token, &d.dq_token, &d.dk_token};
      int64_t* hs[] = {&d.q_head, &d.k_head, &d.oq_head, &d.ok_head, &d.dq_head, &d.dk_head};
      for (int i = 0; i < 6; ++i) {
        const int64_t heads = i % 2 ? d.heads_k : d.heads_q;
        *hs[i] = d.head_dim + pick({0, 0, 0, 8, -1});
        *s[i] = (heads > 0 ? heads : 1) * *hs[i] + pick({0, 0, 0, 8, 1, -4});
        if (rng() % 8 == 0) { *s[i] = *hs[i]; *hs[i] = *s[i] * (d.tokens > 0 ? d.tokens : 1); }
        if (rng() % 16 == 0 && i < 2) *s[i] = *hs[i] = 0;
      }
      ge_qk_handle_t h = nullptr;
      const ge_status_t st = ge_qk_validate(&d);
      CHECK(ge_qk_create(&d, &h) == st);
      if (h) {
        size_t bytes = 0;
        CHECK(ge_qk_workspace_size(h, &bytes) == GE_OK);
        ge_qk_args_t a{};
        a.q = fake(); a.k = fake(); a.q_out = fake(); a.k_out = fake(); a.positions = fake(); a.inv_freq = (const float*)fake();
        a.gain_q = fake(); a.gain_k = fake(); a.dq_out = fake(); a.dk_out = fake(); a.dq = fake(); a.dk = fake();
        a.dgain_q = (float*)fake(); a.dgain_k = (float*)fake(); a.amplitude = 1.0f;
        if (rng() % 8 == 0) a.q_out = const_cast<void*>(a.q);
        next += uintptr_t(1) << 44;
        g_ws = next; g_ws_bytes = bytes;
        a.workspace = reinterpret_cast<void*>(g_ws); a.workspace_bytes = bytes;
        for (ge_status_t run : {ge_qk_forward(h, &a, nullptr), ge_qk_backward(h, &a, nullptr)}) {
          CHECK(run == GE_OK || run == GE_ERR_INVALID_ARG);
          ok += run == GE_OK;
        }
        ge_qk_destroy(h);
      }
    }
    if (it % 8 == 0) {
      const int n = (int)(rng() % (rng() % 8 ? 40 : 700));
      std::vector<ge_clip_tensor_t> t(n);
      std::vector<const void*> in(n);
      std::vector<void*> out(n);
      for (int i = 0; i < n; ++i) {
        t[i].numel = (int64_t)(rng() % 4 ? rng() % 100000 : rng() % 3);
        t[i].dtype = (int32_t)pick({0, 2});
        next += uintptr_t(1) << 24;
        in[i] = reinterpret_cast<void*>(next + (t[i].dtype ? 4 : 2) * (rng() % 8));
        next += uintptr_t(1) << 24;
        out[i] = rng() % 3 ? reinterpret_cast<void*>(next) : const_cast<void*>(in[i]);
      }
      ge_clip_handle_t h = nullptr;
      CHECK(ge_clip_create(t.data(), n, &h) == GE_OK);
      size_t bytes = 0;
      CHECK(ge_clip_workspace_size(h, &bytes) == GE_OK);
      ge_clip_args_t a{};
      a.in = in.data(); a.out = rng() % 4 ? out.data() : nullptr;
      next += uintptr_t(1) << 40;
      a.norm = reinterpret_cast<float*>(next);
      next += uintptr_t(1) << 40;
      g_ws = next; g_ws_bytes = bytes;
      a.workspace = reinterpret_cast<void*>(g_ws); a.workspace_bytes = bytes; a.max_norm = 1.0f; a.eps = 1e-6f;
      CHECK(ge_clip_run(h, &a, nullptr) == GE_OK);
      ++ok;
      int at = -1;
      for (int i = 0; i < n; ++i)
        if (t[i].numel > 0) at = i;
      if (at >= 0 && a.out) {                 // an output over another input
        out[at] = a.norm;
        CHECK(ge_clip_run(h, &a, nullptr) == GE_ERR_INVALID_ARG);
      }
      ge_clip_destroy(h);
    }
  }
  std::printf("fuzz ok: %ld calls, %ld launches\n", ok, g_launches);
  return ok > 0 ? 0 : 1;
}
