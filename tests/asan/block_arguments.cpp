// Arguments of the block operators' C-ABI, one call each, on the host under the sanitizers: stand-ins for
// the HIP runtime (a gfx950 that is current) and for the launches, which only count.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <vector>

#include "../../gemm_epilogue_transformer_tiled_amd/csrc/ge_block_internal.h"
#include "../../include/ge_block.h"

extern "C" hipError_t hipGetDevice(int* d) { *d = 0; return hipSuccess; }
#undef hipGetDeviceProperties
extern "C" hipError_t hipGetDeviceProperties(hipDeviceProp_t* p, int) {
  std::memset(p, 0, sizeof *p);
  std::strcpy(p->gcnArchName, "gfx950:sramecc+:xnack-");
  return hipSuccess;
}
extern "C" hipError_t hipGetDevicePropertiesR0600(hipDeviceProp_t* p, int d) { return hipGetDeviceProperties(p, d); }
extern "C" hipError_t hipGetLastError(void) { return hipSuccess; }

static int g_launches = 0;
static void* at(int i) { return reinterpret_cast<void*>((uintptr_t)(i + 1) << 40); }
// What the launches use of the workspace, which lies at at(30): tickets, and everything else.
struct Use { int64_t lo, hi; };
static std::vector<Use> g_tickets, g_data;
static void use(std::vector<Use>& v, const void* p, size_t bytes) {
  const int64_t lo = (int64_t)(reinterpret_cast<uintptr_t>(p) - reinterpret_cast<uintptr_t>(at(30)));
  if (lo >= 0 && lo < (int64_t(1) << 40) && bytes > 0) v.push_back(Use{lo, lo + (int64_t)bytes});
}
static hipError_t product(int tile, const ge::FfnLaunch& l, bool pair) {
  ++g_launches;
  const ge::FfnTileInfo ti = ge::ffn_tile_info(tile);
  if (l.splits > 1) {
    use(g_tickets, l.ctr, (size_t)l.tiles * ge::kFfnCtrStride * 4);
    use(g_data, l.part, (size_t)l.tiles * l.splits * ti.bm * (pair ? ti.bn_pair * 2 : ti.bn) * 4);
  }
  for (int i = 0; i < l.n; ++i)
    for (const void* y : {l.prod[i].Y, l.prod[i].Y2, l.prod[i].Y3}) use(g_data, y, (size_t)l.prod[i].M * l.prod[i].N * 2);
  return hipSuccess;
}
namespace ge {
hipError_t launch_ffn_pair(int tile, int, bool, const FfnLaunch& l, hipStream_t) { return product(tile, l, true); }
hipError_t launch_ffn_grad(int tile, int, bool, const FfnLaunch& l, hipStream_t) { return product(tile, l, false); }
hipError_t launch_ffn_plain(int, int tile, bool, const FfnLaunch& l, hipStream_t) { return product(tile, l, false); }
hipError_t launch_ffn_few(bool pair, int, bool, const FfnFew& p, hipStream_t) {
  ++g_launches;
  if (p.splits > 1) {
    use(g_tickets, p.ctr, (size_t)p.tiles * kFfnCtrStride * 4);
    use(g_data, p.part, (size_t)p.tiles * p.splits * (pair ? 2 : 1) * kFfnFewRows * kFfnFewCols * 4);
  }
  use(g_data, p.Y, (size_t)p.M * p.N * 2);
  return hipSuccess;
}
hipError_t launch_qk(const QkKind& k, const QkParams& p, hipStream_t) {
  ++g_launches;
  if (k.backward && k.norm) use(g_data, p.part, (size_t)p.workgroups * 2 * p.head_dim * 4);
  return hipSuccess;
}
hipError_t launch_qk_gains(const float*, int, int, float*, float*, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_clip_norm(const ClipTable&, int grid, int, double* part, hipStream_t) {
  ++g_launches;
  use(g_data, part, (size_t)grid * 8);
  return hipSuccess;
}
hipError_t launch_clip_finish(const double*, int, float*, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_clip_scale(const ClipTable&, int, int, const double*, int, float, float, float*, hipStream_t) {
  ++g_launches;
  return hipSuccess;
}
}  // namespace ge

static int g_failed = 0;
#define EXPECT(call, want)                                                                     \
  do {                                                                                         \
    const int got = (call);                                                                    \
    if (got != (want)) {                                                                       \
      std::printf("line %d: %s is %d, not %d\n", __LINE__, #call, got, (int)(want));           \
      ++g_failed;                                                                              \
    }                                                                                          \
  } while (0)

// The gain gradients of a side that has heads are asked for, those of one without are not.
static void gain_gradients() {
  for (int side = 0; side < 2; ++side) {
    const int64_t hq = side ? 0 : 2, hk = side ? 2 : 0, D = 64, T = 10;
    ge_qk_desc_t d{};
    d.tokens = T; d.heads_q = hq; d.heads_k = hk;
    for (int64_t* s : {&d.q_head, &d.k_head, &d.oq_head, &d.ok_head, &d.dq_head, &d.dk_head}) *s = D;
    for (int64_t* s : {&d.q_token, &d.k_token, &d.oq_token, &d.ok_token, &d.dq_token, &d.dk_token}) *s = 2 * D;
    d.head_dim = D; d.rot_dim = D; d.pairs = GE_PAIRS_HALF; d.norm = 1; d.dtype = GE_DT_BF16; d.pos64 = 1; d.eps = 1e-6f;
    ge_qk_handle_t h = nullptr;
    EXPECT(ge_qk_create(&d, &h), GE_OK);
    size_t bytes = 0;
    EXPECT(ge_qk_workspace_size(h, &bytes), GE_OK);
    ge_qk_args_t a{};
    a.q = at(0); a.k = at(1); a.positions = at(2); a.inv_freq = (const float*)at(3); a.gain_q = at(4); a.gain_k = at(5);
    a.dq_out = at(6); a.dk_out = at(7); a.dq = at(8); a.dk = at(9); a.workspace = at(10); a.workspace_bytes = bytes;
    a.amplitude = 1.0f;
    g_launches = 0;
    EXPECT(ge_qk_backward(h, &a, nullptr), GE_ERR_INVALID_ARG);          // both missing
    (side ? a.dgain_q : a.dgain_k) = (float*)at(11);
    EXPECT(ge_qk_backward(h, &a, nullptr), GE_ERR_INVALID_ARG);          // the one that is needed is missing
    EXPECT(g_launches, 0);
    a.dgain_q = a.dgain_k = nullptr;
    (side ? a.dgain_k : a.dgain_q) = (float*)at(11);
    EXPECT(ge_qk_backward(h, &a, nullptr), GE_OK);
    EXPECT(g_launches, 2);
    a.dgain_q = a.dgain_k = (float*)at(11);                              // one place for two results
    EXPECT(ge_qk_backward(h, &a, nullptr), GE_ERR_INVALID_ARG);
    ge_qk_destroy(h);
  }
}

// One workspace of the largest size, calls of several handles in turn: nothing but tickets is left where any
// of them has tickets.
static void shared_workspace() {
  g_tickets.clear();
  g_data.clear();
  int overlaps = 0;
  for (int64_t M : {1, 16, 27, 64, 333, 777, 4100})
    for (int64_t d : {64, 264, 1032, 4096})
      for (int64_t h : {136, 2856, 11008, 131072}) {
        ge_ffn_desc_t f{};
        f.M = M; f.d = d; f.h = h; f.act = GE_ACT_SILU; f.w_layout = GE_LAYOUT_KN;
        f.ldx = f.ldy = f.ldr = f.lddy = f.lddx = f.ldwd = f.lddwd = d;
        f.ldg = f.ldw = f.lddw = h;
        ge_ffn_handle_t p = nullptr;
        EXPECT(ge_ffn_create(&f, &p), GE_OK);
        size_t forward = 0, backward = 0;
        EXPECT(ge_ffn_workspace_size(p, 0, &forward), GE_OK);
        EXPECT(ge_ffn_workspace_size(p, 1, &backward), GE_OK);
        ge_ffn_args_t a{};
        a.X = at(0); a.Wg = at(1); a.Wu = at(2); a.Wd = at(3); a.Y = at(4); a.G = at(5); a.U = at(6); a.dY = at(7);
        a.dX = at(8); a.dWg = at(9); a.dWu = at(10); a.dWd = at(11);
        a.workspace = at(30);
        a.workspace_bytes = forward;
        EXPECT(ge_ffn_forward(p, &a, nullptr), GE_OK);
        a.workspace_bytes = backward;
        EXPECT(ge_ffn_backward(p, &a, nullptr), GE_OK);
        ge_ffn_destroy(p);
      }
  for (int64_t T : {1, 100, 20000}) {
    ge_qk_desc_t d{};
    d.tokens = T; d.heads_q = 4; d.heads_k = 2;
    for (int64_t* s : {&d.q_head, &d.k_head, &d.oq_head, &d.ok_head, &d.dq_head, &d.dk_head}) *s = 64;
    for (int64_t* s : {&d.q_token, &d.k_token, &d.oq_token, &d.ok_token, &d.dq_token, &d.dk_token}) *s = 256;
    d.head_dim = 64; d.rot_dim = 64; d.pairs = GE_PAIRS_HALF; d.norm = 1; d.dtype = GE_DT_BF16; d.pos64 = 1;
    ge_qk_handle_t h = nullptr;
    EXPECT(ge_qk_create(&d, &h), GE_OK);
    ge_qk_args_t a{};
    a.q = at(0); a.k = at(1); a.positions = at(2); a.inv_freq = (const float*)at(3); a.gain_q = at(4); a.gain_k = at(5);
    a.dq_out = at(6); a.dk_out = at(7); a.dq = at(8); a.dk = at(9); a.dgain_q = (float*)at(10); a.dgain_k = (float*)at(11);
    a.workspace = at(30); a.amplitude = 1.0f;
    EXPECT(ge_qk_workspace_size(h, &a.workspace_bytes), GE_OK);
    EXPECT(ge_qk_backward(h, &a, nullptr), GE_OK);
    ge_qk_destroy(h);
  }
  {
    ge_clip_tensor_t t[2] = {{1000, GE_DT_BF16}, {50000000, GE_DT_FP32}};
    const void* in[2] = {at(0), at(1)};
    void* out[2] = {at(2), at(3)};
    ge_clip_handle_t h = nullptr;
    EXPECT(ge_clip_create(t, 2, &h), GE_OK);
    ge_clip_args_t a{};
    a.in = in; a.out = out; a.norm = (float*)at(4); a.workspace = at(30); a.max_norm = 1.0f; a.eps = 1e-6f;
    EXPECT(ge_clip_workspace_size(h, &a.workspace_bytes), GE_OK);
    EXPECT(ge_clip_run(h, &a, nullptr), GE_OK);
    ge_clip_destroy(h);
  }
  for (const Use& t : g_tickets)
    for (const Use& d : g_data) overlaps += t.lo < d.hi && d.lo < t.hi;
  EXPECT(overlaps, 0);
  EXPECT((int)(g_tickets.size() > 20 && g_data.size() > 100), 1);
}

int main() {
  gain_gradients();
  shared_workspace();
  std::printf(g_failed ? "%d wrong\n" : "arguments ok\n", g_failed);
  return g_failed ? 1 : 0;
}
