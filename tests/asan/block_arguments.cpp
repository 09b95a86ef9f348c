// Arguments of the block operators' C-ABI, one call each, on the host under the sanitizers: stand-ins for
// the HIP runtime (a gfx950 that is current) and for the launches, which only count.
#include <hip/hip_runtime.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>

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
namespace ge {
hipError_t launch_ffn_pair(int, int, bool, const FfnLaunch&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_ffn_grad(int, int, bool, const FfnLaunch&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_ffn_plain(int, int, bool, const FfnLaunch&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_ffn_few(bool, int, bool, const FfnFew&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_qk(const QkKind&, const QkParams&, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_qk_gains(const float*, int, int, float*, float*, hipStream_t) { ++g_launches; return hipSuccess; }
hipError_t launch_clip_norm(const ClipTable&, int, int, double*, hipStream_t) { ++g_launches; return hipSuccess; }
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

static void* at(int i) { return reinterpret_cast<void*>((uintptr_t)(i + 1) << 40); }

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

int main() {
  gain_gradients();
  std::printf(g_failed ? "%d wrong\n" : "arguments ok\n", g_failed);
  return g_failed ? 1 : 0;
}
