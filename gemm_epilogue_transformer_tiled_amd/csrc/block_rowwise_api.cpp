// C-ABI of the query/key norm with rotation and of gradient clipping (include/ge_block.h).
// Host code only; the handles hold host memory only.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "../../include/ge_block.h"
#include "block_host.h"
#include "ge_block_internal.h"

using ge::block::aligned;
using ge::block::ceil_div;
using ge::block::Matrix;

// ---------------------------------------------------------------------------------------------
// query/key norm with rotation
// ---------------------------------------------------------------------------------------------
struct ge_qk_plan {
  ge_qk_desc_t desc;
  int device;
  int group, tokens_per_wg, head_splits, q_splits, grid_forward, grid_backward;
  int64_t turns;
};

namespace {

constexpr int kMostTokens = 16;          // of one turn
static_assert(ge::kQkMaxAngles >= ge::kQkThreads, "a turn's angles: about one a thread, or one token's (up to 256)");
constexpr int64_t kMaxTokens = int64_t(1) << 40, kMaxHeads = int64_t(1) << 20, kMaxStride = int64_t(1) << 40;

// Heads of tokens as rows of elements: the larger stride separates rows.  Exact for the layouts
// that keep heads of a token (or tokens of a head) together.
Matrix as_matrix(const void* p, int64_t tokens, int64_t heads, int64_t st, int64_t sh, int64_t d, int64_t size) {
  if (tokens == 0 || heads == 0) return Matrix{p, 0, 0, 0, size};
  if (tokens == 1) st = 0;
  if (heads == 1) sh = 0;
  if (st >= sh) return Matrix{p, tokens, (heads - 1) * sh + d, st, size};
  return Matrix{p, heads, (tokens - 1) * st + d, sh, size};
}

// At most `most` workgroups, fewer where that gives each the same number of turns.
int64_t even_grid(int64_t turns, int64_t most) { return turns > 0 ? ceil_div(turns, ceil_div(turns, most)) : 0; }

// Whether the strides of an output keep its heads apart.
bool apart(int64_t tokens, int64_t heads, int64_t st, int64_t sh, int64_t d) {
  if (tokens == 0 || heads == 0 || (tokens == 1 && heads == 1)) return true;
  if (tokens <= 1) return sh >= d;
  if (heads <= 1) return st >= d;
  const int64_t lo = std::min(st, sh), hi = std::max(st, sh), n_lo = st <= sh ? tokens : heads;
  return lo >= d && hi >= (n_lo - 1) * lo + d;
}

bool wide(const ge_qk_desc_t& d, const void* const* ptrs, int n_ptrs, const int64_t* strides, int n_strides) {
  if (d.head_dim % 8 || d.rot_dim % 8) return false;
  for (int i = 0; i < n_ptrs; ++i)
    if (!aligned(ptrs[i], 16)) return false;
  // offsets within a turn's tokens: 24-bit factors, 31-bit byte offsets
  for (int i = 0; i < n_strides; i += 2) {
    if (strides[i] % 8 || strides[i + 1] % 8 || strides[i] >= (1 << 24) || strides[i + 1] >= (1 << 24)) return false;
    if (strides[i] * kMostTokens + strides[i + 1] * std::max(d.heads_q, d.heads_k) >= (int64_t(1) << 28)) return false;
  }
  return true;
}

// [tickets' room, unused][partial gain gradients]
size_t gain_bytes(const ge_qk_plan* h) {
  return h->desc.norm ? ge::kTicketBytes + (size_t)std::max(h->grid_backward, 1) * 2 * (size_t)h->desc.head_dim * 4 : 0;
}

struct Side {           // q or k
  const void* x;
  void* y;
  const void* dy;
  int64_t heads, xt, xh, yt, yh, dt, dh;
};

// Fills the launch parameters and checks pointers and overlaps; false: invalid.
bool fill(const ge_qk_plan* h, const ge_qk_args_t* a, bool backward, ge::QkParams& p, ge::QkKind& kind) {
  const ge_qk_desc_t& d = h->desc;
  const int64_t size = d.dtype == GE_DT_BF16 ? 2 : 4;
  const bool need_x = !backward || d.norm;
  const Side sides[2] = {
      {a->q, backward ? a->dq : a->q_out, a->dq_out, d.heads_q, d.q_token, d.q_head, backward ? d.dq_token : d.oq_token,
       backward ? d.dq_head : d.oq_head, d.oq_token, d.oq_head},
      {a->k, backward ? a->dk : a->k_out, a->dk_out, d.heads_k, d.k_token, d.k_head, backward ? d.dk_token : d.ok_token,
       backward ? d.dk_head : d.ok_head, d.ok_token, d.ok_head}};
  Matrix in[8], out[6];
  int n_in = 0, n_out = 0;
  const void* ptrs[6];
  int64_t strides[12];
  int n_ptrs = 0, n_strides = 0;
  // which output may be which input, element for element: the same pointer and strides
  bool same[6][8] = {};
  for (int w = 0; w < 2; ++w) {
    const Side& s = sides[w];
    p.heads[w] = (int32_t)s.heads;
    p.x[w] = s.x; p.y[w] = s.y; p.dy[w] = s.dy;
    p.xt[w] = s.xt; p.xh[w] = s.xh; p.yt[w] = s.yt; p.yh[w] = s.yh; p.dt[w] = s.dt; p.dh[w] = s.dh;
    if (s.heads == 0 || d.tokens == 0) continue;
    if (!s.y || !aligned(s.y, size)) return false;
    const int o = n_out++;
    out[o] = as_matrix(s.y, d.tokens, s.heads, s.yt, s.yh, d.head_dim, size);
    ptrs[n_ptrs++] = s.y; strides[n_strides++] = s.yt; strides[n_strides++] = s.yh;
    if (need_x) {
      if (!s.x || !aligned(s.x, size)) return false;
      same[o][n_in] = s.x == s.y && s.xt == s.yt && s.xh == s.yh;
      in[n_in++] = as_matrix(s.x, d.tokens, s.heads, s.xt, s.xh, d.head_dim, size);
      ptrs[n_ptrs++] = s.x; strides[n_strides++] = s.xt; strides[n_strides++] = s.xh;
    }
    if (backward) {
      if (!s.dy || !aligned(s.dy, size)) return false;
      same[o][n_in] = s.dy == s.y && s.dt == s.yt && s.dh == s.yh;
      in[n_in++] = as_matrix(s.dy, d.tokens, s.heads, s.dt, s.dh, d.head_dim, size);
      ptrs[n_ptrs++] = s.dy; strides[n_strides++] = s.dt; strides[n_strides++] = s.dh;
    }
    if (d.norm) {
      const void* gain = w ? a->gain_k : a->gain_q;
      if (!gain || !aligned(gain, size)) return false;
      in[n_in++] = Matrix{gain, 1, d.head_dim, d.head_dim, size};
      p.gain[w] = gain;
    }
  }
  if (d.tokens > 0 && d.rot_dim > 0 && n_out > 0) {
    const int64_t ps = d.pos64 ? 8 : 4;
    if (!a->positions || !aligned(a->positions, ps) || !a->inv_freq || !aligned(a->inv_freq, 4)) return false;
    in[n_in++] = Matrix{a->positions, 1, d.tokens, d.tokens, ps};
    in[n_in++] = Matrix{a->inv_freq, 1, d.rot_dim / 2, d.rot_dim / 2, 4};
  }
  if (backward && d.norm) {
    float* const dgain[2] = {a->dgain_q, a->dgain_k};
    for (int w = 0; w < 2; ++w) {
      float* const g = dgain[w];
      if (!g && sides[w].heads > 0) return false;
      if (!g) continue;
      if (!aligned(g, 4)) return false;
      out[n_out++] = Matrix{g, 1, d.head_dim, d.head_dim, 4};
    }
    if (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < gain_bytes(h)) return false;
    out[n_out++] = Matrix{a->workspace, 1, (int64_t)gain_bytes(h), (int64_t)gain_bytes(h), 1};
  }
  if (!std::isfinite(a->amplitude)) return false;
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (!same[o][i] && ge::block::overlap(out[o], in[i])) return false;
    for (int q = 0; q < o; ++q)
      if (ge::block::overlap(out[o], out[q])) return false;
  }
  p.positions = a->positions;
  p.inv_freq = a->inv_freq;
  if (backward && d.norm) p.part = reinterpret_cast<float*>(static_cast<unsigned char*>(a->workspace) + ge::kTicketBytes);
  p.tokens = d.tokens;
  p.turns = h->turns;
  p.head_dim = d.head_dim;
  p.rot_dim = d.rot_dim;
  p.group = h->group;
  p.tokens_per_wg = h->tokens_per_wg;
  p.head_splits = h->head_splits;
  p.q_splits = h->q_splits;
  p.workgroups = backward ? h->grid_backward : h->grid_forward;
  p.pos64 = d.pos64 != 0;
  p.eps = d.eps;
  p.amplitude = a->amplitude;
  kind = ge::QkKind{d.dtype == GE_DT_BF16, wide(d, ptrs, n_ptrs, strides, n_strides), d.pairs == GE_PAIRS_HALF,
                    d.norm != 0, backward};
  return true;
}

}  // namespace

extern "C" {

ge_status_t ge_qk_validate(const ge_qk_desc_t* d) {
  if (!d) return GE_ERR_INVALID_ARG;
  if (d->tokens < 0 || d->heads_q < 0 || d->heads_k < 0) return GE_ERR_INVALID_ARG;
  if (d->pairs != GE_PAIRS_HALF && d->pairs != GE_PAIRS_INTERLEAVED) return GE_ERR_INVALID_ARG;
  if ((d->norm | 1) != 1 || (d->pos64 | 1) != 1) return GE_ERR_INVALID_ARG;
  if (d->dtype != GE_DT_BF16 && d->dtype != GE_DT_FP32 && d->dtype != GE_DT_FP8_E4M3) return GE_ERR_INVALID_ARG;
  if (!(d->eps >= 0.0f) || !std::isfinite(d->eps)) return GE_ERR_INVALID_ARG;
  if (d->head_dim < 1 || d->rot_dim < 0 || d->rot_dim > d->head_dim) return GE_ERR_INVALID_ARG;
  const int64_t strides[] = {d->q_token, d->q_head, d->k_token, d->k_head, d->oq_token, d->oq_head,
                             d->ok_token, d->ok_head, d->dq_token, d->dq_head, d->dk_token, d->dk_head};
  for (int64_t s : strides)
    if (s < 0) return GE_ERR_INVALID_ARG;
  if (d->dtype == GE_DT_FP8_E4M3) return GE_ERR_UNSUPPORTED;
  if (d->head_dim % 2 || d->head_dim > 512 || d->rot_dim % 2) return GE_ERR_UNSUPPORTED;
  if (d->tokens > kMaxTokens || d->heads_q > kMaxHeads || d->heads_k > kMaxHeads) return GE_ERR_UNSUPPORTED;
  for (int64_t s : strides)
    if (s > kMaxStride) return GE_ERR_UNSUPPORTED;
  // every byte offset in 62 bits
  for (int i = 0; i < 12; i += 2) {
    const int64_t heads = (i / 2) % 2 ? d->heads_k : d->heads_q;
    if ((double)d->tokens * (double)strides[i] + (double)heads * (double)strides[i + 1] > 1e18) return GE_ERR_UNSUPPORTED;
  }
  if (!apart(d->tokens, d->heads_q, d->oq_token, d->oq_head, d->head_dim) ||
      !apart(d->tokens, d->heads_k, d->ok_token, d->ok_head, d->head_dim) ||
      !apart(d->tokens, d->heads_q, d->dq_token, d->dq_head, d->head_dim) ||
      !apart(d->tokens, d->heads_k, d->dk_token, d->dk_head, d->head_dim))
    return GE_ERR_INVALID_ARG;
  return GE_OK;
}

ge_status_t ge_qk_create(const ge_qk_desc_t* d, ge_qk_handle_t* handle) {
  if (!handle) return GE_ERR_INVALID_ARG;
  *handle = nullptr;
  const ge_status_t st = ge_qk_validate(d);
  if (st != GE_OK) return st;
  int device = 0;
  if (!ge::block::current_gfx950(&device)) return GE_ERR_DEVICE;
  ge_qk_plan* p = new (std::nothrow) ge_qk_plan();
  if (!p) return GE_ERR_HIP;
  p->desc = *d;
  p->device = device;
  p->group = 1;
  while (p->group * 8 < d->head_dim) p->group *= 2;
  const int64_t heads = d->heads_q + d->heads_k, groups = ge::kQkThreads / p->group;
  if (d->tokens * heads <= 1024 * groups) {
    // few heads in all: one head per group of lanes, so that every compute unit has work
    p->tokens_per_wg = 1;
    p->q_splits = (int)ceil_div(d->heads_q, groups);
    p->head_splits = p->q_splits + (int)ceil_div(d->heads_k, groups);
    if (p->head_splits < 2) p->head_splits = 1;        // (one of the two has no heads)
  } else {
    // a workgroup turns about one angle per thread, then all heads of those tokens; fewer tokens
    // where that would leave less than four workgroups for a compute unit
    const int rot2 = std::max(d->rot_dim / 2, 1);
    const int64_t most = std::min<int64_t>(std::max(ge::kQkThreads / rot2, 1), kMostTokens);
    p->tokens_per_wg = (int)std::min(most, std::max<int64_t>(1, d->tokens / 1024));
    p->head_splits = 1;
    p->q_splits = 0;
  }
  const int64_t turns = heads > 0 ? ceil_div(d->tokens, p->tokens_per_wg) * p->head_splits : 0;
  p->turns = turns;
  // As many workgroups as are resident (six on a compute unit), each with the same number of turns:
  // their gains and addresses are set up once (16384 tokens of 40 heads of 128: 82 us with a workgroup
  // for every turn, 76 with 1536).
  p->grid_forward = (int)even_grid(turns, 1536);
  // with the norm every workgroup leaves partial sums: at least four turns each, or 512 workgroups
  p->grid_backward = d->norm ? (int)std::min<int64_t>(turns, std::min<int64_t>(ge::kQkMaxBackwardGrid,
                                                                               std::max<int64_t>(512, turns / 4)))
                             : p->grid_forward;
  *handle = p;
  return GE_OK;
}

void ge_qk_destroy(ge_qk_handle_t h) { delete h; }

ge_status_t ge_qk_workspace_size(ge_qk_handle_t h, size_t* bytes) {
  if (!h || !bytes) return GE_ERR_INVALID_ARG;
  *bytes = gain_bytes(h);
  return GE_OK;
}

ge_status_t ge_qk_forward(ge_qk_handle_t h, const ge_qk_args_t* a, void* stream) {
  if (!h || !a) return GE_ERR_INVALID_ARG;
  ge::QkParams p{};
  ge::QkKind kind{};
  if (!fill(h, a, false, p, kind)) return GE_ERR_INVALID_ARG;
  if (!ge::block::is_current(h->device)) return GE_ERR_DEVICE;
  return ge::launch_qk(kind, p, static_cast<hipStream_t>(stream)) == hipSuccess ? GE_OK : GE_ERR_HIP;
}

ge_status_t ge_qk_backward(ge_qk_handle_t h, const ge_qk_args_t* a, void* stream) {
  if (!h || !a) return GE_ERR_INVALID_ARG;
  ge::QkParams p{};
  ge::QkKind kind{};
  if (!fill(h, a, true, p, kind)) return GE_ERR_INVALID_ARG;
  if (!ge::block::is_current(h->device)) return GE_ERR_DEVICE;
  hipStream_t s = static_cast<hipStream_t>(stream);
  if (ge::launch_qk(kind, p, s) != hipSuccess) return GE_ERR_HIP;
  if (h->desc.norm && ge::launch_qk_gains(p.part, h->grid_backward, p.head_dim, a->dgain_q, a->dgain_k, s) != hipSuccess)
    return GE_ERR_HIP;
  return GE_OK;
}

}  // extern "C"

// ---------------------------------------------------------------------------------------------
// gradient norm and clipping
// ---------------------------------------------------------------------------------------------
struct ge_clip_plan {
  ge_clip_tensor_t* t;
  int32_t n, live;            // tensors, and those that are not empty
  int policy;                 // ge::ClipPolicy
  int device;
};

namespace {

// [tickets' room, unused][partial sums]
constexpr size_t kClipBytes = ge::kTicketBytes + ge::kClipPartials * sizeof(double);

int64_t clip_launches(const ge_clip_plan* h) { return ceil_div(h->live, ge::kClipTensors); }

struct Range {
  uintptr_t lo, hi;
  bool out;
  bool operator<(const Range& o) const { return lo < o.lo; }
};

}  // namespace

extern "C" {

ge_status_t ge_clip_create(const ge_clip_tensor_t* tensors, int32_t n, ge_clip_handle_t* handle) {
  if (!handle) return GE_ERR_INVALID_ARG;
  *handle = nullptr;
  if (n < 0 || (n > 0 && !tensors)) return GE_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (tensors[i].numel < 0 || (tensors[i].dtype != GE_DT_BF16 && tensors[i].dtype != GE_DT_FP32 &&
                                 tensors[i].dtype != GE_DT_FP8_E4M3))
      return GE_ERR_INVALID_ARG;
  int64_t all = 0, live = 0, bytes = 0;
  for (int32_t i = 0; i < n; ++i) {
    if (tensors[i].dtype == GE_DT_FP8_E4M3) return GE_ERR_UNSUPPORTED;
    if (tensors[i].numel >= (int64_t(1) << 45) || (all += tensors[i].numel) >= (int64_t(1) << 45)) return GE_ERR_UNSUPPORTED;
    live += tensors[i].numel > 0;
    bytes += tensors[i].numel * (tensors[i].dtype == GE_DT_BF16 ? 2 : 4);
  }
  // each launch and, in the workspace, each of its workgroups has a partial sum
  if (live > (int64_t)ge::kClipTensors * 256) return GE_ERR_UNSUPPORTED;
  int device = 0;
  if (!ge::block::current_gfx950(&device)) return GE_ERR_DEVICE;
  ge_clip_plan* p = new (std::nothrow) ge_clip_plan();
  if (!p) return GE_ERR_HIP;
  p->t = new (std::nothrow) ge_clip_tensor_t[n > 0 ? n : 1];
  if (!p->t) {
    delete p;
    return GE_ERR_HIP;
  }
  std::copy(tensors, tensors + n, p->t);
  p->n = n;
  p->live = (int32_t)live;
  p->policy = ge::clip_policy(bytes);
  p->device = device;
  *handle = p;
  return GE_OK;
}

void ge_clip_destroy(ge_clip_handle_t h) {
  if (!h) return;
  delete[] h->t;
  delete h;
}

ge_status_t ge_clip_workspace_size(ge_clip_handle_t h, size_t* bytes) {
  if (!h || !bytes) return GE_ERR_INVALID_ARG;
  *bytes = kClipBytes;
  return GE_OK;
}

ge_status_t ge_clip_run(ge_clip_handle_t h, const ge_clip_args_t* a, void* stream) {
  if (!h || !a) return GE_ERR_INVALID_ARG;
  if (!(a->max_norm >= 0.0f) || !(a->eps >= 0.0f) || !std::isfinite(a->eps)) return GE_ERR_INVALID_ARG;
  if (h->n > 0 && !a->in) return GE_ERR_INVALID_ARG;
  if (!a->out && !a->norm) return GE_ERR_INVALID_ARG;
  if (a->norm && !aligned(a->norm, 4)) return GE_ERR_INVALID_ARG;
  const size_t ws = kClipBytes;
  if (!a->workspace || !aligned(a->workspace, 16) || a->workspace_bytes < ws) return GE_ERR_INVALID_ARG;
  // outputs (and the norm and the workspace) overlap nothing but their own input, exactly
  {
    Range* r = new (std::nothrow) Range[2 * (size_t)h->live + 2];
    if (!r) return GE_ERR_HIP;
    size_t n = 0;
    bool ok = true;
    for (int32_t i = 0; i < h->n && ok; ++i) {
      if (h->t[i].numel == 0) continue;
      const size_t size = h->t[i].dtype == GE_DT_BF16 ? 2 : 4, bytes = (size_t)h->t[i].numel * size;
      const uintptr_t in = reinterpret_cast<uintptr_t>(a->in[i]), out = a->out ? reinterpret_cast<uintptr_t>(a->out[i]) : 0;
      ok = in && in % size == 0 && (!a->out || (out && out % size == 0));
      if (in != out) r[n++] = Range{in, in + bytes, false};
      if (a->out) r[n++] = Range{out, out + bytes, true};
    }
    const uintptr_t w = reinterpret_cast<uintptr_t>(a->workspace), nm = reinterpret_cast<uintptr_t>(a->norm);
    r[n++] = Range{w, w + ws, true};
    if (a->norm) r[n++] = Range{nm, nm + 4, true};
    if (ok) {
      std::sort(r, r + n);
      uintptr_t end_in = 0, end_out = 0;
      for (size_t i = 0; i < n && ok; ++i) {
        ok = r[i].lo >= end_out && (!r[i].out || r[i].lo >= end_in);
        (r[i].out ? end_out : end_in) = std::max(r[i].out ? end_out : end_in, r[i].hi);
      }
    }
    delete[] r;
    if (!ok) return GE_ERR_INVALID_ARG;
  }
  if (!ge::block::is_current(h->device)) return GE_ERR_DEVICE;

  hipStream_t s = static_cast<hipStream_t>(stream);
  double* part = reinterpret_cast<double*>(static_cast<unsigned char*>(a->workspace) + ge::kTicketBytes);
  const int64_t launches = clip_launches(h);
  const int most = launches > 0 ? (int)(ge::kClipPartials / launches) : 0;   // workgroups of one norm launch
  // pass 0: partial sums of every launch's tensors; pass 1: the norm and the scaled values
  int nparts = 0;
  for (int pass = 0; pass < 2; ++pass) {
    if (pass == 1 && (!a->out || launches == 0)) {
      if (a->norm && ge::launch_clip_finish(part, nparts, a->norm, s) != hipSuccess) return GE_ERR_HIP;
      break;
    }
    // the clipping pass takes the launches' tables in reverse: last read, first met
    for (int64_t l = 0; l < launches; ++l) {
      const int64_t which = pass == 0 ? l : launches - 1 - l;
      ge::ClipTable t{};
      int64_t chunks = 0, seen = 0;
      for (int32_t i = 0; i < h->n; ++i) {
        if (h->t[i].numel == 0) continue;
        if (seen++ / ge::kClipTensors != which) continue;
        t.in[t.n] = a->in[i];
        t.out[t.n] = a->out ? a->out[i] : nullptr;
        t.numel[t.n] = h->t[i].numel;
        t.chunk0[t.n] = (uint32_t)chunks;
        if (h->t[i].dtype == GE_DT_FP32) t.fp32[t.n >> 5] |= 1u << (t.n & 31);
        chunks += ceil_div(h->t[i].numel, ge::kClipChunk);
        ++t.n;
      }
      t.chunk0[t.n] = (uint32_t)chunks;
      const int grid = (int)std::min<int64_t>(chunks, pass == 0 ? most : ge::kClipPartials);
      hipError_t e;
      if (pass == 0) {
        e = ge::launch_clip_norm(t, grid, h->policy, part + nparts, s);
        nparts += grid;
      } else {
        e = ge::launch_clip_scale(t, grid, h->policy, part, nparts, a->max_norm, a->eps, l == 0 ? a->norm : nullptr, s);
      }
      if (e != hipSuccess) return GE_ERR_HIP;
    }
  }
  return GE_OK;
}

}  // extern "C"
