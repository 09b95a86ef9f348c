// Host helpers of the transformer-block operators' C-ABI: device and argument checks.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>
#include <cstring>

namespace ge {
namespace block {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The current device, if it is a gfx950.  What a device is does not change: its properties (some
// 20 us to ask for) are read once.
inline bool current_gfx950(int* device) {
  static std::atomic<int> known[64];                   // 0: not asked, 1: gfx950, 2: another
  if (hipGetDevice(device) != hipSuccess) {
    (void)hipGetLastError();
    return false;
  }
  const bool kept = *device >= 0 && *device < 64;
  int k = kept ? known[*device].load(std::memory_order_relaxed) : 0;
  if (k == 0) {
    hipDeviceProp_t prop;
    if (hipGetDeviceProperties(&prop, *device) != hipSuccess) {
      (void)hipGetLastError();
      return false;
    }
    k = std::strncmp(prop.gcnArchName, "gfx950", 6) == 0 ? 1 : 2;
    if (kept) known[*device].store(k, std::memory_order_relaxed);
  }
  return k == 1;
}
inline bool is_current(int device) {
  int now = -1;
  if (hipGetDevice(&now) != hipSuccess) {
    (void)hipGetLastError();
    return false;
  }
  return now == device;
}

// rows x cols elements of `size` bytes at p, row pitch ld elements.
struct Matrix {
  const void* p;
  int64_t rows, cols, ld;
  int64_t size = 2;
  bool empty() const { return rows <= 0 || cols <= 0; }
};

// Whether two matrices may share an element.  Exact for equal pitches (column blocks of one
// wider matrix do not overlap); for different pitches any overlap of their address ranges counts.
inline bool overlap(const Matrix& a, const Matrix& b) {
  if (a.empty() || b.empty()) return false;
  const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
  const uintptr_t ea = pa + (uintptr_t)(((a.rows - 1) * a.ld + a.cols) * a.size);
  const uintptr_t eb = pb + (uintptr_t)(((b.rows - 1) * b.ld + b.cols) * b.size);
  if (ea <= pb || eb <= pa) return false;
  if (a.ld * a.size != b.ld * b.size || a.rows == 1 || b.rows == 1) return true;
  const int64_t pitch = a.ld * a.size;
  int64_t r = (int64_t)(pb - pa) % pitch;              // b's first column within a's rows
  if (r < 0) r += pitch;
  return r < a.cols * a.size || r + b.cols * b.size > pitch;
}

// Every non-empty matrix has a 16-byte aligned pointer, and no output overlaps an input or
// another output, except input `same_in` with output `same_out` (the same matrix).
inline bool usable(const Matrix* in, int n_in, const Matrix* out, int n_out, int same_in, int same_out) {
  for (int i = 0; i < n_in; ++i)
    if (!in[i].empty() && (!in[i].p || !aligned(in[i].p, 16))) return false;
  for (int o = 0; o < n_out; ++o) {
    if (!out[o].empty() && (!out[o].p || !aligned(out[o].p, 16))) return false;
    for (int i = 0; i < n_in; ++i)
      if (!(i == same_in && o == same_out) && overlap(in[i], out[o])) return false;
    for (int q = 0; q < o; ++q)
      if (overlap(out[q], out[o])) return false;
  }
  return true;
}

}  // namespace block
}  // namespace ge
