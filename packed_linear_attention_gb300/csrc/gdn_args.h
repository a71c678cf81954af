// gdn_args.h — checks of arguments that the C entry points share (host code).
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/gdn.h"
#include "gdn_internal.h"

namespace gdn {
namespace args {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline bool known_dtype(int32_t t) { return t == GDN_F32 || t == GDN_BF16; }
inline size_t item_size(int32_t dtype) { return dtype == GDN_BF16 ? 2 : 4; }

// Rows of `heads` heads: pointer, alignment and stride.
inline bool rows_ok(const void* p, int64_t stride, int32_t heads, int32_t head_dim, int32_t dtype) {
  return p && aligned(p, 16) && stride >= (int64_t)heads * head_dim &&
         stride % (int64_t)(16 / item_size(dtype)) == 0 && stride <= (int64_t)1 << 40;
}

struct Span {
  uintptr_t lo, hi;
};
// The bytes that `tokens` rows of a strided tensor reach over.
inline Span span_of(const void* p, int64_t tokens, int64_t stride, int64_t row, size_t item) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, tokens > 0 ? lo + (uintptr_t)((tokens - 1) * stride + row) * item : lo};
}
inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }

// Two strided tensors share memory unless their rows lie beside one another in rows of the
// same stride (column ranges of one array).
inline bool rows_overlap(const void* p, int64_t ps, int64_t prow, const void* q, int64_t qs,
                  int64_t qrow, int64_t tokens, size_t item) {
  if (!overlap(span_of(p, tokens, ps, prow, item), span_of(q, tokens, qs, qrow, item)))
    return false;
  if (ps != qs) return true;
  const int64_t stride = ps * (int64_t)item;
  int64_t d = (int64_t)(reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p)) % stride;
  if (d < 0) d += stride;
  return d < prow * (int64_t)item || d + qrow * (int64_t)item > stride;
}

// Runs `launch` with the handle's device current.
template <class F>
gdn_status on_device(const gdn_handle* h, F launch) {
  const int device = gdn::handle_device(h);
  int prev = 0;
  if (cudaGetDevice(&prev) != cudaSuccess) return GDN_ERR_CUDA;
  if (prev != device && cudaSetDevice(device) != cudaSuccess) return GDN_ERR_CUDA;
  const int e = launch();
  if (prev != device) cudaSetDevice(prev);
  return e == 0 ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace args
}  // namespace gdn
