// seq_checks.h -- argument checks and workspace layouts that the C ABI files of
// the language-model operators share (host only).
#pragma once

#include <cmath>
#include <cstdint>

#include "fa.h"
#include "seq_kernels.h"

namespace fa {
namespace {

inline bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline size_t up256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// a * b * ... of positive ints, or -1 past 2^40
inline long long product(const int* x, int n) {
  long long r = 1;
  for (int i = 0; i < n; ++i) {
    if (x[i] < 1) return -1;
    if (r > (1LL << 40) / x[i]) return -1;
    r *= x[i];
  }
  return r;
}
template <typename... I>
bool sizes_ok(I... x) {
  const int v[] = {x...};
  return product(v, sizeof...(x)) > 0;
}
inline bool scale_ok(float scale) { return std::isfinite(scale) && scale > 0.f; }
inline bool dtype_ok(fa_dtype dt) { return dt == FA_DTYPE_F32 || dt == FA_DTYPE_BF16; }

// partial results [splits][rows] of dv entries and their lse
struct PartLayout {
  int splits_a, splits_b;
  size_t off_lse, bytes;
};
inline PartLayout part_layout(int sa, int sb, long long rows, int dv) {
  PartLayout w{sa, sb, 0, 0};
  const size_t n = static_cast<size_t>(sa + sb) * rows;
  w.off_lse = up256(n * dv * 4);
  w.bytes = w.off_lse + up256(n * 4);
  return w;
}

// the sequences' 64-key tiles, times the most ranges they are cut into, stay below 2^31
inline bool tiles_ok(int n_seq, long long n_keys) { return n_seq * ((n_keys + 63) / 64) * 305 <= 0x7fffffffLL; }

// tokens a sequence can hold in its pages, or -1
inline long long paged_keys(int page_size, int max_pages) {
  const long long n = static_cast<long long>(page_size) * max_pages;
  return n <= 0x7fffff00LL ? n : -1;
}

inline fa_status of(cudaError_t e) { return e == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

}  // namespace
}  // namespace fa
