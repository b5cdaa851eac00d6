// ops.h -- shared pieces of the operators of include/rnnt_ops.h (internal).
#pragma once
#include <cstdio>
#include <cstdlib>

#include "../../include/rnnt_ops.h"
#include "kernels.h"
#include "profile.h"

namespace rnnt {

inline bool op_dtype(int d) { return d == RNNT_F32 || d == RNNT_BF16; }
inline int op_size(int d) { return d == RNNT_F32 ? 4 : 2; }
inline bool aligned_to(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

#define OPS_CHECK(expr)                                                                  \
  do {                                                                                   \
    cudaError_t e_ = (expr);                                                             \
    if (e_ != cudaSuccess) {                                                             \
      if (getenv("RNNT_VERBOSE"))                                                        \
        fprintf(stderr, "rnnt: %s -> %s (%s:%d)\n", #expr, cudaGetErrorString(e_),       \
                __FILE__, __LINE__);                                                     \
      return RNNT_ERR_CUDA;                                                              \
    }                                                                                    \
  } while (0)

// Launch with an optional profiling bracket (see include/rnnt_profile.h).
#define OPS_LAUNCH(name, expr)          \
  do {                                  \
    rnnt::ProfScope ps_(name, st);      \
    OPS_CHECK(expr);                    \
  } while (0)

__device__ __forceinline__ void report(int32_t* status, int code) {
  if (status) atomicOr(status, status_bit(code));
}

template <typename T> __device__ __forceinline__ T from_f(float x);
template <> __device__ __forceinline__ float from_f<float>(float x) { return x; }
template <> __device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Division of 0 <= n < 2^31 by a fixed d (round-up reciprocal): a multiply-high,
// an add and a shift in place of the twenty instructions of a 32-bit division.
struct FastDiv {
  uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
  FastDiv f{d, 0, 0};
  while ((1ull << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
  return f;
}
__device__ __forceinline__ int operator/(int n, const FastDiv& f) {
  return (int)((__umulhi((uint32_t)n, f.mul) + (uint32_t)n) >> f.shift);
}

}  // namespace rnnt
