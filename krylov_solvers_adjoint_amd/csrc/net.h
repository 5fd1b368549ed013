// Definitions shared by the network operators (layer norm, the gated
// feed-forward unit, the gated delta rule): element types, unaligned vector
// access, cross-lane sums.
#pragma once

#include <new>

#include "common.h"

// Products and sums of these operators may be fused (one rounding instead of
// two); the solver's kernels, whose results follow the textbook expression
// bit for bit, do not include this file.
#pragma clang fp contract(fast)

namespace sla {
namespace net {

template <typename T, int N>
struct VecOf {
  // any element-aligned address: rows of odd widths start anywhere, and
  // gfx950's global loads and stores take such addresses at full width
  typedef T type __attribute__((ext_vector_type(N), aligned(sizeof(T))));
};

// One 16-byte load or store of T.
template <typename T>
constexpr int kVec = int(16 / sizeof(T));

// N consecutive elements p[0..N) of which the first `have` exist (the others
// read as zero), widened to fp32.
template <int N, typename T>
__device__ __forceinline__ void load_f32(const T* __restrict__ p, int64_t have, float (&out)[N]) {
  if (have >= N) {
    const auto v = *reinterpret_cast<const typename VecOf<T, N>::type*>(p);
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = float(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = i < have ? float(p[i]) : 0.f;
  }
}

// ... and back, rounded once to T (nearest even).
template <int N, typename T>
__device__ __forceinline__ void store_f32(T* __restrict__ p, int64_t have, const float (&in)[N]) {
  if (have >= N) {
    typename VecOf<T, N>::type v;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = T(in[i]);
    *reinterpret_cast<typename VecOf<T, N>::type*>(p) = v;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < have) p[i] = T(in[i]);
  }
}

// Sum over groups of W neighbouring lanes, in every lane of the group.
template <int W, typename V>
__device__ __forceinline__ V lane_sum(V v) {
#pragma unroll
  for (int d = 1; d < W; d <<= 1) v += __shfl_xor(v, d, kWave);
  return v;
}

typedef float f32x4 __attribute__((ext_vector_type(4)));

__host__ __device__ inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline size_t type_size(sla_type t) { return t == SLA_F32 ? 4 : 2; }

inline bool valid_type(sla_type t) { return t == SLA_F32 || t == SLA_F16 || t == SLA_BF16; }

}  // namespace net
}  // namespace sla

#define SLA_NET_REQUIRE(cond, ...)                                             \
  do {                                                                         \
    if (!(cond)) {                                                             \
      ::sla::set_error(__VA_ARGS__);                                           \
      return SLA_ERR_ARG;                                                      \
    }                                                                          \
  } while (0)

// No exception leaves a C entry.
#define SLA_NET_BEGIN try {
#define SLA_NET_END                                                            \
  }                                                                            \
  catch (const std::bad_alloc&) {                                              \
    ::sla::set_error("host out of memory");                                    \
    return SLA_ERR_OOM;                                                        \
  }                                                                            \
  catch (...) {                                                                \
    ::sla::set_error("internal error");                                        \
    return SLA_ERR_DEVICE;                                                     \
  }
