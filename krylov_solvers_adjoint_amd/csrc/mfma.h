// What kernels on the matrix cores are made of: fragments, transposed reads from
// LDS, direct loads into it, stores of whole rows.
#pragma once

#include <type_traits>

#include "net.h"

namespace sla {
namespace net {
namespace {

// 16 bytes of an operand: a lane's factor of one matrix instruction (8 16-bit
// values of 32 k) or of four (4 fp32 values of 16 k).
template <typename T>
struct Unit {
  static constexpr int kN = 16 / int(sizeof(T));
  typedef T Vec __attribute__((ext_vector_type(16 / sizeof(T))));
  typedef typename VecOf<T, 16 / sizeof(T)>::type Loose;
};

// acc (4 columns 4 h + r of row l) += rows of `a` times rows of `b`.
__device__ __forceinline__ void mma16(f32x4& acc, Unit<__bf16>::Vec a, Unit<__bf16>::Vec b) {
  acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b, a, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma16(f32x4& acc, Unit<_Float16>::Vec a, Unit<_Float16>::Vec b) {
  acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(b, a, acc, 0, 0, 0);
}
__device__ __forceinline__ void mma16(f32x4& acc, Unit<float>::Vec a, Unit<float>::Vec b) {
#pragma unroll
  for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(b[j], a[j], acc, 0, 0, 0);
}

typedef __attribute__((address_space(3))) void* LdsPtr;
typedef __fp16 HalfQuad __attribute__((__vector_size__(8)));

// Four k of one column out of an LDS tile stored [k][row]: the 16 lanes of a
// group read four lines of 16 values and get a column each.
template <typename T>
__device__ __forceinline__ typename VecOf<T, 4>::type read_column(const char* p) {
  typedef T V4 __attribute__((ext_vector_type(4)));
  V4 v;
  if constexpr (std::is_same<T, __bf16>::value)
    v = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) V4*)p);
  else
    v = __builtin_bit_cast(V4, __builtin_amdgcn_ds_read_tr16_b64_v4f16(
                                   (__attribute__((address_space(3))) HalfQuad*)p));
  return v;
}

// An offset that lies out of every buffer: the load gives zeros.
constexpr int kOutside = int(0x80000000u);

// 16 bytes a lane from p + at to lds + 16 lane (p and lds: one for the wave).
// In assembly, so that the compiler does not take every LDS read behind it for
// one that has to wait for it; the kernel waits by count (arrive).
__device__ __forceinline__ void send(const char* p, int at, char* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  typedef int Words __attribute__((ext_vector_type(4)));
  const uint64_t q = reinterpret_cast<uint64_t>(p);
  const Words rsrc = {int(q), int(q >> 32) & 0xffff, 0x7fffffff, 0x00020000};
  const int m0 = int(reinterpret_cast<uintptr_t>((LdsPtr)lds));
  // m0 is written: the compiler, which keeps it to itself, warns and takes note
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :: "s"(m0), "v"(at), "s"(rsrc) : "memory", "m0");
#pragma clang diagnostic pop
#endif
}
// Waits until at most N direct loads are under way and the wave's LDS reads
// are done, then for the other waves.
template <int N>
__device__ __forceinline__ void landed() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// The wave's first element of a step, in scalar registers.
__device__ __forceinline__ const char* uniform(const char* q) {
  const uint64_t p = reinterpret_cast<uint64_t>(q);
  return reinterpret_cast<const char*>(
      uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(p >> 32)))) << 32 |
      uint32_t(__builtin_amdgcn_readfirstlane(int(p))));
}

// Two neighbouring tiles' quads of 16-bit columns, x and y of lane (l, h), as
// eight columns in a row: of tile h % 2, from 8 (h / 2) on, and back.  A store
// then writes 64 bytes of each of 16 rows instead of 32: of 16384 x 1024 x 4096
// bf16, da and db (0.4 GB beside the product) take 326 us instead of 363, h 286
// instead of 295, dx and dW 248 and 245 instead of 253 and 256.
typedef uint32_t Pair __attribute__((ext_vector_type(2)));
typedef uint32_t Quads __attribute__((ext_vector_type(4)));
__device__ __forceinline__ Quads side_by_side(Pair x, Pair y) {
  Quads q;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto s = __builtin_amdgcn_permlane16_swap(x[i], y[i], false, false);
    q[i] = s[0];
    q[2 + i] = s[1];
  }
  return q;
}
template <typename T>
__device__ __forceinline__ Pair packed(const float (&u)[4]) {
  typedef T V4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(Pair, V4{T(u[0]), T(u[1]), T(u[2]), T(u[3])});
}

template <typename F>
sla_status with_type(sla_type t, F&& f) {
  if (t == SLA_F32) return f(float());
  if (t == SLA_F16) return f(_Float16());
  return f(__bf16());
}

}  // namespace
}  // namespace net
}  // namespace sla
