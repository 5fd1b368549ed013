// The gated feed-forward unit and its gradients.
//
//   a = x Wg^T   b = x Wu^T   h = f(a) b          f: silu, gelu or relu
//   da = dh b f'(a)           db = dh f(a)
//   dx = da Wg + db Wu        dWg = da^T x        dWu = db^T x
//
// Both projections, the activation and the product are one kernel: a
// workgroup's tile holds the same columns of a and of b, so h leaves from the
// accumulators and a and b never reach memory.  Backward computes a and b
// again with the same kernel (its epilogue turns them into da and db) rather
// than keep them.  da and db are rounded once to the inputs' type, the factors'
// type of the products that follow: keeping fp32 would halve nothing and
// double the bytes, and the 16-bit matrix instructions take 16-bit factors.
// All sums are fp32.
#include "net.h"

namespace sla {
namespace net {
namespace {

constexpr int kFfnBlock = 256;
constexpr int kBM = 128, kBN = 128, kBK = 32;

enum { EPI_GATE, EPI_GATE_GRAD, EPI_STORE };

__device__ __forceinline__ void activation(int act, float a, float& f, float& df) {
  if (act == SLA_ACT_SILU) {
    const float s = 1.f / (1.f + expf(-a));
    f = a * s;
    df = s * (1.f + a * (1.f - s));
  } else if (act == SLA_ACT_GELU) {
    const float c = 0.5f * (1.f + erff(a * 0.70710678118654752f));
    f = a * c;
    df = c + a * (0.39894228040143268f * expf(-0.5f * a * a));
  } else {
    f = a > 0.f ? a : a * 0.f;  // NaN stays NaN
    df = a > 0.f ? 1.f : 0.f;
  }
}

// One product C[M][N] = sum over `parts` segments of A_s[M][K] B_s[N][K]^T.
// AT: A is stored [k][row] (lda elements from one k to the next) instead of
// [row][k]; BT: likewise.
struct Product {
  const void *A[2], *B[2];
  int64_t lda, ldb;
  int64_t M, N, K;
  int parts;
  const void* dh;    // EPI_GATE_GRAD [M][N]
  int64_t lddh;
  void* C[2];        // EPI_GATE: h; EPI_GATE_GRAD: da, db; EPI_STORE: one per blockIdx.z
  int64_t ldc;
  int act;
};

template <typename T>
struct Mfma;
template <>
struct Mfma<__bf16> {
  typedef __bf16 Frag __attribute__((ext_vector_type(8)));
  static constexpr int kPad = 8;
  static __device__ __forceinline__ f32x4 run(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mfma<_Float16> {
  typedef _Float16 Frag __attribute__((ext_vector_type(8)));
  static constexpr int kPad = 8;
  static __device__ __forceinline__ f32x4 run(Frag a, Frag b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  }
};
template <>
struct Mfma<float> {
  typedef float Frag __attribute__((ext_vector_type(8)));
  static constexpr int kPad = 4;
  static __device__ __forceinline__ f32x4 run(Frag a, Frag b, f32x4 c) {
#pragma unroll
    for (int j = 0; j < 8; ++j) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], c, 0, 0, 0);
    return c;
  }
};

// A kBM (or kBN) x kBK piece of an operand, on its way to LDS through
// registers: 16 elements a thread, zero outside the matrix.
template <typename T, bool TRANS>
struct Piece {
  typename VecOf<T, 8>::type v[2];
  __device__ __forceinline__ void fetch(const T* p, int64_t ld, int64_t rows, int64_t k0,
                                        int64_t K) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = threadIdx.x + i * kFfnBlock;
      int64_t line, along, lines, length;
      if constexpr (TRANS) {
        line = k0 + at / 16, along = at % 16 * 8, lines = K, length = rows;
      } else {
        line = at / 4, along = k0 + at % 4 * 8, lines = rows, length = K;
      }
      const T* q = p + line * ld + along;
      const int64_t have = line < lines ? length - along : 0;
      if (have >= 8) {
        v[i] = *reinterpret_cast<const typename VecOf<T, 8>::type*>(q);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = j < have ? q[j] : T(0.f);
      }
    }
  }
  __device__ __forceinline__ void put(T* lds, int ldl) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int at = threadIdx.x + i * kFfnBlock;
      if constexpr (TRANS) {
#pragma unroll
        for (int j = 0; j < 8; ++j) lds[(at % 16 * 8 + j) * ldl + at / 16] = v[i][j];
      } else {
        T* d = lds + (at / 4) * ldl + at % 4 * 8;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = v[i][j];
      }
    }
  }
};

// 128 x 128 tiles, 4 waves of 64 x 64.  EPI_GATE*: the tile's columns are 64
// of a and the same 64 of b, half of each in every wave.
template <typename T, bool AT, bool BT, int EPI>
__global__ __launch_bounds__(kFfnBlock) void k_ffn_product(Product g) {
  using MM = Mfma<T>;
  constexpr bool kGate = EPI != EPI_STORE;
  constexpr int LD = kBK + MM::kPad, kCols = kGate ? kBN / 2 : kBN;
  __shared__ __align__(16) T As[kBM * LD];
  __shared__ __align__(16) T Bs[kBN * LD];
  const int t = threadIdx.x, w = t / kWave, l = t % 16, h = (t % kWave) / 16;
  const int wm = w / 2, wn = w % 2;
  const int64_t m0 = int64_t(blockIdx.y) * kBM, n0 = int64_t(blockIdx.x) * kCols;
  const int z = blockIdx.z;
  f32x4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  // row of the B tile of this wave's column tile j
  auto brow = [&](int j) {
    return kGate ? (j / 2) * (kBN / 2) + wn * 32 + (j % 2) * 16 : wn * 64 + j * 16;
  };
  for (int s = 0; s < g.parts; ++s) {
    const T* A = (const T*)g.A[kGate ? 0 : s + z] + m0 * (AT ? 1 : g.lda);
    const T* B0 = (const T*)g.B[kGate ? 0 : s] + n0 * (BT ? 1 : g.ldb);
    const T* B1 = (const T*)g.B[1] + n0 * g.ldb;  // kGate only
    for (int64_t k0 = 0; k0 < g.K; k0 += kBK) {
      Piece<T, AT> pa;
      Piece<T, BT> pb;
      pa.fetch(A + k0 * 0, g.lda, g.M - m0, k0, g.K);
      if constexpr (kGate) {
        // lines 0..63 from Wg, 64..127 from Wu
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int at = t + i * kFfnBlock;
          const int64_t line = at / 4 % 64, along = k0 + at % 4 * 8;
          const T* q = (i ? B1 : B0) + line * g.ldb + along;
          const int64_t have = n0 + line < g.N ? g.K - along : 0;
          if (have >= 8) {
            pb.v[i] = *reinterpret_cast<const typename VecOf<T, 8>::type*>(q);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) pb.v[i][j] = j < have ? q[j] : T(0.f);
          }
        }
      } else {
        pb.fetch(B0, g.ldb, g.N - n0, k0, g.K);
      }
      __syncthreads();
      pa.put(As, LD);
      pb.put(Bs, LD);
      __syncthreads();
      typename MM::Frag fa[4], fb[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        fa[i] = *reinterpret_cast<const typename MM::Frag*>(As + (wm * 64 + i * 16 + l) * LD + 8 * h);
        fb[i] = *reinterpret_cast<const typename MM::Frag*>(Bs + (brow(i) + l) * LD + 8 * h);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = MM::run(fa[i], fb[j], acc[i][j]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t row = m0 + wm * 64 + i * 16 + 4 * h + r;
      if (row >= g.M) continue;
#pragma unroll
      for (int j = 0; j < (kGate ? 2 : 4); ++j) {
        const int64_t col = n0 + brow(j) + l;
        if (col >= g.N) continue;
        if constexpr (EPI == EPI_STORE) {
          ((T*)g.C[z])[row * g.ldc + col] = T(acc[i][j][r]);
        } else {
          float f, df;
          activation(g.act, acc[i][j][r], f, df);
          const float b = acc[i][j + 2][r];
          if constexpr (EPI == EPI_GATE) {
            ((T*)g.C[0])[row * g.ldc + col] = T(f * b);
          } else {
            const float d = float(((const T*)g.dh)[row * g.lddh + col]);
            ((T*)g.C[0])[row * g.ldc + col] = T(d * b * df);
            ((T*)g.C[1])[row * g.ldc + col] = T(d * f);
          }
        }
      }
    }
}

template <typename T, bool AT, bool BT, int EPI>
sla_status launch_product(const Product& g, int outputs, hipStream_t stream) {
  if (g.M == 0 || g.N == 0) return SLA_OK;
  const int64_t gx = div_up(g.N, EPI == EPI_STORE ? kBN : kBN / 2), gy = div_up(g.M, kBM);
  SLA_NET_REQUIRE(gx < (int64_t(1) << 31) && gy < 65536, "gated_ffn: a matrix is too large");
  k_ffn_product<T, AT, BT, EPI><<<dim3(int(gx), int(gy), outputs), kFfnBlock, 0, stream>>>(g);
  LAUNCH_CHECK();
  return SLA_OK;
}

sla_status ffn_args(const char* who, int64_t rows, int64_t inner, int64_t outer, int64_t ldx,
                    sla_type type, int act) {
  SLA_NET_REQUIRE(valid_type(type), "%s: unknown type", who);
  SLA_NET_REQUIRE(act == SLA_ACT_SILU || act == SLA_ACT_GELU || act == SLA_ACT_RELU,
                  "%s: unknown activation", who);
  SLA_NET_REQUIRE(rows >= 0 && rows < (int64_t(1) << 22), "%s: rows out of range", who);
  SLA_NET_REQUIRE(inner >= 1 && inner < (int64_t(1) << 22) && outer >= 1 &&
                      outer < (int64_t(1) << 22), "%s: inner or outer out of range", who);
  SLA_NET_REQUIRE(ldx >= inner, "%s: row stride below inner", who);
  return SLA_OK;
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

using namespace sla;
using namespace sla::net;

extern "C" {

sla_status sla_gated_ffn(const void* x, int64_t ldx, const void* w_gate, const void* w_up,
                         int64_t rows, int64_t inner, int64_t outer, sla_type type, int act,
                         void* h, hipStream_t stream) {
  clear_error();
  SLA_TRY(ffn_args("sla_gated_ffn", rows, inner, outer, ldx, type, act));
  if (rows == 0) return SLA_OK;
  SLA_NET_REQUIRE(x && w_gate && w_up && h, "sla_gated_ffn: an argument is NULL");
  return with_type(type, [&](auto te) -> sla_status {
    using T = decltype(te);
    Product g{};
    g.A[0] = x;
    g.B[0] = w_gate;
    g.B[1] = w_up;
    g.lda = ldx;
    g.ldb = inner;
    g.M = rows, g.N = outer, g.K = inner, g.parts = 1;
    g.C[0] = h;
    g.ldc = outer;
    g.act = act;
    return launch_product<T, false, false, EPI_GATE>(g, 1, stream);
  });
}

sla_status sla_gated_ffn_work(int64_t rows, int64_t inner, int64_t outer, sla_type type,
                              int64_t* bytes_host) {
  clear_error();
  SLA_TRY(ffn_args("sla_gated_ffn_work", rows, inner, outer, inner, type, SLA_ACT_SILU));
  SLA_NET_REQUIRE(bytes_host, "sla_gated_ffn_work: bytes_host is NULL");
  *bytes_host = 2 * rows * outer * int64_t(type_size(type));
  return SLA_OK;
}

sla_status sla_gated_ffn_grad(const void* dh, int64_t lddh, const void* x, int64_t ldx,
                              const void* w_gate, const void* w_up, int64_t rows, int64_t inner,
                              int64_t outer, sla_type type, int act, void* dx, void* dw_gate,
                              void* dw_up, void* work, int64_t work_bytes, hipStream_t stream) {
  clear_error();
  SLA_TRY(ffn_args("sla_gated_ffn_grad", rows, inner, outer, ldx, type, act));
  SLA_NET_REQUIRE(lddh >= outer, "sla_gated_ffn_grad: row stride of dh below outer");
  SLA_NET_REQUIRE(rows == 0 || (dh && x && w_gate && w_up),
                  "sla_gated_ffn_grad: an argument is NULL");
  SLA_NET_REQUIRE((dw_gate == nullptr) == (dw_up == nullptr),
                  "sla_gated_ffn_grad: both weights' gradients or neither");
  const int64_t size = rows * outer * int64_t(type_size(type));
  SLA_NET_REQUIRE(rows == 0 || (work && work_bytes >= 2 * size),
                  "sla_gated_ffn_grad: workspace too small (sla_gated_ffn_work)");
  return with_type(type, [&](auto te) -> sla_status {
    using T = decltype(te);
    Product g{};
    g.A[0] = x;
    g.B[0] = w_gate;
    g.B[1] = w_up;
    g.lda = ldx;
    g.ldb = inner;
    g.M = rows, g.N = outer, g.K = inner, g.parts = 1;
    g.dh = dh;
    g.lddh = lddh;
    g.C[0] = work;
    g.C[1] = (char*)work + size;
    g.ldc = outer;
    g.act = act;
    SLA_TRY((launch_product<T, false, false, EPI_GATE_GRAD>(g, 1, stream)));
    if (dx) {
      Product p{};
      p.A[0] = g.C[0], p.A[1] = g.C[1];
      p.B[0] = w_gate, p.B[1] = w_up;
      p.lda = outer, p.ldb = inner;
      p.M = rows, p.N = inner, p.K = outer, p.parts = 2;
      p.C[0] = dx;
      p.ldc = inner;
      SLA_TRY((launch_product<T, false, true, EPI_STORE>(p, 1, stream)));
    }
    if (dw_gate) {
      Product p{};
      p.A[0] = g.C[0], p.A[1] = g.C[1];
      p.B[0] = p.B[1] = x;
      p.lda = outer, p.ldb = ldx;
      p.M = outer, p.N = inner, p.K = rows, p.parts = 1;
      p.C[0] = dw_gate, p.C[1] = dw_up;
      p.ldc = inner;
      SLA_TRY((launch_product<T, true, true, EPI_STORE>(p, 2, stream)));
    }
    return SLA_OK;
  });
}

}  // extern "C"
