#include "linear.h"
#include "product.h"

namespace sla {
namespace net {
namespace {

// The gradients of narrow projections (inner <= KP, outer <= NP) in one pass over
// x and dy: a wave takes kRows rows at a time, makes z, dz and dx of them and adds
// to dW and db, all on its own; the waves are joined at the end.
//
// The matrix instructions leave a row's four neighbouring columns in a lane,
// which is what the next product's factor looks like (16-bit: two tiles'
// quads, W^T laid out to match), so dz goes from z's sums into dx's product
// without leaving the registers.  For dW dz and x are turned by way of LDS.
//
// Bound by the fp32 matrix instructions (10^6 x 64 x 64 with silu: 25 Gflop, 160 us
// at their rate, beside 768 MB, 154 us): 275 to 290 us, where the four general
// kernels took 490; bf16 98 us for 384 MB (3.9 TB/s); without an activation 164 and 95.
template <typename T, int NP, int KP>
struct Narrow {
  static constexpr bool kHalf = sizeof(T) == 2;
  static constexpr int kUnit = kHalf ? 32 : 16;              // k of one fragment
  static constexpr int RT = kHalf ? 2 : 1, kRows = 16 * RT;  // tiles of rows a wave takes
  static constexpr int NJ = NP / 16, KJ = KP / 16, NS = NP / kUnit, KS = KP / kUnit;
  static constexpr int kLineN = NP + (kHalf ? 8 : 4), kLineK = KP + (kHalf ? 8 : 4);
  static constexpr int kWeight = NP * KP * int(sizeof(T));   // bytes of W in fragments
  static constexpr int kTurn = kRows * (kLineN + kLineK) * int(sizeof(T));
  static constexpr int kSums = NP * KP * 4;                  // of a wave's dW
  static constexpr int kBytes = 2 * kWeight + 4 * kTurn > 4 * kSums ? 2 * kWeight + 4 * kTurn
                                                                     : 4 * kSums;
  static constexpr int kPart = NP * KP + NP;                 // floats that a workgroup leaves
};
// Four elements from p on, of which `have` exist (WHOLE: all).
template <bool WHOLE, int N, typename T>
__device__ __forceinline__ typename VecOf<T, N>::type some(const T* p, int have) {
  typedef typename VecOf<T, N>::type V;
  if (WHOLE || have >= N) return *reinterpret_cast<const V*>(p);
  V v;
#pragma unroll
  for (int j = 0; j < N; ++j) v[j] = j < have ? p[j] : T(0.f);
  return v;
}
// SLOPE: there is an activation.  A kernel of its own for dz = dy: as a fourth way
// of the branch over the activations, one that hands dy's registers on untouched, it
// has made the compiler (-O3) leave out the copies to dz on one of the two edges that
// lead to it (seen in the assembly of a 64 x 64 fp16 kernel, whose dx was wrong).
template <typename T, int NP, int KP, bool WHOLE, bool SLOPE>
__global__ __launch_bounds__(256, 2) void k_narrow_grad(NarrowGrad g) {
  typedef Narrow<T, NP, KP> L;
  typedef typename Unit<T>::Vec Vec;
  typedef T V4 __attribute__((ext_vector_type(4)));
  constexpr int RT = L::RT, NJ = L::NJ, KJ = L::KJ, NS = L::NS, KS = L::KS, kN = Unit<T>::kN;
  extern __shared__ __align__(16) char smem[];
  const int t = threadIdx.x, w = t / kWave, l = t % 16, h = t % kWave / 16, lane = t % kWave;
  Vec* const wz = (Vec*)smem;                       // [NJ][KS][lane]
  Vec* const wx = (Vec*)(smem + L::kWeight);        // [KJ][NS][lane]
  T* const tz = (T*)(smem + 2 * L::kWeight + w * L::kTurn);
  T* const tx = tz + L::kRows * L::kLineN;
  const T* W = (const T*)g.w;
  for (int i = w; SLOPE && i < NJ * KS; i += 4) {
    const int n = i / KS * 16 + l, k = i % KS * L::kUnit + h * kN;
    Vec v;
#pragma unroll
    for (int r = 0; r < kN; ++r)
      v[r] = n < g.outer && k + r < g.inner ? W[n * g.inner + k + r] : T(0.f);
    wz[i * kWave + lane] = v;
  }
  for (int i = w; i < KJ * NS; i += 4) {
    const int k = i / NS * 16 + l;
    Vec v;
#pragma unroll
    for (int r = 0; r < kN; ++r) {
      const int n = i % NS * L::kUnit + r / 4 * 16 + 4 * h + r % 4;
      v[r] = n < g.outer && k < g.inner ? W[n * g.inner + k] : T(0.f);
    }
    wx[i * kWave + lane] = v;
  }
  f32x4 bias[NJ];
  Product p{};
  p.bias = SLOPE ? g.bias : nullptr;
  p.bias_f32 = g.bias_f32;
#pragma unroll
  for (int j = 0; j < NJ; ++j) bias[j] = bias_of<T>(p, 16 * j + 4 * h, g.outer - 16 * j - 4 * h);
  const float up = L::kHalf && g.scale ? g.scale[0] : 1.f;
  const float down = L::kHalf && g.scale ? g.scale[1] : 1.f;
  f32x4 dw[NJ][KJ];
  float db[NJ][4];
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) db[j][r] = 0.f;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int c = 0; c < KJ; ++c) dw[j][c] = f32x4{0, 0, 0, 0};
  Vec xs[RT][KS];
  typename VecOf<T, 4>::type dy[RT][NJ];
  const int64_t turns = div_up(g.rows, L::kRows), waves = int64_t(gridDim.x) * 4;
  auto load = [&](int64_t turn) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int64_t r = turn * L::kRows + 16 * i + l, row = r < g.rows ? r : g.rows - 1;
      const T* px = (const T*)g.x + row * g.ldx;
      const T* pd = (const T*)g.dy + row * g.lddy;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int k = s * L::kUnit + h * kN;
        const auto v = some<WHOLE, kN>(px + k, g.inner - k);
#pragma unroll
        for (int q = 0; q < kN; ++q) xs[i][s][q] = v[q];
      }
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        dy[i][j] = some<WHOLE, 4>(pd + 16 * j + 4 * h, g.outer - 16 * j - 4 * h);
      if (turn + 1 == turns && r >= g.rows) {   // behind the last row: nothing
#pragma unroll
        for (int s = 0; s < KS; ++s) xs[i][s] = Vec{};
#pragma unroll
        for (int j = 0; j < NJ; ++j) dy[i][j] = typename VecOf<T, 4>::type{};
      }
    }
  };
  __syncthreads();
  int64_t turn = int64_t(blockIdx.x) * 4 + w;
  if (turn < turns) load(turn);
  for (; turn < turns; turn += waves) {
    // dz in place of z's sums, rounded to T
    V4 dz[RT][NJ];
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      f32x4 z[NJ];
      if constexpr (SLOPE) {
#pragma unroll
        for (int j = 0; j < NJ; ++j) z[j] = bias[j];
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          Vec b[NJ];
#pragma unroll
          for (int j = 0; j < NJ; ++j) b[j] = wz[(j * KS + s) * kWave + lane];
          mma_row(z, xs[i][s], b);
        }
      }
      auto make = [&](auto act) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float v = float(dy[i][j][r]);
            if constexpr (act.value != kActNone) {
              float f, df;
              activation<act.value, L::kHalf>(z[j][r], f, df);
              v = v * up * df;
            }
            // z of a column that does not exist is NaN where x is not finite
            if (!WHOLE && 16 * j + 4 * h + r >= g.outer) v = 0.f;
            dz[i][j][r] = T(v);
            db[j][r] += v;   // (not rounded to T)
            // summed here: behind the branch all of v would have to wait in registers
            asm volatile("" : "+v"(db[j][r]));
          }
      };
      if constexpr (!SLOPE) make(std::integral_constant<int, kActNone>());
      else if (g.act == SLA_ACT_SILU) make(std::integral_constant<int, SLA_ACT_SILU>());
      else if (g.act == SLA_ACT_GELU) make(std::integral_constant<int, SLA_ACT_GELU>());
      else make(std::integral_constant<int, SLA_ACT_RELU>());
    }
    if (g.want_w) {   // turned by way of LDS (the wave's own: no barrier)
#pragma unroll
      for (int i = 0; i < RT; ++i) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          *(V4*)(tz + (16 * i + l) * L::kLineN + 16 * j + 4 * h) = dz[i][j];
#pragma unroll
        for (int s = 0; s < KS; ++s)
          *(Vec*)(tx + (16 * i + l) * L::kLineK + s * L::kUnit + h * kN) = xs[i][s];
      }
    }
    const int64_t now = turn;
    if (turn + waves < turns) load(turn + waves);
    if (g.dx) {
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        f32x4 o[KJ];
#pragma unroll
        for (int c = 0; c < KJ; ++c) o[c] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          Vec a, b[KJ];
#pragma unroll
          for (int r = 0; r < kN; ++r) a[r] = dz[i][s * kN / 4 + r / 4][r % 4];
#pragma unroll
          for (int c = 0; c < KJ; ++c) b[c] = wx[(c * NS + s) * kWave + lane];
          mma_row(o, a, b);
        }
        const int64_t row = now * L::kRows + 16 * i + l;
        if (row < g.rows) {
          T* to = (T*)g.dx + row * g.inner + 4 * h;
#pragma unroll
          for (int c = 0; c < KJ; ++c) {
            const float v[4] = {o[c][0] * down, o[c][1] * down, o[c][2] * down, o[c][3] * down};
            store_f32<4>(to + 16 * c, WHOLE ? 4 : g.inner - 16 * c - 4 * h, v);
          }
        }
      }
    }
    if (g.want_w) {
      asm volatile("" ::: "memory");
      auto column = [&](const T* from, int line) {
        Vec v;
        if constexpr (L::kHalf) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const auto c = read_column<T>(
                (const char*)(from + (8 * h + 4 * q + (l >> 2)) * line + (l & 3) * 4));
#pragma unroll
            for (int r = 0; r < 4; ++r) v[4 * q + r] = c[r];
          }
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = from[(4 * h + r) * line + l];
        }
        return v;
      };
      Vec b[KJ];
#pragma unroll
      for (int c = 0; c < KJ; ++c) b[c] = column(tx + 16 * c, L::kLineK);
#pragma unroll
      for (int j = 0; j < NJ; ++j) mma_row(dw[j], column(tz + 16 * j, L::kLineN), b);
      asm volatile("" ::: "memory");
    }
  }
  if (!g.part) return;
  // the four waves' sums in order, as [n][k]
  __syncthreads();
  f32x4* const mine = (f32x4*)smem + w * NJ * KJ * kWave + lane;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int c = 0; c < KJ; ++c) mine[(j * KJ + c) * kWave] = dw[j][c];
  __syncthreads();
  float* out = g.part + int64_t(blockIdx.x) * L::kPart;
  for (int i = t; i < NJ * KJ * kWave; i += 256) {
    const f32x4* q = (const f32x4*)smem + i;
    constexpr int kNext = NJ * KJ * kWave;
    const f32x4 v = (q[0] + q[kNext]) + (q[2 * kNext] + q[3 * kNext]);
    const int j = i / kWave / KJ, c = i / kWave % KJ, ll = i % 16, hh = i % kWave / 16;
    *(f32x4*)(out + (16 * j + ll) * KP + 16 * c + 4 * hh) = v;
  }
  __syncthreads();
  float* const sums = (float*)smem;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float v = lane_sum<16>(db[j][r]);
      if (l == 0) sums[w * NP + 16 * j + 4 * h + r] = v;
    }
  __syncthreads();
  if (t < NP)
    out[NP * KP + t] = (sums[t] + sums[NP + t]) + (sums[2 * NP + t] + sums[3 * NP + t]);
}
// dW [outer][inner] and db [outer] from the workgroups' sums, in their order.
constexpr int kJoinLines = 16;
template <typename T, typename B>
__global__ __launch_bounds__(kWave* kJoinLines) void k_narrow_join(
    const float* __restrict__ part, int groups, int np, int kp, int outer, int inner,
    const float* __restrict__ scale, T* __restrict__ dw, B* __restrict__ db) {
  __shared__ float join[kJoinLines][kWave];
  const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
  const int i = blockIdx.x * kWave + lane, all = np * kp + np;
  float s = 0.f;
  if (i < all) {
#pragma unroll 8
    for (int k = w; k < groups; k += kJoinLines) s += part[int64_t(k) * all + i];
  }
  join[w][lane] = s;
  __syncthreads();
  if (w || i >= all) return;
  s = 0.f;
  for (int k = 0; k < kJoinLines; ++k) s += join[k][lane];
  if (scale) s *= scale[1];
  if (i < np * kp) {
    if (dw && i / kp < outer && i % kp < inner) dw[i / kp * inner + i % kp] = T(s);
  } else if (db && i - np * kp < outer) {
    db[i - np * kp] = B(s);
  }
}

template <typename T, int NP, int KP>
sla_status start_narrow(const NarrowGrad& g, hipStream_t stream) {
  constexpr int lds = Narrow<T, NP, KP>::kBytes;
  const bool whole = g.outer == NP && g.inner == KP, slope = g.act != SLA_ACT_NONE;
  auto* kernel = whole ? (slope ? k_narrow_grad<T, NP, KP, true, true>
                                : k_narrow_grad<T, NP, KP, true, false>)
                       : (slope ? k_narrow_grad<T, NP, KP, false, true>
                                : k_narrow_grad<T, NP, KP, false, false>);
  SLA_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, lds));
  kernel<<<narrow_groups(g.rows), 256, lds, stream>>>(g);
  LAUNCH_CHECK();
  return SLA_OK;
}
template <typename T>
sla_status pick_narrow(const NarrowGrad& g, hipStream_t stream) {
  if (narrow_pad(g.outer) == 32)
    return narrow_pad(g.inner) == 32 ? start_narrow<T, 32, 32>(g, stream)
                                     : start_narrow<T, 32, 64>(g, stream);
  return narrow_pad(g.inner) == 32 ? start_narrow<T, 64, 32>(g, stream)
                                   : start_narrow<T, 64, 64>(g, stream);
}

}  // namespace

sla_status launch_narrow(const NarrowGrad& g, sla_type type, hipStream_t stream) {
  return with_type(type, [&](auto te) -> sla_status {
    using T = decltype(te);
    SLA_TRY(pick_narrow<T>(g, stream));
    if (!g.part) return SLA_OK;
    const int np = narrow_pad(g.outer), kp = narrow_pad(g.inner), groups = narrow_groups(g.rows);
    const int grid = int(div_up(np * kp + np, kWave));
    if (g.bias_f32)
      k_narrow_join<T, float><<<grid, kWave * kJoinLines, 0, stream>>>(
          g.part, groups, np, kp, g.outer, g.inner, g.scale, (T*)g.dw, (float*)g.db);
    else
      k_narrow_join<T, T><<<grid, kWave * kJoinLines, 0, stream>>>(
          g.part, groups, np, kp, g.outer, g.inner, g.scale, (T*)g.dw, (T*)g.db);
    LAUNCH_CHECK();
    return SLA_OK;
  });
}

}  // namespace net
}  // namespace sla
