// A projection with its bias, activation and residual in the epilogue, and its
// gradients.
//
//   z = x W^T + bias   y = residual + f(z)           f: none, silu, gelu or relu
//   dz = dy f'(z)      dx = dz W   dW = dz^T x   dbias = sum_rows dz
//
// The residual's gradient is dy.  Without an activation dz is dy; with one, z is
// computed again (its product's epilogue makes dz of it) rather than kept.  dz
// is then rounded once to the inputs' type, the type of the factors of the
// products that follow, which adds half a step to dx and dW; fp16's is held
// times a power of two that the largest |dy| gives, for its range (no activation
// is steeper than 1.13).  All sums are fp32.
#include "product.h"

namespace sla {
namespace net {
namespace {

// Column sums of dz: a team of lanes has 16 bytes a lane of a row, the other
// teams of the workgroup and the slabs of rows take rows in turn; teams and slabs
// are joined in order.
constexpr int kColumnSlabs = 512;
template <typename T, int TEAM>
__global__ __launch_bounds__(256) void k_column_sums(const T* __restrict__ dz, int64_t ld,
                                                     int64_t rows, int64_t cols,
                                                     float* __restrict__ part) {
  constexpr int V = kVec<T>, kTeams = 256 / TEAM;
  __shared__ float join[kTeams][V][TEAM];
  const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
  const int64_t c = (int64_t(blockIdx.x) * TEAM + lane) * V, have = cols - c;
  float s[V];
#pragma unroll
  for (int j = 0; j < V; ++j) s[j] = 0.f;
  if (have > 0) {
    const int64_t turn = int64_t(gridDim.y) * kTeams;
    int64_t r = int64_t(blockIdx.y) * kTeams + team;
    for (; r + 3 * turn < rows; r += 4 * turn) {   // four rows' loads travel at once
      float v[4][V];
#pragma unroll
      for (int k = 0; k < 4; ++k) load_f32<V>(dz + (r + k * turn) * ld + c, have, v[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int j = 0; j < V; ++j) s[j] += v[k][j];
    }
    for (; r < rows; r += turn) {
      float v[V];
      load_f32<V>(dz + r * ld + c, have, v);
#pragma unroll
      for (int j = 0; j < V; ++j) s[j] += v[j];
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) join[team][j][lane] = s[j];
  __syncthreads();
  if (team == 0 && have > 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      s[j] = 0.f;
      for (int k = 0; k < kTeams; ++k) s[j] += join[k][j][lane];
    }
    store_f32<V>(part + int64_t(blockIdx.y) * cols + c, have, s);
  }
}
constexpr int kJoinLines = 16;
template <typename W>
__global__ __launch_bounds__(kWave* kJoinLines) void k_column_join(
    const float* __restrict__ part, int slabs, int64_t cols, const float* __restrict__ scale,
    W* __restrict__ out) {
  __shared__ float join[kJoinLines][kWave];
  const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
  const int64_t c = int64_t(blockIdx.x) * kWave + lane;
  float s = 0.f;
  if (c < cols) {
#pragma unroll 8
    for (int i = w; i < slabs; i += kJoinLines) s += part[int64_t(i) * cols + c];
  }
  join[w][lane] = s;
  __syncthreads();
  if (w == 0 && c < cols) {
    s = 0.f;
    for (int k = 0; k < kJoinLines; ++k) s += join[k][lane];
    out[c] = W(scale ? s * scale[1] : s);
  }
}

int column_team(int64_t cols, int es) {
  const int64_t lanes = div_up(cols, 16 / es);
  return lanes <= 4 ? 4 : lanes <= 16 ? 16 : 64;
}
int column_slabs(int64_t rows, int64_t cols, int es) {
  const int team = column_team(cols, es);
  const int64_t tiles = div_up(cols, team * 16 / es), want = div_up(2048, tiles);
  const int64_t least = div_up(rows, 4 * (256 / team));   // four rows a team
  const int64_t most = least < want ? least : want;
  return int(most < 1 ? 1 : most < kColumnSlabs ? most : kColumnSlabs);
}
template <typename T>
void start_column_sums(const T* dz, int64_t ld, int64_t rows, int64_t cols, float* part,
                       hipStream_t stream) {
  const int team = column_team(cols, int(sizeof(T)));
  const dim3 grid(int(div_up(cols, team * kVec<T>)), column_slabs(rows, cols, int(sizeof(T))));
  if (team == 4) k_column_sums<T, 4><<<grid, 256, 0, stream>>>(dz, ld, rows, cols, part);
  else if (team == 16) k_column_sums<T, 16><<<grid, 256, 0, stream>>>(dz, ld, rows, cols, part);
  else k_column_sums<T, 64><<<grid, 256, 0, stream>>>(dz, ld, rows, cols, part);
}

// The gradients of narrow projections (inner <= KP, outer <= NP) in one pass over
// x and dy: a wave takes kRows rows at a time, makes z, dz and dx of them and adds
// to dW and db, all on its own; the waves are joined at the end.
//
// The matrix instructions leave a row's four neighbouring columns in a lane,
// which is what the next product's factor looks like (16-bit: two tiles'
// quads, W^T laid out to match), so dz goes from z's sums into dx's product
// without leaving the registers.  For dW dz and x are turned by way of LDS.
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
struct NarrowGrad {
  const void *x, *dy, *w, *bias;
  int64_t ldx, lddy, rows;
  int inner, outer, bias_f32, act, want_w;
  const float* scale;
  void* dx;
  float* part;   // [workgroups][kPart]; may be none
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
template <typename T, int NP, int KP, bool WHOLE>
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
  const bool slope = g.act != SLA_ACT_NONE;
  for (int i = w; i < NJ * KS; i += 4) {
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
  p.bias = slope ? g.bias : nullptr;
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
#pragma unroll
      for (int j = 0; j < NJ; ++j) z[j] = bias[j];
      if (slope) {
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
            float f, df;
            activation<act.value, L::kHalf>(z[j][r], f, df);
            const float e = float(dy[i][j][r]);
            dz[i][j][r] = T(act.value == kActNone ? e : e * up * df);
          }
      };
      if (g.act == SLA_ACT_SILU) make(std::integral_constant<int, SLA_ACT_SILU>());
      else if (g.act == SLA_ACT_GELU) make(std::integral_constant<int, SLA_ACT_GELU>());
      else if (g.act == SLA_ACT_RELU) make(std::integral_constant<int, SLA_ACT_RELU>());
      else make(std::integral_constant<int, kActNone>());
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) db[j][r] += float(dz[i][j][r]);
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

// Where one pass pays: the tiles of the general products read x and dy three
// times.
constexpr int64_t kNarrow = 64, kNarrowRows = 4096;
constexpr int kNarrowGroups = 512;
bool narrow(int64_t rows, int64_t inner, int64_t outer) {
  return inner <= kNarrow && outer <= kNarrow && rows >= kNarrowRows;
}
int narrow_pad(int64_t n) { return n <= 32 ? 32 : 64; }
int narrow_groups(int64_t rows) {
  const int64_t n = div_up(rows, 128);
  return int(n < kNarrowGroups ? n : kNarrowGroups);
}
template <typename T, int NP, int KP>
sla_status start_narrow(const NarrowGrad& g, hipStream_t stream) {
  constexpr int lds = Narrow<T, NP, KP>::kBytes;
  const bool whole = g.outer == NP && g.inner == KP;
  auto* kernel = whole ? k_narrow_grad<T, NP, KP, true> : k_narrow_grad<T, NP, KP, false>;
  SLA_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, lds));
  kernel<<<narrow_groups(g.rows), 256, lds, stream>>>(g);
  LAUNCH_CHECK();
  return SLA_OK;
}
template <typename T>
sla_status launch_narrow(const NarrowGrad& g, hipStream_t stream) {
  if (narrow_pad(g.outer) == 32)
    return narrow_pad(g.inner) == 32 ? start_narrow<T, 32, 32>(g, stream)
                                     : start_narrow<T, 32, 64>(g, stream);
  return narrow_pad(g.inner) == 32 ? start_narrow<T, 64, 32>(g, stream)
                                   : start_narrow<T, 64, 64>(g, stream);
}

sla_status linear_args(const char* who, int64_t rows, int64_t inner, int64_t outer, int64_t ldx,
                       sla_type type, sla_type btype, int act) {
  SLA_NET_REQUIRE(valid_type(type) && (btype == type || btype == SLA_F32),
                  "%s: unknown or mixed types", who);
  SLA_NET_REQUIRE(act == SLA_ACT_SILU || act == SLA_ACT_GELU || act == SLA_ACT_RELU ||
                      act == SLA_ACT_NONE, "%s: unknown activation", who);
  SLA_NET_REQUIRE(rows >= 0 && rows < (int64_t(1) << 31), "%s: rows out of range", who);
  SLA_NET_REQUIRE(inner >= 1 && inner < (int64_t(1) << 22) && outer >= 1 &&
                      outer < (int64_t(1) << 22), "%s: inner or outer out of range", who);
  SLA_NET_REQUIRE(ldx >= inner, "%s: row stride below inner", who);
  return SLA_OK;
}

// Splits of dW's sums at most: one workgroup's share of a million rows would
// take a millisecond.
constexpr int kWeightSplits = 1024;
int64_t up256(int64_t n) { return div_up(n, 256) * 256; }

// The gradient's workspace: dz (with an activation), fp16's scale and what it
// comes from, the columns' partial sums, the sums of a split product.
struct LinearSizes {
  int64_t forward, dz, scale, columns, sums, grad;
};
LinearSizes linear_sizes(int64_t rows, int64_t inner, int64_t outer, sla_type type, int act) {
  const int es = int(type_size(type));
  LinearSizes z{};
  z.forward = split_bytes(rows, outer, inner, 1, 1, 0, es);
  z.scale = act != SLA_ACT_NONE && type == SLA_F16 ? 256 + up256(kBoundGroups * 12) : 0;
  if (narrow(rows, inner, outer)) {
    const int64_t np = narrow_pad(outer), kp = narrow_pad(inner);
    z.sums = narrow_groups(rows) * (np * kp + np) * 4;
    z.grad = z.scale + z.sums;
    return z;
  }
  z.dz = act == SLA_ACT_NONE ? 0 : up256(rows * outer * es);
  z.columns = up256(column_slabs(rows, outer, es) * outer * 4);
  const int64_t x = split_bytes(rows, inner, outer, 1, 1, 1, es);
  const int64_t w = split_bytes(outer, inner, rows, 1, 1, 2, es, kWeightSplits);
  z.sums = x > w ? x : w;
  if (act != SLA_ACT_NONE && z.forward > z.sums) z.sums = z.forward;
  z.grad = z.dz + z.scale + z.columns + z.sums;
  return z;
}

}  // namespace
}  // namespace net
}  // namespace sla

using namespace sla;
using namespace sla::net;

extern "C" {

sla_status sla_linear_work(int64_t rows, int64_t inner, int64_t outer, sla_type type, int act,
                           int64_t* forward_bytes_host, int64_t* grad_bytes_host) {
  SLA_NET_BEGIN
  clear_error();
  SLA_TRY(linear_args("sla_linear_work", rows, inner, outer, inner, type, type, act));
  const LinearSizes z = linear_sizes(rows, inner, outer, type, act);
  if (forward_bytes_host) *forward_bytes_host = z.forward;
  if (grad_bytes_host) *grad_bytes_host = z.grad;
  return SLA_OK;
  SLA_NET_END
}

sla_status sla_linear(const void* x, int64_t ldx, const void* weight, const void* bias,
                      sla_type btype, const void* residual, int64_t ldr, int64_t rows,
                      int64_t inner, int64_t outer, sla_type type, int act, void* y, void* work,
                      int64_t work_bytes, hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  SLA_TRY(linear_args("sla_linear", rows, inner, outer, ldx, type, btype, act));
  SLA_NET_REQUIRE(!residual || ldr >= outer, "sla_linear: row stride of the residual below outer");
  if (rows == 0) return SLA_OK;
  SLA_NET_REQUIRE(x && weight && y, "sla_linear: an argument is NULL");
  const LinearSizes z = linear_sizes(rows, inner, outer, type, act);
  SLA_NET_REQUIRE(z.forward == 0 || (work && work_bytes >= z.forward),
                  "sla_linear: workspace too small (sla_linear_work)");
  return with_type(type, [&](auto te) -> sla_status {
    using T = decltype(te);
    Product g{};
    g.who = "sla_linear";
    g.A[0] = x, g.B[0] = weight;
    g.lda = ldx, g.ldb = inner;
    g.M = rows, g.N = outer, g.K = inner, g.parts = g.outputs = 1;
    g.dh = residual;
    g.lddh = ldr;
    g.bias = bias;
    g.bias_f32 = btype == SLA_F32;
    g.C[0] = y;
    g.ldc = outer;
    g.act = act;
    g.part = (float*)work;
    return launch_product<T, false, false, EPI_LINEAR>(g, stream);
  });
  SLA_NET_END
}

sla_status sla_linear_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                           const void* weight, const void* bias, sla_type btype, int64_t rows,
                           int64_t inner, int64_t outer, sla_type type, int act, void* dx,
                           void* dweight, void* dbias, void* work, int64_t work_bytes,
                           hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  SLA_TRY(linear_args("sla_linear_grad", rows, inner, outer, ldx, type, btype, act));
  SLA_NET_REQUIRE(lddy >= outer, "sla_linear_grad: row stride of dy below outer");
  SLA_NET_REQUIRE(rows == 0 || (dy && x && weight), "sla_linear_grad: an argument is NULL");
  const LinearSizes z = linear_sizes(rows, inner, outer, type, act);
  SLA_NET_REQUIRE(work && work_bytes >= z.grad,
                  "sla_linear_grad: workspace too small (sla_linear_work)");
  if (!dx && !dweight && !dbias) return SLA_OK;
  float* scale = z.scale && rows ? (float*)((char*)work + z.dz) : nullptr;
  float* columns = (float*)((char*)work + z.dz + z.scale);
  float* sums = (float*)((char*)work + z.dz + z.scale + z.columns);
  return with_type(type, [&](auto te) -> sla_status {
    using T = decltype(te);
    const void* dz = dy;
    int64_t lddz = lddy;
    if (scale) {
      const int groups = int(rows < 4 * kBoundGroups ? div_up(rows, 4) : kBoundGroups);
      const Lines none = {nullptr, 0, 0, 1};
      k_bound<<<groups, kProductBlock, 0, stream>>>(
          Lines{(const _Float16*)dy, lddy, rows, int(outer)}, none, none, none, scale + 64);
      LAUNCH_CHECK();
      k_scale<true><<<1, kWave, 0, stream>>>(scale + 64, groups, scale);
      LAUNCH_CHECK();
    }
    if (narrow(rows, inner, outer)) {
      const bool joined = dweight || dbias;
      const NarrowGrad g = {x, dy, weight, bias, ldx, lddy, rows, int(inner), int(outer),
                            btype == SLA_F32, act, dweight != nullptr, scale, dx,
                            joined ? sums : nullptr};
      SLA_TRY(launch_narrow<T>(g, stream));
      if (joined) {
        const int np = narrow_pad(outer), kp = narrow_pad(inner), groups = narrow_groups(rows);
        const int grid = int(div_up(np * kp + np, kWave));
        if (btype == SLA_F32)
          k_narrow_join<T, float><<<grid, kWave * kJoinLines, 0, stream>>>(
              sums, groups, np, kp, int(outer), int(inner), scale, (T*)dweight, (float*)dbias);
        else
          k_narrow_join<T, T><<<grid, kWave * kJoinLines, 0, stream>>>(
              sums, groups, np, kp, int(outer), int(inner), scale, (T*)dweight, (T*)dbias);
        LAUNCH_CHECK();
      }
      return SLA_OK;
    }
    if (act != SLA_ACT_NONE && rows) {
      Product g{};
      g.who = "sla_linear_grad";
      g.A[0] = x, g.B[0] = weight;
      g.lda = ldx, g.ldb = inner;
      g.M = rows, g.N = outer, g.K = inner, g.parts = g.outputs = 1;
      g.dh = dy;
      g.lddh = lddy;
      g.bias = bias;
      g.bias_f32 = btype == SLA_F32;
      g.C[0] = work;
      g.ldc = outer;
      g.act = act;
      g.scale = scale;
      g.part = sums;
      SLA_TRY((launch_product<T, false, false, EPI_SLOPE>(g, stream)));
      dz = work;
      lddz = outer;
    }
    if (dx) {
      Product p{};
      p.who = "sla_linear_grad";
      p.A[0] = dz, p.B[0] = weight;
      p.lda = lddz, p.ldb = inner;
      p.M = rows, p.N = inner, p.K = outer, p.parts = p.outputs = 1;
      p.part = sums;
      p.scale = scale;
      p.C[0] = dx;
      p.ldc = inner;
      SLA_TRY((launch_product<T, false, true, EPI_STORE>(p, stream)));
    }
    if (dweight) {
      Product p{};
      p.who = "sla_linear_grad";
      p.A[0] = dz, p.B[0] = x;
      p.lda = lddz, p.ldb = ldx;
      p.M = outer, p.N = inner, p.K = rows, p.parts = p.outputs = 1;
      p.part = sums;
      p.scale = scale;
      p.most = kWeightSplits;
      p.C[0] = dweight;
      p.ldc = inner;
      SLA_TRY((launch_product<T, true, true, EPI_STORE>(p, stream)));
    }
    if (dbias) {
      const int slabs = column_slabs(rows, outer, int(sizeof(T)));
      start_column_sums<T>((const T*)dz, lddz, rows, outer, columns, stream);
      LAUNCH_CHECK();
      const int grid = int(div_up(outer, kWave));
      if (btype == SLA_F32)
        k_column_join<float><<<grid, kWave * kJoinLines, 0, stream>>>(columns, slabs, outer, scale, (float*)dbias);
      else
        k_column_join<T><<<grid, kWave * kJoinLines, 0, stream>>>(columns, slabs, outer, scale, (T*)dbias);
      LAUNCH_CHECK();
    }
    return SLA_OK;
  });
  SLA_NET_END
}

}  // extern "C"
