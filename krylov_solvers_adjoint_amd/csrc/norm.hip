// Layer norm and its gradients.
//
//   mean = sum_c x_c / C      rstd = 1 / sqrt(sum_c (x_c - mean)^2 / C + eps)
//   n_c  = (x_c - mean) rstd  y_c  = n_c w_c + b_c
//   t_c  = dy_c w_c
//   dx_c = rstd (t_c - sum(t)/C - n_c sum(t n)/C)
//   dw_c = sum_rows dy_c n_c  db_c = sum_rows dy_c
//
// Bound by memory: forward reads x and writes y, backward reads x and dy and
// writes dx, once each.  A row lives in the registers of a team of lanes (8
// to 64 lanes of a wave, or a whole workgroup), so the centred second moment
// and both backward sums need no second read.  The forward pass keeps mean
// and rstd (8 bytes a row).
//
// The mean is found in two steps.  c = x_0 + mean(x - x_0), x_0 the row's first
// element, lies next to the mean even if that is far from zero, but no closer
// than the rounding of the largest |x - x_0|.  The differences d = x - c are
// exact next to c, their own mean corrects it, and the variance is
// mean(d^2) - mean(d)^2, whose second term is a rounding's square.  So a
// constant row is exactly zero, a row close to a far mean keeps its digits, and
// so does one whose first element is the outlier (differences to x_0 = 1e4
// alone had left 4.5e-4 of the other 8191 elements).
//
// The gradient gets 1 / sqrt(var + eps) and the mean in one number: from x_0, or
// from zero if that is nearer (the other number is negative then).  A mean far
// from both belongs to a row whose deviations are of that size too.
//
// Measured: 10^6 x 64 fp32 forward 90 us (5.7 TB/s) and backward 151 + 5 (5.1
// TB/s); 16384 x 1024 bf16 16 and 22 + 5 us; 4096 x 16384 fp32 (the wide
// kernels) 168 and 429 us, 3.2 and 1.9 TB/s of what has to move.
//
// The weight's gradient: every thread keeps its columns' sums over all the
// rows its workgroup walks, the teams of a workgroup are joined through LDS,
// and a second kernel sums the workgroups' partials in a fixed order: no
// atomics, so the same inputs give the same bits.
#include "net.h"

namespace sla {
namespace net {
namespace {

constexpr int kNormBlock = 256;

// Sum over a team of TEAM threads, in every thread of it.  Teams of more than
// a wave are the whole workgroup and go through LDS (`red`, one float per
// wave; the caller alternates between two such arrays, so that one barrier
// is enough).
template <int TEAM, typename V>
__device__ __forceinline__ V team_sum(V v, V* red) {
  if constexpr (TEAM <= kWave) {
    return lane_sum<TEAM>(v);
  } else {
    v = lane_sum<kWave>(v);
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = v;
    __syncthreads();
    V s = 0;
#pragma unroll
    for (int i = 0; i < TEAM / kWave; ++i) s += red[i];
    return s;
  }
}
// Two sums behind one barrier.
template <int TEAM>
__device__ __forceinline__ float2 team_sums(float a, float b, float2* red) {
  if constexpr (TEAM <= kWave) {
    return make_float2(lane_sum<TEAM>(a), lane_sum<TEAM>(b));
  } else {
    a = lane_sum<kWave>(a);
    b = lane_sum<kWave>(b);
    if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = make_float2(a, b);
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < TEAM / kWave; ++i) s.x += red[i].x, s.y += red[i].y;
    return s;
  }
}

// A row's statistics as the gradient keeps them: the mean from x0 or from zero,
// 1 / sqrt(var + eps), negative in the second case.
__device__ __forceinline__ float2 pack_stats(double mean, float x0, float rstd) {
  const double far = mean - double(x0);
  return fabs(mean) < fabs(far) ? make_float2(float(mean), -rstd) : make_float2(float(far), rstd);
}
// The same for a mean c + more.
__device__ __forceinline__ float2 pack_stats(float c, float more, float x0, float rstd) {
  const float far = c - x0;
  return fabsf(c) < fabsf(far) ? make_float2(c + more, -rstd) : make_float2(far + more, rstd);
}
struct Stats {
  float from, mean, rstd;
  __device__ __forceinline__ float normal(float x) const { return (x - from - mean) * rstd; }
};
template <typename T>
__device__ __forceinline__ Stats row_stats(const float2& s, const T* x) {
  const bool zero = __float_as_uint(s.y) >> 31;
  return {zero ? 0.f : float(x[0]), s.x, zero ? -s.y : s.y};
}

template <typename T, typename W, int TEAM, int NV>
__global__ __launch_bounds__(kNormBlock) void k_layer_norm(
    const T* __restrict__ x, int64_t ldx, int64_t rows, int cols, const W* __restrict__ w,
    const W* __restrict__ b, float eps, T* __restrict__ y, float2* __restrict__ stats) {
  constexpr int V = kVec<T>;
  constexpr int kTeams = kNormBlock / TEAM;
  __shared__ float red[kNormBlock / kWave];
  __shared__ float2 reds[kNormBlock / kWave];
  const int lane = threadIdx.x % TEAM;
  const float inv = 1.f / float(cols);
  float wv[NV][V], bv[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TEAM + lane) * V;
    if (w) load_f32<V>(w + c, cols - c, wv[j]);
    if (b) load_f32<V>(b + c, cols - c, bv[j]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!w) wv[j][i] = 1.f;
      if (!b) bv[j][i] = 0.f;
    }
  }
  // every thread runs the same number of turns: a workgroup-wide team has
  // barriers inside
  for (int64_t r0 = int64_t(blockIdx.x) * kTeams; r0 < rows; r0 += int64_t(gridDim.x) * kTeams) {
    const int64_t r = r0 + threadIdx.x / TEAM;
    const bool on = r < rows;
    const T* xr = x + (on ? r : r0) * ldx;
    float v[NV][V];
    float s = 0.f;
    const float x0 = float(xr[0]);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TEAM + lane) * V;
      load_f32<V>(xr + c, cols - c, v[j]);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TEAM + lane) * V;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (c + i < cols) s += v[j][i] - x0;
    }
    const float mid = x0 + team_sum<TEAM>(s, red) * inv;
    float e = 0.f, q = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TEAM + lane) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        v[j][i] -= mid;
        if (c + i < cols) {
          e += v[j][i];
          q += v[j][i] * v[j][i];
        }
      }
    }
    const float2 eq = team_sums<TEAM>(e, q, reds);
    const float more = eq.x * inv, var = eq.y * inv - more * more;
    const float rstd = 1.f / sqrtf((var < 0.f ? 0.f : var) + eps);
    if (!on) continue;
    if (stats && lane == 0) stats[r] = pack_stats(mid, more, x0, rstd);
    T* yr = y + r * cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TEAM + lane) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] = (v[j][i] - more) * rstd * wv[j][i] + bv[j][i];
      store_f32<V>(yr + c, cols - c, v[j]);
    }
  }
}

// part: [2][gridDim.x][cols] sums of dw and db over the workgroup's rows.
template <typename T, typename W, int TEAM, int NV>
__global__ __launch_bounds__(kNormBlock) void k_layer_norm_grad(
    const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx, int64_t rows,
    int cols, const W* __restrict__ w, const float2* __restrict__ stats, T* __restrict__ dx,
    float* __restrict__ part) {
  constexpr int V = kVec<T>;
  constexpr int kTeams = kNormBlock / TEAM;
  // the joined sums of the teams: one team's columns at a time
  __shared__ float join[kTeams > 1 ? kNormBlock * V : 1];
  __shared__ float red[2][kNormBlock / kWave];
  const int lane = threadIdx.x % TEAM;
  const float inv = 1.f / float(cols);
  float wv[NV][V], aw[NV][V], ab[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (j * TEAM + lane) * V;
    if (w) load_f32<V>(w + c, cols - c, wv[j]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (!w) wv[j][i] = 1.f;
      aw[j][i] = ab[j][i] = 0.f;
    }
  }
  for (int64_t r0 = int64_t(blockIdx.x) * kTeams; r0 < rows; r0 += int64_t(gridDim.x) * kTeams) {
    const int64_t r = r0 + threadIdx.x / TEAM;
    const bool on = r < rows;
    const int64_t rr = on ? r : r0;
    const Stats st = row_stats(stats[rr], x + rr * ldx);
    float n[NV][V], g[NV][V];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TEAM + lane) * V;
      load_f32<V>(x + rr * ldx + c, cols - c, n[j]);
      // a team past the last row adds nothing to the sums
      load_f32<V>(dy + rr * lddy + c, on ? cols - c : 0, g[j]);
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TEAM + lane) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        n[j][i] = on && c + i < cols ? st.normal(n[j][i]) : 0.f;
        aw[j][i] += g[j][i] * n[j][i];
        ab[j][i] += g[j][i];
        g[j][i] *= wv[j][i];
        s1 += g[j][i];
        s2 += g[j][i] * n[j][i];
      }
    }
    if (!dx) continue;
    s1 = team_sum<TEAM>(s1, red[0]) * inv;
    s2 = team_sum<TEAM>(s2, red[1]) * inv;
    if (!on) continue;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TEAM + lane) * V;
#pragma unroll
      for (int i = 0; i < V; ++i) g[j][i] = st.rstd * (g[j][i] - s1 - n[j][i] * s2);
      store_f32<V>(dx + r * cols + c, cols - c, g[j]);
    }
  }
  if (!part) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* out = part + (int64_t(which) * gridDim.x + blockIdx.x) * cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * TEAM + lane) * V;
      float t[V];
#pragma unroll
      for (int i = 0; i < V; ++i) t[i] = which ? ab[j][i] : aw[j][i];
      if constexpr (kTeams > 1) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < V; ++i) join[i * kNormBlock + threadIdx.x] = t[i];
        __syncthreads();
        if (threadIdx.x < TEAM) {
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float s = 0.f;
            for (int k = 0; k < kTeams; ++k) s += join[i * kNormBlock + k * TEAM + lane];
            t[i] = s;
          }
          store_f32<V>(out + c, cols - c, t);
        }
      } else {
        store_f32<V>(out + c, cols - c, t);
      }
    }
  }
}

// Rows wider than a workgroup's registers: the row is read again for each
// pass (it comes from the cache), and the columns' sums are left to
// k_norm_columns.  A thread adds up cols / 256 values one after the other, so
// these sums are fp64 (in fp32 2e7 columns were 3.8e-6 off).  The gradient sums
// the mean again in place of the rounded one it gets: n is the same number in
// both directions.
template <typename T>
__device__ __forceinline__ double wide_mean(const T* __restrict__ x, int64_t cols, double* red) {
  double s = 0;
#pragma unroll 8   // loads under way at a time
  for (int64_t c = threadIdx.x; c < cols; c += kNormBlock) s += double(float(x[c]));
  return team_sum<kNormBlock>(s, red) / double(cols);
}
template <typename T>
__device__ __forceinline__ float wide_normal(T x, double mean, float rstd) {
  return float(double(float(x)) - mean) * rstd;
}
template <typename T, typename W>
__global__ __launch_bounds__(kNormBlock) void k_layer_norm_wide(
    const T* __restrict__ x, int64_t ldx, int64_t cols, const W* __restrict__ w,
    const W* __restrict__ b, float eps, T* __restrict__ y, float2* __restrict__ stats) {
  __shared__ double red[2][kNormBlock / kWave];
  const int64_t r = blockIdx.x;
  const T* xr = x + r * ldx;
  const double mean = wide_mean(xr, cols, red[0]);
  double q = 0;
#pragma unroll 8
  for (int64_t c = threadIdx.x; c < cols; c += kNormBlock) {
    const double d = double(float(xr[c])) - mean;
    q += d * d;
  }
  const double var = team_sum<kNormBlock>(q, red[1]) / double(cols);
  const float rstd = float(1 / sqrt(var + double(eps)));
  if (stats && threadIdx.x == 0) stats[r] = pack_stats(mean, float(xr[0]), rstd);
#pragma unroll 8
  for (int64_t c = threadIdx.x; c < cols; c += kNormBlock)
    y[r * cols + c] = T(wide_normal(xr[c], mean, rstd) * (w ? float(w[c]) : 1.f) +
                        (b ? float(b[c]) : 0.f));
}

template <typename T, typename W>
__global__ __launch_bounds__(kNormBlock) void k_layer_norm_grad_wide(
    const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx, int64_t cols,
    const W* __restrict__ w, const float2* __restrict__ stats, T* __restrict__ dx) {
  __shared__ double red[3][kNormBlock / kWave];
  const int64_t r = blockIdx.x;
  const float rstd = fabsf(stats[r].y);
  const double mean = wide_mean(x + r * ldx, cols, red[2]);
  double a1 = 0, a2 = 0;
#pragma unroll 8
  for (int64_t c = threadIdx.x; c < cols; c += kNormBlock) {
    const float t = float(dy[r * lddy + c]) * (w ? float(w[c]) : 1.f);
    a1 += double(t);
    a2 += double(t * wide_normal(x[r * ldx + c], mean, rstd));
  }
  const float s1 = float(team_sum<kNormBlock>(a1, red[0]) / double(cols));
  const float s2 = float(team_sum<kNormBlock>(a2, red[1]) / double(cols));
#pragma unroll 8
  for (int64_t c = threadIdx.x; c < cols; c += kNormBlock) {
    const float t = float(dy[r * lddy + c]) * (w ? float(w[c]) : 1.f);
    dx[r * cols + c] = T(rstd * (t - s1 - wide_normal(x[r * ldx + c], mean, rstd) * s2));
  }
}

// The wide rows' means for k_norm_columns.
template <typename T>
__global__ __launch_bounds__(kNormBlock) void k_norm_means(const T* __restrict__ x, int64_t ldx,
                                                           int64_t cols, double* __restrict__ mean) {
  __shared__ double red[kNormBlock / kWave];
  const double m = wide_mean(x + blockIdx.x * ldx, cols, red);
  if (threadIdx.x == 0) mean[blockIdx.x] = m;
}
// Column sums of the wide rows: a thread per column, a slab of rows per
// workgroup row (the partials of k_layer_norm_grad's layout).
template <typename T>
__global__ __launch_bounds__(kNormBlock) void k_norm_columns(
    const T* __restrict__ dy, int64_t lddy, const T* __restrict__ x, int64_t ldx, int64_t rows,
    int64_t cols, const float2* __restrict__ stats, const double* __restrict__ mean,
    float* __restrict__ part) {
  const int64_t c = int64_t(blockIdx.x) * kNormBlock + threadIdx.x;
  if (c >= cols) return;
  float aw = 0.f, ab = 0.f;
  for (int64_t r = blockIdx.y; r < rows; r += gridDim.y) {
    const float g = float(dy[r * lddy + c]);
    aw += g * wide_normal(x[r * ldx + c], mean[r], fabsf(stats[r].y));
    ab += g;
  }
  part[int64_t(blockIdx.y) * cols + c] = aw;
  part[(int64_t(gridDim.y) + blockIdx.y) * cols + c] = ab;
}

// dw and db from `slabs` partial rows each: 16 columns by 64 lines of
// threads, so that a line reads 64 bytes and the longest chain of loads is
// slabs / 64.  A workgroup walks the columns: one for every 16 of them would be
// a launch of 2^32 threads from 2^26 columns on, and the runtime starts such a
// launch without its upper bits.
constexpr int kJoinCols = 16, kJoinLines = 64, kJoinGroups = 1 << 16;
template <typename W>
__global__ __launch_bounds__(kJoinCols* kJoinLines) void k_norm_join(
    const float* __restrict__ part, int slabs, int64_t cols, W* __restrict__ dw,
    W* __restrict__ db) {
  __shared__ float s[kJoinLines][kJoinCols + 1];
  const int cc = threadIdx.x % kJoinCols, line = threadIdx.x / kJoinCols;
  const float* p = part + int64_t(blockIdx.y) * slabs * cols;
  W* out = blockIdx.y ? db : dw;
  for (int64_t c0 = int64_t(blockIdx.x) * kJoinCols; c0 < cols;
       c0 += int64_t(gridDim.x) * kJoinCols) {
    const int64_t c = c0 + cc;
    float v = 0.f;
    if (c < cols) {
#pragma unroll 4
      for (int i = line; i < slabs; i += kJoinLines) v += p[int64_t(i) * cols + c];
    }
    s[line][cc] = v;
    __syncthreads();
#pragma unroll
    for (int d = kJoinLines / 2; d > 0; d >>= 1) {
      if (line < d) s[line][cc] += s[line + d][cc];
      __syncthreads();
    }
    if (line == 0 && c < cols && out) out[c] = W(s[0][cc]);
    __syncthreads();
  }
}

// The team for rows of `cols` elements: the smallest that holds a row in one
// or two 16-byte vectors a lane, then up to 8 vectors a lane.
struct NormPlan {
  int team, nv;  // nv == 0: the wide kernels
};
NormPlan norm_plan(int64_t cols, int vec) {
  const int64_t v = div_up(cols, vec);
  if (v <= 8) return {8, 1};
  if (v <= 16) return {16, 1};
  if (v <= 32) return {32, 1};
  if (v <= 64) return {64, 1};
  if (v <= 128) return {64, 2};
  if (v <= 256) return {64, 4};
  if (v <= 512) return {256, 2};
  if (v <= 1024) return {256, 4};
  if (v <= 2048) return {256, 8};
  return {256, 0};
}

int norm_grid(int64_t rows, const NormPlan& p, int per_cu) {
  const int64_t want = div_up(rows, kNormBlock / p.team);
  const int64_t most = int64_t(device_cus()) * per_cu;
  return int(want < most ? want : most);
}

constexpr int kFwdPerCu = 8, kGradPerCu = 4;
constexpr int kWideSlabs = 64;

int norm_slabs(int64_t rows, int64_t cols, int vec) {
  const NormPlan p = norm_plan(cols, vec);
  if (p.nv) return norm_grid(rows, p, kGradPerCu);
  return int(rows < kWideSlabs ? rows : kWideSlabs);
}

// The workspace: the partial sums, behind them the wide rows' means.
int64_t slab_bytes(int slabs, int64_t cols) { return int64_t(slabs) * cols * 8; }
int64_t norm_bytes(int64_t rows, int64_t cols, int vec) {
  return slab_bytes(norm_slabs(rows, cols, vec), cols) +
         (norm_plan(cols, vec).nv ? 0 : rows * int64_t(sizeof(double)));
}

template <typename F>
sla_status with_team(const NormPlan& p, F&& f) {
  if (p.team == 8) return f(std::integral_constant<int, 8>(), std::integral_constant<int, 1>());
  if (p.team == 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
  if (p.team == 32) return f(std::integral_constant<int, 32>(), std::integral_constant<int, 1>());
  if (p.team == 64) {
    if (p.nv == 1) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>());
    if (p.nv == 2) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 2>());
    return f(std::integral_constant<int, 64>(), std::integral_constant<int, 4>());
  }
  if (p.nv == 2) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 2>());
  if (p.nv == 4) return f(std::integral_constant<int, 256>(), std::integral_constant<int, 4>());
  return f(std::integral_constant<int, 256>(), std::integral_constant<int, 8>());
}

// f(element, weight): the weight is of x's type or fp32.
template <typename F>
sla_status with_types(sla_type t, sla_type wt, F&& f) {
  if (t == SLA_F32) return f(float(), float());
  if (t == SLA_F16) return wt == SLA_F32 ? f(_Float16(), float()) : f(_Float16(), _Float16());
  return wt == SLA_F32 ? f(__bf16(), float()) : f(__bf16(), __bf16());
}

sla_status norm_args(const char* who, int64_t rows, int64_t cols, int64_t ld, sla_type t,
                     sla_type wt) {
  SLA_NET_REQUIRE(valid_type(t) && (wt == t || wt == SLA_F32), "%s: unknown or mixed types", who);
  SLA_NET_REQUIRE(rows >= 0 && rows < (int64_t(1) << 31), "%s: rows out of range", who);
  SLA_NET_REQUIRE(cols >= 1 && cols < (int64_t(1) << 31), "%s: cols out of range", who);
  SLA_NET_REQUIRE(ld >= cols, "%s: row stride %lld below cols %lld", who, (long long)ld,
                  (long long)cols);
  return SLA_OK;
}

}  // namespace
}  // namespace net
}  // namespace sla

using namespace sla;
using namespace sla::net;

extern "C" {

sla_status sla_layer_norm(const void* x, int64_t ldx, int64_t rows, int64_t cols, sla_type type,
                          const void* weight, const void* bias, sla_type wtype, double eps,
                          void* y, float* stats, hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  SLA_TRY(norm_args("sla_layer_norm", rows, cols, ldx, type, wtype));
  SLA_NET_REQUIRE(eps >= 0 && eps < 1e30, "sla_layer_norm: eps must be non-negative");
  if (rows == 0) return SLA_OK;
  SLA_NET_REQUIRE(x && y, "sla_layer_norm: x or y is NULL");
  return with_types(type, wtype, [&](auto te, auto we) -> sla_status {
    using T = decltype(te);
    using W = decltype(we);
    const NormPlan p = norm_plan(cols, kVec<T>);
    if (p.nv == 0) {
      k_layer_norm_wide<T, W><<<int(rows), kNormBlock, 0, stream>>>(
          (const T*)x, ldx, cols, (const W*)weight, (const W*)bias, float(eps), (T*)y,
          (float2*)stats);
      LAUNCH_CHECK();
      return SLA_OK;
    }
    return with_team(p, [&](auto team, auto nv) -> sla_status {
      k_layer_norm<T, W, team.value, nv.value>
          <<<norm_grid(rows, p, kFwdPerCu), kNormBlock, 0, stream>>>(
              (const T*)x, ldx, rows, int(cols), (const W*)weight, (const W*)bias, float(eps),
              (T*)y, (float2*)stats);
      LAUNCH_CHECK();
      return SLA_OK;
    });
  });
  SLA_NET_END
}

sla_status sla_layer_norm_work(int64_t rows, int64_t cols, sla_type type, int64_t* bytes_host) {
  SLA_NET_BEGIN
  clear_error();
  SLA_TRY(norm_args("sla_layer_norm_work", rows, cols, cols, type, type));
  SLA_NET_REQUIRE(bytes_host, "sla_layer_norm_work: bytes_host is NULL");
  *bytes_host = norm_bytes(rows, cols, int(16 / type_size(type)));
  return SLA_OK;
  SLA_NET_END
}

sla_status sla_layer_norm_grad(const void* dy, int64_t lddy, const void* x, int64_t ldx,
                               int64_t rows, int64_t cols, sla_type type, const void* weight,
                               sla_type wtype, const float* stats, void* dx, void* dweight,
                               void* dbias, void* work, int64_t work_bytes, hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  SLA_TRY(norm_args("sla_layer_norm_grad", rows, cols, ldx < lddy ? ldx : lddy, type, wtype));
  const bool sums = dweight || dbias;
  SLA_NET_REQUIRE(rows == 0 || (dy && x && stats), "sla_layer_norm_grad: dy, x or stats is NULL");
  return with_types(type, wtype, [&](auto te, auto we) -> sla_status {
    using T = decltype(te);
    using W = decltype(we);
    const int slabs = norm_slabs(rows, cols, kVec<T>);
    SLA_NET_REQUIRE(!sums || slabs == 0 || (work && work_bytes >= norm_bytes(rows, cols, kVec<T>)),
                    "sla_layer_norm_grad: workspace too small (sla_layer_norm_work)");
    float* part = sums ? (float*)work : nullptr;
    const NormPlan p = norm_plan(cols, kVec<T>);
    if (rows && p.nv == 0) {
      if (dx) {
        k_layer_norm_grad_wide<T, W><<<int(rows), kNormBlock, 0, stream>>>(
            (const T*)dy, lddy, (const T*)x, ldx, cols, (const W*)weight, (const float2*)stats,
            (T*)dx);
        LAUNCH_CHECK();
      }
      if (sums) {
        double* means = (double*)((char*)work + slab_bytes(slabs, cols));
        k_norm_means<T><<<int(rows), kNormBlock, 0, stream>>>((const T*)x, ldx, cols, means);
        LAUNCH_CHECK();
        k_norm_columns<T><<<dim3(int(div_up(cols, kNormBlock)), slabs), kNormBlock, 0, stream>>>(
            (const T*)dy, lddy, (const T*)x, ldx, rows, cols, (const float2*)stats, means, part);
        LAUNCH_CHECK();
      }
    } else if (rows) {
      SLA_TRY(with_team(p, [&](auto team, auto nv) -> sla_status {
        k_layer_norm_grad<T, W, team.value, nv.value><<<slabs, kNormBlock, 0, stream>>>(
            (const T*)dy, lddy, (const T*)x, ldx, rows, int(cols), (const W*)weight,
            (const float2*)stats, (T*)dx, part);
        LAUNCH_CHECK();
        return SLA_OK;
      }));
    }
    if (sums) {
      const int64_t want = div_up(cols, kJoinCols);
      const int groups = int(want < kJoinGroups ? want : kJoinGroups);
      k_norm_join<W><<<dim3(groups, 2), kJoinCols * kJoinLines, 0, stream>>>(
          part, slabs, cols, (W*)dweight, (W*)dbias);
      LAUNCH_CHECK();
    }
    return SLA_OK;
  });
  SLA_NET_END
}

}  // extern "C"
