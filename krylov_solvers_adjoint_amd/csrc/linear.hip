// A projection with its bias, activation and residual in the epilogue, and its
// gradients.
//
//   z = x W^T + bias   y = residual + f(z)           f: none, silu, gelu or relu
//   dz = dy f'(z)      dx = dz W   dW = dz^T x   dbias = sum_rows dz
//
// The residual's gradient is dy.  Without an activation dz is dy; with one, z is
// computed again (its product's epilogue makes dz of it) rather than kept.  dz
// is then rounded once to the inputs' type, the type of the factors of the
// products that follow, which adds half a step to dx and dW, and to the terms of
// dbias, which are read from it (in the one-pass kernel they are summed before the
// rounding); fp16's is held times a power of two that the largest |dy| gives, for
// its range (no activation is steeper than 1.13).  All sums are fp32.
//
// Measured: 16384 x 4096 x 1024 bf16 with a residual 124 us forward (1.1 PFLOP/s),
// dx 135, dW 124 + 12 (two splits); 5000 x 771 x 1403 fp16 41 to 48 us a product:
// the sizes ask for 128 tiles (440 of them, 26 us at widths that are multiples of
// 8), whose stores of odd rows take 7 us more; padded copies of the operands
// changed nothing.  4 x 4096 x 1024 bf16: 8 us, 64 workgroups that read 8.4 MB.
#include "linear.h"
#include "product.h"

namespace sla {
namespace net {
namespace {

// Column sums of dz: a team of lanes has 16 bytes a lane of a row, the other
// teams of the workgroup and the slabs of rows take rows in turn; teams and slabs
// are joined in order.  10^6 x 64 fp32: 40 us (6.4 TB/s); lanes of one row a wave
// had left 48 of 64 idle, 312 us.
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

sla_status linear_args(const char* who, int64_t rows, int64_t inner, int64_t outer, int64_t ldx,
                       sla_type type, sla_type btype, int act) {
  SLA_NET_REQUIRE(valid_type(type) && (btype == type || btype == SLA_F32),
                  "%s: unknown or mixed types", who);
  SLA_NET_REQUIRE(act == SLA_ACT_SILU || act == SLA_ACT_GELU || act == SLA_ACT_RELU ||
                      act == SLA_ACT_NONE, "%s: unknown activation", who);
  // more would be 2^32 threads in tiles of 128 rows
  SLA_NET_REQUIRE(rows >= 0 && rows <= (int64_t(1) << 31) - 128, "%s: rows out of range", who);
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
  // (few rows: one launch that keeps its sums on the chip)
  z.forward = rows <= kFewRows ? 0 : split_bytes(rows, outer, inner, 1, 1, 0, es);
  z.scale = act != SLA_ACT_NONE && type == SLA_F16 ? 256 + up256(kBoundGroups * 12) : 0;
  if (narrow(rows, inner, outer)) {
    z.sums = narrow_bytes(rows, inner, outer);
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
      const NarrowGrad g = {x, dy, weight, bias, ldx, lddy, rows, int(inner), int(outer),
                            btype == SLA_F32, act, dweight != nullptr, scale, dx, dweight, dbias,
                            dweight || dbias ? sums : nullptr};
      SLA_TRY(launch_narrow(g, type, stream));
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
