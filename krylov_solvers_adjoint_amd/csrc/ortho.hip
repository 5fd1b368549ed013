// Newton-Schulz products that orthogonalise a matrix.
//
//   X = M / (|M|_F + eps), then for every step
//   A = X X^T    B = b A + c A A    X <- a X + B X       (rows <= cols)
//   A = X^T X    B = b A + c A A    X <- a X + X B       (rows > cols)
//
// A step maps every singular value s to a s + b s^3 + c s^5 and leaves the
// singular vectors.  Small singular values grow by a factor of a a step, and
// every rounding on the way with them: factors of 16 bits would leave errors of
// a^steps half steps.  The factors are therefore held in two fp16 parts, hi and
// the rest lo, 22 bits, and the products of fp16's matrix instructions hi hi +
// hi lo + lo hi take their place, with sums in fp32 (lo lo, 2^-22 of a term, is
// left out): three instructions where the fp32 ones take sixteen times as long.
// X, A and B are held times 2^12, 2^10 and 2^8: entries up to 16, 64 and 256
// fit (X's and A's entries are at most the largest singular value and its
// square), and lo's last bit lies 2^-36, 2^-34 and 2^-32 below one.
//
// Planes are padded to multiples of 32 with zeros, which every product keeps.
#include "product.h"

namespace sla {
namespace net {
namespace {

constexpr int kNormGroups = 256;   // partial sums of a matrix at most
constexpr int kPad = 32;
constexpr float kUpX = 4096.f;

int64_t padded(int64_t n) { return div_up(n, kPad) * kPad; }

// Sums of squares in fp64 (fp32's squares would leave its range): a workgroup
// takes rows in turn, a second kernel joins them in order.
template <typename T>
__global__ __launch_bounds__(256) void k_ortho_norm(const T* __restrict__ m, int64_t ld,
                                                    int64_t rows, int64_t cols,
                                                    double* __restrict__ parts) {
  __shared__ double red[4];
  const T* p = m + int64_t(blockIdx.y) * rows * ld;
  double s = 0;
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = threadIdx.x * 4; c < cols; c += 1024) {
      float v[4];
      load_f32<4>(p + r * ld + c, cols - c, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) s += double(v[j]) * double(v[j]);
    }
  s = lane_sum<kWave>(s);
  if (threadIdx.x % kWave == 0) red[threadIdx.x / kWave] = s;
  __syncthreads();
  if (threadIdx.x == 0)
    parts[int64_t(blockIdx.y) * gridDim.x + blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// X times 2^12 in two planes [rows][ldx], zeros where the padding is.  steps ==
// 0 leaves X itself, rounded.
template <typename T>
__global__ __launch_bounds__(256) void k_ortho_enter(const T* __restrict__ m, int64_t ld,
                                                     int64_t rows, int64_t cols, double eps,
                                                     const double* __restrict__ parts, int groups,
                                                     _Float16* __restrict__ hi,
                                                     _Float16* __restrict__ lo, int64_t prows,
                                                     int64_t pcols, T* __restrict__ out) {
  const double* q = parts + int64_t(blockIdx.y) * groups;
  double sum = 0;
  for (int i = threadIdx.x % kWave; i < groups; i += kWave) sum += q[i];
  sum = lane_sum<kWave>(sum);
  const double up = (out ? 1.0 : double(kUpX)) / (sqrt(sum) + eps);
  const int64_t quads = pcols / 4;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < prows * quads;
       i += int64_t(gridDim.x) * 256) {
    const int64_t r = i / quads, c = i % quads * 4;
    const int64_t have = r < rows ? cols - c : 0;
    float v[4], h[4], l[4];
    load_f32<4>(m + (int64_t(blockIdx.y) * rows + (have > 0 ? r : 0)) * ld + (have > 0 ? c : 0),
                have, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // the quotient once rounded to fp32; nothing is divided where nothing is
      const float x = j < have ? float(double(v[j]) * up) : 0.f;
      v[j] = x;
      h[j] = float(_Float16(x));
      l[j] = x - h[j];
    }
    if (out) {
      if (have > 0) store_f32<4>(out + (int64_t(blockIdx.y) * rows + r) * cols + c, have, v);
    } else {
      const int64_t at = (int64_t(blockIdx.y) * prows + r) * pcols + c;
      store_f32<4>(hi + at, 4, h);
      store_f32<4>(lo + at, 4, l);
    }
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
struct OrthoPlan {
  int64_t count, rows, cols, prows, pcols, side;   // side: of A and B
  int64_t plane, square;                           // bytes of X's planes, of A's
  int64_t parts, sums, total;
};
int64_t up256(int64_t n) { return div_up(n, 256) * 256; }

sla_status ortho_plan(const char* who, int64_t count, int64_t rows, int64_t cols, sla_type type,
                      OrthoPlan& p) {
  SLA_NET_REQUIRE(valid_type(type), "%s: unknown type", who);
  SLA_NET_REQUIRE(count >= 0 && count < 65536, "%s: more than 65535 matrices", who);
  SLA_NET_REQUIRE(rows >= 1 && rows <= 65536 && cols >= 1 && cols <= 65536,
                  "%s: rows or cols out of range (1 to 65536)", who);
  p.count = count, p.rows = rows, p.cols = cols;
  p.prows = padded(rows), p.pcols = padded(cols);
  p.side = p.prows < p.pcols ? p.prows : p.pcols;
  p.plane = up256(count * p.prows * p.pcols * 2);
  p.square = up256(count * p.side * p.side * 2);
  p.parts = up256(count * kNormGroups * 8);
  const int64_t a = split_bytes(p.side, p.side, rows > cols ? p.prows : p.pcols, 3, int(count),
                                rows > cols ? 2 : 0, 2);
  const int64_t b = split_bytes(p.side, p.side, p.side, 3, int(count), 0, 2);
  const int64_t c = split_bytes(p.prows, p.pcols, p.side, 3, int(count), rows > cols ? 0 : 1, 2);
  p.sums = up256(a > b ? (a > c ? a : c) : (b > c ? b : c));
  p.total = 4 * p.plane + 4 * p.square + p.parts + p.sums;
  return SLA_OK;
}

}  // namespace
}  // namespace net
}  // namespace sla

using namespace sla;
using namespace sla::net;

extern "C" {

sla_status sla_orthogonalise_work(int64_t count, int64_t rows, int64_t cols, sla_type type,
                                  int64_t* bytes_host) {
  SLA_NET_BEGIN
  clear_error();
  OrthoPlan p;
  SLA_TRY(ortho_plan("sla_orthogonalise_work", count, rows, cols, type, p));
  SLA_NET_REQUIRE(bytes_host, "sla_orthogonalise_work: bytes_host is NULL");
  *bytes_host = p.total;
  return SLA_OK;
  SLA_NET_END
}

sla_status sla_orthogonalise(const void* m, int64_t ldm, int64_t count, int64_t rows,
                             int64_t cols, sla_type type, int steps, const double* coefficients,
                             double eps, void* x, void* work, int64_t work_bytes,
                             hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  OrthoPlan p;
  SLA_TRY(ortho_plan("sla_orthogonalise", count, rows, cols, type, p));
  SLA_NET_REQUIRE(ldm >= cols, "sla_orthogonalise: row stride below cols");
  SLA_NET_REQUIRE(steps >= 0 && steps <= 64, "sla_orthogonalise: 0 to 64 steps");
  SLA_NET_REQUIRE(steps == 0 || coefficients, "sla_orthogonalise: coefficients is NULL");
  for (int i = 0; i < 3 * steps; ++i)
    SLA_NET_REQUIRE(coefficients[i] >= -64 && coefficients[i] <= 64,
                    "sla_orthogonalise: a coefficient is outside of -64 .. 64");
  SLA_NET_REQUIRE(eps >= 0 && eps < 1e30, "sla_orthogonalise: eps must be non-negative");
  if (count == 0) return SLA_OK;
  SLA_NET_REQUIRE(m && x, "sla_orthogonalise: m or x is NULL");
  SLA_NET_REQUIRE(work && work_bytes >= p.total,
                  "sla_orthogonalise: workspace too small (sla_orthogonalise_work)");
  char* at = (char*)work;
  auto take = [&](int64_t bytes) {
    char* q = at;
    at += bytes;
    return (_Float16*)q;
  };
  _Float16 *X[2][2], *A[2], *B[2];
  for (auto& plane : X)
    for (auto& q : plane) q = take(p.plane);
  for (auto& q : A) q = take(p.square);
  for (auto& q : B) q = take(p.square);
  double* parts = (double*)take(p.parts);
  float* sums = (float*)at;
  const int groups = int(rows < kNormGroups ? rows : kNormGroups);
  SLA_TRY(with_type(type, [&](auto te) -> sla_status {
    using T = decltype(te);
    k_ortho_norm<T><<<dim3(groups, int(count)), 256, 0, stream>>>((const T*)m, ldm, rows, cols,
                                                                  parts);
    LAUNCH_CHECK();
    const int64_t want = div_up(p.prows * p.pcols / 4, 256);
    k_ortho_enter<T><<<dim3(int(want < 4096 ? want : 4096), int(count)), 256, 0, stream>>>(
        (const T*)m, ldm, rows, cols, eps, parts, groups, X[0][0], X[0][1], p.prows, p.pcols,
        steps ? nullptr : (T*)x);
    LAUNCH_CHECK();
    return SLA_OK;
  }));
  const bool tall = rows > cols;
  for (int i = 0; i < steps; ++i) {
    const double* c = coefficients + 3 * i;
    _Float16 **from = X[i % 2], **to = X[(i + 1) % 2];
    Product g{};
    g.who = "sla_orthogonalise";
    g.parts = 3;
    g.outputs = int(count);
    g.part = sums;
    auto factors = [](Product& q, _Float16** a, _Float16** b) {
      q.A[0] = q.A[1] = a[0], q.A[2] = a[1];
      q.B[0] = q.B[2] = b[0], q.B[1] = b[1];
    };
    auto square = [&](Product& q) {
      q.M = q.N = q.ldc = p.side;
      q.zc = p.side * p.side;
    };
    Product q = g;   // A
    factors(q, from, from);
    q.lda = q.ldb = p.pcols;
    q.za = q.zb = p.prows * p.pcols;
    q.K = tall ? p.prows : p.pcols;
    square(q);
    q.C[0] = A[0], q.C[1] = A[1];
    q.beta = 0x1p-14f;
    if (tall) SLA_TRY((launch_product<_Float16, true, true, EPI_POLY>(q, stream)));
    else SLA_TRY((launch_product<_Float16, false, false, EPI_POLY>(q, stream)));

    q = g;   // B (A is symmetric: its rows are its columns)
    factors(q, A, A);
    q.lda = q.ldb = p.side;
    q.za = q.zb = p.side * p.side;
    q.K = p.side;
    square(q);
    q.C[0] = B[0], q.C[1] = B[1];
    q.D[0] = A[0], q.D[1] = A[1];
    q.alpha = float(c[1] * 0x1p-2);
    q.beta = float(c[2] * 0x1p-12);
    SLA_TRY((launch_product<_Float16, false, false, EPI_POLY>(q, stream)));

    q = g;   // X
    q.M = p.prows, q.N = p.pcols, q.K = p.side;
    q.ldc = p.pcols;
    q.zc = p.prows * p.pcols;
    q.D[0] = from[0], q.D[1] = from[1];
    q.alpha = float(c[0]);
    q.beta = 0x1p-8f;
    q.C[0] = to[0], q.C[1] = to[1];
    if (i + 1 == steps) {
      q.last = x;
      q.last_type = type;
      q.last_rows = rows, q.last_cols = cols;
      q.alpha *= 1 / kUpX, q.beta *= 1 / kUpX;
    }
    if (tall) {
      factors(q, from, B);
      q.lda = p.pcols, q.za = p.prows * p.pcols;
      q.ldb = p.side, q.zb = p.side * p.side;
      SLA_TRY((launch_product<_Float16, false, false, EPI_POLY>(q, stream)));
    } else {
      factors(q, B, from);
      q.lda = p.side, q.za = p.side * p.side;
      q.ldb = p.pcols, q.zb = p.prows * p.pcols;
      SLA_TRY((launch_product<_Float16, false, true, EPI_POLY>(q, stream)));
    }
  }
  return SLA_OK;
  SLA_NET_END
}

}  // extern "C"
