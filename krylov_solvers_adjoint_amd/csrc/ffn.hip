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
// That adds half a step to dx and dW (2.35e-3 instead of 1.7e-3 in bf16).
// fp16 has not the range besides: products of a small dh fell below 2^-24, of
// a large one passed 65504, where dx and dW are ordinary numbers.  Its da and
// db are held times a power of two, taken from a bound on the largest of them
// (k_bound), and dx and dW are multiplied back.  All sums are fp32.
#include "product.h"

namespace sla {
namespace net {
namespace {


sla_status ffn_args(const char* who, int64_t rows, int64_t inner, int64_t outer, int64_t ldx,
                    sla_type type, int act) {
  SLA_NET_REQUIRE(valid_type(type), "%s: unknown type", who);
  SLA_NET_REQUIRE(act == SLA_ACT_SILU || act == SLA_ACT_GELU || act == SLA_ACT_RELU,
                  "%s: unknown activation", who);
  SLA_NET_REQUIRE(rows >= 0 && rows < (int64_t(1) << 31), "%s: rows out of range", who);
  SLA_NET_REQUIRE(inner >= 1 && inner < (int64_t(1) << 22) && outer >= 1 &&
                      outer < (int64_t(1) << 22), "%s: inner or outer out of range", who);
  SLA_NET_REQUIRE(ldx >= inner, "%s: row stride below inner", who);
  return SLA_OK;
}

// The workspace: da, db, fp16's scale and what it comes from, then the sums of a
// split product (dx and the weights' gradients use the same place one after the
// other).
constexpr int64_t kScaleBytes = 256 + kBoundGroups * 12;
int64_t factor_bytes(int64_t rows, int64_t outer, int es) {
  return div_up(rows * outer * es, 256) * 256;
}
int64_t grad_bytes(int64_t rows, int64_t inner, int64_t outer, int es) {
  const int64_t x = split_bytes(rows, inner, outer, 2, 1, 1, es);
  const int64_t w = split_bytes(outer, inner, rows, 1, 2, 2, es);
  return 2 * factor_bytes(rows, outer, es) + kScaleBytes + (x > w ? x : w);
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
  SLA_NET_BEGIN
  clear_error();
  SLA_TRY(ffn_args("sla_gated_ffn", rows, inner, outer, ldx, type, act));
  if (rows == 0) return SLA_OK;
  SLA_NET_REQUIRE(x && w_gate && w_up && h, "sla_gated_ffn: an argument is NULL");
  return with_type(type, [&](auto te) -> sla_status {
    using T = decltype(te);
    Product g{};
    g.who = "sla_gated_ffn";
    g.A[0] = x;
    g.B[0] = w_gate;
    g.B[1] = w_up;
    g.lda = ldx;
    g.ldb = inner;
    g.M = rows, g.N = outer, g.K = inner, g.parts = g.outputs = 1;
    g.C[0] = h;
    g.ldc = outer;
    g.act = act;
    return launch_product<T, false, false, EPI_GATE>(g, stream);
  });
  SLA_NET_END
}

sla_status sla_gated_ffn_work(int64_t rows, int64_t inner, int64_t outer, sla_type type,
                              int64_t* bytes_host) {
  SLA_NET_BEGIN
  clear_error();
  SLA_TRY(ffn_args("sla_gated_ffn_work", rows, inner, outer, inner, type, SLA_ACT_SILU));
  SLA_NET_REQUIRE(bytes_host, "sla_gated_ffn_work: bytes_host is NULL");
  *bytes_host = grad_bytes(rows, inner, outer, int(type_size(type)));
  return SLA_OK;
  SLA_NET_END
}

sla_status sla_gated_ffn_grad(const void* dh, int64_t lddh, const void* x, int64_t ldx,
                              const void* w_gate, const void* w_up, int64_t rows, int64_t inner,
                              int64_t outer, sla_type type, int act, void* dx, void* dw_gate,
                              void* dw_up, void* work, int64_t work_bytes, hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  SLA_TRY(ffn_args("sla_gated_ffn_grad", rows, inner, outer, ldx, type, act));
  SLA_NET_REQUIRE(lddh >= outer, "sla_gated_ffn_grad: row stride of dh below outer");
  SLA_NET_REQUIRE(rows == 0 || (dh && x && w_gate && w_up),
                  "sla_gated_ffn_grad: an argument is NULL");
  SLA_NET_REQUIRE((dw_gate == nullptr) == (dw_up == nullptr),
                  "sla_gated_ffn_grad: both weights' gradients or neither");
  const int es = int(type_size(type));
  const int64_t size = factor_bytes(rows, outer, es);
  SLA_NET_REQUIRE(rows == 0 || (work && work_bytes >= grad_bytes(rows, inner, outer, es)),
                  "sla_gated_ffn_grad: workspace too small (sla_gated_ffn_work)");
  return with_type(type, [&](auto te) -> sla_status {
    using T = decltype(te);
    Product g{};
    g.who = "sla_gated_ffn";
    g.A[0] = x;
    g.B[0] = w_gate;
    g.B[1] = w_up;
    g.lda = ldx;
    g.ldb = inner;
    g.M = rows, g.N = outer, g.K = inner, g.parts = g.outputs = 1;
    g.dh = dh;
    g.lddh = lddh;
    g.C[0] = work;
    g.C[1] = (char*)work + size;
    g.ldc = outer;
    g.act = act;
    float* scale = nullptr;
    if (std::is_same<T, _Float16>::value && rows) {
      scale = (float*)((char*)work + 2 * size);
      const int64_t lines = rows > outer ? rows : outer;
      const int groups = int(lines < 4 * kBoundGroups ? div_up(lines, 4) : kBoundGroups);
      const Lines ld = {(const _Float16*)dh, lddh, rows, int(outer)};
      const Lines lx = {(const _Float16*)x, ldx, rows, int(inner)};
      const Lines lg = {(const _Float16*)w_gate, inner, outer, int(inner)};
      const Lines lu = {(const _Float16*)w_up, inner, outer, int(inner)};
      k_bound<<<groups, kProductBlock, 0, stream>>>(ld, lx, lg, lu, scale + 64);
      LAUNCH_CHECK();
      k_scale<false><<<1, kWave, 0, stream>>>(scale + 64, groups, scale);
      LAUNCH_CHECK();
    }
    g.scale = scale;
    SLA_TRY((launch_product<T, false, false, EPI_GATE_GRAD>(g, stream)));
    float* part = (float*)((char*)work + 2 * size + kScaleBytes);
    if (dx) {
      Product p{};
      p.who = g.who;
      p.A[0] = g.C[0], p.A[1] = g.C[1];
      p.B[0] = w_gate, p.B[1] = w_up;
      p.lda = outer, p.ldb = inner;
      p.M = rows, p.N = inner, p.K = outer, p.parts = 2, p.outputs = 1;
      p.part = part;
      p.scale = scale;
      p.C[0] = dx;
      p.ldc = inner;
      SLA_TRY((launch_product<T, false, true, EPI_STORE>(p, stream)));
    }
    if (dw_gate) {
      Product p{};
      p.who = g.who;
      p.A[0] = g.C[0], p.A[1] = g.C[1];
      p.B[0] = p.B[1] = x;
      p.lda = outer, p.ldb = ldx;
      p.M = outer, p.N = inner, p.K = rows, p.parts = 1, p.outputs = 2;
      p.part = part;
      p.scale = scale;
      p.C[0] = dw_gate, p.C[1] = dw_up;
      p.ldc = inner;
      SLA_TRY((launch_product<T, true, true, EPI_STORE>(p, stream)));
    }
    return SLA_OK;
  });
  SLA_NET_END
}

}  // extern "C"
