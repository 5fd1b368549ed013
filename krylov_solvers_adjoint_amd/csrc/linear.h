// The projection's gradients in one pass over x and dy, for narrow projections of
// many rows (linear_narrow.hip).
#pragma once

#include "net.h"

namespace sla {
namespace net {

struct NarrowGrad {
  const void *x, *dy, *w, *bias;   // the weight and bias as sla_linear takes them
  int64_t ldx, lddy, rows;
  int inner, outer, bias_f32, act, want_w;
  const float* scale;
  void* dx;
  void *dw, *db;   // may be none, each
  float* part;     // the workgroups' sums; none if neither dw nor db is wanted
};

// Where one pass pays: the general products read x and dy three times, in four
// launches or more.  64 x 64, bias, silu, one pass against them: 64 rows fp32 15.3
// and 16.2 us, 1000 rows 19 and 27, 10^5 rows 47 and 80; bf16 12.6 and 13.7, 13.5
// and 22, 28 and 48; 16 rows 14.7 and 14.8.  Up to 64 x 128 and 128 x 64 one pass was
// faster too (10^6 rows fp32 414 us against 495 and 354 against 484, bf16 274 against
// 263 and 192 against 273), but its kernels took 100 s more to compile: left out for
// that alone.
constexpr int64_t kNarrow = 64, kNarrowRows = 64;
constexpr int kNarrowGroups = 512;
inline bool narrow(int64_t rows, int64_t inner, int64_t outer) {
  return inner <= kNarrow && outer <= kNarrow && rows >= kNarrowRows;
}
inline int narrow_pad(int64_t n) { return n <= 32 ? 32 : 64; }
inline int narrow_groups(int64_t rows) {
  const int64_t n = div_up(rows, 128);
  return int(n < kNarrowGroups ? n : kNarrowGroups);
}
inline int64_t narrow_bytes(int64_t rows, int64_t inner, int64_t outer) {
  const int64_t np = narrow_pad(outer), kp = narrow_pad(inner);
  return narrow_groups(rows) * (np * kp + np) * 4;
}
sla_status launch_narrow(const NarrowGrad& g, sla_type type, hipStream_t stream);

}  // namespace net
}  // namespace sla
