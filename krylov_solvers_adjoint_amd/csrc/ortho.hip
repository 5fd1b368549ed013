// Newton-Schulz products that orthogonalise a matrix.
//
//   X = M / (|M|_F + eps), then for every step
//   A = X X^T    B = a I + b A + c A A    X <- B X       (rows <= cols)
//   A = X^T X    B = a I + b A + c A A    X <- X B       (rows > cols)
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
// Lines are padded to multiples of 32 with zeros, which every product keeps.
//
// Measured, five steps: 1024 x 4096 321 to 347 us on four machines (A 18 + 6 in seven
// splits, B 12, X 27 a step; 70 Gflop, three times that for the parts: 0.65 PFLOP/s), 4096 x 4096 4.07 ms
// (1.0 PFLOP/s), 1403 x 515 169 us.  X of 1024 x 4096 without its parts, timed in a
// copy: products alone 17 us (10 at the instructions' rate, launch and first loads
// the rest), loads and LDS reads beside them 6, the way out 4.  Short products are
// bound by launches and by what a CU has under way (128 KB) against the way from
// the last cache: B of 1024 x 1024 takes 12 us for 3 Gflop.
#include "mfma.h"

namespace sla {
namespace net {
namespace {

constexpr int kNormGroups = 256;   // partial sums of a matrix at most
constexpr int kPad = 32;
constexpr float kUpX = 4096.f;
constexpr int kMostSteps = 64;

int64_t padded(int64_t n) { return div_up(n, kPad) * kPad; }

// Where element c of a line lies: 32 elements' hi parts, then their lo parts.
// So the 32 k of a step are one cache line of a row.
__host__ __device__ constexpr int64_t part_at(int64_t c) { return c / 32 * 64 + c % 32; }

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
                                                     _Float16* __restrict__ planes,
                                                     int64_t prows, int64_t pcols,
                                                     T* __restrict__ out) {
  const double* q = parts + int64_t(blockIdx.y) * groups;
  double sum = 0;
  for (int i = threadIdx.x % kWave; i < groups; i += kWave) sum += q[i];
  sum = lane_sum<kWave>(sum);
  const double up = (out ? 1.0 : double(kUpX)) / (sqrt(sum) + eps);
  const uint32_t units = uint32_t(pcols / 8);   // of 8 columns; prows * units < 2^32
  const uint32_t all = uint32_t(prows) * units;
  for (uint32_t i = blockIdx.x * 256 + threadIdx.x; i < all; i += gridDim.x * 256) {
    const int64_t r = i / units, c = i % units * 8;
    const int64_t have = r < rows ? cols - c : 0;
    float v[8];
    load_f32<8>(m + (int64_t(blockIdx.y) * rows + (have > 0 ? r : 0)) * ld + (have > 0 ? c : 0),
                have, v);
    typedef _Float16 V8 __attribute__((ext_vector_type(8)));
    V8 h, l;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // the quotient once rounded to fp32; nothing is divided where nothing is
      const float x = j < have ? float(double(v[j]) * up) : 0.f;
      v[j] = x;
      h[j] = _Float16(x);
      l[j] = _Float16(x - float(h[j]));
    }
    if (out) {
      if (have > 0) store_f32<8>(out + (int64_t(blockIdx.y) * rows + r) * cols + c, have, v);
    } else {
      V8* to = (V8*)(planes + (int64_t(blockIdx.y) * prows + r) * 2 * pcols + part_at(c));
      to[0] = h;
      to[4] = l;
    }
  }
}

// One product of two-part factors in tiles of B x B.
struct Poly {
  const _Float16 *A, *B;         // AT: stored [k][row], else [row][k]; BT: likewise
  int64_t lda, ldb, za, zb;      // halves from line to line, from matrix to matrix
  int64_t M, N, K;               // multiples of 32
  const _Float16* D;             // laid out as C; may be none
  float alpha, beta, diagonal;   // C = alpha D + beta A B^T + diagonal I
  _Float16* C;
  int64_t ldc, zc;
  void* last;                    // where the result leaves rounded, [..][last_rows][last_cols]
  int last_type;
  int64_t last_rows, last_cols;
  int gx, gy, lower;             // tiles; lower: C is symmetric, its upper tiles are mirrored
  int splits;                    // of k; > 1: sums go to part, as the lanes hold them
  float* part;
};

// 32 k of W rows of one plane in LDS, in slots of 16 bytes.  Stored by row: a
// row's four slots are exchanged by the row; stored by k: pairs of a line's
// slots are exchanged by the line, so that the four lines and their
// neighbours 8 k further that half a wave reads at a time lie in different
// banks.  256 threads fill it by direct loads.
template <int W, bool TRANS>
struct Plane {
  static constexpr int kBytes = 64 * W, kLoads = W / 64, kLine = W / 8;
  static __device__ __forceinline__ int turn(int k) {
    return W == 128 ? (k & 3) | (k >> 3 & 1) << 2 : (k >> 1 & 1) | (k >> 3 & 1) << 1;
  }
  // load i of thread t: its offset in bytes from the step's first element
  static __device__ __forceinline__ int offset(int i, int t, int64_t ld, int64_t rows) {
    const int s = i * 256 + t;
    if constexpr (TRANS) {
      const int k = s / kLine, along = (s % kLine ^ 2 * turn(k)) * 8;
      return along < rows ? int((k * ld + part_at(along)) * 2) : kOutside;
    } else {
      const int row = s / 4;
      return row < rows ? int((row * ld + (s % 4 ^ (row >> 1 & 3)) * 8) * 2) : kOutside;
    }
  }
  // the lane's part of rows `base` + 16 j ...: kept addresses, j a constant
  struct Reader {
    int at[TRANS ? 4 : 1];
    __device__ __forceinline__ Reader(int base) {
      const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
      if constexpr (TRANS) {
        const int k = 8 * h + (l >> 2);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          at[j] = k * W * 2 + ((base / 16 + j) ^ turn(k)) * 32 + (l & 3) * 8;
      } else {
        at[0] = (base + l) * 64 + (h ^ (l >> 1 & 3)) * 16;
      }
    }
    __device__ __forceinline__ Unit<_Float16>::Vec read(const char* lds, int j) const {
      typedef Unit<_Float16>::Vec Vec;
      if constexpr (TRANS) {
        Vec v;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const auto c = read_column<_Float16>(lds + at[TRANS ? j : 0] + 4 * q * W * 2);
#pragma unroll
          for (int r = 0; r < 4; ++r) v[4 * q + r] = c[r];
        }
        return v;
      } else {
        return *reinterpret_cast<const Vec*>(lds + at[0] + j * 1024);
      }
    }
  };
};

// Tile `id` of all matrices' tiles.
__device__ __forceinline__ void place_poly(const Poly& g, int id, int& m, int& n, int& z) {
  const int tiles = g.lower ? g.gy * (g.gy + 1) / 2 : g.gx * g.gy;
  z = id / tiles;
  id -= z * tiles;
  if (g.lower) {
    m = int((sqrtf(8.f * float(id) + 1.f) - 1.f) * 0.5f);
    while (m * (m + 1) / 2 > id) --m;
    while ((m + 1) * (m + 2) / 2 <= id) ++m;
    n = id - m * (m + 1) / 2;
  } else {
    const int width = 8 * g.gx, group = id / width;
    const int rows = g.gy - group * 8 < 8 ? g.gy - group * 8 : 8;
    id -= group * width;
    m = group * 8 + id % rows;
    n = id / rows;
  }
  m = __builtin_amdgcn_readfirstlane(m);
  n = __builtin_amdgcn_readfirstlane(n);
  z = __builtin_amdgcn_readfirstlane(z);
}
// The workgroup's: each XCD gets a run of neighbouring tiles.
__device__ __forceinline__ void find_poly(const Poly& g, int& m, int& n, int& z, int& tile,
                                          int& split) {
  const int total = gridDim.x, b = blockIdx.x;
  const int xcd = b % kXcds, q = total / kXcds, r = total % kXcds;
  const int id = xcd * q + (xcd < r ? xcd : r) + b / kXcds;
  const int tiles = total / g.splits;   // of all matrices; an XCD has few splits' k
  tile = __builtin_amdgcn_readfirstlane(id % tiles);
  split = __builtin_amdgcn_readfirstlane(id / tiles);
  place_poly(g, tile, m, n, z);
}

// NR x NJ tiles of a wave's sums leave, from (row, col) on.  Planes leave 16
// bytes a lane; the mirrored ones by way of LDS (`lds`: kMirrorBytes of the
// wave's own).
template <int NR, int NJ>
constexpr int kMirrorBytes = 2 * 16 * NJ * (16 * NR + 8) * 2;
template <typename T, int NR, int NJ>
__device__ __forceinline__ void leave_rounded(const Poly& g, int64_t row, int64_t col, int z,
                                              const f32x4 (&u)[NR][NJ]) {
  const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int64_t r = row + 16 * i + l;
    if (r >= g.last_rows) continue;
    T* to = (T*)g.last + (z * g.last_rows + r) * g.last_cols;
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const int64_t c = col + 16 * j + 4 * h;
      const float v[4] = {u[i][j][0], u[i][j][1], u[i][j][2], u[i][j][3]};
      store_f32<4>(to + c, g.last_cols - c, v);
    }
  }
}
template <int NR, int NJ>
__device__ __forceinline__ void leave_poly(const Poly& g, int64_t row, int64_t col, int z,
                                           bool mirror, f32x4 (&u)[NR][NJ], char* lds) {
  typedef _Float16 V4 __attribute__((ext_vector_type(4)));
  const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
  // pairs of tiles, 32 columns, exist or not as a whole
  const int64_t first = z * g.zc + (row + l) * g.ldc + 2 * col + 16 * (h % 2) + 8 * (h / 2);
  auto is = [&](int i, int j) { return row + 16 * i < g.M && col + 16 * j < g.N; };
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) u[i][j][r] *= g.beta;
  if (g.D) {
    Quads d[2][NR][NJ / 2];
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < NJ; j += 2)
          d[p][i][j / 2] = *reinterpret_cast<const Quads*>(
              g.D + (is(i, j) ? first + 16 * i * g.ldc + 32 * j : 0) + 32 * p);
#pragma unroll
    for (int p = 1; p >= 0; --p)   // the small part first
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int j = 0; j < NJ; j += 2) {
          const Quads x = d[p][i][j / 2], y = side_by_side(Pair{x[0], x[1]}, Pair{x[2], x[3]});
          const V4 a = __builtin_bit_cast(V4, Pair{y[0], y[1]});
          const V4 b = __builtin_bit_cast(V4, Pair{y[2], y[3]});
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            u[i][j][r] += g.alpha * float(a[r]);
            u[i][j + 1][r] += g.alpha * float(b[r]);
          }
        }
  }
  if (g.diagonal != 0.f) {
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (row + 16 * i + l == col + 16 * j + 4 * h + r) u[i][j][r] += g.diagonal;
  }
  if (g.last) {
    if (g.last_type == SLA_F32) leave_rounded<float>(g, row, col, z, u);
    else if (g.last_type == SLA_F16) leave_rounded<_Float16>(g, row, col, z, u);
    else leave_rounded<__bf16>(g, row, col, z, u);
    return;
  }
  constexpr int kLine = 16 * NR + 8;   // halves of a mirrored line
#pragma unroll
  for (int i = 0; i < NR; ++i)
#pragma unroll
    for (int j = 0; j < NJ; j += 2) {
      Pair hi[2], lo[2];
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        V4 a, b;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          a[r] = _Float16(u[i][j + n][r]);
          b[r] = _Float16(u[i][j + n][r] - float(a[r]));
        }
        hi[n] = __builtin_bit_cast(Pair, a);
        lo[n] = __builtin_bit_cast(Pair, b);
        if (mirror) {
          _Float16* q = (_Float16*)lds + (16 * (j + n) + 4 * h) * kLine + 16 * i + l;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            q[r * kLine] = a[r];
            q[(16 * NJ + r) * kLine] = b[r];
          }
        }
      }
      if (is(i, j)) {
        Quads* to = reinterpret_cast<Quads*>(g.C + first + 16 * i * g.ldc + 32 * j);
        to[0] = side_by_side(hi[0], hi[1]);
        to[4] = side_by_side(lo[0], lo[1]);
      }
    }
  if (mirror) {
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the wave's own writes
    constexpr int kUnits = 2 * NR;                         // of 8 rows in a mirrored line
#pragma unroll
    for (int n = 0; n < 2 * 16 * NJ * kUnits / kWave; ++n) {
      const int s = n * kWave + threadIdx.x % kWave, line = s / kUnits, unit = s % kUnits;
      const int64_t c = col + line % (16 * NJ), r = row + unit * 8;
      if (c < g.N && r < g.M)
        *reinterpret_cast<Quads*>(g.C + z * g.zc + c * g.ldc + part_at(r) +
                                  line / (16 * NJ) * 32) =
            *reinterpret_cast<const Quads*>((const _Float16*)lds + line * kLine + unit * 8);
    }
  }
}

// Direct loads as send() makes them, from a buffer in scalar registers: 16 bytes
// a lane from offset at + part to lds + 16 lane.
typedef int Buffer __attribute__((ext_vector_type(4)));
__device__ __forceinline__ Buffer buffer_of(const char* p, int bytes) {
  const uint64_t q = reinterpret_cast<uint64_t>(uniform(p));
  return Buffer{int(q), int(q >> 32) & 0xffff, bytes, 0x00020000};
}
__device__ __forceinline__ void send_part(const Buffer& from, int at, int part, int lds) {
#if defined(__HIP_DEVICE_COMPILE__)
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
               :: "s"(lds), "v"(at), "s"(from), "n"(part) : "memory", "m0");
#pragma clang diagnostic pop
#endif
}

// KG groups of four waves take the steps of 32 k in turn, each with a ring of
// kDepth steps in LDS, and are added up at the end.  A wave has a quarter of the
// tile; the fragments of a step are read while the one before is multiplied.
template <int B, int KG>
struct PolyRing {
  static constexpr int kStep = 4 * 64 * B;                       // bytes of the four planes
  static constexpr int kDepth = KG * 4 * kStep <= 131072 ? 4 : 2;
  static constexpr int kBytes = KG * kDepth * kStep;
};
template <int B, int KG, bool AT, bool BT>
__global__ __launch_bounds__(256 * KG) void k_ortho_product(Poly g) {
  typedef Plane<B, AT> PA;
  typedef Plane<B, BT> PB;
  typedef Unit<_Float16>::Vec Vec;
  typedef PolyRing<B, KG> Ring;
  constexpr int kDepth = Ring::kDepth, NI = B / 32, NJ = B / 32, kLoads = PA::kLoads;
  constexpr int kSends = 4 * kLoads;
  extern __shared__ __align__(1024) char smem[];
  const int t = threadIdx.x % 256;
  const int group = KG == 1 ? 0 : __builtin_amdgcn_readfirstlane(int(threadIdx.x) / 256);
  const int w = __builtin_amdgcn_readfirstlane(t / kWave);
  char* const ring = smem + group * kDepth * Ring::kStep;
  const int lds0 = __builtin_amdgcn_readfirstlane(
      int(reinterpret_cast<uintptr_t>((LdsPtr)(ring + w * 1024))));
  int m, n, z, tile, split;
  find_poly(g, m, n, z, tile, split);
  const int64_t m0 = int64_t(m) * B, n0 = int64_t(n) * B;
  const int all = int(g.K / 32), each = (all + g.splits - 1) / g.splits;
  const int begin = split * each, steps = begin + each < all ? begin + each : all;
  const int turns = begin < steps ? (steps - begin + KG - 1) / KG : 0;
  int oa[kLoads], ob[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    oa[i] = PA::offset(i, t, g.lda, g.M - m0);
    ob[i] = PB::offset(i, t, g.ldb, g.N - n0);
  }
  const char* a = (const char*)(g.A + z * g.za + (AT ? 2 * m0 : m0 * g.lda));
  const char* b = (const char*)(g.B + z * g.zb + (BT ? 2 * n0 : n0 * g.ldb));
  const int64_t ka = AT ? 64 * g.lda : 128, kb = BT ? 64 * g.ldb : 128;   // bytes of a step
  // the loads of turn i; behind the last one zeros come in their place (a buffer
  // without bytes)
  Buffer from_a, from_b;
  int to = 0;
  auto aim = [&](int i, int slot) {
    const int step = begin + i * KG + group;
    const int bytes = step < steps ? 0x7fffffff : 0;
    from_a = buffer_of(a + step * ka, bytes);
    from_b = buffer_of(b + step * kb, bytes);
    to = lds0 + slot * Ring::kStep;
  };
  auto send_one = [&](int n) {   // one of kSends: both parts of a line one after the other
    const int p = n % 2, j = n / 4;
    if (n / 2 % 2) send_part(from_b, ob[j], 64 * p, to + (2 + p) * PA::kBytes + j * 4096);
    else send_part(from_a, oa[j], 64 * p, to + p * PA::kBytes + j * 4096);
  };
  const typename PA::Reader ra((w / 2) * (B / 2));
  const typename PB::Reader rb((w % 2) * (B / 2));
  f32x4 acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
  Vec fa[2][2][NI], fb[2][2][NJ];
  constexpr int kReads = 2 * (NI + NJ);
  auto read_one = [&](const char* from, int f, int n) {   // one of kReads: what comes first first
    const int p = n / (NI + NJ), k = n % (NI + NJ);
    if (k < NJ) fb[f][p][k] = rb.read(from + (2 + p) * PA::kBytes, k);
    else fa[f][p][k - NJ] = ra.read(from + p * PA::kBytes, k - NJ);
  };
#pragma unroll
  for (int i = 0; i < kDepth; ++i) {
    aim(i, i);
#pragma unroll
    for (int n = 0; n < kSends; ++n) send_one(n);
  }
  landed<(kDepth - 1) * kSends>();
#pragma unroll
  for (int n = 0; n < kReads; ++n) read_one(ring, 0, n);
  // One wave a SIMD issues everything itself: the reads and loads go between
  // the products, a few instructions in the shadow of two of them.
  constexpr int kSlots = NI * NJ * 3 / 2, kItems = kReads + kSends;
  for (int i = 0; i < turns; i += kDepth) {
#pragma unroll
    for (int d = 0; d < kDepth; ++d) {
      if (i + d >= turns) break;
      const int f = d % 2;
      // the next turn's tiles have come and every wave has read this one's
      landed<(kDepth - 2) * kSends>();
      aim(i + d + kDepth, d);
      const char* next = ring + (d + 1) % kDepth * Ring::kStep;
#pragma unroll
      for (int n = 0; n < kSlots; ++n) {
#pragma unroll
        for (int k = n * kItems / kSlots; k < (n + 1) * kItems / kSlots; ++k) {
          if (k % 3 == 2) send_one(k / 3);
          else read_one(next, f ^ 1, k - k / 3);
        }
#pragma unroll
        for (int k = 2 * n; k < 2 * n + 2; ++k) {
          // four sums or more between two products of one
          constexpr int kRows = NJ >= 4 ? 1 : 2, kTurn = 3 * kRows * NJ;
          const int q = k % kTurn / (kRows * NJ), c = k % (kRows * NJ);
          const int row = k / kTurn * kRows + c / NJ, col = c % NJ;
          mma16(acc[row][col], fa[f][q == 2][row], fb[f][q == 1][col]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // the last loads must not come in after the workgroup has given its LDS back
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __syncthreads();

  constexpr int kOwn = NI / KG;   // rows of tiles that a group finishes
  if constexpr (KG == 2) {
    f32x4* give = (f32x4*)smem + (group * 4 + w) * kOwn * NJ * kWave + t % kWave;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        give[(i * NJ + j) * kWave] = group ? acc[i][j] : acc[kOwn + i][j];
    __syncthreads();
    const f32x4* take = (const f32x4*)smem + ((group ^ 1) * 4 + w) * kOwn * NJ * kWave + t % kWave;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const f32x4 o = take[(i * NJ + j) * kWave];
        acc[i][j] = group ? o + acc[kOwn + i][j] : acc[i][j] + o;
      }
    __syncthreads();
  }
  f32x4 own[kOwn][NJ];
#pragma unroll
  for (int i = 0; i < kOwn; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) own[i][j] = acc[i][j];
  if (g.splits > 1) {
    const int64_t tiles = gridDim.x / g.splits;   // of all matrices
    f32x4* part = (f32x4*)g.part +
                  ((int64_t(split) * tiles + tile) * 4 + w) * NI * NJ * kWave + t % kWave;
#pragma unroll
    for (int i = 0; i < kOwn; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) part[((i + group * kOwn) * NJ + j) * kWave] = own[i][j];
    return;
  }
  leave_poly<kOwn, NJ>(g, m0 + (w / 2) * (B / 2) + 16 * group * kOwn, n0 + (w % 2) * (B / 2), z,
                       g.lower && m != n, own,
                       smem + (group * 4 + w) * kMirrorBytes<kOwn, NJ>);
}

// The sums of a split product, in the order of the splits: a wave has a row of
// a quarter's tiles.
template <int B>
__global__ __launch_bounds__(kWave) void k_ortho_join(Poly g) {
  constexpr int NI = B / 32, NJ = B / 32;
  __shared__ __align__(16) char lds[kMirrorBytes<1, NJ>];
  const int tiles = gridDim.x / (4 * NI);
  const int tile = blockIdx.x / (4 * NI), w = blockIdx.x / NI % 4, i = blockIdx.x % NI;
  int m, n, z;
  place_poly(g, tile, m, n, z);
  const f32x4* part = (const f32x4*)g.part + (int64_t(tile) * 4 + w) * NI * NJ * kWave +
                      i * NJ * kWave + threadIdx.x;
  f32x4 sum[1][NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) sum[0][j] = part[j * kWave];
#pragma unroll 4
  for (int k = 1; k < g.splits; ++k) {
    part += int64_t(tiles) * 4 * NI * NJ * kWave;
#pragma unroll
    for (int j = 0; j < NJ; ++j) sum[0][j] += part[j * kWave];
  }
  leave_poly<1, NJ>(g, int64_t(m) * B + (w / 2) * (B / 2) + 16 * i,
                    int64_t(n) * B + (w % 2) * (B / 2), z, g.lower && m != n, sum, lds);
}

// Small matrices (12 of 128 x 64 fp32: 25 us, of which a step takes 4, a chain of
// five barriers): one workgroup has a matrix in LDS, the smaller side as rows
// (at most S, the other side at most N), through all steps.  A wave has 16 x 16
// tiles of the products; results wait in registers until every wave has read
// the factors that they replace.
struct Steps {
  float a[kMostSteps], b[kMostSteps], c[kMostSteps];
};
template <int S, int N>
struct Small {
  static constexpr int kLineX = N + 16, kLineQ = S + 16;   // halves; 32 bytes against the banks
  static constexpr int kPlaneX = S * kLineX, kPlaneQ = S * kLineQ;
  static constexpr int kBytes = 2 * (kPlaneX + kPlaneQ) * 2;
  static constexpr int kSquare = S / 16 * (S / 16) / 16, kWide = S / 16 * (N / 16) / 16;
};
constexpr int kSmallBlock = 1024;
template <typename T, int S, int N>
__global__ __launch_bounds__(kSmallBlock) void k_ortho_small(const T* __restrict__ m, int64_t ld,
                                                             int rows, int cols, double eps,
                                                             int steps, Steps by,
                                                             T* __restrict__ x) {
  typedef Small<S, N> L;
  typedef Unit<_Float16>::Vec Vec;
  typedef _Float16 V4 __attribute__((ext_vector_type(4)));
  extern __shared__ __align__(16) char smem[];
  __shared__ double red[kSmallBlock / kWave];
  _Float16* const X = (_Float16*)smem;
  _Float16* const Q = X + 2 * L::kPlaneX;
  const int t = threadIdx.x, l = t % 16, h = t % kWave / 16;
  const int w = __builtin_amdgcn_readfirstlane(t / kWave);
  const bool tall = rows > cols;
  const int side = tall ? cols : rows, wide = tall ? rows : cols;
  const int tiles = (wide + 31) / 32 * 2;   // tiles along X's rows
  m += blockIdx.x * rows * ld;
  x += int64_t(blockIdx.x) * rows * cols;
  double sum = 0;
  for (int i = t; i < rows * cols; i += kSmallBlock) {
    const double v = double(float(m[i / cols * ld + i % cols]));
    sum += v * v;
  }
  sum = lane_sum<kWave>(sum);
  if (t % kWave == 0) red[w] = sum;
  for (int i = t; i < 2 * L::kPlaneX / 8; i += kSmallBlock) ((Vec*)X)[i] = Vec{};
  __syncthreads();
  sum = 0;
#pragma unroll
  for (int i = 0; i < kSmallBlock / kWave; ++i) sum += red[i];
  if (steps == 0) {
    const double by_norm = 1 / (sqrt(sum) + eps);
    for (int i = t; i < rows * cols; i += kSmallBlock)
      x[i] = T(float(double(float(m[i / cols * ld + i % cols])) * by_norm));
    return;
  }
  const double up = double(kUpX) / (sqrt(sum) + eps);
  for (int i = t; i < rows * cols; i += kSmallBlock) {
    const int r = i / cols, c = i % cols;
    const float v = float(double(float(m[r * ld + c])) * up);
    _Float16* to = X + (tall ? c * L::kLineX + r : r * L::kLineX + c);
    to[0] = _Float16(v);
    to[L::kPlaneX] = _Float16(v - float(to[0]));
  }
  __syncthreads();
  // a line's part of 8 k; 8 k of a column
  auto row_of = [&](const _Float16* p, int line, int base, int k) {
    return *reinterpret_cast<const Vec*>(p + (base + l) * line + k + 8 * h);
  };
  auto column_of = [&](const _Float16* p, int line, int base, int k) {
    Vec v;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const auto c = read_column<_Float16>(
          (const char*)(p + (k + 8 * h + 4 * q + (l >> 2)) * line + base + (l & 3) * 4));
#pragma unroll
      for (int r = 0; r < 4; ++r) v[4 * q + r] = c[r];
    }
    return v;
  };
  // the three products of two-part factors, a sum each
  auto multiply = [&](f32x4 (&acc)[3], const Vec (&a)[2], const Vec (&b)[2]) {
    mma16(acc[0], a[0], b[0]);
    mma16(acc[1], a[0], b[1]);
    mma16(acc[2], a[1], b[0]);
  };
  auto put = [&](_Float16* to, int plane, const f32x4& v) {
    V4 a, b;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      a[r] = _Float16(v[r]);
      b[r] = _Float16(v[r] - float(a[r]));
    }
    *(V4*)to = a;
    *(V4*)(to + plane) = b;
  };
  const int squares = (side + 15) / 16;   // tiles along A's rows that hold anything
  const int ks = (side + 31) / 32 * 32;
  for (int step = 0; step < steps; ++step) {
    f32x4 sq[L::kSquare];
#pragma unroll
    for (int n = 0; n < L::kSquare; ++n) {   // A
      const int tile = w + 16 * n, i = tile / (S / 16), j = tile % (S / 16);
      f32x4 acc[3] = {};
      if (i < squares && j < squares)
        for (int k = 0; k < 16 * tiles; k += 32) {
          Vec a[2], b[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            a[p] = row_of(X + p * L::kPlaneX, L::kLineX, 16 * i, k);
            b[p] = row_of(X + p * L::kPlaneX, L::kLineX, 16 * j, k);
          }
          multiply(acc, a, b);
        }
      sq[n] = (acc[0] + (acc[1] + acc[2])) * 0x1p-14f;
      put(Q + (16 * i + l) * L::kLineQ + 16 * j + 4 * h, L::kPlaneQ, sq[n]);
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < L::kSquare; ++n) {   // B
      const int tile = w + 16 * n, i = tile / (S / 16), j = tile % (S / 16);
      f32x4 acc[3] = {};
      if (i < squares && j < squares)
        for (int k = 0; k < ks; k += 32) {
          Vec a[2], b[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            a[p] = row_of(Q + p * L::kPlaneQ, L::kLineQ, 16 * i, k);
            b[p] = row_of(Q + p * L::kPlaneQ, L::kLineQ, 16 * j, k);
          }
          multiply(acc, a, b);
        }
      sq[n] = sq[n] * (by.b[step] * 0x1p-2f) +
              (acc[0] + (acc[1] + acc[2])) * (by.c[step] * 0x1p-12f);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (16 * i + l == 16 * j + 4 * h + r) sq[n][r] += by.a[step] * 0x1p8f;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < L::kSquare; ++n) {
      const int tile = w + 16 * n, i = tile / (S / 16), j = tile % (S / 16);
      put(Q + (16 * i + l) * L::kLineQ + 16 * j + 4 * h, L::kPlaneQ, sq[n]);
    }
    __syncthreads();
    f32x4 out[L::kWide];
#pragma unroll
    for (int n = 0; n < L::kWide; ++n) {   // X
      const int tile = w + 16 * n, i = tile % (S / 16), j = tile / (S / 16);
      f32x4 acc[3] = {};
      if (i < squares && j < tiles)
        for (int k = 0; k < ks; k += 32) {
          Vec a[2], b[2];
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            a[p] = row_of(Q + p * L::kPlaneQ, L::kLineQ, 16 * i, k);
            b[p] = column_of(X + p * L::kPlaneX, L::kLineX, 16 * j, k);
          }
          multiply(acc, a, b);
        }
      out[n] = (acc[0] + (acc[1] + acc[2])) * 0x1p-8f;
    }
    const bool last = step + 1 == steps;
    if (!last) __syncthreads();
#pragma unroll
    for (int n = 0; n < L::kWide; ++n) {
      const int tile = w + 16 * n, i = tile % (S / 16), j = tile / (S / 16);
      if (j >= tiles) continue;
      const int r = 16 * i + l, c = 16 * j + 4 * h;
      if (!last) {
        put(X + r * L::kLineX + c, L::kPlaneX, out[n]);
      } else if (r < side) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (c + q < wide)
            x[tall ? (c + q) * cols + r : r * cols + c + q] = T(out[n][q] * (1 / kUpX));
      }
    }
    if (!last) __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
// Tiles of 128 where they fill the card: 1024 x 4096 in all 342 us instead of 401
// with 64 (one machine, side by side), 2048 x 2048 795 instead of 905, 4096 x 4096 4.07 ms instead of 5.8.  Fewer
// long sums are split (A of 1024 x 4096: 18 + 6 us instead of 34 in tiles of 64), short
// ones not (K = 1024: 14 + 6 instead of 12).
constexpr int64_t kTilesFor128 = 200, kTilesToSplit = 24, kLongSums = 2048;
// Tiles and splits of a product.
struct PolyPlan {
  int tile, splits;
  int64_t tiles, bytes;
};
PolyPlan plan_poly(int64_t M, int64_t N, int64_t K, bool lower, int64_t count) {
  auto tiles_of = [&](int64_t b) {
    const int64_t gy = div_up(M, b), gx = div_up(N, b);
    return (lower ? gy * (gy + 1) / 2 : gx * gy) * count;
  };
  PolyPlan p{64, 1, tiles_of(64), 0};
  const int64_t t = tiles_of(128), steps = K / 32;
  if (t >= kTilesFor128) {
    p = {128, 1, t, 0};
  } else if (t >= kTilesToSplit && K > kLongSums) {
    const int64_t s = 256 / t < steps / 4 ? 256 / t : steps / 4;
    if (s > 1) p = {128, int(s), t, s * t * 128 * 128 * 4};
  }
  return p;
}

template <typename T, int S, int N>
sla_status start_small(const void* m, int64_t ldm, int64_t count, int64_t rows, int64_t cols,
                       double eps, int steps, const Steps& by, void* x, hipStream_t stream) {
  auto* kernel = k_ortho_small<T, S, N>;
  SLA_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                  hipFuncAttributeMaxDynamicSharedMemorySize,
                                  Small<S, N>::kBytes));
  kernel<<<int(count), kSmallBlock, Small<S, N>::kBytes, stream>>>(
      (const T*)m, ldm, int(rows), int(cols), eps, steps, by, (T*)x);
  LAUNCH_CHECK();
  return SLA_OK;
}
// Whether one workgroup's LDS holds a matrix.  Against the general products, five
// steps: 64 x 64 20 us and 68, 128 x 128 77 and 80 (64 of them 80 and 97, 400 of them
// 173 and 343), 64 x 512 86 and 81; no workspace.
bool small_ortho(int64_t rows, int64_t cols) {
  const int64_t side = rows < cols ? rows : cols, wide = rows < cols ? cols : rows;
  return (side <= 64 && wide <= 512) || (side <= 128 && wide <= 128);
}

struct OrthoPlan {
  int64_t count, rows, cols, prows, pcols, side;   // side: of A and B
  int64_t plane, square;                           // bytes of X's planes, of A's
  int64_t parts, total;
};
int64_t up256(int64_t n) { return div_up(n, 256) * 256; }

sla_status ortho_plan(const char* who, int64_t count, int64_t rows, int64_t cols, sla_type type,
                      OrthoPlan& p) {
  SLA_NET_REQUIRE(valid_type(type), "%s: unknown type", who);
  SLA_NET_REQUIRE(count >= 0 && count < 65536, "%s: more than 65535 matrices", who);
  SLA_NET_REQUIRE(rows >= 1 && rows <= 65536 && cols >= 1 && cols <= 65536,
                  "%s: rows or cols out of range (1 to 65536)", who);
  p = {};
  if (small_ortho(rows, cols)) return SLA_OK;   // needs no workspace
  p.count = count, p.rows = rows, p.cols = cols;
  p.prows = padded(rows), p.pcols = padded(cols);
  p.side = p.prows < p.pcols ? p.prows : p.pcols;
  p.plane = up256(count * p.prows * p.pcols * 4);
  p.square = up256(count * p.side * p.side * 4);
  p.parts = up256(count * kNormGroups * 8);
  const int64_t a = plan_poly(p.side, p.side, rows > cols ? p.prows : p.pcols, true, count).bytes;
  const int64_t b = plan_poly(p.side, p.side, p.side, true, count).bytes;
  const int64_t c = plan_poly(p.prows, p.pcols, p.side, false, count).bytes;
  const int64_t sums = a > b ? (a > c ? a : c) : (b > c ? b : c);
  p.total = 2 * p.plane + 2 * p.square + p.parts + sums;
  return SLA_OK;
}

template <int B, int KG, bool AT, bool BT>
sla_status start_poly(Poly& g, const PolyPlan& p, hipStream_t stream) {
  g.gx = int(div_up(g.N, B)), g.gy = int(div_up(g.M, B));
  g.splits = p.splits;
  SLA_NET_REQUIRE(p.tiles * p.splits * 256 * KG < (int64_t(1) << 31),
                  "sla_orthogonalise: too large");
  auto* kernel = k_ortho_product<B, KG, AT, BT>;
  constexpr int lds = PolyRing<B, KG>::kBytes;
  SLA_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, lds));
  kernel<<<int(p.tiles * p.splits), 256 * KG, lds, stream>>>(g);
  LAUNCH_CHECK();
  if (p.splits > 1) {
    k_ortho_join<B><<<int(p.tiles * 4 * (B / 32)), kWave, 0, stream>>>(g);
    LAUNCH_CHECK();
  }
  return SLA_OK;
}
template <bool AT, bool BT>
sla_status launch_poly(Poly& g, int64_t count, hipStream_t stream) {
  const PolyPlan p = plan_poly(g.M, g.N, g.K, g.lower, count);
  if (p.tile == 128) return start_poly<128, 1, AT, BT>(g, p, stream);
  return start_poly<64, 2, AT, BT>(g, p, stream);
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
  SLA_NET_REQUIRE(steps >= 0 && steps <= kMostSteps, "sla_orthogonalise: 0 to 64 steps");
  SLA_NET_REQUIRE(steps == 0 || coefficients, "sla_orthogonalise: coefficients is NULL");
  for (int i = 0; i < 3 * steps; ++i)
    SLA_NET_REQUIRE(coefficients[i] >= -64 && coefficients[i] <= 64,
                    "sla_orthogonalise: a coefficient is outside of -64 .. 64");
  SLA_NET_REQUIRE(eps >= 0 && eps < 1e30, "sla_orthogonalise: eps must be non-negative");
  if (count == 0) return SLA_OK;
  SLA_NET_REQUIRE(m && x, "sla_orthogonalise: m or x is NULL");
  SLA_NET_REQUIRE(p.total == 0 || (work && work_bytes >= p.total),
                  "sla_orthogonalise: workspace too small (sla_orthogonalise_work)");
  if (small_ortho(rows, cols)) {
    Steps by{};
    for (int i = 0; i < steps; ++i) {
      by.a[i] = float(coefficients[3 * i]);
      by.b[i] = float(coefficients[3 * i + 1]);
      by.c[i] = float(coefficients[3 * i + 2]);
    }
    const int64_t side = rows < cols ? rows : cols, wide = rows < cols ? cols : rows;
    return with_type(type, [&](auto te) -> sla_status {
      using T = decltype(te);
      if (side > 64)
        return start_small<T, 128, 128>(m, ldm, count, rows, cols, eps, steps, by, x, stream);
      if (wide > 128)
        return start_small<T, 64, 512>(m, ldm, count, rows, cols, eps, steps, by, x, stream);
      return start_small<T, 64, 128>(m, ldm, count, rows, cols, eps, steps, by, x, stream);
    });
  }
  char* at = (char*)work;
  auto take = [&](int64_t bytes) {
    char* q = at;
    at += bytes;
    return (_Float16*)q;
  };
  _Float16* X[2] = {take(p.plane), nullptr};
  X[1] = take(p.plane);
  _Float16* const A = take(p.square);
  _Float16* const B = take(p.square);
  double* parts = (double*)take(p.parts);
  const int groups = int(rows < kNormGroups ? rows : kNormGroups);
  SLA_TRY(with_type(type, [&](auto te) -> sla_status {
    using T = decltype(te);
    k_ortho_norm<T><<<dim3(groups, int(count)), 256, 0, stream>>>((const T*)m, ldm, rows, cols,
                                                                  parts);
    LAUNCH_CHECK();
    const int64_t want = div_up(p.prows * p.pcols / 8, 256);
    k_ortho_enter<T><<<dim3(int(want < 1024 ? want : 1024), int(count)), 256, 0, stream>>>(
        (const T*)m, ldm, rows, cols, eps, parts, groups, X[0], p.prows, p.pcols,
        steps ? nullptr : (T*)x);
    LAUNCH_CHECK();
    return SLA_OK;
  }));
  const bool tall = rows > cols;
  for (int i = 0; i < steps; ++i) {
    const double* c = coefficients + 3 * i;
    _Float16 *from = X[i % 2], *to = X[(i + 1) % 2];
    const int64_t ldx = 2 * p.pcols, zx = p.prows * ldx, lda = 2 * p.side, za = p.side * lda;
    Poly g{};   // A
    g.part = (float*)at;
    g.A = g.B = from;
    g.lda = g.ldb = ldx;
    g.za = g.zb = zx;
    g.M = g.N = p.side;
    g.ldc = lda;
    g.zc = za;
    g.lower = 1;
    g.K = tall ? p.prows : p.pcols;
    g.C = A;
    g.beta = 0x1p-14f;
    if (tall) SLA_TRY((launch_poly<true, true>(g, count, stream)));
    else SLA_TRY((launch_poly<false, false>(g, count, stream)));

    g.A = g.B = A;   // B (A is symmetric: its rows are its columns)
    g.lda = g.ldb = lda;
    g.za = g.zb = za;
    g.K = p.side;
    g.C = B;
    g.D = A;
    g.alpha = float(c[1] * 0x1p-2);
    g.beta = float(c[2] * 0x1p-12);
    g.diagonal = float(c[0] * 0x1p8);
    SLA_TRY((launch_poly<false, false>(g, count, stream)));

    g.M = p.prows, g.N = p.pcols;   // X
    g.ldc = ldx;
    g.zc = zx;
    g.lower = 0;
    g.D = nullptr;
    g.diagonal = 0.f;
    g.C = to;
    g.beta = 0x1p-8f;
    if (i + 1 == steps) {
      g.last = x;
      g.last_type = type;
      g.last_rows = rows, g.last_cols = cols;
      g.beta *= 1 / kUpX;
    }
    if (tall) {
      g.A = from, g.lda = ldx, g.za = zx;
      g.B = B, g.ldb = lda, g.zb = za;
      SLA_TRY((launch_poly<false, false>(g, count, stream)));
    } else {
      g.A = B, g.lda = lda, g.za = za;
      g.B = from, g.ldb = ldx, g.zb = zx;
      SLA_TRY((launch_poly<false, true>(g, count, stream)));
    }
  }
  return SLA_OK;
  SLA_NET_END
}

}  // extern "C"
