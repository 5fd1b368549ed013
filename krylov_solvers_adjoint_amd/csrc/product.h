// Matrix products on the matrix cores, for the operators that are made of them:
// tiles staged through LDS, split sums, and what becomes of a tile's sums on
// their way out (the epilogues).
#pragma once

#include "mfma.h"

namespace sla {
namespace net {
namespace {


constexpr int kProductBlock = 256;
// Bytes of k a step covers (64 bytes: 32 16-bit values or 16 fp32), and the
// steps in LDS at a time.  Direct loads need the distance: with two steps of
// 128 bytes (as many bytes in all) every step waited for memory: dx and dW of
// 16384 x 1024 x 4096 took 316 and 330 us against 256 each.
template <bool DIRECT>
struct Ring {
  static constexpr int kStep = DIRECT ? 64 : 128, kDepth = DIRECT ? 4 : 2;
};

// What leaves for the sums a, b (and d, an array of the outputs' shape, where
// there is one):
//   GATE f(a) b   GATE_GRAD d b f'(a) and d f(a)   STORE a
//   LINEAR d + f(a + bias)   SLOPE d f'(a + bias)
enum { EPI_GATE, EPI_GATE_GRAD, EPI_STORE, EPI_LINEAR, EPI_SLOPE };
constexpr int kActNone = 3;   // beside the SLA_ACT_* (LINEAR alone)
constexpr bool two_weights(int epi) { return epi == EPI_GATE || epi == EPI_GATE_GRAD; }
constexpr bool takes_d(int epi) {
  return epi == EPI_GATE_GRAD || epi == EPI_LINEAR || epi == EPI_SLOPE;
}

// f(a) and f'(a).  FAST (16-bit tensors): exp and the reciprocal by their
// instructions (1 ulp each), and gelu's erfc(x) exp(x^2) (x >= 0) as t times a
// polynomial in t = 1 / (1 + 0.44 x), fitted to the least relative error over
// 0 .. 9.5, where exp(-x^2) ends: 5.2e-6 (1.1e-5 of f at a = -13, with exp's),
// a fortieth of fp16's half step.  The error has to be relative: f(a) falls
// with the tail, and a form that is good to 1.5e-7 of erf had left f(-6) eight
// half steps off.  The library's expf, erff and divide took 7 us of a 256 x
// 256 tile's 41.
template <int ACT, bool FAST>
__device__ __forceinline__ void activation(float a, float& f, float& df) {
  constexpr float kLog2e = 1.4426950408889634f;
  if constexpr (ACT == SLA_ACT_SILU) {
    float s;
    if constexpr (FAST) s = __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * a));
    else s = 1.f / (1.f + expf(-a));
    f = a * s;
    df = s * (1.f + a * (1.f - s));
  } else if constexpr (ACT == SLA_ACT_GELU) {
    float c, e;   // the normal distribution's integral, exp(-a^2 / 2)
    if constexpr (FAST) {
      e = __builtin_amdgcn_exp2f(-0.5f * kLog2e * a * a);
      const float x = fabsf(a) * 0.70710678118654752f;
      const float t = __builtin_amdgcn_rcpf(1.f + 0.44f * x);
      const float p = t * (0.248561018f + t * (0.242569534f + t * (0.263586435f +
                      t * (0.0407308007f + t * (0.350652906f + t * -0.14610586f)))));
      c = 0.5f * p * e;
      c = a < 0.f ? c : 1.f - c;
    } else {
      e = expf(-0.5f * a * a);
      c = 0.5f * erfcf(a * -0.70710678118654752f);   // 1 + erf() would cancel in the tail
    }
    f = a * c;
    df = c + a * (0.39894228040143268f * e);
  } else if constexpr (ACT == kActNone) {
    f = a;
    df = 1.f;
  } else {
    f = a < 0.f ? 0.f : a;  // 0 at -inf; NaN stays NaN, the slope's too
    df = a > 0.f ? 1.f : a <= 0.f ? 0.f : a;
  }
}

// One product C[M][N] = sum over `parts` segments of A_s[M][K] B_s[N][K]^T.
// AT: A is stored [k][row] (lda elements from one k to the next) instead of
// [row][k]; BT: likewise.
struct Product {
  const void *A[2], *B[2];
  int64_t lda, ldb;
  int64_t M, N, K;
  int parts, outputs;
  const void* dh;    // d [M][N] (EPI_LINEAR: may be none)
  int64_t lddh;
  const void* bias;  // EPI_LINEAR, EPI_SLOPE [N]: may be none
  int bias_f32;      // it is fp32, not of the operands' type
  void* C[2];        // EPI_GATE_GRAD: da, db; EPI_STORE: one per output; else one
  const float* scale;   // fp16 gradients: {what is held times it, its inverse}
  int64_t ldc;
  int act;
  const char* who;   // the entry, for its errors
  // filled by the launch
  int splits;        // of the steps; > 1: fp32 sums go to part [output][split][M][N]
  float* part;
  int gx, gy;        // tiles along N and M
  int most;          // splits at most (0: kMostSplits)
};
constexpr int kMostSplits = 32;

// A row of sums; fp32's four instructions a factor in turns over the sums: one
// on the sum of the one before would wait for it.
template <int NJ, typename V>
__device__ __forceinline__ void mma_row(f32x4 (&acc)[NJ], const V& a, const V (&b)[NJ]) {
  if constexpr (sizeof(a[0]) == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[j] = __builtin_amdgcn_mfma_f32_16x16x4f32(b[j][k], a[k], acc[j], 0, 0, 0);
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j) mma16(acc[j], a, b[j]);
  }
}

// A step's piece of an operand in LDS: W rows by STEP bytes of k, in 16-byte
// slots.  TRANS: lines of W rows, a line for each k; else lines of k, a line
// for each row.  So that a wave's fragment read touches every bank evenly the
// slots of a row's line are exchanged by the row (the offset of a read then
// depends on the lane alone), and the lines of k are moved apart: a read of 16
// lines of 32 bytes (16-bit: k = 8 h + r, or 4 more) or 4 of 64 (fp32: k = 4 h)
// finds them at different banks.  Direct loads (PAIR) write 1024 bytes in one
// piece: there the lines k and k + 4, never read together, are neighbours.
template <typename T, int W, bool TRANS, int THREADS, int STEP, bool PAIR>
struct Tile {
  static constexpr int kN = Unit<T>::kN;
  static constexpr int kLineSlots = TRANS ? W / kN : STEP / 16;
  static constexpr int kLoads = W * STEP / 16 / THREADS;   // slots a thread fills
  static constexpr int kSteps = STEP / int(sizeof(T));
  static constexpr int kThreads = THREADS, kRows = W;
  static constexpr bool kTrans = TRANS;
  typedef T Element;
  typedef typename Unit<T>::Vec Vec;
  static_assert(!(TRANS && PAIR) || (W == 256 && sizeof(T) == 2), "a pair of lines a load");

  static constexpr __device__ int line_at(int k) {
    if (sizeof(T) == 4) return k * W * 4 + 64 * (k >> 2);
    if (PAIR) return ((k >> 3) * 4 + (k & 3)) * (W * 4 + 32) + (k >> 2 & 1) * (W * 2);
    return k * (W * 2 + 32) + 128 * (k >> 3);
  }
  static constexpr int kBytes =
      TRANS ? (line_at(kSteps - 1) + W * int(sizeof(T)) + 127) / 128 * 128 : W * STEP;
  // the slot of a row's line that holds unit u of k
  static __device__ __forceinline__ int slot_of(int row, int u) {
    return STEP == 128 ? u ^ (row & 7) : u ^ (row >> 1 & 3);
  }

  // what slot i (of this thread's) holds: line and the first element along it
  static __device__ __forceinline__ void source(int i, int& line, int& along) {
    const int s = i * THREADS + int(threadIdx.x);
    line = s / kLineSlots;
    const int u = s % kLineSlots;
    if constexpr (TRANS) {
      if (PAIR) line = line / 8 * 8 + line % 2 * 4 + line / 2 % 4;
      along = u * kN;
    } else {
      along = slot_of(line, u) * kN;
    }
  }
  // where the slot lies; for direct loads the place of the wave's first one
  static __device__ __forceinline__ int place(int i) {
    const int s = i * THREADS + int(threadIdx.x);
    if constexpr (!TRANS) return s * 16;
    else return line_at(s / kLineSlots) + s % kLineSlots * 16;
  }
  static __device__ __forceinline__ int place(int i, int wave) {
    const int n = i * (THREADS / kWave) + wave;
    return TRANS ? n * (W * 4 + 32) : n * 1024;
  }
  // rows base + l (base a multiple of 16), sub-step s (of 64 bytes) of the step
  static __device__ __forceinline__ Vec read(const char* lds, int base, int s) {
    const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
    if constexpr (!TRANS) {
      return *reinterpret_cast<const Vec*>(lds + (base + l) * STEP + slot_of(l, 4 * s + h) * 16);
    } else if constexpr (sizeof(T) == 2) {
      Vec v;
      const char* p = lds + line_at(8 * h + (l >> 2)) + (l & 3) * 8;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const auto c = read_column<T>(p + base * 2 + line_at(32 * s + 4 * q));
#pragma unroll
        for (int j = 0; j < 4; ++j) v[4 * q + j] = c[j];
      }
      return v;
    } else {
      Vec v;
      const char* p = lds + line_at(4 * h) + l * 4;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = *reinterpret_cast<const T*>(p + base * 4 + line_at(16 * s + j));
      return v;
    }
  }
};

// Where a step's operand lies: its first element, the elements from one line
// to the next, how many rows and k there are from it on, and the length of a
// whole line.
struct Source {
  const char* p;
  int64_t ld, rows, ks, line;
};

// Memory to LDS without a register in between, for operands whose lines are
// whole aligned 16-byte units (the launch checks it).  Rows that do not exist
// and k behind the end read as zero: their offset lies out of the buffer's
// range.  `at`: each load's offset from the step's first element, kept from
// step to step.
template <typename TI, int FROM, int COUNT>
__device__ __forceinline__ void stage_offsets(int* at, const Source& s) {
#pragma unroll
  for (int i = FROM; i < FROM + COUNT; ++i) {
    int line, along;
    TI::source(i, line, along);
    if (!TI::kTrans) line -= FROM * TI::kThreads / TI::kLineSlots;
    at[i] = (TI::kTrans ? along : line) < s.rows
                ? int((line * s.ld + along) * int64_t(16 / TI::kN)) : kOutside;
  }
}
// Load i of a step whose first element is p and that has `ks` k (none: zeros).
template <typename TI>
__device__ __forceinline__ void stage(char* lds, const char* p, int at, int i, int ks) {
  int line, along;
  TI::source(i, line, along);
  const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  send(p, (TI::kTrans ? line : along) < ks ? at : kOutside, lds + TI::place(i, wave));
}

// ... and by way of registers, for any shape and alignment.  No lane branches
// (the join of one would wait for its load): a unit that passes the end of its
// line is read from further in front, a line that does not exist is another
// one, and mend() puts that right when the loads have come.
template <typename TI, int FROM, int COUNT>
__device__ __forceinline__ void fetch(typename TI::Vec* v, const Source& s) {
  typedef typename TI::Element T;
  const int64_t length = TI::kTrans ? s.rows : s.ks, lines = TI::kTrans ? s.ks : s.rows;
  const bool units = s.line >= TI::kN;
#pragma unroll
  for (int i = FROM; i < FROM + COUNT; ++i) {
    int line, along;
    TI::source(i, line, along);
    if (!TI::kTrans) line -= FROM * TI::kThreads / TI::kLineSlots;
    const T* q = (const T*)s.p + (line < lines ? line : lines - 1) * s.ld;
    if (units) {
      const int64_t last = length - TI::kN;
      const auto u = *reinterpret_cast<const typename Unit<T>::Loose*>(
          q + (along < last ? int64_t(along) : last));
#pragma unroll
      for (int j = 0; j < TI::kN; ++j) v[i][j] = u[j];
    } else {
#pragma unroll
      for (int j = 0; j < TI::kN; ++j) {
        const T x = q[along + j < length ? along + j : 0];
        v[i][j] = along + j < length ? x : T(0.f);
      }
    }
  }
}
// What fetch() read in place of what does not exist becomes zero; for a step
// that lies inside its operand nothing is to be done.  Rows that do not exist
// may hold anything: nobody stores what is made of them.
template <typename TI, int FROM, int COUNT>
__device__ __forceinline__ void mend(typename TI::Vec* v, const Source& s) {
  typedef uint32_t Words __attribute__((ext_vector_type(4)));
  const int64_t length = TI::kTrans ? s.rows : s.ks;
  constexpr int64_t kWhole = TI::kTrans ? int64_t(TI::kRows) : int64_t(TI::kSteps);
  if (length >= kWhole && s.ks >= TI::kSteps) return;
  const int over = int((TI::kN - length % TI::kN) % TI::kN);   // elements a cut unit was moved by
  const bool units = s.line >= TI::kN;
#pragma unroll
  for (int i = FROM; i < FROM + COUNT; ++i) {
    int line, along;
    TI::source(i, line, along);
    Words w = __builtin_bit_cast(Words, v[i]);
    if (units) {
      // down by `over` elements
      constexpr int kWord = 4 / int(sizeof(typename TI::Element));
      Words m = w;
      if (over / kWord & 1) m = Words{m[1], m[2], m[3], 0};
      if (over / kWord & 2) m = Words{m[2], m[3], 0, 0};
      if (over % kWord)
        m = Words{m[0] >> 16 | m[1] << 16, m[1] >> 16 | m[2] << 16, m[2] >> 16 | m[3] << 16,
                  m[3] >> 16};
      const bool cut = along < length && along + TI::kN > length, past = along >= length;
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = past ? 0u : cut ? m[j] : w[j];
    }
    if (TI::kTrans && line >= s.ks) w = Words{0, 0, 0, 0};
    v[i] = __builtin_bit_cast(typename TI::Vec, w);
  }
}

// The workgroup's tile.  Workgroups go to the 8 XCDs in turn: each XCD gets a
// run of neighbouring tiles (8 tiles of M by as many of N as it has), whose
// operands its L2 then holds once.
struct Where {
  int m, n, z, split;
};
__device__ __forceinline__ Where find_tile(const Product& g) {
  const int total = gridDim.x, b = blockIdx.x;
  const int xcd = b % kXcds, q = total / kXcds, r = total % kXcds;
  int id = xcd * q + (xcd < r ? xcd : r) + b / kXcds;
  Where w;
  const int tiles = g.gx * g.gy;
  const int zs = id / tiles;
  id -= zs * tiles;
  w.z = __builtin_amdgcn_readfirstlane(zs / g.splits);
  w.split = __builtin_amdgcn_readfirstlane(zs % g.splits);
  const int width = 8 * g.gx, group = id / width;
  const int rows = g.gy - group * 8 < 8 ? g.gy - group * 8 : 8;
  id -= group * width;
  w.m = __builtin_amdgcn_readfirstlane(group * 8 + id % rows);
  w.n = __builtin_amdgcn_readfirstlane(id / rows);
  return w;
}

// f(ACT) with the product's activation as a constant.
template <int EPI, typename F>
__device__ __forceinline__ void with_activation(const Product& g, F&& f) {
  if (EPI == EPI_LINEAR && g.act == kActNone) f(std::integral_constant<int, kActNone>());
  else if (EPI == EPI_STORE || g.act == SLA_ACT_SILU) f(std::integral_constant<int, SLA_ACT_SILU>());
  else if (g.act == SLA_ACT_GELU) f(std::integral_constant<int, SLA_ACT_GELU>());
  else f(std::integral_constant<int, SLA_ACT_RELU>());
}

// What a product's results are multiplied with on their way out.
template <typename T, int EPI>
__device__ __forceinline__ float scale_of(const Product& g) {
  if constexpr (std::is_same<T, _Float16>::value && EPI != EPI_GATE && EPI != EPI_LINEAR)
    return g.scale ? g.scale[EPI == EPI_STORE] : 1.f;   // (no rows: none)
  return 1.f;
}
// Four columns of the bias, of which `have` exist.
template <typename T>
__device__ __forceinline__ f32x4 bias_of(const Product& g, int64_t col, int64_t have) {
  float b[4] = {0.f, 0.f, 0.f, 0.f};
  if (g.bias && have > 0) {
    if (g.bias_f32) load_f32<4>((const float*)g.bias + col, have, b);
    else load_f32<4>((const T*)g.bias + col, have, b);
  }
  return f32x4{b[0], b[1], b[2], b[3]};
}
// What becomes of four columns of a row (b: the other weight's sums, or the
// bias): u, and v for db.
template <typename T, int EPI, int ACT>
__device__ __forceinline__ void result(const float (&d)[4], const f32x4& a, const f32x4& b,
                                       float scale, float (&u)[4], float (&v)[4]) {
  if constexpr (EPI == EPI_STORE) {
#pragma unroll
    for (int r = 0; r < 4; ++r) u[r] = a[r] * scale;
  } else if constexpr (EPI == EPI_LINEAR || EPI == EPI_SLOPE) {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float f, df;
      activation<ACT, sizeof(T) == 2>(a[r] + b[r], f, df);
      u[r] = EPI == EPI_LINEAR ? f + d[r] : d[r] * scale * df;
    }
  } else {
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      float f, df;
      activation<ACT, sizeof(T) == 2>(a[r], f, df);
      if constexpr (EPI == EPI_GATE) {
        u[r] = f * b[r];
      } else {
        const float e = d[r] * scale;
        u[r] = e * b[r] * df;
        v[r] = e * f;
      }
    }
  }
}
// They leave at element `at` of C; the first `have` of them exist.
template <typename T, int EPI, int ACT>
__device__ __forceinline__ void leave(const Product& g, int64_t at, const float (&d)[4],
                                      int64_t have, int z, const f32x4& a, const f32x4& b) {
  float u[4], v[4];
  result<T, EPI, ACT>(d, a, b, scale_of<T, EPI>(g), u, v);
  store_f32<4>((T*)(EPI == EPI_STORE && z ? g.C[1] : g.C[0]) + at, have, u);
  if constexpr (EPI == EPI_GATE_GRAD) store_f32<4>((T*)g.C[1] + at, have, v);
}

// Tiles of B x B in waves of WM x WN.  EPI_GATE*: the tile's columns are B / 2
// of a and the same B / 2 of b, half of each wave's columns are of either.
//
// A few steps' tiles are in LDS (Ring).  A wave multiplies a row of 16 x WN at
// a time and reads the fragments NI - 1 rows ahead of their use, between the
// products of the rows, so that the matrix cores and the LDS work side by
// side.  The step's only barrier comes behind the read of its tiles' last
// fragment: from there on the next tiles' fragments are read and this one's
// place is filled with a later step's.
//
// Bound by the matrix cores at the card's power limit (the same products of
// zeros take three quarters of the time) and, for tiles of 256, by the LDS
// reads beside them: 8192 x 2048 x 2 x 8192 bf16 478 us, 1.15 PFLOP/s, where
// the instructions alone reach 1.8 on such data; fp32 85 % of its 0.154.
template <typename T, int B, int WM, int WN, bool AT, bool BT, int EPI, bool DIRECT>
__global__ __launch_bounds__(kWave* B* B / WM / WN, 2) void k_product(Product g) {
  constexpr bool kGate = two_weights(EPI);
  constexpr int kThreads = kWave * (B / WM) * (B / WN);
  constexpr int NI = WM / 16, NJ = WN / 16, kCols = kGate ? B / 2 : B;
  constexpr int kStep = Ring<DIRECT>::kStep, kDepth = Ring<DIRECT>::kDepth;
  constexpr int kRows = kStep / 64 * NI;   // rows of products in a step
  using TA = Tile<T, B, AT, kThreads, kStep, DIRECT>;
  using TB = Tile<T, B, BT, kThreads, kStep, DIRECT>;
  typedef typename Unit<T>::Vec Vec;
  extern __shared__ __align__(1024) char smem[];
  auto place = [&](int n) { return smem + n % kDepth * (TA::kBytes + TB::kBytes); };
  const int t = threadIdx.x, l = t % 16, h = t % kWave / 16;
  const int w = __builtin_amdgcn_readfirstlane(t / kWave), wm = w / (B / WN), wn = w % (B / WN);
  const Where at = find_tile(g);
  const int64_t m0 = int64_t(at.m) * B, n0 = int64_t(at.n) * kCols;
  const int steps = int(div_up(g.K, TA::kSteps)), all = steps * g.parts;
  const int each = (all + g.splits - 1) / g.splits;
  const int from = at.split * each, to = from + each < all ? from + each : all;
  f32x4 acc[NI][NJ];
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = f32x4{0, 0, 0, 0};

  auto source_a = [&](int it) {
    const int seg = it >= steps;
    const int64_t k0 = int64_t(it - seg * steps) * TA::kSteps;
    const T* p = (const T*)(kGate || !(seg + at.z) ? g.A[0] : g.A[1]) +
                 (AT ? k0 * g.lda + m0 : m0 * g.lda + k0);
    return Source{(const char*)p, g.lda, g.M - m0, g.K - k0, AT ? g.M : g.K};
  };
  auto source_b = [&](int it, int which) {
    const int seg = it >= steps;
    const int64_t k0 = int64_t(it - seg * steps) * TB::kSteps;
    const T* p = (const T*)((kGate ? which : seg) ? g.B[1] : g.B[0]) +
                 (BT ? k0 * g.ldb + n0 : n0 * g.ldb + k0);
    return Source{(const char*)p, g.ldb, g.N - n0, g.K - k0, BT ? g.N : g.K};
  };
  // the wave's rows of the B tile: column tile j
  auto brow = [&](int j) {
    return kGate ? (j / (NJ / 2)) * (B / 2) + wn * (WN / 2) + j % (NJ / 2) * 16 : wn * WN + j * 16;
  };
  constexpr int HB = TB::kLoads / 2;
  int ta[DIRECT ? TA::kLoads : 1], tb[DIRECT ? TB::kLoads : 1];
  if constexpr (DIRECT) {
    stage_offsets<TA, 0, TA::kLoads>(ta, source_a(0));
    if constexpr (kGate) {
      stage_offsets<TB, 0, HB>(tb, source_b(0, 0));
      stage_offsets<TB, HB, HB>(tb, source_b(0, 0));
    } else {
      stage_offsets<TB, 0, TB::kLoads>(tb, source_b(0, 0));
    }
  }
  Vec ra[DIRECT ? 1 : TA::kLoads], rb[DIRECT ? 1 : TB::kLoads];
  // DIRECT: the loads of a step, one at a time (the wave's issue would wait
  // for a burst of them); behind the last step zeros come in their place
  constexpr int kSends = TA::kLoads + TB::kLoads;
  const char *pa = nullptr, *pb = nullptr, *pu = nullptr;
  int ks = 0;
  auto aim = [&](int it) {
    if constexpr (DIRECT) {
      const bool live = it < to;
      it = live ? it : from;
      const Source a = source_a(it);
      pa = uniform(a.p);
      pb = uniform(source_b(it, 0).p);
      if (kGate) pu = uniform(source_b(it, 1).p);
      ks = live ? int(a.ks < TA::kSteps ? a.ks : TA::kSteps) : 0;
    }
  };
  auto send_one = [&](char* lds, int n) {
    if (n < TA::kLoads) {
      stage<TA>(lds, pa, ta[DIRECT ? n : 0], n, ks);
    } else {
      const int i = n - TA::kLoads;
      stage<TB>(lds + TA::kBytes, kGate && i >= HB ? pu : pb, tb[DIRECT ? i : 0], i, ks);
    }
  };
  auto load = [&](int it) {   // not DIRECT: the step's tiles into registers
    if (it >= to) return;
    fetch<TA, 0, TA::kLoads>(ra, source_a(it));
    if constexpr (kGate) {
      fetch<TB, 0, HB>(rb, source_b(it, 0));
      fetch<TB, HB, HB>(rb, source_b(it, 1));
    } else {
      fetch<TB, 0, TB::kLoads>(rb, source_b(it, 0));
    }
  };
  auto put = [&](char* lds, int it) {
    if constexpr (!DIRECT) {
      mend<TA, 0, TA::kLoads>(ra, source_a(it));
      if constexpr (kGate) {
        mend<TB, 0, HB>(rb, source_b(it, 0));
        mend<TB, HB, HB>(rb, source_b(it, 1));
      } else {
        mend<TB, 0, TB::kLoads>(rb, source_b(it, 0));
      }
#pragma unroll
      for (int i = 0; i < TA::kLoads; ++i)
        *reinterpret_cast<Vec*>(lds + TA::place(i)) = ra[i];
#pragma unroll
      for (int i = 0; i < TB::kLoads; ++i)
        *reinterpret_cast<Vec*>(lds + TA::kBytes + TB::place(i)) = rb[i];
    }
  };
  Vec fa[NI], fb[2][NJ];
  auto read_a = [&](const char* lds, int r) {   // row r of a step
    fa[r % NI] = TA::read(lds, wm * WM + 16 * (r % NI), r / NI);
  };
  auto read_b = [&](const char* lds, int s, int to_s, int j) {
    fb[to_s][j] = TB::read(lds + TA::kBytes, brow(j), s);
  };
  if (from < to) {
    if constexpr (DIRECT) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        aim(from + d);
#pragma unroll
        for (int n = 0; n < kSends; ++n) send_one(place(d), n);
      }
      landed<(kDepth - 1) * kSends>();
    } else {
      load(from);
      put(place(0), from);
      if (from + 1 < to) {
        load(from + 1);
        put(place(1), from + 1);
      }
      load(from + 2);
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) read_b(place(0), 0, 0, j);
#pragma unroll
    for (int i = 0; i < NI - 1; ++i) read_a(place(0), i);
    // Step `it`, whose tiles are at place u; behind the last step the
    // fragments read are not used.
    auto step = [&](auto u, int it) {
      char* const cur = place(u.value);
      char* const nxt = place(u.value + 1);
      constexpr int kFlip = kRows == NI ? u.value % 2 : 0;   // which fb the step begins with
      constexpr int kTurn = kRows - NI + 1;   // from this row on: the next tile's fragments
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        if (r == kTurn) {
          // the next step's tiles have come (the loads of those behind it may
          // be under way) and every wave has read this step's
          if constexpr (DIRECT) {
            landed<(kDepth - 2) * kSends>();
            aim(it + kDepth);
          } else {
            __syncthreads();
            if (it + 2 < to) {
              put(cur, it + 2);
              load(it + 3);
            }
          }
        }
        if (r < kTurn) read_a(cur, r + NI - 1);
        else read_a(nxt, r + NI - 1 - kRows);
        if (kRows > NI && r < NI) {
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            if ((j < NI ? j : NI - 1) == r) read_b(cur, 1, 1, j);
        }
        if (r >= kTurn) {
          constexpr int kLeft = NI - 1;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
            if (j % kLeft == r - kTurn) read_b(nxt, 0, kRows == NI ? kFlip ^ 1 : 0, j);
          if constexpr (DIRECT) {
            constexpr int kEach = (kSends + kLeft - 1) / kLeft;
#pragma unroll
            for (int n = 0; n < kSends; ++n)
              if (n / kEach == r - kTurn) send_one(cur, n);
          }
        }
        mma_row(acc[r % NI], fa[r % NI], fb[kRows == NI ? kFlip : r / NI]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    for (int it = from; it < to; it += kDepth) {
      step(std::integral_constant<int, 0>(), it);
      if (it + 1 < to) step(std::integral_constant<int, 1>(), it + 1);
      if constexpr (kDepth == 4) {
        if (it + 2 < to) step(std::integral_constant<int, 2>(), it + 2);
        if (it + 3 < to) step(std::integral_constant<int, 3>(), it + 3);
      }
    }
    // the last loads must not come in after the workgroup has given its LDS back
    if constexpr (DIRECT) asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }

  // the lane's first quad; the others lie 16 rows or 16 columns further
  const int64_t row0 = m0 + wm * WM + l, col0 = n0 + 4 * h;
  auto finish = [&](auto act, auto whole) {
    int64_t at_c = row0 * g.ldc + col0;
    float* part = g.splits > 1 ? g.part + (int64_t(at.z) * g.splits + at.split) * g.M * g.N +
                                     row0 * g.N + col0 : nullptr;
    constexpr int kQuads = kGate ? NJ / 2 : NJ;
    auto has = [&](int j) { return whole.value ? int64_t(4) : g.N - col0 - brow(j); };
    // whole 16-bit tiles: two quads at a time
    constexpr bool kWide = whole.value && sizeof(T) == 2 && kQuads % 2 == 0;
    typedef typename std::conditional<sizeof(T) == 2, T, _Float16>::type Half;   // T, if kWide
    typedef typename VecOf<Half, 8>::type Loose8;
    const int wide = brow(h % 2) - brow(0) + 8 * (h / 2) - 4 * h;   // from the lane's first quad
    // dh of all rows is asked for before the first row leaves
    typename VecOf<T, 4>::type dh[takes_d(EPI) ? NI : 1][kQuads];
    const bool has_d = EPI != EPI_LINEAR || g.dh;
    if (takes_d(EPI) && !part && !has_d) {
#pragma unroll
      for (int i = 0; i < (takes_d(EPI) ? NI : 1); ++i)
#pragma unroll
        for (int j = 0; j < kQuads; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) dh[i][j][r] = T(0.f);
    }
    f32x4 bias[EPI == EPI_LINEAR || EPI == EPI_SLOPE ? kQuads : 1];
    if constexpr (EPI == EPI_LINEAR || EPI == EPI_SLOPE) {
      if (!part) {
#pragma unroll
        for (int j = 0; j < kQuads; ++j) bias[j] = bias_of<T>(g, col0 + brow(j), has(j));
      }
    }
    if constexpr (takes_d(EPI)) if (!part && has_d) {
      const T* p = (const T*)g.dh + row0 * g.lddh + col0;
      if constexpr (kWide) {
        Quads q[NI][kQuads / 2];
#pragma unroll
        for (int i = 0; i < NI; ++i, p += 16 * g.lddh)
#pragma unroll
          for (int j = 0; j < kQuads; j += 2) {
            const Loose8 x = *reinterpret_cast<const Loose8*>(p + brow(j) + wide);
            q[i][j / 2] = __builtin_bit_cast(Quads, x);
          }
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int j = 0; j < kQuads; j += 2) {
            const Quads x = q[i][j / 2], y = side_by_side(Pair{x[0], x[1]}, Pair{x[2], x[3]});
            typedef Half V4 __attribute__((ext_vector_type(4)));
            const V4 a = __builtin_bit_cast(V4, Pair{y[0], y[1]});
            const V4 b = __builtin_bit_cast(V4, Pair{y[2], y[3]});
#pragma unroll
            for (int r = 0; r < 4; ++r) dh[i][j][r] = T(a[r]), dh[i][j + 1][r] = T(b[r]);
          }
      } else {
#pragma unroll
        for (int i = 0; i < NI; ++i, p += 16 * g.lddh)
#pragma unroll
          for (int j = 0; j < kQuads; ++j) {
            const int64_t have = whole.value || row0 + 16 * i < g.M ? has(j) : 0;
            if (have >= 4) {
              dh[i][j] = *reinterpret_cast<const typename VecOf<T, 4>::type*>(p + brow(j));
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r) dh[i][j][r] = r < have ? p[brow(j) + r] : T(0.f);
            }
          }
      }
    }
    if constexpr (kWide) {
      if (kGate || !part) {
        T* c0 = (T*)(EPI == EPI_STORE && at.z ? g.C[1] : g.C[0]) + at_c + wide;
        T* c1 = (T*)(kGate ? g.C[1] : g.C[0]) + at_c + wide;
        const float scale = scale_of<T, EPI>(g);
#pragma unroll
        for (int i = 0; i < NI; ++i, c0 += 16 * g.ldc, c1 += 16 * g.ldc)
#pragma unroll
          for (int j = 0; j < kQuads; j += 2) {
            Pair u2[2], v2[2];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              float d[4] = {0.f, 0.f, 0.f, 0.f}, u[4], v[4] = {0.f, 0.f, 0.f, 0.f};
              if constexpr (takes_d(EPI)) {
#pragma unroll
                for (int r = 0; r < 4; ++r) d[r] = float(dh[i][j + n][r]);
              }
              if constexpr (EPI == EPI_LINEAR || EPI == EPI_SLOPE)
                result<T, EPI, act.value>(d, acc[i][j + n], bias[j + n], scale, u, v);
              else
                result<T, EPI, act.value>(d, acc[i][j + n],
                                          acc[i][kGate ? j + n + NJ / 2 : j + n], scale, u, v);
              u2[n] = packed<Half>(u);
              v2[n] = packed<Half>(v);
            }
            *reinterpret_cast<Loose8*>(c0 + brow(j)) =
                __builtin_bit_cast(Loose8, side_by_side(u2[0], u2[1]));
            if constexpr (EPI == EPI_GATE_GRAD)
              *reinterpret_cast<Loose8*>(c1 + brow(j)) =
                  __builtin_bit_cast(Loose8, side_by_side(v2[0], v2[1]));
          }
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (whole.value || row0 + 16 * i < g.M) {
#pragma unroll
        for (int j = 0; j < kQuads; ++j) {
          const int64_t have = has(j);
          if (!whole.value && have <= 0) continue;
          float u[4];
          if (!kGate && part) {
#pragma unroll
            for (int r = 0; r < 4; ++r) u[r] = acc[i][j][r];
            store_f32<4>(part + brow(j), have, u);
          } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) u[r] = takes_d(EPI) ? float(dh[i][j][r]) : 0.f;
            if constexpr (EPI == EPI_LINEAR || EPI == EPI_SLOPE)
              leave<T, EPI, act.value>(g, at_c + brow(j), u, have, at.z, acc[i][j], bias[j]);
            else
              leave<T, EPI, act.value>(g, at_c + brow(j), u, have, at.z, acc[i][j],
                                       acc[i][kGate ? j + NJ / 2 : j]);
          }
        }
      }
      at_c += 16 * g.ldc;
      if (!kGate && part) part += 16 * g.N;
    }
  };
  with_activation<EPI>(g, [&](auto act) {
    if (m0 + B <= g.M && n0 + kCols <= g.N) finish(act, std::true_type());
    else finish(act, std::false_type());
  });
}

// The sums of a split product, in the order of the splits, rounded once.
// LINES > 1: for many splits of few sums; a line of threads takes every
// LINES-th split, the first line joins them.
template <typename T, int EPI, int LINES>
__global__ __launch_bounds__(kProductBlock) void k_join(Product g) {
  constexpr int kWidth = kProductBlock / LINES;
  __shared__ f32x4 lines[LINES > 1 ? LINES : 1][LINES > 1 ? kWidth : 1];
  const int at = threadIdx.x % kWidth, line = threadIdx.x / kWidth;
  const int64_t size = g.M * g.N, quads = div_up(size, 4);
  const int64_t i = (int64_t(blockIdx.x) * kWidth + at) * 4;
  if (LINES == 1 && i >= quads * 4) return;
  float s[4] = {0.f, 0.f, 0.f, 0.f}, u[4];
  if (i < size) {
    const float* p = g.part + int64_t(blockIdx.y) * g.splits * size + i;
    if (line < g.splits) load_f32<4>(p + line * size, size - i, s);
#pragma unroll 4
    for (int k = line + LINES; k < g.splits; k += LINES) {
      load_f32<4>(p + k * size, size - i, u);
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += u[j];
    }
  }
  if constexpr (LINES > 1) {
    lines[line][at] = f32x4{s[0], s[1], s[2], s[3]};
    __syncthreads();
    if (line || i >= size) return;
#pragma unroll
    for (int k = 1; k < LINES; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += lines[k][at][j];
  }
  const float scale = scale_of<T, EPI>(g);
  if constexpr (EPI == EPI_STORE) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] *= scale;
  } else {
    with_activation<EPI>(g, [&](auto act) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (i + j >= size) break;
        const int64_t row = size < (int64_t(1) << 32) ? uint32_t(i + j) / uint32_t(g.N)
                                                       : (i + j) / g.N;
        const int64_t col = i + j - row * g.N;
        const float d[4] = {g.dh ? float(((const T*)g.dh)[row * g.lddh + col]) : 0.f, 0.f, 0.f,
                            0.f};
        float o[4], o2[4];
        result<T, EPI, act.value>(d, f32x4{s[j], 0, 0, 0}, bias_of<T>(g, col, 1), scale, o, o2);
        s[j] = o[0];
      }
    });
  }
  store_f32<4>((T*)g.C[blockIdx.y] + i, size - i, s);
}

// fp16's da and db: |da| <= 1.13 |dh| |b| and |db| <= |dh| |a| (no activation is
// steeper than 1.13 or larger than its argument), and |a|, |b| <= the norm of a
// row of x times that of a row of the weights.  A wave takes lines of one of
// the four arrays at a time; values that are not finite count nothing (what is
// made of them is not finite either).  parts: three maxima a workgroup.  Reading
// the arrays is the work: 49 us for the 184 MB of 16384 x 1024 x 4096 (3.8 TB/s),
// of 1090 for the training step; 222 us for 1.6e7 rows of 16 and 16 (4.6 TB/s),
// which a wave a line had made 6 ms.
constexpr int kBoundGroups = 1024;
struct Lines {
  const _Float16* p;
  int64_t ld, count;
  int width;
};
// The largest value (or sum of squares of a line) of the lines a wave walks, in
// any of its lanes: teams of lanes, as many as hold a line in 16 bytes each.
__device__ __forceinline__ float lines_max(const Lines& s, int64_t wave, int64_t waves,
                                           bool square) {
  const int lane = threadIdx.x % kWave;
  int team = 1;
  while (team < kWave && team * 8 < s.width) team *= 2;
  const int per = kWave / team;
  float best = 0.f;
  for (int64_t i = wave * per + lane / team; i < s.count; i += waves * per) {
    const _Float16* p = s.p + i * s.ld;
    float m = 0.f;
    for (int64_t c = lane % team * 8; c < s.width; c += team * 8) {
      float v[8];
      load_f32<8>(p + c, s.width - c, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (square) m += v[j] * v[j];
        else m = fmaxf(m, fabsf(v[j]) <= 65504.f ? fabsf(v[j]) : 0.f);
      }
    }
    if (square)
      for (int d = 1; d < team; d *= 2) m += __shfl_xor(m, d, kWave);
    best = m < __builtin_inff() ? fmaxf(best, m) : best;
  }
  return best;
}
__attribute__((unused)) __global__ __launch_bounds__(kProductBlock) void k_bound(Lines dh, Lines x, Lines wg, Lines wu,
                                                         float* __restrict__ parts) {
  constexpr int kWaves = kProductBlock / kWave;
  __shared__ float best[3][kWaves];
  const int w = threadIdx.x / kWave;
  const int64_t wave = int64_t(blockIdx.x) * kWaves + w, waves = int64_t(gridDim.x) * kWaves;
  float m[3] = {lines_max(dh, wave, waves, false), lines_max(x, wave, waves, true),
                fmaxf(lines_max(wg, wave, waves, true), lines_max(wu, wave, waves, true))};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) m[k] = fmaxf(m[k], __shfl_xor(m[k], d, kWave));
    if (threadIdx.x % kWave == 0) best[k][w] = m[k];
  }
  __syncthreads();
  if (threadIdx.x < 3) {
    float v = 0.f;
    for (int i = 0; i < kWaves; ++i) v = fmaxf(v, best[threadIdx.x][i]);
    parts[3 * blockIdx.x + threadIdx.x] = v;
  }
}
// The power of two that brings the bound to 2^14 .. 2^15, and its inverse.
// SINGLE: of the first maximum alone.
template <bool SINGLE>
__global__ __launch_bounds__(kWave) void k_scale(const float* __restrict__ parts, int groups,
                                                 float* __restrict__ scale) {
  float m[3] = {0.f, 0.f, 0.f};
  for (int i = threadIdx.x; i < groups; i += kWave)
#pragma unroll
    for (int k = 0; k < 3; ++k) m[k] = fmaxf(m[k], parts[3 * i + k]);
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) m[k] = fmaxf(m[k], __shfl_xor(m[k], d, kWave));
  if (threadIdx.x == 0) {
    const float bound = SINGLE ? 1.13f * m[0] : 1.13f * m[0] * sqrtf(m[1]) * sqrtf(m[2]);
    const int up = bound > 0.f ? 14 - ilogbf(bound) : 0;
    scale[0] = ldexpf(1.f, up);
    scale[1] = ldexpf(1.f, -up);
  }
}

// The projections of few rows (at most 16 RT): reading the weights is the
// work.  A workgroup has 16 columns of each weight; its waves take turns
// along k, fragments straight from memory, and are joined through LDS.  4 x
// 1024 x 2 x 4096 bf16: 5.2 us (16.8 MB), against 36 us with tiles of 128; 4 x 4096 x
// 1024 with one weight 8.0 us (8.4 MB), 64 workgroups (of 16 waves each: 8.4).
constexpr int kFewWaves = 4;
template <typename T, int RT, int EPI>
__global__ __launch_bounds__(kWave* kFewWaves) void k_few(Product g) {
  constexpr int NB = two_weights(EPI) ? 2 : 1;
  typedef typename Unit<T>::Vec Vec;
  constexpr int kN = Unit<T>::kN, kSpan = 4 * kN;   // k of one fragment
  __shared__ f32x4 sums[kFewWaves][RT][NB][kWave];
  const int t = threadIdx.x, w = t / kWave, l = t % 16, h = t % kWave / 16;
  const int64_t n0 = int64_t(blockIdx.x) * 16;
  auto line = [](const void* p, int64_t ld, int64_t row, int64_t rows) {
    return (const T*)p + (row < rows ? row : rows - 1) * ld;
  };
  const T* b0 = line(g.B[0], g.ldb, n0 + l, g.N);
  const T* b1 = NB == 2 ? line(g.B[1], g.ldb, n0 + l, g.N) : nullptr;
  const T* a[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) a[i] = line(g.A[0], g.lda, 16 * i + l, g.M);
  const int K = int(g.K);
  f32x4 acc[RT][NB];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i][0] = acc[i][NB - 1] = f32x4{0, 0, 0, 0};
  // a wave takes two neighbouring spans (128 bytes of a row) at a time
  auto load = [&](int k, auto whole, Vec (&u)[2][NB], Vec (&x)[2][RT]) {
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int kk = k + s * kSpan + h * kN;
      auto unit = [&](const T* p) {
        Vec v;
        if constexpr (whole.value) {
          const auto q = *reinterpret_cast<const typename Unit<T>::Loose*>(p + kk);
#pragma unroll
          for (int j = 0; j < kN; ++j) v[j] = q[j];
        } else {
#pragma unroll
          for (int j = 0; j < kN; ++j) v[j] = kk + j < K ? p[kk + j] : T(0.f);
        }
        return v;
      };
      u[s][0] = unit(b0);
      if constexpr (NB == 2) u[s][1] = unit(b1);
#pragma unroll
      for (int i = 0; i < RT; ++i) x[s][i] = unit(a[i]);
    }
  };
  auto multiply = [&](const Vec (&u)[2][NB], const Vec (&x)[2][RT]) {
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        mma16(acc[i][0], x[s][i], u[s][0]);
        if constexpr (NB == 2) mma16(acc[i][1], x[s][i], u[s][1]);
      }
  };
  constexpr int kStep = 2 * kSpan, kTurn = kFewWaves * kStep;
  int k = kStep * w;
  for (; k + 3 * kTurn + kStep <= K; k += 4 * kTurn) {  // four turns' loads travel at once
    Vec u[4][2][NB], x[4][2][RT];
#pragma unroll
    for (int n = 0; n < 4; ++n) load(k + n * kTurn, std::true_type(), u[n], x[n]);
#pragma unroll
    for (int n = 0; n < 4; ++n) multiply(u[n], x[n]);
  }
  for (; k < K; k += kTurn) {
    Vec u[2][NB], x[2][RT];
    if (k + kStep <= K) load(k, std::true_type(), u, x);
    else load(k, std::false_type(), u, x);
    multiply(u, x);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    sums[w][i][0][t % kWave] = acc[i][0];
    if constexpr (NB == 2) sums[w][i][1][t % kWave] = acc[i][1];
  }
  __syncthreads();
  for (int i = w; i < RT; i += kFewWaves) {
    const int64_t row = 16 * i + l, col = n0 + 4 * h;
    if (row >= g.M || col >= g.N) continue;
    f32x4 s[2];
#pragma unroll
    for (int b = 0; b < NB; ++b)
      s[b] = (sums[0][i][b][t % kWave] + sums[1][i][b][t % kWave]) +
             (sums[2][i][b][t % kWave] + sums[3][i][b][t % kWave]);
    if constexpr (NB == 1) s[1] = bias_of<T>(g, col, g.N - col);
    float d[4] = {0.f, 0.f, 0.f, 0.f};
    if (takes_d(EPI) && (EPI != EPI_LINEAR || g.dh))
      load_f32<4>((const T*)g.dh + row * g.lddh + col, g.N - col, d);
    with_activation<EPI>(g, [&](auto act) {
      leave<T, EPI, act.value>(g, row * g.ldc + col, d, g.N - col, 0, s[0], s[1]);
    });
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Tiles and splits of a product: the pair with the least estimated time.  With
// n workgroups on a CU, at most `slots` of them at once, a step of 128 bytes of
// k takes wait (per round of slots) + n share, as measured from n = 1 to 6:
//   fp32     64: 0.93, 1.37, 1.89, 2.37, 3.07, 3.57 us   128: 2.53, 4.19, -, 8.44
//   16 bit   64: 0.60, 0.66, 0.78, 0.94, 1.32, 1.47 us   128: 1.07, 1.31, 2.20, 2.53
//           256: 1.54, 3.00, 4.63, 6.01 us
// so the large tile wins as soon as it fills the card, the small one where
// there is little to do; a split costs the writing and reading of its sums.
// fp32 operands stored [k][row] (`turned` of the two) are read from LDS a word
// at a time: 2.0 us instead of 1.37 with both of them (64, n = 2).
struct ProductPlan {
  int tile, splits;
};
// Threads of a launch: the runtime starts one of 2^32 and more without its upper
// bits.  Tiles of 64 columns or more stay below for every matrix that fits the
// card; only long narrow ones have to take a larger tile for it.
constexpr int64_t kMostThreads = (int64_t(1) << 32) - 1;
ProductPlan plan_product(int64_t M, int64_t N, int64_t K, int parts, int outputs, bool gate,
                         int turned, int es, bool direct, int most = 0) {
  struct Kind {
    int tile, slots;
    double wait, share, start;   // us; start: before and behind the steps
  };
  static const Kind kind16[] = {{256, 1, 0.0, 1.5, 8.0}, {128, 2, 0.83, 0.24, 5.5},
                                {64, 4, 0.48, 0.115, 4.0}};
  static const Kind kind32[] = {{256, 1, 0, 0, 0}, {128, 2, 0.87, 1.66, 5.0},
                                {64, 4, 0.42, 0.5, 5.0}};
  const Kind* kinds = es == 4 ? kind32 : kind16;
  const int64_t steps = div_up(K, 128 / es) * parts, cus = device_cus();
  ProductPlan best{64, 1};
  double least = 1e30;
  for (int i = es == 4 || !direct ? 1 : 0; i < 3; ++i) {
    const Kind& k = kinds[i];
    const int64_t tiles = div_up(M, k.tile) * div_up(N, gate ? k.tile / 2 : k.tile) * outputs;
    const int64_t threads = k.tile == 256 ? 512 : 256;
    for (int s = 1; s <= (gate ? 1 : most ? most : kMostSplits) && s <= (steps + 3) / 4;
         s += s < kMostSplits ? 1 : s / 8) {
      if (tiles * s * threads > kMostThreads) break;
      const int64_t n = div_up(tiles * s, cus);
      const double rounds = double(div_up(n, k.slots));
      const double wait = k.wait + (es == 4 ? 0.3 * turned : 0.0);
      double time = double(div_up(steps, s)) * (rounds * wait + double(n) * k.share) +
                    rounds * k.start;
      if (s > 1) time += 5.0 + double(s + 1) * double(M * N * outputs) * 4 / 4e6;
      if (time < least) least = time, best = {k.tile, s};
    }
  }
  return best;
}

inline int64_t split_bytes(int64_t M, int64_t N, int64_t K, int parts, int outputs, int turned, int es,
                    int limit = 0) {
  int64_t most = 0;
  for (int direct = 0; direct < 2; ++direct) {
    const ProductPlan p = plan_product(M, N, K, parts, outputs, false, turned, es, direct, limit);
    const int64_t b = p.splits > 1 ? p.splits * outputs * M * N * 4 : 0;
    if (b > most) most = b;
  }
  return most;
}

// Whether an operand's lines are whole aligned 16-byte units that 31 bits of
// a tile's offsets reach.
inline bool whole_units(const void* p, int64_t ld, int64_t along, int es) {
  const int64_t n = 16 / es;
  return reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % n == 0 && along % n == 0 &&
         ld * es * 256 < (int64_t(1) << 31);
}

template <typename T, int B, int WM, int WN, bool AT, bool BT, int EPI, bool DIRECT>
sla_status run_product(Product& g, hipStream_t stream) {
  constexpr int kThreads = kWave * (B / WM) * (B / WN);
  constexpr int kStep = Ring<DIRECT>::kStep;
  constexpr int lds = Ring<DIRECT>::kDepth * (Tile<T, B, AT, kThreads, kStep, DIRECT>::kBytes +
                                              Tile<T, B, BT, kThreads, kStep, DIRECT>::kBytes);
  const int64_t gx = div_up(g.N, two_weights(EPI) ? B / 2 : B), gy = div_up(g.M, B);
  SLA_NET_REQUIRE(gx * gy * g.outputs * g.splits * kThreads <= kMostThreads,
                  "%s: a matrix is too large", g.who);
  g.gx = int(gx), g.gy = int(gy);
  auto* kernel = k_product<T, B, WM, WN, AT, BT, EPI, DIRECT>;
  if (lds > 65536)
    SLA_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                    hipFuncAttributeMaxDynamicSharedMemorySize, lds));
  kernel<<<int(gx * gy) * g.outputs * g.splits, kThreads, lds, stream>>>(g);
  LAUNCH_CHECK();
  return SLA_OK;
}

constexpr int64_t kFewRows = 64;
template <typename T, int EPI>
sla_status launch_few(const Product& g, hipStream_t stream) {
  const int grid = int(div_up(g.N, 16));
  if (g.M <= 16) k_few<T, 1, EPI><<<grid, kWave * kFewWaves, 0, stream>>>(g);
  else if (g.M <= 32) k_few<T, 2, EPI><<<grid, kWave * kFewWaves, 0, stream>>>(g);
  else k_few<T, 4, EPI><<<grid, kWave * kFewWaves, 0, stream>>>(g);
  LAUNCH_CHECK();
  return SLA_OK;
}

template <typename T, bool AT, bool BT, int EPI>
sla_status launch_product(Product& g, hipStream_t stream) {
  constexpr bool kGate = two_weights(EPI);
  constexpr int es = int(sizeof(T));
  if (g.M == 0 || g.N == 0) return SLA_OK;
  if constexpr (EPI != EPI_STORE)
    if (g.M <= kFewRows) return launch_few<T, EPI>(g, stream);
  const int64_t ka = AT ? g.M : g.K, kb = BT ? g.N : g.K;
  const bool direct =
      es == 2 && whole_units(g.A[0], g.lda, ka, es) && whole_units(g.B[0], g.ldb, kb, es) &&
      (!g.A[1] || whole_units(g.A[1], g.lda, ka, es)) &&
      (!g.B[1] || whole_units(g.B[1], g.ldb, kb, es));
  const ProductPlan p = plan_product(g.M, g.N, g.K, g.parts, g.outputs, kGate, int(AT) + int(BT),
                                     es, direct, g.most);
  g.splits = p.splits;
  if (p.tile == 64) SLA_TRY((run_product<T, 64, 32, 32, AT, BT, EPI, false>(g, stream)));
  if (p.tile == 128) SLA_TRY((run_product<T, 128, 64, 64, AT, BT, EPI, false>(g, stream)));
  if constexpr (es == 2)
    if (p.tile == 256) SLA_TRY((run_product<T, 256, 128, 64, AT, BT, EPI, true>(g, stream)));
  if (g.splits > 1) {
    if (g.splits > kMostSplits)
      k_join<T, EPI, 16><<<dim3(int(div_up(g.M * g.N, 4 * kProductBlock / 16)), g.outputs),
                           kProductBlock, 0, stream>>>(g);
    else
      k_join<T, EPI, 1><<<dim3(int(div_up(g.M * g.N, 4 * kProductBlock)), g.outputs),
                          kProductBlock, 0, stream>>>(g);
    LAUNCH_CHECK();
  }
  return SLA_OK;
}

}  // namespace
}  // namespace net
}  // namespace sla
