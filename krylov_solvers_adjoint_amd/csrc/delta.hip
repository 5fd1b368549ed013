// The gated delta rule: a matrix state per sequence and head, decayed by
// exp(g_t), corrected towards v_t at k_t, and read at q_t.
//
//   D_t = exp(g_t) S_{t-1}
//   m_t = v_t - D_t^T k_t                      (what the state got wrong)
//   S_t = D_t + k_t (beta_t m_t)^T
//   o_t = scale S_t^T q_t
//
// Whole sequences run in chunks of 64 tokens.  With G the running sum of g
// inside a chunk, S the state before it and d_ij = exp(G_i - G_j) (i >= j),
//
//   A_ij = d_ij k_i.k_j   (i > j)      P_ij = scale d_ij q_i.k_j   (i >= j)
//   R    = v - exp(G) (k S)            what the chunk's tokens see of S
//   (I + A B) M = R,  N = B M,  B = diag(beta)
//   o    = scale exp(G) (q S) + P N
//   S'   = exp(G_L) S + (exp(G_L - G) k)^T N
//
// With E = A (I + B A)^-1 (strictly lower), (I + A B)^-1 = I - E B and
// (I + B A)^-1 = I - B E, so one 64 x 64 matrix gives both M = R - E (B R)
// forward and, for the adjoint system, X = Y - E^T (B Y) backward; nothing
// is ever divided by beta, which may be zero.
//
// Backward, with dS the gradient of the state behind the chunk:
//
//   Y  = P^T do + exp(G_L - G) (k dS)      X = Y - E^T (B Y)    (= dL/dN)
//   dS_before = exp(G_L) dS + (scale exp(G) q)^T do - (exp(G) k)^T (B X)
//   dv = B X         dbeta_i = X_i . M_i
//   dP_ij = scale d_ij do_i.N_j            dA_ij = d_ij beta_i X_i.N_j
//   dq = scale exp(G) (do S^T) + dP k
//   u  = - exp(G) B (X S^T) - dA k         w = dP^T q - dA^T k + exp(G_L - G) (N dS^T)
//   dk = u + w       dg_t = sum over i >= t > j of H_ij + sum over i >= t of a_i
//                           + sum over j < t of b_j + exp(G_L) <S, dS>
//   H_ij = do_i.N_j P_ij - beta_i X_i.N_j A_ij
//   a_i  = scale exp(G_i) q_i.(do S^T)_i - exp(G_i) beta_i k_i.(X S^T)_i
//   b_j  = exp(G_L - G_j) k_j.(N dS^T)_j
//
// Work that does not depend on the state (k_delta_prepare, k_delta_out,
// k_delta_grads) runs over all chunks at once; what does (k_delta_states,
// k_delta_adjoint) walks a sequence's chunks, a workgroup for every 32
// columns of the state, which never mix.
//
// Everything is held in fp32 whatever the tokens' type: the state, its
// gradient, dg and dbeta leave in fp32, and a matrix product of rounded 16-bit
// factors would leave them three digits.  The products run on the bf16 matrix
// instructions all the same, 16 times the rate of the fp32 ones: an fp32
// factor is cut into three bf16 parts of 8 bits each, which hold all its 24
// (fp16 needs two, bf16 is one), and a product takes the pairs of parts whose
// orders add up to at most 2: what is left out of a term is 2^-24 of it on
// average, 2^-21 at most.  (An infinite factor becomes NaN, and what is not
// finite may reach earlier tokens of its chunk: zeros of the triangles meet it
// in the products.)  That holds
// for results that are rounded to 16 bits (o, dq, dk) too: they are sums of
// terms that cancel, behind a token that erases above all, and terms of two
// parts (cut off at 2^-16) had left 0.015 of a state of 1e3 in o.  G is
// summed in fp64: its differences are exponents.  A gate that resets the state
// (-infinity, a type's lowest value) would take the later gates' digits out of
// that sum, or make its differences infinite less infinite: gates below
// kGateFloor count as kGateFloor, whose exp is the same zero.
//
// An operand of the 16 x 16 x 32 instruction holds, in lane (l, h) = (lane %
// 16, lane / 16), eight k of row (column) l; which eight is free as long as
// both operands agree.  Here they are 4 h .. 4 h + 3 and 16 more, because the
// results of two instructions, rows 4 h .. 4 h + 3 of column l each, are then
// an operand of the next one as they stand: a wave that holds all rows of 16
// columns of the state walks through a chunk in its registers, without a
// barrier between the products.  Operands stored the other way round are
// turned by the transposed LDS read.
#include <type_traits>

#include "net.h"

namespace sla {
namespace net {
namespace {

constexpr int kChunk = 64;
constexpr int kDeltaBlock = 256;
constexpr int kSlice = 32;              // columns of the state a parallel kernel takes at a time
constexpr int kLdC = kChunk + 4;        // LDS row of 64 floats (padded against bank conflicts)
constexpr int kWalk = 64;               // columns of the state per walking workgroup
// exp() of a gate at the floor is 0 in fp32 (from -104 on), and stays 0 beside
// any growth of a chunk's 63 other gates that exp() holds (88 each); 64 such
// gates leave the fp64 sum 33 bits behind the point.
constexpr float kGateFloor = -8192.f;
__device__ __forceinline__ float floored(float g) { return g < kGateFloor ? kGateFloor : g; }  // NaN stays

struct DeltaShape {
  int64_t total;      // tokens
  int64_t seqlen;     // tokens of every sequence (no offsets)
  int64_t chunks;     // chunks of all sequences, or their upper bound (offsets)
  int nseq, hk, hv, dk, dv, dvp;  // dvp: dv rounded up to a slice
  float scale;
  // offsets: first token and first chunk of each sequence [nseq + 1]; nullptr otherwise
  const int32_t* tok;
  const int32_t* first;
};

template <typename T>
struct DeltaIn {
  const T *q, *k, *v;
  int64_t ldq, ldk, ldv;   // elements from one token to the next
  const float *g, *beta;   // [total][hv]
};

// What the forward pass keeps for the backward pass (and what its own kernels
// exchange), by chunk and value head.
struct DeltaKept {
  double* G;   // [64] running sums of g
  float* E;    // [64][64]
  float* P;    // [64][64]
  // As the walk's waves hold them, so that a store is 1 KB in one piece: for
  // every 16 columns and every 16 rows (tokens; rows of the state) 64 lanes by
  // 4, lane (l, h) rows 4 h .. 4 h + 3 of column l.
  float* M;    // [dvp / 16][4][64][4]
  float* S;    // [dvp / 16][dk padded / 16][64][4] the state before the chunk
};

struct Place {
  int seq, len;          // sequence, tokens of the chunk
  int64_t tok;           // first token
};

__device__ __forceinline__ int64_t first_chunk(const DeltaShape& s, int seq) {
  return s.first ? s.first[seq] : seq * div_up(s.seqlen, kChunk);
}
__device__ __forceinline__ int64_t first_token(const DeltaShape& s, int seq) {
  return s.tok ? s.tok[seq] : seq * s.seqlen;
}

// False for a chunk number past the last one (the grid covers an upper bound).
__device__ __forceinline__ bool find_chunk(const DeltaShape& s, int64_t c, Place& p) {
  int lo = 0;
  if (s.first) {
    if (c >= s.first[s.nseq]) return false;
    int hi = s.nseq;  // first[lo] <= c < first[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (s.first[mid] <= c) lo = mid;
      else hi = mid;
    }
  } else {
    lo = int(c / div_up(s.seqlen, kChunk));
  }
  const int64_t off = (c - first_chunk(s, lo)) * kChunk;
  p.seq = lo;
  p.tok = first_token(s, lo) + off;
  const int64_t left = first_token(s, lo + 1) - p.tok;
  p.len = left < kChunk ? int(left) : kChunk;
  return true;
}

// acc += A B for one 16 x 16 tile in fp32; lane l gives row (and column)
// l % 16 and, of every 16 values of k, the four from 4 (l / 16).  The
// result's lane l holds rows 4 (l / 16) + r of column l % 16.
// AT: A is stored [k][row] instead of [row][k]; BT: B as [k][col] instead of [col][k].
template <int K, bool AT, bool BT>
__device__ __forceinline__ void mma(f32x4& acc, const float* A, int lda, const float* B, int ldb) {
  const int l = threadIdx.x % 16, h = (threadIdx.x % kWave) / 16;
#pragma unroll 4
  for (int k = 0; k < K; k += 16) {
    f32x4 a, b;
    if constexpr (AT) {
#pragma unroll
      for (int j = 0; j < 4; ++j) a[j] = A[(k + 4 * h + j) * lda + l];
    } else {
      a = *reinterpret_cast<const f32x4*>(A + l * lda + k + 4 * h);
    }
    if constexpr (BT) {
#pragma unroll
      for (int j = 0; j < 4; ++j) b[j] = B[(k + 4 * h + j) * ldb + l];
    } else {
      b = *reinterpret_cast<const f32x4*>(B + l * ldb + k + 4 * h);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) acc = __builtin_amdgcn_mfma_f32_16x16x4f32(a[j], b[j], acc, 0, 0, 0);
  }
}

// ---------------------------------------------------------------------------
// Parts and operands
// ---------------------------------------------------------------------------
typedef uint32_t U2 __attribute__((ext_vector_type(2)));
typedef uint32_t U4 __attribute__((ext_vector_type(4)));
typedef __bf16 Frag __attribute__((ext_vector_type(8)));

template <typename T>
constexpr int kParts = sizeof(T) == 4 ? 3 : (std::is_same<T, _Float16>::value ? 2 : 1);

// The upper halves of two words, a's lowest.
__device__ __forceinline__ uint32_t upper(uint32_t a, uint32_t b) {
  return __builtin_amdgcn_perm(b, a, 0x07060302);
}
// The parts of n (2, 4 or 8) values, two to a word: each is the value less the
// ones before, cut off after 8 bits; the differences are exact.
template <int PARTS, int N>
__device__ __forceinline__ void split(const float (&x)[N], uint32_t (&p)[PARTS][N / 2]) {
  float r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) r[i] = x[i];
#pragma unroll
  for (int k = 0; k < PARTS; ++k) {
#pragma unroll
    for (int i = 0; i < N; i += 2)
      p[k][i / 2] = upper(__float_as_uint(r[i]), __float_as_uint(r[i + 1]));
    if (k + 1 < PARTS) {
#pragma unroll
      for (int i = 0; i < N; ++i) r[i] -= __uint_as_float(__float_as_uint(r[i]) & 0xffff0000u);
    }
  }
}
template <typename T>
using Eight = typename VecOf<T, 8>::type;
template <typename T>
__device__ __forceinline__ void split(const Eight<T>& v, uint32_t (&p)[kParts<T>][4]) {
  if constexpr (std::is_same<T, __bf16>::value) {
    const U4 u = __builtin_bit_cast(U4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[0][i] = u[i];
  } else {
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = float(v[i]);
    split<kParts<T>, 8>(x, p);
  }
}
// An operand's parts.
template <int PARTS>
struct Op {
  Frag f[PARTS];
};
__device__ __forceinline__ Frag frag(const uint32_t (&w)[4]) {
  const U4 u = {w[0], w[1], w[2], w[3]};
  return __builtin_bit_cast(Frag, u);
}
// ... of the results of two instructions (rows 4 h + r of each are the k).
template <int PARTS>
__device__ __forceinline__ Op<PARTS> operand(const f32x4& a, const f32x4& b) {
  const float x[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  uint32_t p[PARTS][4];
  split<PARTS, 8>(x, p);
  Op<PARTS> o;
#pragma unroll
  for (int k = 0; k < PARTS; ++k) o.f[k] = frag(p[k]);
  return o;
}
// ... of values that T holds exactly.
template <typename T>
__device__ __forceinline__ Op<kParts<T>> operand_of(const f32x4& a, const f32x4& b) {
  return operand<kParts<T>>(a, b);
}
// acc += a b, the small pairs first.
template <int NA, int NB>
__device__ __forceinline__ void mul(f32x4& acc, const Op<NA>& a, const Op<NB>& b) {
  constexpr int kTop = NA + NB - 2 < 2 ? NA + NB - 2 : 2;
#pragma unroll
  for (int s = kTop; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.f[i], b.f[s - i], acc, 0, 0, 0);
}

// The same for N sums with one factor in common, in turns: an instruction on
// the sum of the one before would wait for it.
template <int N, int NA, int NB>
__device__ __forceinline__ void mul_turns(f32x4* acc, const Op<NA> (&a)[N], const Op<NB>& b) {
  constexpr int kTop = NA + NB - 2 < 2 ? NA + NB - 2 : 2;
#pragma unroll
  for (int s = kTop; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB) {
#pragma unroll
        for (int n = 0; n < N; ++n)
          acc[n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[n].f[i], b.f[s - i], acc[n], 0, 0, 0);
      }
}

typedef __bf16 Quad __attribute__((ext_vector_type(4)));
__device__ __forceinline__ Frag join(const Quad& a, const Quad& b) {
  return Frag{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}
__device__ __forceinline__ Quad turned(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) Quad*)p);
}
// Rows l of an LDS array of rows of k (p: row 0, first of the 32 k; two reads
// of 8 bytes, free of conflicts if the rows are an odd number of those apart).
template <int PARTS>
__device__ __forceinline__ Op<PARTS> row_op(const char* p, int stride, int part) {
  const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
  Op<PARTS> o;
#pragma unroll
  for (int k = 0; k < PARTS; ++k) {
    const char* q = p + k * part + l * stride + 8 * h;
    o.f[k] = join(*reinterpret_cast<const Quad*>(q), *reinterpret_cast<const Quad*>(q + 32));
  }
  return o;
}
// Columns l of 32 lines of k (p: line 0, first of the 16 columns; free of
// conflicts if the lines are 32 bytes apart modulo 128).
__device__ __forceinline__ Quad turned(const char* p, int stride) {
  const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
  return turned(p + (4 * h + (l >> 2)) * stride + (l & 3) * 8);
}
template <int PARTS>
__device__ __forceinline__ Op<PARTS> col_op(const char* p, int stride, int part) {
  Op<PARTS> o;
#pragma unroll
  for (int k = 0; k < PARTS; ++k)
    o.f[k] = join(turned(p + k * part, stride), turned(p + k * part + 16 * stride, stride));
  return o;
}
// The chunk's rows of k and q are read both ways: their lines are not spread
// apart, but the 8-byte units of a line are exchanged by key(line), which
// sends both the same unit of 16 lines and four units of four neighbouring
// lines to 16 different places modulo 128 bytes.
__device__ __forceinline__ int key(int line) { return (line & 3) << 2 | (line >> 2 & 3); }
// Tokens 16 i + l, k = 32 b .. of [64][DK] rows.
template <int PARTS, int DK>
__device__ __forceinline__ Op<PARTS> token_rows(const char* p, int i, int b) {
  const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
  Op<PARTS> o;
#pragma unroll
  for (int k = 0; k < PARTS; ++k) {
    const char* q = p + k * kChunk * DK * 2 + (16 * i + l) * DK * 2;
    o.f[k] = join(*reinterpret_cast<const Quad*>(q + ((8 * b + h) ^ key(l)) * 8),
                  *reinterpret_cast<const Quad*>(q + ((8 * b + 4 + h) ^ key(l)) * 8));
  }
  return o;
}
// Columns 16 a + l, k = the tokens 32 b ..
template <int PARTS, int DK>
__device__ __forceinline__ Op<PARTS> token_cols(const char* p, int a, int b) {
  const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
  const int line = 4 * h + (l >> 2);
  Op<PARTS> o;
#pragma unroll
  for (int k = 0; k < PARTS; ++k) {
    const char* q = p + k * kChunk * DK * 2 + (32 * b + line) * DK * 2 +
                    ((4 * a + (l & 3)) ^ key(line)) * 8;
    o.f[k] = join(turned(q), turned(q + 16 * DK * 2));
  }
  return o;
}

// ... as they are: columns 16 a + l of the tokens 16 i + 4 h + r.
template <int PARTS, int DK>
__device__ __forceinline__ f32x4 token_tile(const char* p, int a, int i) {
  const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
  const int line = 4 * h + (l >> 2);
  f32x4 x = {0, 0, 0, 0};
#pragma unroll
  for (int k = PARTS - 1; k >= 0; --k) {
    const Quad v = turned(p + k * kChunk * DK * 2 + (16 * i + line) * DK * 2 +
                          ((4 * a + (l & 3)) ^ key(line)) * 8);
    x += f32x4{float(v[0]), float(v[1]), float(v[2]), float(v[3])};
  }
  return x;
}

// A lower triangle of 64 x 64 in 16 x 16 blocks: line i has 16 (i / 16 + 1)
// columns, and the lines are an odd number of 32 bytes apart.
__device__ __forceinline__ constexpr int tri_stride(int t) {
  return t == 0 ? 32 : t == 3 ? 160 : 96;
}
__device__ __forceinline__ constexpr int tri_at(int t) {   // of line 16 t
  return t == 0 ? 0 : t == 1 ? 512 : t == 2 ? 2048 : 3584;
}
constexpr int kTri = 6144;   // bytes of a part
// Operand with rows j = 16 tj + l and k = i = 32 kb .. (the triangle turned).
template <int PARTS>
__device__ __forceinline__ Op<PARTS> tri_turned(const char* p, int tj, int kb) {
  Op<PARTS> o;
  const Quad zero = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < PARTS; ++k) {
    const char* q = p + k * kTri + 32 * tj;
    const int t = 2 * kb;
    o.f[k] = join(t >= tj ? turned(q + tri_at(t), tri_stride(t)) : zero,
                  t + 1 >= tj ? turned(q + tri_at(t + 1), tri_stride(t + 1)) : zero);
  }
  return o;
}
// The same triangle stored turned, line j with its 64 - 16 (j / 16) rows i:
// what a wave holds of a block, four rows of a column a lane, is 8 bytes of it.
__device__ __forceinline__ constexpr int upper_stride(int t) { return tri_stride(3 - t); }
__device__ __forceinline__ constexpr int upper_at(int t) {   // of line 16 t
  return t == 0 ? 0 : t == 1 ? 2560 : t == 2 ? 4096 : 5632;
}
// Operand with rows i = 16 ti + l and k = j = 32 kb ...
template <int PARTS>
__device__ __forceinline__ Op<PARTS> upper_rows(const char* p, int ti, int kb) {
  Op<PARTS> o;
  const Quad zero = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < PARTS; ++k) {
    const int t = 2 * kb;
    const char* q = p + k * kTri + 32 * (ti - t);
    o.f[k] = join(t <= ti ? turned(q + upper_at(t), upper_stride(t)) : zero,
                  t + 1 <= ti ? turned(q + upper_at(t + 1) - 32, upper_stride(t + 1)) : zero);
  }
  return o;
}
// Operand with rows j = 16 tj + l and k = i = 32 kb ...
template <int PARTS>
__device__ __forceinline__ Op<PARTS> upper_turned(const char* p, int tj, int kb) {
  const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
  Op<PARTS> o;
  const Quad zero = {0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < PARTS; ++k) {
    const char* q = p + k * kTri + upper_at(tj) + l * upper_stride(tj) + 32 * (2 * kb - tj) + 8 * h;
    o.f[k] = join(2 * kb >= tj ? *reinterpret_cast<const Quad*>(q) : zero,
                  2 * kb + 1 >= tj ? *reinterpret_cast<const Quad*>(q + 32) : zero);
  }
  return o;
}

// A chunk's rows of WIDTH elements (zero past `len` rows and `have` columns),
// 8 elements a load, held in registers between the load and the LDS store so
// that the next chunk's rows travel while this one is worked on.
// WHOLE: the columns are a multiple of 8.
template <typename T, int WIDTH, bool WHOLE>
struct Rows {
  static constexpr int kLoads = kChunk * WIDTH / 8 / kDeltaBlock;
  static_assert(kLoads >= 1, "a load per thread");
  Eight<T> v[kLoads];
  uint32_t in;   // load i is of an existing row and column: bit i
  // No lane branches: a load of what does not exist goes to row 0 instead, and
  // put() drops it (a branch's join would wait for each load in turn).
  __device__ __forceinline__ void fetch(const T* p, int64_t ld, int len, int have) {
    in = 0;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = threadIdx.x + i * kDeltaBlock;
      const int row = at / (WIDTH / 8), col = at % (WIDTH / 8) * 8;
      const bool on = row < len && col < have;
      in |= uint32_t(on) << i;
      if constexpr (WHOLE) {
        v[i] = *reinterpret_cast<const Eight<T>*>(p + (on ? row * ld + col : 0));
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool here = on && col + j < have;
          const T x = p[here ? row * ld + col + j : 0];
          v[i][j] = here ? x : T(0.f);
        }
      }
    }
  }
  // its parts, kChunk * WIDTH * 2 bytes each
  __device__ __forceinline__ void put(char* lds) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = threadIdx.x + i * kDeltaBlock;
      const int row = at / (WIDTH / 8), unit = at % (WIDTH / 8) * 2;
      uint32_t p[kParts<T>][4];
      split<T>(v[i], p);
      const uint32_t keep = 0u - (in >> i & 1u);
#pragma unroll
      for (int k = 0; k < kParts<T>; ++k) {
#pragma unroll
        for (int j = 0; j < 4; ++j) p[k][j] &= keep;
        char* d = lds + k * kChunk * WIDTH * 2 + row * WIDTH * 2;
        *reinterpret_cast<U2*>(d + (unit ^ key(row)) * 8) = U2{p[k][0], p[k][1]};
        *reinterpret_cast<U2*>(d + (unit + 1 ^ key(row)) * 8) = U2{p[k][2], p[k][3]};
      }
    }
  }
};
// A 64 x 64 lower triangle of fp32, four elements a load.
struct Square {
  f32x4 v[4];
  __device__ __forceinline__ void fetch(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      v[i] = *reinterpret_cast<const f32x4*>(p + (threadIdx.x + i * kDeltaBlock) * 4);
  }
  template <typename F>
  __device__ __forceinline__ void put(F&& at, int part) const {   // at(row, col): where
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = (threadIdx.x + i * kDeltaBlock) / 16, col = threadIdx.x % 16 * 4;
      const float x[4] = {v[i][0], v[i][1], v[i][2], v[i][3]};
      uint32_t p[3][2];
      split<3, 4>(x, p);
      char* d = at(row, col);
      if (d) {
#pragma unroll
        for (int k = 0; k < 3; ++k) *reinterpret_cast<U2*>(d + k * part) = U2{p[k][0], p[k][1]};
      }
    }
  }
  __device__ __forceinline__ void put_tri(char* lds) const {
    put([&](int row, int col) -> char* {
      const int t = row / 16;
      return col / 16 <= t ? lds + tri_at(t) + row % 16 * tri_stride(t) + col * 2 : nullptr;
    }, kTri);
  }
};

// The sequences' tokens and chunks from the caller's offsets, in one
// workgroup.  Offsets that fall or leave [0, total] cannot be refused here
// (they are on the device): each is taken as the largest of its
// predecessors and itself, clamped, so that no kernel leaves the arrays.
// The tokens before the first and behind the last sequence belong to none:
// their outputs are zero.
struct Gap {
  void* p;
  int64_t width;  // bytes of a token
};
struct Gaps {
  Gap g[5];
};
__device__ __forceinline__ void clear_gaps(const int32_t* tok, int nseq, int64_t total,
                                           const Gaps& gaps) {
  const int64_t head = tok[0], tail = tok[nseq];
  for (int n = 0; n < 5; ++n) {
    if (!gaps.g[n].p) continue;
    uint16_t* p = (uint16_t*)gaps.g[n].p;
    const int64_t w = gaps.g[n].width / 2;
    for (int64_t i = threadIdx.x; i < head * w; i += kDeltaBlock) p[i] = 0;
    for (int64_t i = tail * w + threadIdx.x; i < total * w; i += kDeltaBlock) p[i] = 0;
  }
}
__global__ __launch_bounds__(kDeltaBlock) void k_delta_plan(const int32_t* __restrict__ cu,
                                                            int nseq, int64_t total, int32_t* tok,
                                                            int32_t* first, Gaps gaps) {
  if (threadIdx.x < kWave) {
    // 64 offsets at a time: their running maximum, then the chunks up to each
    int carry = 0, chunks = 0;
    for (int b = 0; b <= nseq; b += kWave) {
      const int i = b + int(threadIdx.x);
      int v = i <= nseq ? cu[i] : 0;
      v = v < 0 ? 0 : (v > total ? int(total) : v);
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const int u = __shfl_up(v, d, kWave);
        if (int(threadIdx.x) >= d && u > v) v = u;
      }
      if (b > 0 && v < carry) v = carry;
      int before = __shfl_up(v, 1, kWave);
      if (threadIdx.x == 0) before = b == 0 ? v : carry;
      int n = (v - before + kChunk - 1) / kChunk;  // chunks of sequence i - 1
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const int u = __shfl_up(n, d, kWave);
        if (int(threadIdx.x) >= d) n += u;
      }
      if (i <= nseq) {
        tok[i] = v;
        first[i] = chunks + n;
      }
      carry = __shfl(v, kWave - 1, kWave);
      chunks += __shfl(n, kWave - 1, kWave);
    }
  }
  __syncthreads();
  clear_gaps(tok, nseq, total, gaps);
}
__global__ __launch_bounds__(kDeltaBlock) void k_delta_gaps(const int32_t* tok, int nseq,
                                                            int64_t total, Gaps gaps) {
  clear_gaps(tok, nseq, total, gaps);
}

// E, P and G of every chunk and value head.  Wave w works on rows 16 w ..
// 16 w + 15.  E is solved in 16 x 16 blocks: the diagonal blocks by
// substitution (a column a lane), the others as
//   Z = sum_{J <= K < I} A_IK T_KJ,  E_IJ = Z - E_II (B_I Z),  T_IJ = -B_I E_IJ,
// a block column per wave, with T = I - B E the inverse so far.  Bound by the
// latency of the substitution and its barriers, four workgroups a CU: 93 us
// for 4 x 4096 tokens and 16 heads of 128 in bf16 (whose 200 MB take 40).
template <typename T, int DK>
struct PrepareLds {
  static constexpr int kRow = kParts<T> * kChunk * DK * 2;
  static constexpr int kSquare = kChunk * kLdC * 4;
  static constexpr int kFirst = 2 * kRow > 2 * kSquare ? 2 * kRow : 2 * kSquare;
  static constexpr int kBytes = kFirst + kSquare + kChunk * 12;
};
template <typename T, int DK, bool WHOLE>
__global__ __launch_bounds__(kDeltaBlock) void k_delta_prepare(DeltaShape s, DeltaIn<T> in,
                                                               DeltaKept kept) {
  using L = PrepareLds<T, DK>;
  constexpr int NP = kParts<T>;
  extern __shared__ __align__(16) char smem[];
  char* kf = smem;                        // k's and q's parts
  char* qf = smem + L::kRow;
  float* A = (float*)(smem + L::kFirst);  // [64][kLdC]
  float* E = (float*)smem;                // over k and q once they are used up
  float* Tm = E + kChunk * kLdC;
  double* G = (double*)(A + kChunk * kLdC);
  float* beta = (float*)(G + kChunk);
  Place p;
  if (!find_chunk(s, blockIdx.x, p)) return;
  const int vh = blockIdx.y, kh = vh / (s.hv / s.hk);
  const int t = threadIdx.x, w = t / kWave, l = t % 16, h = (t % kWave) / 16;
  {
    Rows<T, DK, WHOLE> kr, qr;
    kr.fetch(in.k + p.tok * in.ldk + int64_t(kh) * s.dk, in.ldk, p.len, s.dk);
    qr.fetch(in.q + p.tok * in.ldq + int64_t(kh) * s.dk, in.ldq, p.len, s.dk);
    kr.put(kf);
    qr.put(qf);
  }
  if (t < kChunk) {
    const int64_t at = (p.tok + t) * s.hv + vh;
    double g = t < p.len ? double(floored(in.g[at])) : 0.0;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const double u = __shfl_up(g, d, kWave);
      if (t >= d) g += u;
    }
    G[t] = g;
    beta[t] = t < p.len ? in.beta[at] : 0.f;
  }
  __syncthreads();
  const int64_t slot = int64_t(blockIdx.x) * s.hv + vh;
  if (t < kChunk) kept.G[slot * kChunk + t] = G[t];
  float* Pg = kept.P + slot * kChunk * kChunk;
  for (int J = 0; J < 4; ++J) {
    f32x4 kk = {0, 0, 0, 0}, qk = {0, 0, 0, 0};
    if (J <= w) {
#pragma unroll
      for (int b = 0; b < DK / 32; ++b) {
        const Op<NP> kj = token_rows<NP, DK>(kf, J, b);
        mul(kk, token_rows<NP, DK>(kf, w, b), kj);
        mul(qk, token_rows<NP, DK>(qf, w, b), kj);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 16 * w + 4 * h + r, j = 16 * J + l;
      const float d = j <= i ? expf(float(G[i] - G[j])) : 0.f;
      A[i * kLdC + j] = j < i ? d * kk[r] : 0.f;
      Pg[i * kChunk + j] = j <= i ? s.scale * d * qk[r] : 0.f;
    }
  }
  __syncthreads();
  // diagonal block w: column l (the four lane groups do the same)
  {
    float e[16], tc[16];
    const float* Ab = A + (16 * w) * kLdC + 16 * w;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float x = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (j < i) x += Ab[i * kLdC + j] * tc[j];
      e[i] = x;
      tc[i] = (i == l ? 1.f : 0.f) - beta[16 * w + i] * x;
    }
    if (h == 0) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        E[(16 * w + i) * kLdC + 16 * w + l] = e[i];
        Tm[(16 * w + i) * kLdC + 16 * w + l] = tc[i];
      }
    }
  }
  __syncthreads();
  // block column w: its blocks below the diagonal, in order
  for (int I = w + 1; I < 4; ++I) {
    f32x4 z = {0, 0, 0, 0};
    for (int K = w; K < I; ++K)
      mma<16, false, true>(z, A + 16 * I * kLdC + 16 * K, kLdC, Tm + 16 * K * kLdC + 16 * w, kLdC);
    // B_I Z through this wave's own block of Tm
    float* Tb = Tm + 16 * I * kLdC + 16 * w;
#pragma unroll
    for (int r = 0; r < 4; ++r) Tb[(4 * h + r) * kLdC + l] = beta[16 * I + 4 * h + r] * z[r];
    __builtin_amdgcn_wave_barrier();
    f32x4 y = {0, 0, 0, 0};
    mma<16, false, true>(y, E + 16 * I * kLdC + 16 * I, kLdC, Tb, kLdC);
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float e = z[r] - y[r];
      E[(16 * I + 4 * h + r) * kLdC + 16 * w + l] = e;
      Tb[(4 * h + r) * kLdC + l] = -beta[16 * I + 4 * h + r] * e;
    }
    __builtin_amdgcn_wave_barrier();
  }
  __syncthreads();
  float* Eg = kept.E + slot * kChunk * kChunk;
  for (int i = t; i < kChunk * kChunk; i += kDeltaBlock) {
    const int row = i / kChunk, col = i % kChunk;
    Eg[i] = col < row ? E[row * kLdC + col] : 0.f;
  }
}

// Per-token factors of a chunk, computed by its first 64 threads.
struct alignas(16) Factors {
  float beta[kChunk];
  float in[kChunk];    // exp(G)
  float out[kChunk];   // exp(G_L - G)
  float all;           // exp(G_L)
};
__device__ __forceinline__ void set_factors(Factors& f, double g, double end, float beta) {
  const int t = threadIdx.x;
  if (t < kChunk) {
    f.beta[t] = beta;
    f.in[t] = expf(float(g));
    f.out[t] = expf(float(end - g));
    if (t == 0) f.all = expf(float(end));
  }
}
__device__ __forceinline__ void set_factors(Factors& f, const DeltaShape& s, const double* G,
                                            const float* beta, const Place& p, int vh) {
  const int t = threadIdx.x;
  if (t < kChunk)
    set_factors(f, G[t], G[kChunk - 1], t < p.len ? beta[(p.tok + t) * s.hv + vh] : 0.f);
}

__device__ __forceinline__ Place chunk_of(int seq, int64_t first, int64_t end, int64_t c) {
  Place p;
  p.seq = seq;
  p.tok = first + c * kChunk;
  const int64_t left = end - p.tok;
  p.len = left < kChunk ? int(left) : kChunk;
  return p;
}

// A wave's 16 columns of [dk][dv] arrays of a sequence and head, rows 16 a +
// 4 h + r in f32x4 number a.
template <int DK>
__device__ __forceinline__ void load_state(f32x4 (&S)[DK / 16], const float* p, const DeltaShape& s,
                                           int64_t head, int c0) {
  const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
#pragma unroll
  for (int a = 0; a < DK / 16; ++a)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * a + 4 * h + r, col = c0 + l;
      S[a][r] = p && row < s.dk && col < s.dv ? p[(head * s.dk + row) * s.dv + col] : 0.f;
    }
}
template <int DK>
__device__ __forceinline__ void store_state(const f32x4 (&S)[DK / 16], float* p,
                                            const DeltaShape& s, int64_t head, int c0) {
  const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
#pragma unroll
  for (int a = 0; a < DK / 16; ++a)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * a + 4 * h + r, col = c0 + l;
      if (row < s.dk && col < s.dv) p[(head * s.dk + row) * s.dv + col] = S[a][r];
    }
}
// A chunk's rows of 64 columns of v or do, as they are, in LDS.
template <typename T>
struct Values {
  static constexpr int kBytes = kChunk * kWalk * int(sizeof(T));
  static constexpr int kLoads = kChunk * kWalk / 8 / kDeltaBlock;
  Eight<T> v[kLoads];
  // have: columns from the first on; whole: a multiple of 8 of them
  __device__ __forceinline__ void fetch(const T* p, int64_t ld, int len, int have, bool whole) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = threadIdx.x + i * kDeltaBlock;
      const int row = at / (kWalk / 8), col = at % (kWalk / 8) * 8;
      const bool on = row < len && col < have;
      if (whole) {
        const Eight<T> x = *reinterpret_cast<const Eight<T>*>(p + (on ? row * ld + col : 0));
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = on ? x[j] : T(0.f);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool here = on && col + j < have;
          const T x = p[here ? row * ld + col + j : 0];
          v[i][j] = here ? x : T(0.f);
        }
      }
    }
  }
  __device__ __forceinline__ void put(char* lds) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      *reinterpret_cast<Eight<T>*>(lds + (threadIdx.x + i * kDeltaBlock) * 8 *
                                             int(sizeof(T))) = v[i];
  }
  // tokens 16 i + 4 h + r of columns col + l
  static __device__ __forceinline__ f32x4 tile(const char* lds, int col, int i) {
    const int l = threadIdx.x % 16, h = threadIdx.x % kWave / 16;
    f32x4 x;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        x[r] = *reinterpret_cast<const T*>(lds + ((16 * i + 4 * h + r) * kWalk + col + l) * 4);
    } else {
      typedef T V4 __attribute__((ext_vector_type(4)));
      const V4 v = __builtin_bit_cast(V4, turned(lds + 16 * i * kWalk * 2 + col * 2, kWalk * 2));
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] = float(v[r]);
    }
    return x;
  }
};
__device__ __forceinline__ f32x4 quad(const float* p, int i) {   // [16 i + 4 h ..]
  return *reinterpret_cast<const f32x4*>(p + 16 * i + 4 * (threadIdx.x % kWave / 16));
}

// The walks' workgroups: four waves that bring k, E and the like of the next
// chunk into LDS, and behind them waves that walk, 16 columns each, so that neither memory's
// latency nor the cutting of k and E lies in the chain from chunk to chunk.
// Two chunks' worth where LDS holds them; else the bringing waves keep the next
// chunk in registers and store it when the walking ones have read this one's.
constexpr int kWalkBlock = kDeltaBlock + kWalk / 16 * kWave;
template <int SLOT>
constexpr int kWalkDepth = 2 * SLOT <= 160 * 1024 ? 2 : 1;
// All LDS accesses of the wave are done, then those of the others; loads and
// stores of memory go on.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
template <int DEPTH, typename F, typename P>
__device__ __forceinline__ void bring(int64_t count, F&& fetch, P&& put) {
  if (count == 0) return;
  fetch(0);
  if constexpr (DEPTH == 2) {
    put(0);
    if (count > 1) fetch(1);
    lds_barrier();
    for (int64_t c = 0; c < count; ++c) {
      if (c + 1 < count) put(int(c + 1) & 1);
      if (c + 2 < count) fetch(c + 2);
      lds_barrier();
    }
  } else {
    for (int64_t c = 0; c < count; ++c) {
      lds_barrier();
      put(0);
      lds_barrier();
      if (c + 1 < count) fetch(c + 1);
    }
  }
}
template <int DEPTH, typename F>
__device__ __forceinline__ void walk(int64_t count, F&& chunk) {   // chunk(c, slot)
  if (DEPTH == 2 && count > 0) lds_barrier();
  for (int64_t c = 0; c < count; ++c) {
    if constexpr (DEPTH == 1) {
      lds_barrier();
      lds_barrier();
    }
    chunk(c, DEPTH == 2 ? int(c) & 1 : 0);
    if constexpr (DEPTH == 2) lds_barrier();
  }
}

// N products whose operands come from LDS, each read while the one before is
// multiplied: first holds those of product 0; behind the last, next() may
// read ahead.  (The fences keep the reads where they are; left alone the
// compiler puts each in front of its use and the wave waits for it.)
template <int N, typename O, typename L, typename U, typename X>
__device__ __forceinline__ void pipe(O (&first), L&& load, U&& use, X&& next) {
  O o[2];
  o[0] = first;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i + 1 < N) o[(i + 1) % 2] = load(i + 1);
    else next();
    __builtin_amdgcn_sched_barrier(0);
    use(i, o[i % 2]);
    __builtin_amdgcn_sched_barrier(0);
  }
}
template <int PARTS, int N>
struct Ops {
  Op<PARTS> o[N];
};
// The tiles a step of a product with the tokens' rows takes.
template <typename T>
constexpr int kTilesAStep = kParts<T> == 1 ? 4 : 2;

// The states' walk forward: M of every chunk and the state before it.  A
// workgroup has 64 columns of a sequence and head, a wave 16 of them and all
// dk rows in registers; k and E are shared in LDS.  Bound by the chain of one
// chunk, 132 matrix instructions of 16 cycles and the cutting of 64 values a
// lane (bf16, dk = 128): 3.9 us a chunk, 250 us for 4 x 4096 tokens and 16
// heads of 128; 2.8 us of them without the stores of S and M.
template <typename T, int DK>
struct StatesLds {
  static constexpr int kE = kParts<T> * kChunk * DK * 2, kEStride = 136;
  static constexpr int kEPart = kChunk * kEStride;
  static constexpr int kV = kE + 3 * kEPart, kFactors = kV + Values<T>::kBytes;
  static constexpr int kSlot = kFactors + int(sizeof(Factors));
  static constexpr int kDepth = kWalkDepth<kSlot>, kBytes = kDepth * kSlot;
};
template <typename T, int DK, bool WHOLE>
__global__ __launch_bounds__(kWalkBlock) void k_delta_states(DeltaShape s, DeltaIn<T> in,
                                                             DeltaKept kept,
                                                             const float* __restrict__ s0,
                                                             float* __restrict__ send) {
  using L = StatesLds<T, DK>;
  constexpr int NP = kParts<T>, RT = DK / 16, KB = DK / 32;
  extern __shared__ __align__(16) char lds[];
  const int slices = int(div_up(s.dvp, kWalk));
  const int t = threadIdx.x;
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int vh = blockIdx.x / slices % s.hv, seq = blockIdx.x / slices / s.hv;
  const int kh = vh / (s.hv / s.hk);
  const int64_t begin = first_chunk(s, seq), count = first_chunk(s, seq + 1) - begin;
  const int64_t first = first_token(s, seq), past = first_token(s, seq + 1);
  const int64_t head = int64_t(seq) * s.hv + vh;
  const int wc = 16 * (w - 4), c0 = blockIdx.x % slices * kWalk + wc;
  if (w < 4) {
    Rows<T, DK, WHOLE> kr;
    Square er;
    Values<T> vr;
    const int col = blockIdx.x % slices * kWalk;
    double g = 0.0, gend = 0.0;
    float be = 0.f;
    bring<L::kDepth>(count, [&](int64_t c) {
      const Place p = chunk_of(seq, first, past, c);
      const int64_t slot = (begin + c) * s.hv + vh;
      kr.fetch(in.k + p.tok * in.ldk + int64_t(kh) * s.dk, in.ldk, p.len, s.dk);
      er.fetch(kept.E + slot * kChunk * kChunk);
      vr.fetch(in.v + p.tok * in.ldv + int64_t(vh) * s.dv + col, in.ldv, p.len, s.dv - col,
               s.dv % 8 == 0);
      if (t < kChunk) {
        g = kept.G[slot * kChunk + t];
        gend = kept.G[slot * kChunk + kChunk - 1];
        be = t < p.len ? in.beta[(p.tok + t) * s.hv + vh] : 0.f;
      }
    }, [&](int n) {
      char* const d = lds + n * L::kSlot;
      kr.put(d);
      er.put([&](int row, int col) { return d + L::kE + row * L::kEStride + col * 2; }, L::kEPart);
      vr.put(d + L::kV);
      set_factors(*(Factors*)(d + L::kFactors), g, gend, be);
    });
    return;
  }
  const bool live = c0 < s.dvp;
  f32x4 S[RT];
  load_state<DK>(S, s0, s, head, c0);
  walk<L::kDepth>(count, [&](int64_t c, int n_) {
    if (!live) return;
    const char* const smem = lds + n_ * L::kSlot;
    const Factors& f = *(const Factors*)(smem + L::kFactors);
    const int64_t slot = (begin + c) * s.hv + vh;
    constexpr int GT = kTilesAStep<T>, kSide = 4 / GT;
    typedef Ops<NP, GT> Tokens;
    auto rows = [&](int i) {   // step i of k S
      Tokens o;
#pragma unroll
      for (int n = 0; n < GT; ++n) o.o[n] = token_rows<NP, DK>(smem, i % kSide * GT + n, i / kSide);
      return o;
    };
    auto cols = [&](int i) {   // step i of k^T N
      Tokens o;
#pragma unroll
      for (int n = 0; n < GT; ++n)
        o.o[n] = token_cols<NP, DK>(smem, i % (RT / GT) * GT + n, i / (RT / GT));
      return o;
    };
    auto tri = [&](int i) {    // rows 0 and 1, 2 and 3 of E's first half, 2 and 3 of its second
      Ops<3, 2> o;
#pragma unroll
      for (int n = 0; n < 2; ++n)
        o.o[n] = row_op<3>(smem + L::kE + 16 * ((i ? 2 : 0) + n) * L::kEStride + i / 2 * 64,
                           L::kEStride, L::kEPart);
      return o;
    };
    float* Sg = kept.S + (slot * s.dvp + c0) * DK + t % kWave * 4;
    Tokens k0 = rows(0);
    Op<3> so[2];
    so[0] = operand<3>(S[0], S[1]);
#pragma unroll
    for (int a = 0; a < RT; ++a) *reinterpret_cast<f32x4*>(Sg + 256 * a) = S[a];
    f32x4 R[4], bR[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) R[i] = f32x4{0, 0, 0, 0};
    Ops<3, 2> e0;
    pipe<KB * kSide>(k0, rows, [&](int i, const Tokens& o) {
      // the next block is cut while this one is multiplied
      if (i % kSide == 0 && i / kSide + 1 < KB)
        so[(i / kSide + 1) % 2] = operand<3>(S[2 * (i / kSide) + 2], S[2 * (i / kSide) + 3]);
      mul_turns(R + i % kSide * GT, o.o, so[i / kSide % 2]);
    }, [&] { e0 = tri(0); });
    Op<3> n[2];
    auto see = [&](int b) {   // R of tokens 32 b ..
#pragma unroll
      for (int i = 2 * b; i < 2 * b + 2; ++i) {
        R[i] = Values<T>::tile(smem + L::kV, wc, i) - quad(f.in, i) * R[i];
        bR[i] = quad(f.beta, i) * R[i];
      }
      n[b] = operand<3>(bR[2 * b], bR[2 * b + 1]);
    };
    see(0);
    float* Mg = kept.M + (slot * s.dvp + c0) * kChunk + t % kWave * 4;
    f32x4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f32x4{0, 0, 0, 0};
    pipe<3>(e0, tri, [&](int i, const Ops<3, 2>& o) {
      if (i == 0) see(1);
      mul_turns(x + (i ? 2 : 0), o.o, n[i / 2]);
    }, [&] { k0 = cols(0); });
    auto correct = [&](int b) {   // M and exp(G_L - G) N of tokens 32 b ..
#pragma unroll
      for (int i = 2 * b; i < 2 * b + 2; ++i) {
        R[i] -= x[i];
        *reinterpret_cast<f32x4*>(Mg + 256 * i) = R[i];
        bR[i] = quad(f.out, i) * (quad(f.beta, i) * R[i]);
      }
      n[b] = operand<3>(bR[2 * b], bR[2 * b + 1]);
    };
    const float all = f.all;
#pragma unroll
    for (int a = 0; a < RT; ++a) S[a] *= all;
    correct(0);
    pipe<RT / GT * 2>(k0, cols, [&](int i, const Tokens& o) {
      if (i == 0) correct(1);
      mul_turns(S + i % (RT / GT) * GT, o.o, n[i / (RT / GT)]);
    }, [] {});
  });
  if (send && live) store_state<DK>(S, send, s, head, c0);
}

// o = scale exp(G) (q S) + P N, a workgroup per chunk and value head, a slice
// of the columns at a time; a wave has 16 tokens, its rows of q and P stay in
// registers.  Bound by reading S and M (96 KB a chunk and head): 162 us for 4 x
// 4096 tokens and 16 heads of 128, 2.8 TB/s.
template <typename T, int DK>
struct OutLds {
  static constexpr int NS = 3;   // parts of the fp32 factors
  static constexpr int kSStride = 2 * DK + 8, kNStride = 136;
  static constexpr int kSPart = kSlice * kSStride, kNPart = kSlice * kNStride;
  static constexpr int kN = NS * kSPart, kFactors = kN + NS * kNPart;
  static constexpr int kBytes = kFactors + int(sizeof(Factors));
};
template <typename T, int DK>
__global__ __launch_bounds__(kDeltaBlock) void k_delta_out(DeltaShape s, DeltaIn<T> in,
                                                           DeltaKept kept, T* __restrict__ o) {
  using L = OutLds<T, DK>;
  constexpr int NP = kParts<T>, NS = L::NS, KB = DK / 32, NT = DK / 16;
  extern __shared__ __align__(16) char smem[];
  Factors& f = *(Factors*)(smem + L::kFactors);
  Place p;
  if (!find_chunk(s, blockIdx.x, p)) return;
  const int vh = blockIdx.y, kh = vh / (s.hv / s.hk);
  const int64_t slot = int64_t(blockIdx.x) * s.hv + vh;
  const int t = threadIdx.x, w = t / kWave, l = t % 16, h = (t % kWave) / 16;
  set_factors(f, s, kept.G + slot * kChunk, in.beta, p, vh);
  // rows 16 w + l of q and P; 4 h and 16 more of every 32 columns
  Op<NP> qo[KB];
  Op<NS> po[2];
  {
    const int row = 16 * w + l;
    const T* q = in.q + (p.tok + row) * in.ldq + int64_t(kh) * s.dk + 4 * h;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      float x[2][4];
#pragma unroll
      for (int n = 0; n < 2; ++n)
        load_f32<4>(q + 32 * b + 16 * n, row < p.len ? s.dk - 32 * b - 16 * n - 4 * h : 0, x[n]);
      qo[b] = operand_of<T>(f32x4{x[0][0], x[0][1], x[0][2], x[0][3]},
                            f32x4{x[1][0], x[1][1], x[1][2], x[1][3]});
    }
    const float* P = kept.P + slot * kChunk * kChunk + row * kChunk + 4 * h;
#pragma unroll
    for (int b = 0; b < 2; ++b)
      po[b] = operand<NS>(*reinterpret_cast<const f32x4*>(P + 32 * b),
                          *reinterpret_cast<const f32x4*>(P + 32 * b + 16));
  }
  const float* Sg = kept.S + slot * s.dvp * DK;
  const float* Mg = kept.M + slot * s.dvp * kChunk;
  constexpr int kLoads = kSlice * DK / 4 / kDeltaBlock;
  f32x4 sv[kLoads], mv[2];
  auto fetch = [&](int c0) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i)
      sv[i] = *reinterpret_cast<const f32x4*>(Sg + int64_t(c0) * DK + (t + i * kDeltaBlock) * 4);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      mv[i] = *reinterpret_cast<const f32x4*>(Mg + int64_t(c0) * kChunk + (t + i * kDeltaBlock) * 4);
  };
  fetch(0);
  for (int c0 = 0; c0 < s.dvp; c0 += kSlice) {
    __syncthreads();
    auto put = [&](const f32x4& x, char* d, int part) {
      const float y[4] = {x[0], x[1], x[2], x[3]};
      uint32_t u[NS][2];
      split<NS, 4>(y, u);
#pragma unroll
      for (int k = 0; k < NS; ++k) *reinterpret_cast<U2*>(d + k * part) = U2{u[k][0], u[k][1]};
    };
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int n = 4 * i + w;   // of the slice's blocks of 16 columns by 16 rows
      put(sv[i], smem + (n / NT * 16 + l) * L::kSStride + (n % NT * 16 + 4 * h) * 2, L::kSPart);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
      put(mv[i] * quad(f.beta, w),
          smem + L::kN + (16 * i + l) * L::kNStride + (16 * w + 4 * h) * 2, L::kNPart);
    __syncthreads();
    if (c0 + kSlice < s.dvp) fetch(c0 + kSlice);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      f32x4 acc = {0, 0, 0, 0};
#pragma unroll
      for (int b = 0; b < KB; ++b)
        mul(acc, qo[b], row_op<NS>(smem + 16 * n * L::kSStride + 64 * b, L::kSStride, L::kSPart));
      acc *= s.scale * quad(f.in, w);
#pragma unroll
      for (int b = 0; b < 2; ++b)
        if (2 * b <= w)
          mul(acc, po[b], row_op<NS>(smem + L::kN + 16 * n * L::kNStride + 64 * b, L::kNStride,
                                     L::kNPart));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * h + r, col = c0 + 16 * n + l;
        if (row < p.len && col < s.dv) o[((p.tok + row) * s.hv + vh) * s.dv + col] = T(acc[r]);
      }
    }
  }
}

// The walk backward: X of every chunk, dv = B X, and the gradient of the
// state behind it; as the walk forward: 5.6 us a chunk, 357 us for 4 x 4096
// tokens and 16 heads of 128 in bf16.  fp16 and fp32 with dk > 64 hold one
// chunk in LDS, not two.
template <typename T, int DK>
struct AdjointLds {
  static constexpr int kQ = kParts<T> * kChunk * DK * 2, kE = 2 * kQ, kP = kE + 3 * kTri;
  static constexpr int kO = kP + 3 * kTri, kFactors = kO + Values<T>::kBytes;
  static constexpr int kSlot = kFactors + int(sizeof(Factors));
  static constexpr int kDepth = kWalkDepth<kSlot>, kBytes = kDepth * kSlot;
};
template <typename T, int DK, bool WHOLE>
__global__ __launch_bounds__(kWalkBlock) void k_delta_adjoint(
    DeltaShape s, DeltaIn<T> in, DeltaKept kept, const T* __restrict__ dout, int64_t ldo,
    const float* __restrict__ dsend, float* __restrict__ X, float* __restrict__ dS,
    T* __restrict__ dv, float* __restrict__ ds0) {
  using L = AdjointLds<T, DK>;
  constexpr int NP = kParts<T>, RT = DK / 16, KB = DK / 32;
  extern __shared__ __align__(16) char lds[];
  const int slices = int(div_up(s.dvp, kWalk));
  const int t = threadIdx.x, l = t % 16, h = (t % kWave) / 16;
  const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x) / kWave);
  const int vh = blockIdx.x / slices % s.hv, seq = blockIdx.x / slices / s.hv;
  const int kh = vh / (s.hv / s.hk);
  const int64_t begin = first_chunk(s, seq), count = first_chunk(s, seq + 1) - begin;
  const int64_t first = first_token(s, seq), past = first_token(s, seq + 1);
  const int64_t head = int64_t(seq) * s.hv + vh;
  const int wc = 16 * (w - 4), c0 = blockIdx.x % slices * kWalk + wc;
  if (w < 4) {
    Rows<T, DK, WHOLE> kr, qr;
    Square er, pr;
    Values<T> orow;
    const int col = blockIdx.x % slices * kWalk;
    double g = 0.0, gend = 0.0;
    float be = 0.f;
    bring<L::kDepth>(count, [&](int64_t i) {
      const int64_t c = count - 1 - i;
      const Place p = chunk_of(seq, first, past, c);
      const int64_t slot = (begin + c) * s.hv + vh;
      kr.fetch(in.k + p.tok * in.ldk + int64_t(kh) * s.dk, in.ldk, p.len, s.dk);
      qr.fetch(in.q + p.tok * in.ldq + int64_t(kh) * s.dk, in.ldq, p.len, s.dk);
      er.fetch(kept.E + slot * kChunk * kChunk);
      pr.fetch(kept.P + slot * kChunk * kChunk);
      orow.fetch(dout + p.tok * ldo + int64_t(vh) * s.dv + col, ldo, p.len, s.dv - col,
                 s.dv % 8 == 0);
      if (t < kChunk) {
        g = kept.G[slot * kChunk + t];
        gend = kept.G[slot * kChunk + kChunk - 1];
        be = t < p.len ? in.beta[(p.tok + t) * s.hv + vh] : 0.f;
      }
    }, [&](int n) {
      char* const d = lds + n * L::kSlot;
      kr.put(d);
      qr.put(d + L::kQ);
      er.put_tri(d + L::kE);
      pr.put_tri(d + L::kP);
      orow.put(d + L::kO);
      set_factors(*(Factors*)(d + L::kFactors), g, gend, be);
    });
    return;
  }
  const bool live = c0 < s.dvp;
  f32x4 D[RT];
  load_state<DK>(D, dsend, s, head, c0);
  walk<L::kDepth>(count, [&](int64_t i_, int n_) {
    if (!live) return;
    const int64_t c = count - 1 - i_;
    const char* const smem = lds + n_ * L::kSlot;
    const Factors& f = *(const Factors*)(smem + L::kFactors);
    const Place p = chunk_of(seq, first, past, c);
    const int64_t slot = (begin + c) * s.hv + vh;
    constexpr int GT = kTilesAStep<T>, kSide = 4 / GT;
    typedef Ops<NP, GT> Tokens;
    auto rows = [&](int i) {   // step i of k dS
      Tokens o;
#pragma unroll
      for (int n = 0; n < GT; ++n) o.o[n] = token_rows<NP, DK>(smem, i % kSide * GT + n, i / kSide);
      return o;
    };
    auto cols = [&](const char* p, int i) {
      Tokens o;
#pragma unroll
      for (int n = 0; n < GT; ++n)
        o.o[n] = token_cols<NP, DK>(p, i % (RT / GT) * GT + n, i / (RT / GT));
      return o;
    };
    auto q_cols = [&](int i) { return cols(smem + L::kQ, i); };   // step i of q^T do
    auto k_cols = [&](int i) { return cols(smem, i); };           // step i of k^T (B X)
    // rows 0 and 1, 2 and 3 of a turned triangle's second half, 0 and 1 of its first
    auto tri_step = [&](const char* p, int i) {
      Ops<3, 2> o;
#pragma unroll
      for (int n = 0; n < 2; ++n) o.o[n] = tri_turned<3>(p, (i == 1 ? 2 : 0) + n, i < 2);
      return o;
    };
    auto tri_p = [&](int i) { return tri_step(smem + L::kP, i); };
    auto tri_e = [&](int i) { return tri_step(smem + L::kE, i); };
    float* Dg = dS + (slot * s.dvp + c0) * DK + t % kWave * 4;
    Tokens k0 = rows(0);
    Op<3> so[2];
    so[0] = operand<3>(D[0], D[1]);
#pragma unroll
    for (int a = 0; a < RT; ++a) *reinterpret_cast<f32x4*>(Dg + 256 * a) = D[a];
    f32x4 Y[4], bY[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) Y[i] = f32x4{0, 0, 0, 0};
    Ops<3, 2> t0;
    pipe<KB * kSide>(k0, rows, [&](int i, const Tokens& o) {
      if (i % kSide == 0 && i / kSide + 1 < KB)
        so[(i / kSide + 1) % 2] = operand<3>(D[2 * (i / kSide) + 2], D[2 * (i / kSide) + 3]);
      mul_turns(Y + i % kSide * GT, o.o, so[i / kSide % 2]);
    }, [&] { t0 = tri_p(0); });
    auto out_grad = [&](int i) { return Values<T>::tile(smem + L::kO, wc, i); };
    const Op<NP> oo[2] = {operand_of<T>(out_grad(0), out_grad(1)),
                          operand_of<T>(out_grad(2), out_grad(3))};
#pragma unroll
    for (int i = 0; i < 4; ++i) Y[i] *= quad(f.out, i);
    pipe<3>(t0, tri_p, [&](int i, const Ops<3, 2>& o) {
      mul_turns(Y + (i == 1 ? 2 : 0), o.o, oo[i < 2]);
    }, [&] { k0 = q_cols(0); });
    {
      auto read_o = [&](int i) { return s.scale * quad(f.in, i) * out_grad(i); };
      Op<3> os[2];
      os[0] = operand<3>(read_o(0), read_o(1));
      const float all = f.all;
#pragma unroll
      for (int a = 0; a < RT; ++a) D[a] *= all;
      pipe<RT / GT * 2>(k0, q_cols, [&](int i, const Tokens& o) {
        if (i == 0) os[1] = operand<3>(read_o(2), read_o(3));
        mul_turns(D + i % (RT / GT) * GT, o.o, os[i / (RT / GT)]);
      }, [&] { t0 = tri_e(0); });
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) bY[i] = quad(f.beta, i) * Y[i];
    Op<3> n[2];
    n[1] = operand<3>(bY[2], bY[3]);
    float* Xg = X + (slot * s.dvp + c0) * kChunk + t % kWave * 4;
    T* const dvp = dv + ((p.tok + 4 * h) * s.hv + vh) * s.dv + c0 + l;
    f32x4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = f32x4{0, 0, 0, 0};
    pipe<3>(t0, tri_e, [&](int i, const Ops<3, 2>& o) {
      if (i == 0) n[0] = operand<3>(bY[0], bY[1]);
      mul_turns(x + (i == 1 ? 2 : 0), o.o, n[i < 2]);
    }, [&] { k0 = k_cols(0); });
    auto solved = [&](int i) {   // X and dv of tokens 16 i ..
      Y[i] -= x[i];
      *reinterpret_cast<f32x4*>(Xg + 256 * i) = Y[i];
      bY[i] = quad(f.beta, i) * Y[i];
      if (dv && c0 + l < s.dv) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (p.len == kChunk || 16 * i + 4 * h + r < p.len)
            dvp[int64_t(16 * i + r) * s.hv * s.dv] = T(bY[i][r]);
      }
      bY[i] *= -quad(f.in, i);
    };
    solved(0);
    solved(1);
    n[0] = operand<3>(bY[0], bY[1]);
    pipe<RT / GT * 2>(k0, k_cols, [&](int i, const Tokens& o) {
      if (i == 0) {
        solved(2);
        solved(3);
        n[1] = operand<3>(bY[2], bY[3]);
      }
      mul_turns(D + i % (RT / GT) * GT, o.o, n[i / (RT / GT)]);
    }, [] {});
  });
  if (ds0 && live) store_state<DK>(D, ds0, s, head, c0);
}

// All gradients of a chunk but the state's and v's, a workgroup per chunk and
// key head, a wave 16 of its tokens: the value heads that share the key head
// are walked one after the other, so the gradients of q and k are summed in
// registers, in one order.  dg sums what crosses a token and nothing else: rows
// less columns of H, from each token on, are 20 us less work, but what does not
// cross cancels in them only up to its roundings, and behind gates of -10 that
// was all dg consisted of (5e-3 off; at -20 noise).  H's off-diagonal blocks
// need the sums of their rows and columns, the diagonal ones those of the rows
// >= t and columns < t of their 16 x 16.  Only products of full precision enter
// dg, none of the cut dP and dA, which go on into dq and dk.  Two workgroups a
// CU (bf16; 128 registers of sums a lane): 486 us for 4 x 4096 tokens and 16 heads
// of 128, of which the reading of 0.8 GB is 160 and the matrix instructions 85;
// the rest is waiting between the five barriers of a slice.
template <typename T, int DK>
struct GradsLds {
  static constexpr int NS = 3;   // parts of the fp32 factors
  // first over the columns of the state, a slice at a time: S (then dS) and
  // X and N, lines of a column each ...
  static constexpr int kSStride = 2 * DK + 32, kSPart = kSlice * kSStride;
  static constexpr int kXStride = 160, kXPart = kSlice * kXStride;
  static constexpr int kX = 3 * kSPart, kN = kX + 3 * kXPart, kFirst = kN + 3 * kXPart;
  // ... then over the chunk's tokens
  static constexpr int kQ = kParts<T> * kChunk * DK * 2, kdP = 2 * kQ, kdA = kdP + NS * kTri;
  static constexpr int kSecond = kdA + NS * kTri;
  static constexpr int kFactors = kFirst > kSecond ? kFirst : kSecond;
  struct Tail {
    Factors f;
    double G[kChunk];
    // sums of H: rows of a block row's off-diagonal blocks, columns of each
    // block, diagonal blocks; a and b
    float rows[kChunk], cols[4][kChunk], own[kChunk], a[kChunk], b[kChunk], part[4];
  };
  static constexpr int kBytes = kFactors + int(sizeof(Tail));
};
template <typename T, int DK, bool WHOLE, bool SHARED>
__global__ __launch_bounds__(kDeltaBlock, kParts<T> == 1 && !SHARED ? 2 : 1) void k_delta_grads(
    DeltaShape s, DeltaIn<T> in, DeltaKept kept, const T* __restrict__ dout, int64_t ldo,
    const float* __restrict__ X, const float* __restrict__ dS, T* __restrict__ dq,
    T* __restrict__ dk, float* __restrict__ dg, float* __restrict__ dbeta) {
  using L = GradsLds<T, DK>;
  constexpr int NP = kParts<T>, NS = L::NS, NT = DK / 16, KB = DK / 32;
  extern __shared__ __align__(16) char smem[];
  typename L::Tail& z = *(typename L::Tail*)(smem + L::kFactors);
  Place p;
  if (!find_chunk(s, blockIdx.x, p)) return;
  const int kh = blockIdx.y, group = s.hv / s.hk;
  const int t = threadIdx.x, l = t % 16, h = (t % kWave) / 16;
  const int w = __builtin_amdgcn_readfirstlane(t / kWave);
  // SHARED: sums over the group, rows 16 w + 4 h + r, columns 16 n + l
  f32x4 aq[SHARED ? NT : 1], ak[SHARED ? NT : 1];
#pragma unroll
  for (int n = 0; n < (SHARED ? NT : 1); ++n) aq[n] = ak[n] = f32x4{0, 0, 0, 0};

  auto leave = [&](const f32x4 (&x)[NT], const f32x4 (&y)[NT]) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * h + r, col = 16 * n + l;
        if (row < p.len && col < s.dk) {
          const int64_t at = ((p.tok + row) * s.hk + kh) * s.dk + col;
          if (dq) dq[at] = T(x[n][r]);
          if (dk) dk[at] = T(y[n][r]);
        }
      }
  };
  for (int vh = kh * group; vh < (SHARED ? (kh + 1) * group : kh * group + 1); ++vh) {
    const int64_t slot = int64_t(blockIdx.x) * s.hv + vh;
    const float* Sg = kept.S + slot * s.dvp * DK;
    const float* Dg = dS + slot * s.dvp * DK;
    const float* Mg = kept.M + slot * s.dvp * kChunk;
    const float* Xg = X + slot * s.dvp * kChunk;
    __syncthreads();
    set_factors(z.f, s, kept.G + slot * kChunk, in.beta, p, vh);
    if (t < kChunk) z.G[t] = kept.G[slot * kChunk + t];
    f32x4 pp[4], pa[4], oS[NT], xS[NT], nD[NT];
#pragma unroll
    for (int j = 0; j < 4; ++j) pp[j] = pa[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int n = 0; n < NT; ++n) oS[n] = xS[n] = nD[n] = f32x4{0, 0, 0, 0};
    float sd = 0.f;                          // <S, dS> of this thread's elements
    f32x4 xm = {0, 0, 0, 0};                 // X . M of tokens 16 w + 4 h .., this lane's columns
    constexpr int kLoads = kSlice * DK / 4 / kDeltaBlock;
    const T* orow = dout + (p.tok + 16 * w + l) * ldo + int64_t(vh) * s.dv + 4 * h;
    auto put = [&](const f32x4& x, char* d, int part) {
      const float y[4] = {x[0], x[1], x[2], x[3]};
      uint32_t u[3][2];
      split<3, 4>(y, u);
#pragma unroll
      for (int k = 0; k < 3; ++k) *reinterpret_cast<U2*>(d + k * part) = U2{u[k][0], u[k][1]};
    };
    f32x4 sv[kLoads], xv[2], mv[2];
    float ov[2][4];
    auto fetch = [&](int c0) {
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        sv[i] = *reinterpret_cast<const f32x4*>(Sg + int64_t(c0) * DK + (t + i * kDeltaBlock) * 4);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t at = int64_t(c0) * kChunk + (t + i * kDeltaBlock) * 4;
        xv[i] = *reinterpret_cast<const f32x4*>(Xg + at);
        mv[i] = *reinterpret_cast<const f32x4*>(Mg + at);
        load_f32<4>(orow + c0 + 16 * i, 16 * w + l < p.len ? s.dv - c0 - 16 * i - 4 * h : 0, ov[i]);
      }
    };
    // this thread's load i of a slice: a quad of column l of one of its blocks
    auto state_at = [&](int i) {
      const int n = 4 * i + w;
      return (n / NT * 16 + l) * L::kSStride + (n % NT * 16 + 4 * h) * 2;
    };
    for (int c0 = 0; c0 < s.dvp; c0 += kSlice) {
      fetch(c0);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        put(sv[i], smem + state_at(i), L::kSPart);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        xm += xv[i] * mv[i];
        char* d = smem + (16 * i + l) * L::kXStride + (16 * w + 4 * h) * 2;
        put(xv[i], d + L::kX, L::kXPart);
        put(mv[i] * quad(z.f.beta, w), d + L::kN, L::kXPart);
      }
      const Op<NP> oo = operand_of<T>(f32x4{ov[0][0], ov[0][1], ov[0][2], ov[0][3]},
                                      f32x4{ov[1][0], ov[1][1], ov[1][2], ov[1][3]});
      __syncthreads();
      // dS takes S's place next
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
        sv[i] = *reinterpret_cast<const f32x4*>(Dg + int64_t(c0) * DK + (t + i * kDeltaBlock) * 4);
      {
        const Op<3> xo = col_op<3>(smem + L::kX + 32 * w, L::kXStride, L::kXPart);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j <= w) {
            const Op<3> nj = col_op<3>(smem + L::kN + 32 * j, L::kXStride, L::kXPart);
            mul(pp[j], oo, nj);
            mul(pa[j], xo, nj);
          }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const Op<3> sn = col_op<3>(smem + 32 * n, L::kSStride, L::kSPart);
          mul(oS[n], oo, sn);
          mul(xS[n], xo, sn);
          if (n % 2) __builtin_amdgcn_sched_barrier(0);   // or all operands are read at once
        }
      }
      const Op<3> no = col_op<3>(smem + L::kN + 32 * w, L::kXStride, L::kXPart);
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        char* d = smem + state_at(i);
        f32x4 was = {0, 0, 0, 0};   // S there
#pragma unroll
        for (int k = 2; k >= 0; --k) {
          const U2 u = *reinterpret_cast<const U2*>(d + k * L::kSPart);
          was += f32x4{__uint_as_float(u[0] << 16), __uint_as_float(u[0] & 0xffff0000u),
                       __uint_as_float(u[1] << 16), __uint_as_float(u[1] & 0xffff0000u)};
        }
        sd += was[0] * sv[i][0] + was[1] * sv[i][1] + (was[2] * sv[i][2] + was[3] * sv[i][3]);
        put(sv[i], d, L::kSPart);
      }
      __syncthreads();
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mul(nD[n], no, col_op<3>(smem + 32 * n, L::kSStride, L::kSPart));
        if (n % 2) __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float x = lane_sum<16>(xm[r]);
      const int row = 16 * w + 4 * h + r;
      if (dbeta && l == 0 && row < p.len) dbeta[(p.tok + row) * s.hv + vh] = x;
    }
    sd = lane_sum<kWave>(sd);
    if (t % kWave == 0) z.part[w] = sd;
    __syncthreads();
    {
      Rows<T, DK, WHOLE> kr, qr;
      kr.fetch(in.k + p.tok * in.ldk + int64_t(kh) * s.dk, in.ldk, p.len, s.dk);
      qr.fetch(in.q + p.tok * in.ldq + int64_t(kh) * s.dk, in.ldq, p.len, s.dk);
      kr.put(smem);
      qr.put(smem + L::kQ);
    }
    __syncthreads();
    const f32x4 fin = quad(z.f.in, w), fout = quad(z.f.out, w), fbe = quad(z.f.beta, w);
    f32x4 row_h = {0, 0, 0, 0}, own = {0, 0, 0, 0};   // H: rows' sums, the diagonal block
    const float* Pg = kept.P + slot * kChunk * kChunk;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float col_h = 0.f;
      if (j <= w) {
        f32x4 kk = {0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < KB; ++b)
          mul(kk, token_rows<NP, DK>(smem, w, b), token_rows<NP, DK>(smem, j, b));
        f32x4 dp, da;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * w + 4 * h + r, col = 16 * j + l;
          const float d = col <= row ? expf(float(z.G[row] - z.G[col])) : 0.f;
          const float bx = col < row ? d * fbe[r] * pa[j][r] : 0.f;
          dp[r] = s.scale * d * pp[j][r];
          da[r] = -bx;
          const float x = col <= row ? pp[j][r] * Pg[row * kChunk + col] - bx * kk[r] : 0.f;
          if (j < w) {
            row_h[r] += x;
            col_h += x;
          } else {
            own[r] = x;
          }
        }
        // line 16 j + l, rows 16 w + 4 h .. of the turned triangle
        const float y[4] = {dp[0], dp[1], dp[2], dp[3]}, x[4] = {da[0], da[1], da[2], da[3]};
        uint32_t u[NS][2], v[NS][2];
        split<NS, 4>(y, u);
        split<NS, 4>(x, v);
        char* d = smem + upper_at(j) + l * upper_stride(j) + 32 * (w - j) + 8 * h;
#pragma unroll
        for (int k = 0; k < NS; ++k) {
          *reinterpret_cast<U2*>(d + L::kdP + k * kTri) = U2{u[k][0], u[k][1]};
          *reinterpret_cast<U2*>(d + L::kdA + k * kTri) = U2{v[k][0], v[k][1]};
        }
      }
      col_h += __shfl_xor(col_h, 16, kWave);
      col_h += __shfl_xor(col_h, 32, kWave);
      if (h == 0) z.cols[w][16 * j + l] = col_h;
    }
    {
      // rows >= 4 h + r of the diagonal block, then columns before it
      float below = own[0] + own[1] + own[2] + own[3], above = 0.f;
#pragma unroll
      for (int d = 1; d < 4; ++d) {
        const float u = __shfl(below, (t + 16 * d) % kWave, kWave);
        if (h + d < 4) above += u;
      }
#pragma unroll
      for (int r = 3; r >= 0; --r) {
        above += own[r];
        const float x = lane_sum<16>(l < 4 * h + r ? above : 0.f), y = lane_sum<16>(row_h[r]);
        if (l == 0) {
          z.own[16 * w + 4 * h + r] = x;
          z.rows[16 * w + 4 * h + r] = y;
        }
      }
    }
    __syncthreads();
    // dq = scale exp(G) (do S^T) + dP k and the like, the state's parts first
    f32x4 a = {0, 0, 0, 0}, b = {0, 0, 0, 0};
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const f32x4 kv = token_tile<NP, DK>(smem, n, w), qv = token_tile<NP, DK>(smem + L::kQ, n, w);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        oS[n][r] *= s.scale * fin[r];
        const float u = fin[r] * fbe[r] * xS[n][r], y = fout[r] * nD[n][r];
        a[r] += qv[r] * oS[n][r] - kv[r] * u;
        b[r] += kv[r] * y;
        xS[n][r] = y - u;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      // (the empty blocks' operands are zero: a branch here would have the
      // compiler move all sums about; dP's first, then dA's: all four operands
      // at a time spill 53 registers instead of 23 and take 60 us more)
      const Op<NS> pr = upper_rows<NS>(smem + L::kdP, w, b);
      const Op<NS> pc = upper_turned<NS>(smem + L::kdP, w, b);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mul(oS[n], pr, token_cols<NP, DK>(smem, n, b));
        mul(xS[n], pc, token_cols<NP, DK>(smem + L::kQ, n, b));
        if (n % 2) __builtin_amdgcn_sched_barrier(0);
      }
      const Op<NS> ar = upper_rows<NS>(smem + L::kdA, w, b);
      const Op<NS> ac = upper_turned<NS>(smem + L::kdA, w, b);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const Op<NP> kn = token_cols<NP, DK>(smem, n, b);
        mul(xS[n], ar, kn);
        mul(xS[n], ac, kn);
        if (n % 2) __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (SHARED) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        aq[n] += oS[n];
        ak[n] += xS[n];
      }
    } else {
      leave(oS, xS);
    }
    if (dg) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float x = lane_sum<16>(a[r]), y = lane_sum<16>(b[r]);
        if (l == 0) {
          z.a[16 * w + 4 * h + r] = x;
          z.b[16 * w + 4 * h + r] = y;
        }
      }
      __syncthreads();
      if (t < kChunk) {
        const int row = kChunk - 1 - t, tile = row / 16;
        // rows >= row: of all tokens (a), of its block row (H)
        float sa = z.a[row], sr = z.rows[row];
        // rows < row: of all tokens (b), of its block column (H)
        float sb = row ? z.b[row - 1] : 0.f, sc = 0.f;
#pragma unroll
        for (int k = 1; k < 4; ++k)
          if (row % 16 && k > tile) sc += z.cols[k][row - 1];
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
          const float u = __shfl_up(sa, d, kWave), v = __shfl_down(sb, d, kWave);
          if (t >= d) sa += u;
          if (t + d < kWave) sb += v;
        }
#pragma unroll
        for (int d = 1; d < 16; d <<= 1) {
          const float u = __shfl_up(sr, d, kWave), v = __shfl_down(sc, d, kWave);
          if (t % 16 >= d) sr += u;
          if (t % 16 + d < 16) sc += v;
        }
        // whole blocks below and before the tile's
        const float f1 = lane_sum<kWave>(row < 16 ? z.cols[2][row] + z.cols[3][row] : 0.f);
        const float f2 = lane_sum<kWave>(row < 32 ? z.cols[3][row] : 0.f);
        const float full = tile == 1 ? f1 : tile == 2 ? f2 : 0.f;
        const float kept_s = z.f.all * ((z.part[0] + z.part[1]) + (z.part[2] + z.part[3]));
        if (row < p.len)
          dg[(p.tok + row) * s.hv + vh] =
              (sa + sb) + ((sr + sc) + (full + z.own[row])) + kept_s;
      }
    }
  }
  if constexpr (SHARED) leave(aq, ak);
}

// One token of every sequence, the state updated in place: a workgroup per
// sequence, value head and 32 columns; 8 lanes of 4 columns by 32 lines of
// rows, each thread's part of the state in registers between its one read
// and its one write.  Bound by reading and writing the state: 101 us for 128 x
// 32 heads of 128 x 128 (537 MB, 5.3 TB/s).  Both sums over the rows (k and q against the state)
// come from that one read, since S_t^T q = exp(g) S^T q + (k.q) beta m.
template <typename T, int NR>
__global__ __launch_bounds__(kDeltaBlock) void k_delta_step(
    const T* __restrict__ q, int64_t ldq, const T* __restrict__ k, int64_t ldk,
    const T* __restrict__ v, int64_t ldv, const float* __restrict__ g,
    const float* __restrict__ beta, float* __restrict__ state, T* __restrict__ o, int64_t first,
    int hk, int hv, int dk, int dv, float scale) {
  __shared__ f32x4 sk[4][8], sq[4][8];
  __shared__ float sqk[4];
  const int t = threadIdx.x, cl = t % 8, line = t / 8, w = t / kWave;
  const int64_t sh = first + blockIdx.x;  // sequence * hv + head
  const int vh = int(sh % hv);
  const int64_t seq = sh / hv;
  const int kh = vh / (hv / hk);
  const int col = int(blockIdx.y) * kSlice + cl * 4;
  const int have = dv - col;
  float* S = state + sh * dk * dv;
  const T* kr = k + seq * ldk + int64_t(kh) * dk;
  const T* qr = q + seq * ldq + int64_t(kh) * dk;
  float st[NR][4], kv[NR], qv[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = line + 32 * i;
    load_f32<4>(S + int64_t(row) * dv + col, row < dk ? have : 0, st[i]);
    kv[i] = row < dk ? float(kr[row]) : 0.f;
    qv[i] = row < dk ? float(qr[row]) : 0.f;
  }
  float vv[4];
  load_f32<4>(v + seq * ldv + int64_t(vh) * dv + col, have, vv);
  const float a = expf(g[sh]), be = beta[sh];
  f32x4 ks = {0, 0, 0, 0}, qs = {0, 0, 0, 0};
  float qk = 0.f;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ks[j] += kv[i] * st[i][j];
      qs[j] += qv[i] * st[i][j];
    }
    qk += kv[i] * qv[i];
  }
#pragma unroll
  for (int d = 8; d < kWave; d <<= 1) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      ks[j] += __shfl_xor(ks[j], d, kWave);
      qs[j] += __shfl_xor(qs[j], d, kWave);
    }
    qk += __shfl_xor(qk, d, kWave);
  }
  if (t % kWave < 8) {
    sk[w][cl] = ks;
    sq[w][cl] = qs;
    if (cl == 0) sqk[w] = qk;
  }
  __syncthreads();
  ks = (sk[0][cl] + sk[1][cl]) + (sk[2][cl] + sk[3][cl]);
  qs = (sq[0][cl] + sq[1][cl]) + (sq[2][cl] + sq[3][cl]);
  qk = (sqk[0] + sqk[1]) + (sqk[2] + sqk[3]);
  float n[4], out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    n[j] = be * (vv[j] - a * ks[j]);
    out[j] = scale * (a * qs[j] + qk * n[j]);
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = line + 32 * i;
#pragma unroll
    for (int j = 0; j < 4; ++j) st[i][j] = a * st[i][j] + kv[i] * n[j];
    if (row < dk) store_f32<4>(S + int64_t(row) * dv + col, have, st[i]);
  }
  if (line == 0) store_f32<4>(o + sh * dv + col, have, out);
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------
constexpr int kMaxDk = 128;
// Workgroups of 256 threads in a launch: the runtime starts a launch of 2^32
// threads and more without its upper bits, and says nothing.
constexpr int64_t kMostGroups = (int64_t(1) << 24) - 1;

int pad_dk(int64_t dk) { return dk <= 64 ? 64 : 128; }
int64_t pad_dv(int64_t dv) { return div_up(dv, kSlice) * kSlice; }

struct DeltaSizes {
  int64_t chunks, kept, grad;   // chunks, bytes
  int64_t G, E, P, M, S, plan;  // offsets into the kept block
  int64_t X, dS;                // offsets into the gradient's block
};

sla_status delta_sizes(const char* who, const sla_delta_dims* d, DeltaSizes& z) {
  SLA_NET_REQUIRE(d, "%s: dims is NULL", who);
  SLA_NET_REQUIRE(valid_type(d->type), "%s: unknown type", who);
  SLA_NET_REQUIRE(d->sequences >= 0 && d->sequences < (1 << 24), "%s: sequences out of range", who);
  SLA_NET_REQUIRE(d->tokens >= 0 && d->tokens < (int64_t(1) << 31), "%s: tokens out of range", who);
  SLA_NET_REQUIRE(d->packed || d->sequences == 0 || d->tokens % d->sequences == 0,
                  "%s: tokens is not a multiple of sequences", who);
  SLA_NET_REQUIRE(d->sequences > 0 || d->tokens == 0, "%s: tokens without a sequence", who);
  SLA_NET_REQUIRE(d->key_heads >= 1 && d->value_heads >= 1 && d->value_heads < 65536 &&
                      d->value_heads % d->key_heads == 0,
                  "%s: value_heads must be a multiple of key_heads", who);
  SLA_NET_REQUIRE(d->key_dim >= 1 && d->key_dim <= kMaxDk, "%s: key_dim must be 1..%d", who,
                  kMaxDk);
  SLA_NET_REQUIRE(d->value_dim >= 1 && d->value_dim <= 4096, "%s: value_dim must be 1..4096", who);
  const int64_t n = d->sequences;
  z.chunks = d->packed ? d->tokens / kChunk + n : (n ? n * div_up(d->tokens / n, kChunk) : 0);
  const int64_t slots = z.chunks * d->value_heads;
  const int64_t dk = pad_dk(d->key_dim), dvp = pad_dv(d->value_dim);
  SLA_NET_REQUIRE(n * d->value_heads * (dvp / kSlice) < (int64_t(1) << 31) &&
                      z.chunks <= kMostGroups,
                  "%s: too many sequences, heads or chunks", who);
  int64_t at = 0;
  auto take = [&at](int64_t bytes) {
    const int64_t here = at;
    at += div_up(bytes, 256) * 256;
    return here;
  };
  z.G = take(slots * kChunk * 8);
  z.E = take(slots * kChunk * kChunk * 4);
  z.P = take(slots * kChunk * kChunk * 4);
  z.M = take(slots * kChunk * dvp * 4);
  z.S = take(slots * dk * dvp * 4);
  z.plan = take(2 * (n + 1) * 4);
  z.kept = at;
  at = 0;
  z.X = take(slots * kChunk * dvp * 4);
  z.dS = take(slots * dk * dvp * 4);
  z.grad = at;
  return SLA_OK;
}

DeltaShape delta_shape(const sla_delta_dims* d, const DeltaSizes& z, char* kept) {
  DeltaShape s;
  s.total = d->tokens;
  s.nseq = int(d->sequences);
  s.seqlen = s.nseq ? d->tokens / s.nseq : 0;
  s.chunks = z.chunks;
  s.hk = int(d->key_heads);
  s.hv = int(d->value_heads);
  s.dk = int(d->key_dim);
  s.dv = int(d->value_dim);
  s.dvp = int(pad_dv(d->value_dim));
  s.scale = float(d->scale);
  s.tok = d->packed ? (const int32_t*)(kept + z.plan) : nullptr;
  s.first = d->packed ? s.tok + s.nseq + 1 : nullptr;
  return s;
}

// The walks' launch has to stay below 2^32 threads too.  (With a token each so
// many sequences would keep 400 GB; without tokens the call copies states.)
sla_status walk_groups(const char* who, const DeltaShape& s) {
  SLA_NET_REQUIRE(int64_t(s.nseq) * s.hv * div_up(s.dvp, kWalk) <= kMostGroups / 2,
                  "%s: too many sequences and heads", who);
  return SLA_OK;
}

DeltaKept delta_kept(const DeltaSizes& z, char* kept) {
  return {(double*)(kept + z.G), (float*)(kept + z.E), (float*)(kept + z.P),
          (float*)(kept + z.M), (float*)(kept + z.S)};
}

// More LDS than the default 64 KB a workgroup needs the kernel's consent.
template <typename K>
sla_status allow_lds(K kernel, int bytes) {
  SLA_TRY_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                  hipFuncAttributeMaxDynamicSharedMemorySize, bytes));
  return SLA_OK;
}

// f(element, padded dk, whether dk is a multiple of 8).
template <typename F>
sla_status with_delta(const sla_delta_dims* d, F&& g) {
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  const bool small = pad_dk(d->key_dim) == 64;
  auto f = [&](auto te, auto width) -> sla_status {
    return d->key_dim % 8 == 0 ? g(te, width, std::true_type()) : g(te, width, std::false_type());
  };
  if (d->type == SLA_F32) return small ? f(float(), D64()) : f(float(), D128());
  if (d->type == SLA_F16) return small ? f(_Float16(), D64()) : f(_Float16(), D128());
  return small ? f(__bf16(), D64()) : f(__bf16(), D128());
}

}  // namespace
}  // namespace net
}  // namespace sla

using namespace sla;
using namespace sla::net;

extern "C" {

sla_status sla_delta_rule_work(const sla_delta_dims* dims, int64_t* kept_bytes_host,
                               int64_t* grad_bytes_host) {
  SLA_NET_BEGIN
  clear_error();
  DeltaSizes z;
  SLA_TRY(delta_sizes("sla_delta_rule_work", dims, z));
  if (kept_bytes_host) *kept_bytes_host = z.kept;
  if (grad_bytes_host) *grad_bytes_host = z.grad;
  return SLA_OK;
  SLA_NET_END
}

sla_status sla_delta_rule(const sla_delta_dims* dims, const void* q, int64_t ldq, const void* k,
                          int64_t ldk, const void* v, int64_t ldv, const float* g,
                          const float* beta, const int32_t* offsets, const float* initial_state,
                          void* o, float* final_state, void* kept, int64_t kept_bytes,
                          hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  DeltaSizes z;
  SLA_TRY(delta_sizes("sla_delta_rule", dims, z));
  if (dims->sequences == 0) return SLA_OK;
  SLA_NET_REQUIRE(dims->tokens == 0 || (q && k && v && g && beta && o),
                  "sla_delta_rule: an input or o is NULL");
  SLA_NET_REQUIRE(!dims->packed || offsets, "sla_delta_rule: offsets is NULL");
  SLA_NET_REQUIRE(ldq >= dims->key_heads * dims->key_dim &&
                      ldk >= dims->key_heads * dims->key_dim &&
                      ldv >= dims->value_heads * dims->value_dim,
                  "sla_delta_rule: a token stride is shorter than its heads");
  SLA_NET_REQUIRE(kept && kept_bytes >= z.kept,
                  "sla_delta_rule: kept block too small (sla_delta_rule_work)");
  const DeltaShape s = delta_shape(dims, z, (char*)kept);
  const DeltaKept w = delta_kept(z, (char*)kept);
  if (dims->packed) {
    Gaps gaps{};
    if (dims->tokens)
      gaps.g[0] = {o, int64_t(s.hv) * s.dv * int64_t(type_size(dims->type))};
    k_delta_plan<<<1, kDeltaBlock, 0, stream>>>(offsets, s.nseq, s.total, (int32_t*)s.tok,
                                                (int32_t*)s.first, gaps);
    LAUNCH_CHECK();
  }
  SLA_TRY(walk_groups("sla_delta_rule", s));
  return with_delta(dims, [&](auto te, auto width, auto whole) -> sla_status {
    using T = decltype(te);
    constexpr int DK = width.value;
    const DeltaIn<T> in = {(const T*)q, (const T*)k, (const T*)v, ldq, ldk, ldv, g, beta};
    if (z.chunks) {
      constexpr int lds = PrepareLds<T, DK>::kBytes;
      SLA_TRY(allow_lds(k_delta_prepare<T, DK, whole.value>, lds));
      k_delta_prepare<T, DK, whole.value><<<dim3(int(z.chunks), s.hv), kDeltaBlock, lds, stream>>>(s, in, w);
      LAUNCH_CHECK();
    }
    {
      constexpr int lds = StatesLds<T, DK>::kBytes;
      SLA_TRY(allow_lds(k_delta_states<T, DK, whole.value>, lds));
      k_delta_states<T, DK, whole.value><<<s.nseq * s.hv * int(div_up(s.dvp, kWalk)), kWalkBlock, lds, stream>>>(
          s, in, w, initial_state, final_state);
      LAUNCH_CHECK();
    }
    if (z.chunks) {
      constexpr int lds = OutLds<T, DK>::kBytes;
      SLA_TRY(allow_lds(k_delta_out<T, DK>, lds));
      k_delta_out<T, DK><<<dim3(int(z.chunks), s.hv), kDeltaBlock, lds, stream>>>(s, in, w, (T*)o);
      LAUNCH_CHECK();
    }
    return SLA_OK;
  });
  SLA_NET_END
}

sla_status sla_delta_rule_grad(const sla_delta_dims* dims, const void* q, int64_t ldq,
                               const void* k, int64_t ldk, const void* v, int64_t ldv,
                               const float* g, const float* beta, const void* kept,
                               int64_t kept_bytes, const void* grad_o, int64_t ldo,
                               const float* grad_final_state, void* dq, void* dk, void* dv,
                               float* dg, float* dbeta, float* grad_initial_state, void* work,
                               int64_t work_bytes, hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  DeltaSizes z;
  SLA_TRY(delta_sizes("sla_delta_rule_grad", dims, z));
  if (dims->sequences == 0) return SLA_OK;
  SLA_NET_REQUIRE(dims->tokens == 0 || (q && k && v && g && beta && grad_o),
                  "sla_delta_rule_grad: an input or grad_o is NULL");
  SLA_NET_REQUIRE(ldq >= dims->key_heads * dims->key_dim &&
                      ldk >= dims->key_heads * dims->key_dim &&
                      ldv >= dims->value_heads * dims->value_dim &&
                      ldo >= dims->value_heads * dims->value_dim,
                  "sla_delta_rule_grad: a token stride is shorter than its heads");
  SLA_NET_REQUIRE(kept && kept_bytes >= z.kept && work && work_bytes >= z.grad,
                  "sla_delta_rule_grad: kept or work block too small (sla_delta_rule_work)");
  const DeltaShape s = delta_shape(dims, z, (char*)kept);
  const DeltaKept w = delta_kept(z, (char*)kept);
  float* X = (float*)((char*)work + z.X);
  float* dS = (float*)((char*)work + z.dS);
  if (dims->packed && dims->tokens) {
    const int64_t es = int64_t(type_size(dims->type));
    Gaps gaps{};
    gaps.g[0] = {dq, s.hk * int64_t(s.dk) * es};
    gaps.g[1] = {dk, s.hk * int64_t(s.dk) * es};
    gaps.g[2] = {dv, s.hv * int64_t(s.dv) * es};
    gaps.g[3] = {dg, int64_t(s.hv) * 4};
    gaps.g[4] = {dbeta, int64_t(s.hv) * 4};
    k_delta_gaps<<<1, kDeltaBlock, 0, stream>>>(s.tok, s.nseq, s.total, gaps);
    LAUNCH_CHECK();
  }
  SLA_TRY(walk_groups("sla_delta_rule_grad", s));
  return with_delta(dims, [&](auto te, auto width, auto whole) -> sla_status {
    using T = decltype(te);
    constexpr int DK = width.value;
    const DeltaIn<T> in = {(const T*)q, (const T*)k, (const T*)v, ldq, ldk, ldv, g, beta};
    {
      constexpr int lds = AdjointLds<T, DK>::kBytes;
      SLA_TRY(allow_lds(k_delta_adjoint<T, DK, whole.value>, lds));
      k_delta_adjoint<T, DK, whole.value><<<s.nseq * s.hv * int(div_up(s.dvp, kWalk)), kWalkBlock, lds, stream>>>(
          s, in, w, (const T*)grad_o, ldo, grad_final_state, X, dS, (T*)dv, grad_initial_state);
      LAUNCH_CHECK();
    }
    if (z.chunks && (dq || dk || dg || dbeta)) {
      constexpr int lds = GradsLds<T, DK>::kBytes;
      auto* kernel = s.hv > s.hk ? k_delta_grads<T, DK, whole.value, true>
                                 : k_delta_grads<T, DK, whole.value, false>;
      SLA_TRY(allow_lds(kernel, lds));
      kernel<<<dim3(int(z.chunks), s.hk), kDeltaBlock, lds, stream>>>(
          s, in, w, (const T*)grad_o, ldo, X, dS, (T*)dq, (T*)dk, dg, dbeta);
      LAUNCH_CHECK();
    }
    return SLA_OK;
  });
  SLA_NET_END
}

sla_status sla_delta_step(const sla_delta_dims* dims, const void* q, int64_t ldq, const void* k,
                          int64_t ldk, const void* v, int64_t ldv, const float* g,
                          const float* beta, float* state, void* o, hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  DeltaSizes z;
  SLA_TRY(delta_sizes("sla_delta_step", dims, z));
  SLA_NET_REQUIRE(!dims->packed && dims->tokens == dims->sequences,
                  "sla_delta_step: one token for each sequence");
  if (dims->sequences == 0) return SLA_OK;
  SLA_NET_REQUIRE(q && k && v && g && beta && state && o, "sla_delta_step: an argument is NULL");
  SLA_NET_REQUIRE(ldq >= dims->key_heads * dims->key_dim &&
                      ldk >= dims->key_heads * dims->key_dim &&
                      ldv >= dims->value_heads * dims->value_dim,
                  "sla_delta_step: a token stride is shorter than its heads");
  auto go = [&](auto te, auto nr) -> sla_status {
    using T = decltype(te);
    const int64_t all = dims->sequences * dims->value_heads;
    for (int64_t first = 0; first < all; first += kMostGroups) {
      const int64_t left = all - first;
      const dim3 grid(int(left < kMostGroups ? left : kMostGroups),
                      int(div_up(dims->value_dim, kSlice)));
      k_delta_step<T, nr.value><<<grid, kDeltaBlock, 0, stream>>>(
          (const T*)q, ldq, (const T*)k, ldk, (const T*)v, ldv, g, beta, state, (T*)o, first,
          int(dims->key_heads), int(dims->value_heads), int(dims->key_dim), int(dims->value_dim),
          float(dims->scale));
      LAUNCH_CHECK();
    }
    return SLA_OK;
  };
  return with_delta(dims, [&](auto te, auto width, auto) {
    return go(te, std::integral_constant<int, width.value / 32>());
  });
  SLA_NET_END
}

}  // extern "C"
