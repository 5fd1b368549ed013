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
//   dk = u + w       dG_i = q_i.dq_i + k_i.(u_i - w_i), and <S', dS> at the chunk's end
//   dg = the sums of dG from each token to the chunk's end
//
// Work that does not depend on the state (k_delta_prepare, k_delta_out,
// k_delta_grads) runs over all chunks at once; what does (k_delta_states,
// k_delta_adjoint) walks a sequence's chunks, a workgroup for every 32
// columns of the state, which never mix.
//
// Everything is held and multiplied in fp32 whatever the tokens' type: the
// state, its gradient, dg and dbeta leave in fp32, and a matrix product of
// rounded 16-bit factors would leave them three digits.  G is summed in
// fp64: its differences are exponents.
#include "net.h"

namespace sla {
namespace net {
namespace {

constexpr int kChunk = 64;
constexpr int kDeltaBlock = 256;
constexpr int kSlice = 32;              // columns of the state per walking workgroup
constexpr int kLdC = kChunk + 4;        // LDS row of 64 floats (padded against bank conflicts)
constexpr int kLdS = kSlice + 4;        // LDS row of a slice

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
  float* M;    // [64][dvp]
  float* S;    // [dk padded][dvp] the state before the chunk
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

// A chunk's rows of `width` elements (zero past `len` rows and `have`
// columns), 8 elements a load, held in registers between the load and the
// LDS store so that the next chunk's rows travel while this one is worked on.
template <typename T, int WIDTH>
struct Rows {
  static constexpr int kLoads = kChunk * WIDTH / 8 / kDeltaBlock;
  static_assert(kLoads >= 1, "a load per thread");
  float v[kLoads][8];
  __device__ __forceinline__ void fetch(const T* p, int64_t ld, int len, int have) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = threadIdx.x + i * kDeltaBlock;
      const int row = at / (WIDTH / 8), col = at % (WIDTH / 8) * 8;
      load_f32<8>(p + row * ld + col, row < len ? have - col : 0, v[i]);
    }
  }
  __device__ __forceinline__ void put(float* lds, int ldl) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int at = threadIdx.x + i * kDeltaBlock;
      float* d = lds + (at / (WIDTH / 8)) * ldl + at % (WIDTH / 8) * 8;
#pragma unroll
      for (int j = 0; j < 8; j += 4)
        *reinterpret_cast<f32x4*>(d + j) = f32x4{v[i][j], v[i][j + 1], v[i][j + 2], v[i][j + 3]};
    }
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
// a block column per wave, with T = I - B E the inverse so far.
template <typename T, int DK>
__global__ __launch_bounds__(kDeltaBlock) void k_delta_prepare(DeltaShape s, DeltaIn<T> in,
                                                               DeltaKept kept) {
  constexpr int LD = DK + 4;
  extern __shared__ __align__(16) char smem[];
  float* kf = (float*)smem;               // [64][LD]
  float* qf = kf + kChunk * LD;           // [64][LD]
  float* A = qf + kChunk * LD;            // [64][kLdC]
  float* E = kf;                          // over k and q once they are used up
  float* Tm = kf + kChunk * kLdC;
  double* G = (double*)(A + kChunk * kLdC);
  float* beta = (float*)(G + kChunk);
  Place p;
  if (!find_chunk(s, blockIdx.x, p)) return;
  const int vh = blockIdx.y, kh = vh / (s.hv / s.hk);
  const int t = threadIdx.x, w = t / kWave, l = t % 16, h = (t % kWave) / 16;
  {
    Rows<T, DK> kr, qr;
    kr.fetch(in.k + p.tok * in.ldk + int64_t(kh) * s.dk, in.ldk, p.len, s.dk);
    qr.fetch(in.q + p.tok * in.ldq + int64_t(kh) * s.dk, in.ldq, p.len, s.dk);
    kr.put(kf, LD);
    qr.put(qf, LD);
  }
  if (t < kChunk) {
    const int64_t at = (p.tok + t) * s.hv + vh;
    double g = t < p.len ? double(in.g[at]) : 0.0;
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
      mma<DK, false, false>(kk, kf + 16 * w * LD, LD, kf + 16 * J * LD, LD);
      mma<DK, false, false>(qk, qf + 16 * w * LD, LD, kf + 16 * J * LD, LD);
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
struct Factors {
  float beta[kChunk];
  float in[kChunk];    // exp(G)
  float out[kChunk];   // exp(G_L - G)
  float all;           // exp(G_L)
};
__device__ __forceinline__ void load_factors(Factors& f, const DeltaShape& s, const double* G,
                                             const float* beta, const Place& p, int vh) {
  const int t = threadIdx.x;
  if (t < kChunk) {
    const double g = G[t], end = G[kChunk - 1];
    f.beta[t] = t < p.len ? beta[(p.tok + t) * s.hv + vh] : 0.f;
    f.in[t] = expf(float(g));
    f.out[t] = expf(float(end - g));
    if (t == 0) f.all = expf(float(end));
  }
}

__device__ __forceinline__ Place chunk_of(const DeltaShape& s, int seq, int64_t c) {
  Place p;
  p.seq = seq;
  p.tok = first_token(s, seq) + c * kChunk;
  const int64_t left = first_token(s, seq + 1) - p.tok;
  p.len = left < kChunk ? int(left) : kChunk;
  return p;
}

// The states' walk forward: M of every chunk and the state before it.
template <typename T, int DK>
__global__ __launch_bounds__(kDeltaBlock) void k_delta_states(DeltaShape s, DeltaIn<T> in,
                                                              DeltaKept kept,
                                                              const float* __restrict__ s0,
                                                              float* __restrict__ send) {
  constexpr int LD = DK + 4, RT = DK / 64;  // 16-row tiles of the state per wave
  extern __shared__ __align__(16) char smem[];
  float* kf = (float*)smem;              // [64][LD]
  float* St = kf + kChunk * LD;          // [32][LD]   the state, transposed
  float* Ef = St + kSlice * LD;          // [64][kLdC]
  float* Rt = Ef + kChunk * kLdC;        // [32][kLdC] beta R, transposed
  float* Nt = Rt + kSlice * kLdC;        // [32][kLdC] exp(G_L - G) N, transposed
  Factors& f = *(Factors*)(Nt + kSlice * kLdC);
  const int slices = s.dvp / kSlice;
  const int c0 = blockIdx.x % slices * kSlice;
  const int vh = blockIdx.x / slices % s.hv, seq = blockIdx.x / slices / s.hv;
  const int kh = vh / (s.hv / s.hk);
  const int t = threadIdx.x, w = t / kWave, l = t % 16, h = (t % kWave) / 16;
  const int64_t begin = first_chunk(s, seq), count = first_chunk(s, seq + 1) - begin;

  // this wave's rows of the state: 16 (w RT + a) + 4 h + r, columns c0 + 16 b + l
  f32x4 S[RT][2];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * (w * RT + a) + 4 * h + r, col = c0 + 16 * b + l;
        S[a][b][r] = s0 && row < s.dk && col < s.dv
                         ? s0[((int64_t(seq) * s.hv + vh) * s.dk + row) * s.dv + col] : 0.f;
      }
  for (int64_t c = 0; c < count; ++c) {
    const Place p = chunk_of(s, seq, c);
    const int64_t slot = (begin + c) * s.hv + vh;
    Rows<T, DK> kr;
    kr.fetch(in.k + p.tok * in.ldk + int64_t(kh) * s.dk, in.ldk, p.len, s.dk);
    Rows<float, kChunk> er;
    er.fetch(kept.E + slot * kChunk * kChunk, kChunk, kChunk, kChunk);
    f32x4 v[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * h + r, col = c0 + 16 * b + l;
        v[b][r] = row < p.len && col < s.dv
                      ? float(in.v[(p.tok + row) * in.ldv + int64_t(vh) * s.dv + col]) : 0.f;
      }
    __syncthreads();  // the last chunk's readers are done
    kr.put(kf, LD);
    er.put(Ef, kLdC);
    load_factors(f, s, kept.G + slot * kChunk, in.beta, p, vh);
    float* Sg = kept.S + slot * DK * s.dvp;
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        *reinterpret_cast<f32x4*>(St + (16 * b + l) * LD + 16 * (w * RT + a) + 4 * h) = S[a][b];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          Sg[int64_t(16 * (w * RT + a) + 4 * h + r) * s.dvp + c0 + 16 * b + l] = S[a][b][r];
      }
    __syncthreads();
    f32x4 R[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x4 ks = {0, 0, 0, 0};
      mma<DK, false, false>(ks, kf + 16 * w * LD, LD, St + 16 * b * LD, LD);
      f32x4 br;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * h + r;
        R[b][r] = v[b][r] - f.in[row] * ks[r];
        br[r] = f.beta[row] * R[b][r];
      }
      *reinterpret_cast<f32x4*>(Rt + (16 * b + l) * kLdC + 16 * w + 4 * h) = br;
    }
    __syncthreads();
    float* Mg = kept.M + slot * kChunk * s.dvp;
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x4 er2 = {0, 0, 0, 0};
      mma<kChunk, false, false>(er2, Ef + 16 * w * kLdC, kLdC, Rt + 16 * b * kLdC, kLdC);
      f32x4 n;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * h + r;
        const float m = R[b][r] - er2[r];
        Mg[int64_t(row) * s.dvp + c0 + 16 * b + l] = m;
        n[r] = f.out[row] * (f.beta[row] * m);
      }
      *reinterpret_cast<f32x4*>(Nt + (16 * b + l) * kLdC + 16 * w + 4 * h) = n;
    }
    __syncthreads();
    const float all = f.all;
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        S[a][b] *= all;
        mma<kChunk, true, false>(S[a][b], kf + 16 * (w * RT + a), LD, Nt + 16 * b * kLdC, kLdC);
      }
  }
  if (!send) return;
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * (w * RT + a) + 4 * h + r, col = c0 + 16 * b + l;
        if (row < s.dk && col < s.dv)
          send[((int64_t(seq) * s.hv + vh) * s.dk + row) * s.dv + col] = S[a][b][r];
      }
}

// o = scale exp(G) (q S) + P N, a workgroup per chunk and value head, a slice
// of the columns at a time.
template <typename T, int DK>
__global__ __launch_bounds__(kDeltaBlock) void k_delta_out(DeltaShape s, DeltaIn<T> in,
                                                           DeltaKept kept, T* __restrict__ o) {
  constexpr int LD = DK + 4;
  extern __shared__ __align__(16) char smem[];
  float* qf = (float*)smem;              // [64][LD]
  float* Pf = qf + kChunk * LD;          // [64][kLdC]
  float* Sf = Pf + kChunk * kLdC;        // [DK][kLdS]
  float* Nf = Sf + DK * kLdS;            // [64][kLdS]
  Factors& f = *(Factors*)(Nf + kChunk * kLdS);
  Place p;
  if (!find_chunk(s, blockIdx.x, p)) return;
  const int vh = blockIdx.y, kh = vh / (s.hv / s.hk);
  const int64_t slot = int64_t(blockIdx.x) * s.hv + vh;
  const int t = threadIdx.x, w = t / kWave, l = t % 16, h = (t % kWave) / 16;
  {
    Rows<T, DK> qr;
    qr.fetch(in.q + p.tok * in.ldq + int64_t(kh) * s.dk, in.ldq, p.len, s.dk);
    Rows<float, kChunk> pr;
    pr.fetch(kept.P + slot * kChunk * kChunk, kChunk, kChunk, kChunk);
    qr.put(qf, LD);
    pr.put(Pf, kLdC);
  }
  load_factors(f, s, kept.G + slot * kChunk, in.beta, p, vh);
  const float* Sg = kept.S + slot * DK * s.dvp;
  const float* Mg = kept.M + slot * kChunk * s.dvp;
  for (int c0 = 0; c0 < s.dvp; c0 += kSlice) {
    __syncthreads();
    for (int i = t; i < DK * kSlice / 4; i += kDeltaBlock) {
      const int row = i / (kSlice / 4), col = i % (kSlice / 4) * 4;
      *reinterpret_cast<f32x4*>(Sf + row * kLdS + col) =
          *reinterpret_cast<const f32x4*>(Sg + int64_t(row) * s.dvp + c0 + col);
    }
    for (int i = t; i < kChunk * kSlice / 4; i += kDeltaBlock) {
      const int row = i / (kSlice / 4), col = i % (kSlice / 4) * 4;
      *reinterpret_cast<f32x4*>(Nf + row * kLdS + col) =
          *reinterpret_cast<const f32x4*>(Mg + int64_t(row) * s.dvp + c0 + col) * f.beta[row];
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x4 acc = {0, 0, 0, 0};
      mma<DK, false, true>(acc, qf + 16 * w * LD, LD, Sf + 16 * b, kLdS);
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[r] *= s.scale * f.in[16 * w + 4 * h + r];
      mma<kChunk, false, true>(acc, Pf + 16 * w * kLdC, kLdC, Nf + 16 * b, kLdS);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * h + r, col = c0 + 16 * b + l;
        if (row < p.len && col < s.dv)
          o[((p.tok + row) * s.hv + vh) * s.dv + col] = T(acc[r]);
      }
    }
  }
}

// The walk backward: X of every chunk and the gradient of the state behind it.
template <typename T, int DK>
__global__ __launch_bounds__(kDeltaBlock) void k_delta_adjoint(
    DeltaShape s, DeltaIn<T> in, DeltaKept kept, const T* __restrict__ dout, int64_t ldo,
    const float* __restrict__ dsend, float* __restrict__ X, float* __restrict__ dS,
    float* __restrict__ ds0) {
  constexpr int LD = DK + 4, RT = DK / 64;
  extern __shared__ __align__(16) char smem[];
  float* kf = (float*)smem;              // [64][LD]
  float* qf = kf + kChunk * LD;          // [64][LD]
  float* Dt = qf + kChunk * LD;          // [32][LD] the state's gradient, transposed
  float* Ef = Dt + kSlice * LD;          // [64][kLdC]
  float* Pf = Ef + kChunk * kLdC;        // [64][kLdC]
  float* Ot = Pf + kChunk * kLdC;        // [32][kLdC] do, then scale exp(G) do, transposed
  float* Yt = Ot + kSlice * kLdC;        // [32][kLdC] beta Y, then -exp(G) beta X, transposed
  Factors& f = *(Factors*)(Yt + kSlice * kLdC);
  const int slices = s.dvp / kSlice;
  const int c0 = blockIdx.x % slices * kSlice;
  const int vh = blockIdx.x / slices % s.hv, seq = blockIdx.x / slices / s.hv;
  const int kh = vh / (s.hv / s.hk);
  const int t = threadIdx.x, w = t / kWave, l = t % 16, h = (t % kWave) / 16;
  const int64_t begin = first_chunk(s, seq), count = first_chunk(s, seq + 1) - begin;
  f32x4 D[RT][2];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * (w * RT + a) + 4 * h + r, col = c0 + 16 * b + l;
        D[a][b][r] = dsend && row < s.dk && col < s.dv
                         ? dsend[((int64_t(seq) * s.hv + vh) * s.dk + row) * s.dv + col] : 0.f;
      }
  for (int64_t c = count - 1; c >= 0; --c) {
    const Place p = chunk_of(s, seq, c);
    const int64_t slot = (begin + c) * s.hv + vh;
    f32x4 o[2];
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * h + r, col = c0 + 16 * b + l;
        o[b][r] = row < p.len && col < s.dv
                      ? float(dout[(p.tok + row) * ldo + int64_t(vh) * s.dv + col]) : 0.f;
      }
    __syncthreads();
    {
      Rows<T, DK> kr, qr;
      kr.fetch(in.k + p.tok * in.ldk + int64_t(kh) * s.dk, in.ldk, p.len, s.dk);
      qr.fetch(in.q + p.tok * in.ldq + int64_t(kh) * s.dk, in.ldq, p.len, s.dk);
      Rows<float, kChunk> er, pr;
      er.fetch(kept.E + slot * kChunk * kChunk, kChunk, kChunk, kChunk);
      pr.fetch(kept.P + slot * kChunk * kChunk, kChunk, kChunk, kChunk);
      kr.put(kf, LD);
      qr.put(qf, LD);
      er.put(Ef, kLdC);
      pr.put(Pf, kLdC);
    }
    load_factors(f, s, kept.G + slot * kChunk, in.beta, p, vh);
    float* Dg = dS + slot * DK * s.dvp;
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        *reinterpret_cast<f32x4*>(Dt + (16 * b + l) * LD + 16 * (w * RT + a) + 4 * h) = D[a][b];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          Dg[int64_t(16 * (w * RT + a) + 4 * h + r) * s.dvp + c0 + 16 * b + l] = D[a][b][r];
      }
#pragma unroll
    for (int b = 0; b < 2; ++b)
      *reinterpret_cast<f32x4*>(Ot + (16 * b + l) * kLdC + 16 * w + 4 * h) = o[b];
    __syncthreads();
    f32x4 Y[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      Y[b] = f32x4{0, 0, 0, 0};
      mma<DK, false, false>(Y[b], kf + 16 * w * LD, LD, Dt + 16 * b * LD, LD);
#pragma unroll
      for (int r = 0; r < 4; ++r) Y[b][r] *= f.out[16 * w + 4 * h + r];
      mma<kChunk, true, false>(Y[b], Pf + 16 * w, kLdC, Ot + 16 * b * kLdC, kLdC);
      f32x4 by;
#pragma unroll
      for (int r = 0; r < 4; ++r) by[r] = f.beta[16 * w + 4 * h + r] * Y[b][r];
      *reinterpret_cast<f32x4*>(Yt + (16 * b + l) * kLdC + 16 * w + 4 * h) = by;
    }
    __syncthreads();
    float* Xg = X + slot * kChunk * s.dvp;
    f32x4 xs[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f32x4 ey = {0, 0, 0, 0};
      mma<kChunk, true, false>(ey, Ef + 16 * w, kLdC, Yt + 16 * b * kLdC, kLdC);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * h + r;
        const float x = Y[b][r] - ey[r];
        Xg[int64_t(row) * s.dvp + c0 + 16 * b + l] = x;
        xs[b][r] = -f.in[row] * (f.beta[row] * x);
        o[b][r] *= s.scale * f.in[row];
      }
    }
    __syncthreads();
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      *reinterpret_cast<f32x4*>(Yt + (16 * b + l) * kLdC + 16 * w + 4 * h) = xs[b];
      *reinterpret_cast<f32x4*>(Ot + (16 * b + l) * kLdC + 16 * w + 4 * h) = o[b];
    }
    __syncthreads();
    const float all = f.all;
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        D[a][b] *= all;
        mma<kChunk, true, false>(D[a][b], kf + 16 * (w * RT + a), LD, Yt + 16 * b * kLdC, kLdC);
        mma<kChunk, true, false>(D[a][b], qf + 16 * (w * RT + a), LD, Ot + 16 * b * kLdC, kLdC);
      }
  }
  if (!ds0) return;
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int b = 0; b < 2; ++b)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * (w * RT + a) + 4 * h + r, col = c0 + 16 * b + l;
        if (row < s.dk && col < s.dv)
          ds0[((int64_t(seq) * s.hv + vh) * s.dk + row) * s.dv + col] = D[a][b][r];
      }
}

// All gradients of a chunk but the state's, a workgroup per chunk and key
// head: the value heads that share the key head are walked one after the
// other, so the gradients of q and k are summed in registers, in one order.
template <typename T, int DK>
__global__ __launch_bounds__(kDeltaBlock) void k_delta_grads(
    DeltaShape s, DeltaIn<T> in, DeltaKept kept, const T* __restrict__ dout, int64_t ldo,
    const float* __restrict__ X, const float* __restrict__ dS, T* __restrict__ dq,
    T* __restrict__ dk, T* __restrict__ dv, float* __restrict__ dg, float* __restrict__ dbeta) {
  constexpr int LD = DK + 4, NT = DK / 16;
  extern __shared__ __align__(16) char smem[];
  // first over the columns of the state, a slice at a time ...
  float* Of = (float*)smem;              // [64][kLdS] do
  float* Xf = Of + kChunk * kLdS;        // [64][kLdS]
  float* Nf = Xf + kChunk * kLdS;        // [64][kLdS]
  float* Sf = Nf + kChunk * kLdS;        // [DK][kLdS]
  float* Df = Sf + DK * kLdS;            // [DK][kLdS]
  // ... then over the chunk's tokens
  float* kf = (float*)smem;              // [64][LD]
  float* qf = kf + kChunk * LD;          // [64][LD]
  float* dP = qf + kChunk * LD;          // [64][kLdC]
  float* dA = dP + kChunk * kLdC;        // [64][kLdC]
  constexpr int kA = 3 * kChunk * kLdS + 2 * DK * kLdS;
  constexpr int kB = 2 * kChunk * LD + 2 * kChunk * kLdC;
  Factors& f = *(Factors*)((float*)smem + (kA > kB ? kA : kB));
  double* G = (double*)(&f + 1);
  double* dG = G + kChunk;
  float* part = (float*)(dG + kChunk);   // [8]
  Place p;
  if (!find_chunk(s, blockIdx.x, p)) return;
  const int kh = blockIdx.y, group = s.hv / s.hk;
  const int t = threadIdx.x, w = t / kWave, l = t % 16, h = (t % kWave) / 16;
  f32x4 aq[NT], ak[NT];  // sums over the group, rows 16 w + 4 h + r, columns 16 n + l
#pragma unroll
  for (int n = 0; n < NT; ++n) aq[n] = ak[n] = f32x4{0, 0, 0, 0};

  for (int vh = kh * group; vh < (kh + 1) * group; ++vh) {
    const int64_t slot = int64_t(blockIdx.x) * s.hv + vh;
    const float* Sg = kept.S + slot * DK * s.dvp;
    const float* Dg = dS + slot * DK * s.dvp;
    const float* Mg = kept.M + slot * kChunk * s.dvp;
    const float* Xg = X + slot * kChunk * s.dvp;
    __syncthreads();
    load_factors(f, s, kept.G + slot * kChunk, in.beta, p, vh);
    if (t < kChunk) G[t] = kept.G[slot * kChunk + t];
    f32x4 pp[4], pa[4], oS[NT], xS[NT], nD[NT];
#pragma unroll
    for (int j = 0; j < 4; ++j) pp[j] = pa[j] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int n = 0; n < NT; ++n) oS[n] = xS[n] = nD[n] = f32x4{0, 0, 0, 0};
    float sd = 0.f;   // <S, dS> of this thread's elements
    float xm = 0.f;   // X . M of row t / 4, a quarter of its columns
    for (int c0 = 0; c0 < s.dvp; c0 += kSlice) {
      __syncthreads();
      {
        const int row = t / 4, col = t % 4 * 8;
        float a[8], m[8], x[8];
        load_f32<8>(dout + (p.tok + row) * ldo + int64_t(vh) * s.dv + c0 + col,
                    row < p.len ? s.dv - c0 - col : 0, a);
        load_f32<8>(Mg + int64_t(row) * s.dvp + c0 + col, 8, m);
        load_f32<8>(Xg + int64_t(row) * s.dvp + c0 + col, 8, x);
        const float be = f.beta[row];
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          xm += x[i] * m[i];
          v[i] = be * x[i];
          Of[row * kLdS + col + i] = a[i];
          Xf[row * kLdS + col + i] = x[i];
          Nf[row * kLdS + col + i] = be * m[i];
        }
        if (dv && row < p.len)
          store_f32<8>(dv + ((p.tok + row) * s.hv + vh) * s.dv + c0 + col, s.dv - c0 - col, v);
      }
      for (int i = t; i < DK * kSlice / 4; i += kDeltaBlock) {
        const int row = i / (kSlice / 4), col = i % (kSlice / 4) * 4;
        const f32x4 a = *reinterpret_cast<const f32x4*>(Sg + int64_t(row) * s.dvp + c0 + col);
        const f32x4 b = *reinterpret_cast<const f32x4*>(Dg + int64_t(row) * s.dvp + c0 + col);
        sd += a[0] * b[0] + a[1] * b[1] + (a[2] * b[2] + a[3] * b[3]);
        *reinterpret_cast<f32x4*>(Sf + row * kLdS + col) = a;
        *reinterpret_cast<f32x4*>(Df + row * kLdS + col) = b;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j <= w) {
          mma<kSlice, false, false>(pp[j], Of + 16 * w * kLdS, kLdS, Nf + 16 * j * kLdS, kLdS);
          mma<kSlice, false, false>(pa[j], Xf + 16 * w * kLdS, kLdS, Nf + 16 * j * kLdS, kLdS);
        }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma<kSlice, false, false>(oS[n], Of + 16 * w * kLdS, kLdS, Sf + 16 * n * kLdS, kLdS);
        mma<kSlice, false, false>(xS[n], Xf + 16 * w * kLdS, kLdS, Sf + 16 * n * kLdS, kLdS);
        mma<kSlice, false, false>(nD[n], Nf + 16 * w * kLdS, kLdS, Df + 16 * n * kLdS, kLdS);
      }
    }
    xm = lane_sum<4>(xm);
    sd = lane_sum<kWave>(sd);
    __syncthreads();
    if (dbeta && t % 4 == 0 && t / 4 < p.len) dbeta[(p.tok + t / 4) * s.hv + vh] = xm;
    if (t % kWave == 0) part[w] = sd;
    {
      Rows<T, DK> kr, qr;
      kr.fetch(in.k + p.tok * in.ldk + int64_t(kh) * s.dk, in.ldk, p.len, s.dk);
      qr.fetch(in.q + p.tok * in.ldq + int64_t(kh) * s.dk, in.ldq, p.len, s.dk);
      kr.put(kf, LD);
      qr.put(qf, LD);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * h + r, col = 16 * j + l;
        const float d = col <= row ? expf(float(G[row] - G[col])) : 0.f;
        dP[row * kLdC + col] = col <= row ? s.scale * d * pp[j][r] : 0.f;
        dA[row * kLdC + col] = col < row ? d * f.beta[row] * pa[j][r] : 0.f;
      }
    __syncthreads();
    float dgr[4] = {0.f, 0.f, 0.f, 0.f};
    float end = 0.f;  // sum over the rows of k_i . exp(G_L - G_i) (N dS^T)_i
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      f32x4 q4, u = {0, 0, 0, 0}, wv = {0, 0, 0, 0}, nd;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * h + r;
        q4[r] = s.scale * f.in[row] * oS[n][r];
        u[r] = f.in[row] * f.beta[row] * xS[n][r];
        nd[r] = f.out[row] * nD[n][r];
      }
      mma<kChunk, false, true>(q4, dP + 16 * w * kLdC, kLdC, kf + 16 * n, LD);
      mma<kChunk, false, true>(u, dA + 16 * w * kLdC, kLdC, kf + 16 * n, LD);
      mma<kChunk, true, true>(wv, dP + 16 * w, kLdC, qf + 16 * n, LD);
      f32x4 wa = {0, 0, 0, 0};
      mma<kChunk, true, true>(wa, dA + 16 * w, kLdC, kf + 16 * n, LD);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * w + 4 * h + r;
        const float kv = kf[row * LD + 16 * n + l], qv = qf[row * LD + 16 * n + l];
        const float away = wv[r] - wa[r] + nd[r];
        dgr[r] += qv * q4[r] - kv * (u[r] + away);
        end += kv * nd[r];
        aq[n][r] += q4[r];
        ak[n][r] += away - u[r];
      }
    }
    if (dg) {
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        dgr[r] = lane_sum<16>(dgr[r]);
        if (l == 0) dG[16 * w + 4 * h + r] = double(dgr[r]);
      }
      end = lane_sum<kWave>(end);
      if (t % kWave == 0) part[4 + w] = end;
      __syncthreads();
      if (t < kChunk) {
        double x = dG[kChunk - 1 - t];
        if (t == 0)
          x += double(f.all) * ((double(part[0]) + part[1]) + (double(part[2]) + part[3])) +
               ((double(part[4]) + part[5]) + (double(part[6]) + part[7]));
#pragma unroll
        for (int d = 1; d < kWave; d <<= 1) {
          const double u = __shfl_up(x, d, kWave);
          if (t >= d) x += u;
        }
        const int row = kChunk - 1 - t;
        if (row < p.len) dg[(p.tok + row) * s.hv + vh] = float(x);
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * w + 4 * h + r, col = 16 * n + l;
      if (row < p.len && col < s.dk) {
        const int64_t at = ((p.tok + row) * s.hk + kh) * s.dk + col;
        if (dq) dq[at] = T(aq[n][r]);
        if (dk) dk[at] = T(ak[n][r]);
      }
    }
}

// One token of every sequence, the state updated in place: a workgroup per
// sequence, value head and 32 columns; 8 lanes of 4 columns by 32 lines of
// rows, each thread's part of the state in registers between its one read
// and its one write.  Both sums over the rows (k and q against the state)
// come from that one read, since S_t^T q = exp(g) S^T q + (k.q) beta m.
template <typename T, int NR>
__global__ __launch_bounds__(kDeltaBlock) void k_delta_step(
    const T* __restrict__ q, int64_t ldq, const T* __restrict__ k, int64_t ldk,
    const T* __restrict__ v, int64_t ldv, const float* __restrict__ g,
    const float* __restrict__ beta, float* __restrict__ state, T* __restrict__ o, int hk, int hv,
    int dk, int dv, float scale) {
  __shared__ f32x4 sk[4][8], sq[4][8];
  __shared__ float sqk[4];
  const int t = threadIdx.x, cl = t % 8, line = t / 8, w = t / kWave;
  const int64_t sh = blockIdx.x;  // sequence * hv + head
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
                      z.chunks < (int64_t(1) << 31),
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

template <typename F>
sla_status with_delta(const sla_delta_dims* d, F&& f) {
  using D64 = std::integral_constant<int, 64>;
  using D128 = std::integral_constant<int, 128>;
  const bool small = pad_dk(d->key_dim) == 64;
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
  clear_error();
  DeltaSizes z;
  SLA_TRY(delta_sizes("sla_delta_rule_work", dims, z));
  if (kept_bytes_host) *kept_bytes_host = z.kept;
  if (grad_bytes_host) *grad_bytes_host = z.grad;
  return SLA_OK;
}

sla_status sla_delta_rule(const sla_delta_dims* dims, const void* q, int64_t ldq, const void* k,
                          int64_t ldk, const void* v, int64_t ldv, const float* g,
                          const float* beta, const int32_t* offsets, const float* initial_state,
                          void* o, float* final_state, void* kept, int64_t kept_bytes,
                          hipStream_t stream) {
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
  return with_delta(dims, [&](auto te, auto width) -> sla_status {
    using T = decltype(te);
    constexpr int DK = width.value, LD = DK + 4;
    const DeltaIn<T> in = {(const T*)q, (const T*)k, (const T*)v, ldq, ldk, ldv, g, beta};
    if (z.chunks) {
      constexpr int lds = (2 * kChunk * LD + kChunk * kLdC) * 4 + kChunk * 12;
      SLA_TRY(allow_lds(k_delta_prepare<T, DK>, lds));
      k_delta_prepare<T, DK><<<dim3(int(z.chunks), s.hv), kDeltaBlock, lds, stream>>>(s, in, w);
      LAUNCH_CHECK();
    }
    {
      constexpr int lds = (kChunk * LD + kSlice * LD + kChunk * kLdC + 2 * kSlice * kLdC) * 4 +
                          int(sizeof(Factors));
      SLA_TRY(allow_lds(k_delta_states<T, DK>, lds));
      k_delta_states<T, DK><<<s.nseq * s.hv * (s.dvp / kSlice), kDeltaBlock, lds, stream>>>(
          s, in, w, initial_state, final_state);
      LAUNCH_CHECK();
    }
    if (z.chunks) {
      constexpr int lds = (kChunk * LD + kChunk * kLdC + (DK + kChunk) * kLdS) * 4 +
                          int(sizeof(Factors));
      SLA_TRY(allow_lds(k_delta_out<T, DK>, lds));
      k_delta_out<T, DK><<<dim3(int(z.chunks), s.hv), kDeltaBlock, lds, stream>>>(s, in, w, (T*)o);
      LAUNCH_CHECK();
    }
    return SLA_OK;
  });
}

sla_status sla_delta_rule_grad(const sla_delta_dims* dims, const void* q, int64_t ldq,
                               const void* k, int64_t ldk, const void* v, int64_t ldv,
                               const float* g, const float* beta, const void* kept,
                               int64_t kept_bytes, const void* grad_o, int64_t ldo,
                               const float* grad_final_state, void* dq, void* dk, void* dv,
                               float* dg, float* dbeta, float* grad_initial_state, void* work,
                               int64_t work_bytes, hipStream_t stream) {
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
  return with_delta(dims, [&](auto te, auto width) -> sla_status {
    using T = decltype(te);
    constexpr int DK = width.value, LD = DK + 4;
    const DeltaIn<T> in = {(const T*)q, (const T*)k, (const T*)v, ldq, ldk, ldv, g, beta};
    {
      constexpr int lds = (2 * kChunk * LD + kSlice * LD + 2 * kChunk * kLdC +
                           2 * kSlice * kLdC) * 4 + int(sizeof(Factors));
      SLA_TRY(allow_lds(k_delta_adjoint<T, DK>, lds));
      k_delta_adjoint<T, DK><<<s.nseq * s.hv * (s.dvp / kSlice), kDeltaBlock, lds, stream>>>(
          s, in, w, (const T*)grad_o, ldo, grad_final_state, X, dS, grad_initial_state);
      LAUNCH_CHECK();
    }
    if (z.chunks && (dq || dk || dv || dg || dbeta)) {
      constexpr int a = 3 * kChunk * kLdS + 2 * DK * kLdS;
      constexpr int b = 2 * kChunk * LD + 2 * kChunk * kLdC;
      constexpr int lds = (a > b ? a : b) * 4 + int(sizeof(Factors)) + 2 * kChunk * 8 + 32;
      SLA_TRY(allow_lds(k_delta_grads<T, DK>, lds));
      k_delta_grads<T, DK><<<dim3(int(z.chunks), s.hk), kDeltaBlock, lds, stream>>>(
          s, in, w, (const T*)grad_o, ldo, X, dS, (T*)dq, (T*)dk, (T*)dv, dg, dbeta);
      LAUNCH_CHECK();
    }
    return SLA_OK;
  });
}

sla_status sla_delta_step(const sla_delta_dims* dims, const void* q, int64_t ldq, const void* k,
                          int64_t ldk, const void* v, int64_t ldv, const float* g,
                          const float* beta, float* state, void* o, hipStream_t stream) {
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
    const dim3 grid(int(dims->sequences * dims->value_heads), int(div_up(dims->value_dim, kSlice)));
    k_delta_step<T, nr.value><<<grid, kDeltaBlock, 0, stream>>>(
        (const T*)q, ldq, (const T*)k, ldk, (const T*)v, ldv, g, beta, state, (T*)o,
        int(dims->key_heads), int(dims->value_heads), int(dims->key_dim), int(dims->value_dim),
        float(dims->scale));
    LAUNCH_CHECK();
    return SLA_OK;
  };
  return with_delta(dims, [&](auto te, auto width) {
    return go(te, std::integral_constant<int, width.value / 32>());
  });
}

}  // extern "C"
