// The gated scan: a linear recurrence with a decay of its own for every
// channel and token, its gradients, and one token against a kept state.
//
//   a_t = exp(g_t)      h_t = a_t h_{t-1} + x_t
//   l_t = dh_t + m_t    m_{t-1} = a_t l_t     (m_T: the final state's gradient)
//   dx_t = l_t          dg_t = m_{t-1} h_{t-1}          ds0 = m_0
//
// Bound by memory: forward reads x and g and writes h, backward reads x, g and
// dh and writes dx and dg, once each.  A span of tokens is a map h -> P h + H
// with P the product of its decays (and, backwards, m -> P m + M): maps are
// joined without a division, so a decay of zero or a product that underflows
// is harmless.  A thread holds kSpan tokens of its channels in registers; the
// spans of a workgroup's block of tokens are joined in the wave by shuffles and
// over the waves through LDS, in a fixed order; then every thread walks its
// tokens again from the state in front of them.  From block to block the state
// is carried in registers, while the next block's loads travel.
//
// The forward pass keeps the state in front of every block (4 bytes a channel
// and block), from which the backward pass makes h again: it needs x then
// instead of h, as many bytes, and h in fp32 instead of rounded.
//
// Where sequences and channels do not fill the card a sequence is cut into
// segments: k_scan_ends finds every segment's map first, the walks begin with
// the maps of the segments on the way joined.  That reads two arrays again.
// Packed sequences, whose lengths the host does not know, are cut by length: a
// table on the device says which workgroup has which segment.
//
// Measured: 4 x 4096 x 2048 bf16 forward 43 us (201 MB, 4.7 TB/s), backward 85 (336
// MB, 4.0); 131072 x 256 fp16 with fp32 gates 34 us for the maps and 53 for the
// walk (268 MB that have to move); 12345 x 999 fp32 in 23 sequences 40 and 69 us
// (148 and 247 MB); 2048 x 4096 single tokens in bf16 18 us (117 MB, which the
// last cache holds in part).
#include <type_traits>

#include "net.h"

namespace sla {
namespace net {
namespace {

constexpr int kSpan = 8;       // tokens a thread holds
constexpr int kMostSegments = 64;
constexpr int kFill = 512;     // workgroups wanted: two on each of the 256 CUs
constexpr int64_t kMostGroups = int64_t(1) << 20;   // of a launch; they walk the items

// exp(g).  fp32 gates: to 2 ulp, the instruction's exp2 with the product's
// rounding error put right; below -200 and above 200 it is 0 and inf as it is, and
// where exp2 has left the range nothing is put right (inf with an error of 0 or below
// would be NaN); NaN stays.  16-bit gates: without that, off by |g| 2^-23.5 of itself, far below
// their own half step (and a |g| is 0.4 at most, so the state is as good).
template <typename G>
__device__ __forceinline__ float decay(G gate) {
  constexpr float kHi = 1.44269502f, kLo = 1.92596303e-08f;   // log2(e)
  float g = float(gate);
  if constexpr (sizeof(G) == 2) return __builtin_amdgcn_exp2f(g * kHi);
  g = g < -200.f ? -200.f : g > 200.f ? 200.f : g;
  const float t = g * kHi;
  const float r = __builtin_fmaf(g, kLo, __builtin_fmaf(g, kHi, -t));
  const float e = __builtin_amdgcn_exp2f(t);
  return e == __builtin_inff() ? e : __builtin_fmaf(e, r * 0.693147182f, e);
}

struct ScanShape {
  int64_t nseq, seqlen, total;   // seqlen: tokens of every sequence (no offsets)
  int64_t channels;
  const int32_t* tok;            // packed: first token of each sequence [nseq + 1]
  int tiles;                     // of channels
  int segments;                  // of every sequence (no table)
  // packed sequences of which the long ones are cut: {sequence, segment, its map's
  // number} of up to `parts` segments of `each` blocks, sequence -1 behind the last
  const int4* table;
  int64_t parts, each;
  int64_t items;
};
constexpr int kGapItems = 8;     // workgroups (of a tile) for the tokens of no sequence

// What a workgroup works on: a sequence's segment and a tile of its channels.
struct Item {
  int64_t seq;
  int tile, seg, segs;    // segs: the sequence's
  int64_t map;            // where the segment's map lies
  int64_t from, len;      // the sequence's tokens
  int64_t first;          // its first block among all blocks
  int64_t b0, b1, blocks; // the segment's blocks, the sequence's
};
template <int BT>
__device__ __forceinline__ Item item_of(const ScanShape& s, int64_t id) {
  Item w;
  w.tile = int(id % s.tiles);
  id /= s.tiles;
  const int64_t all = s.table ? s.parts : s.nseq * s.segments;
  w.map = id;
  if (id >= all) {   // the tokens of no sequence
    w.seq = s.nseq;
    w.seg = int(id - all);
    return w;
  }
  if (s.table) {
    const int4 e = s.table[id];
    w.seq = e.x;
    w.seg = e.y;
    w.map = e.z;
    if (w.seq < 0) return w;
  } else {
    w.seg = int(id % s.segments);
    w.seq = id / s.segments;
  }
  if (s.tok) {
    w.from = s.tok[w.seq];
    w.len = s.tok[w.seq + 1] - w.from;
    w.first = w.from / BT + w.seq;
  } else {
    w.from = w.seq * s.seqlen;
    w.len = s.seqlen;
    w.first = w.seq * div_up(s.seqlen, BT);
  }
  w.blocks = (w.len + BT - 1) / BT;
  // an odd number of blocks: segments that begin at multiples of a large power
  // of two would all begin in the same memory channels
  const int64_t each =
      s.table ? s.each : (w.blocks + s.segments - 1) / s.segments | (s.segments > 1);
  w.segs = s.table ? int((w.blocks + each - 1) / each) : s.segments;
  w.b0 = w.seg * each < w.blocks ? w.seg * each : w.blocks;
  w.b1 = w.b0 + each < w.blocks ? w.b0 + each : w.blocks;
  return w;
}
// Workgroups go to the 8 XCDs in turn: each gets runs of 16 neighbouring items,
// whose tiles share cache lines.  (One long run each would leave the XCDs idle
// that have the short sequences, or nothing but the tokens of none.)
__device__ __forceinline__ int64_t item_id(int64_t items) {
  constexpr int kRun = 16, kTurn = kRun * kXcds;
  const int64_t total = gridDim.x, b = blockIdx.x;
  if (total < items || b >= total / kTurn * kTurn) return b;
  return b / kTurn * kTurn + b % kXcds * kRun + b / kXcds % kRun;
}

// A thread's place: CL lanes have the tile's channels, the others are further
// spans of tokens.
template <int CL, int WAVES, int V>
struct Place {
  static constexpr int kSlices = kWave / CL;            // spans of a wave
  static constexpr int kBlock = WAVES * kSlices * kSpan;  // tokens of a block
  int lane, slice, wave;
  int64_t tile;     // the tile's first channel
  int in;           // the thread's first channel to read, from there on
  bool on;          // whether it is the thread's own (lanes behind the last read another's)
  __device__ __forceinline__ Place(int which, int64_t channels) {
    const int t = threadIdx.x;
    lane = t % CL;
    slice = t % kWave / CL;
    wave = __builtin_amdgcn_readfirstlane(t / kWave);
    tile = int64_t(which) * CL * V;
    const int64_t left = channels - tile;
    on = lane * V < left;
    in = on ? lane * V : int(left) - V;
  }
  __device__ __forceinline__ int64_t channel() const { return tile + in; }
  // the thread's first token of a block
  __device__ __forceinline__ int64_t token(int64_t block) const {
    return block * kBlock + (wave * kSlices + slice) * kSpan;
  }
};

// One array's part of a sequence's tile: where a wave's block begins (in scalar
// registers) and the thread's place behind that, in bytes (31 bits: spans of a
// wave lie less than 2^24 elements apart, or there is one).
template <typename T, int V, typename At>
struct Lane {
  typedef typename VecOf<typename std::remove_const<T>::type, V>::type Value;
  typedef typename std::conditional<std::is_const<T>::value, const Value, Value>::type Vec;
  T* p;            // the sequence's first token, the tile's first channel
  int64_t ld;
  int at;
  __device__ __forceinline__ Lane(T* first, int64_t ld_, const At& me)
      : p(first), ld(ld_), at(int((me.slice * kSpan * ld_ + me.in) * int64_t(sizeof(T)))) {}
  __device__ __forceinline__ T* block(int64_t b, int wave) const {
    const uint64_t q = reinterpret_cast<uint64_t>(
        p + (b * At::kBlock + wave * At::kSlices * kSpan) * ld);
    return reinterpret_cast<T*>(
        uint64_t(uint32_t(__builtin_amdgcn_readfirstlane(int(q >> 32)))) << 32 |
        uint32_t(__builtin_amdgcn_readfirstlane(int(q))));
  }
  __device__ __forceinline__ Vec* token(T* block, int j) const {
    return reinterpret_cast<Vec*>(reinterpret_cast<uintptr_t>(block + j * ld) + uint32_t(at));
  }
};

// The raw values of a thread's span; tokens behind the end read the last one.
template <typename T, int V>
struct Raw {
  typename VecOf<T, V>::type v[kSpan];
  template <typename At>
  __device__ __forceinline__ void load(const Lane<const T, V, At>& from, int64_t b, int64_t len,
                                       const At& me) {
    if ((b + 1) * At::kBlock <= len) {
      const T* q = from.block(b, me.wave);
#pragma unroll
      for (int j = 0; j < kSpan; ++j) v[j] = *from.token(q, j);
    } else {
      const int64_t t = me.token(b);
#pragma unroll
      for (int j = 0; j < kSpan; ++j) {
        const int64_t at = t + j < len ? t + j : len - 1;
        v[j] = *reinterpret_cast<const typename VecOf<T, V>::type*>(from.p + at * from.ld + me.in);
      }
    }
  }
};

// In-wave joins over the slices (CL lanes apart): inclusive from the first
// slice on (UP), or from the last.
template <int CL, int V, bool UP>
__device__ __forceinline__ void join_slices(float (&P)[V], float (&H)[V], int slice) {
#pragma unroll
  for (int d = 1; d < kWave / CL; d <<= 1) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float p = UP ? __shfl_up(P[v], d * CL, kWave) : __shfl_down(P[v], d * CL, kWave);
      const float q = UP ? __shfl_up(H[v], d * CL, kWave) : __shfl_down(H[v], d * CL, kWave);
      const bool has = UP ? slice >= d : slice + d < kWave / CL;
      if (has) {
        H[v] = P[v] * q + H[v];
        P[v] *= p;
      }
    }
  }
}
// ... and what lies before (behind) the own slice alone.
template <int CL, int V, bool UP>
__device__ __forceinline__ void shift_slices(float (&P)[V], float (&H)[V], int slice) {
  if constexpr (CL == kWave) {
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.f, H[v] = 0.f;
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const float p = UP ? __shfl_up(P[v], CL, kWave) : __shfl_down(P[v], CL, kWave);
      const float q = UP ? __shfl_up(H[v], CL, kWave) : __shfl_down(H[v], CL, kWave);
      const bool has = UP ? slice > 0 : slice < kWave / CL - 1;
      P[v] = has ? p : 1.f;
      H[v] = has ? q : 0.f;
    }
  }
}

// A state through `count` segments' maps, forwards or backwards; eight maps'
// loads travel at once (one by one 63 of them took longer than the walk).
template <int V, int STEP>
__device__ __forceinline__ void through(float (&state)[V], const float* ends, int64_t ld,
                                        int count) {
  for (int k = 0; k < count; k += 8) {
    float e[8][2 * V];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float* p = ends + STEP * (k + i < count ? k + i : k) * ld;
#pragma unroll
      for (int v = 0; v < 2 * V; ++v) e[i][v] = p[v];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v)
        state[v] = k + i < count ? e[i][2 * v] * state[v] + e[i][2 * v + 1] : state[v];
  }
}

// Rows of tokens of no sequence become zero.
template <typename T, int CL, int WAVES, int V>
__device__ __forceinline__ void clear_rows(const ScanShape& s, const Item& w, T* out) {
  if (!out) return;
  const Place<CL, WAVES, V> me(w.tile, s.channels);
  const int64_t head = s.tok[0], tail = s.tok[s.nseq], rows = head + s.total - tail;
  if (!me.on) return;
  constexpr int kSlices = WAVES * Place<CL, WAVES, V>::kSlices;
  for (int64_t i = int64_t(w.seg) * kSlices + threadIdx.x / CL; i < rows;
       i += int64_t(kGapItems) * kSlices) {
    typename VecOf<T, V>::type z = {};
    *reinterpret_cast<typename VecOf<T, V>::type*>(
        out + (i < head ? i : tail + i - head) * s.channels + me.channel()) = z;
  }
}

template <typename T, typename G, int CL, int WAVES, int V>
__global__ __launch_bounds__(WAVES* kWave, 4) void k_scan(
    ScanShape s, const T* __restrict__ x, int64_t ldx, const G* __restrict__ g, int64_t ldg,
    const float* __restrict__ s0, T* __restrict__ h, float* __restrict__ last,
    float* __restrict__ kept, const float* __restrict__ ends) {
  typedef Place<CL, WAVES, V> At;
  constexpr int BT = At::kBlock;
  __shared__ float2 agg[2][WAVES][CL * V];
  int buf = 0;
  for (int64_t id = item_id(s.items); id < s.items; id += gridDim.x) {
    const Item w = item_of<BT>(s, id);
    if (w.seq < 0) continue;
    if (w.seq >= s.nseq) {
      clear_rows<T, CL, WAVES, V>(s, w, h);
      continue;
    }
    if (w.seg > 0 && w.b0 == w.b1) continue;
    const At me(w.tile, s.channels);
    const int64_t ch = me.channel();
    float carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = s0 ? s0[w.seq * s.channels + ch + v] : 0.f;
    through<V, 1>(carry, ends + ((w.map - w.seg) * s.channels + ch) * 2, s.channels * 2, w.seg);
    const Lane<const T, V, At> fx(x + w.from * ldx + me.tile, ldx, me);
    const Lane<const G, V, At> fg(g + w.from * ldg + me.tile, ldg, me);
    const Lane<T, V, At> fh(h + w.from * s.channels + me.tile, s.channels, me);
    Raw<T, V> rx;
    Raw<G, V> rg;
    if (w.b0 < w.b1) {
      rx.load(fx, w.b0, w.len, me);
      rg.load(fg, w.b0, w.len, me);
    }
    for (int64_t b = w.b0; b < w.b1; ++b) {
      const bool whole = (b + 1) * BT <= w.len;
      const int left = whole ? kSpan : int(w.len - me.token(b) < kSpan ? w.len - me.token(b) : kSpan);
      float a[kSpan][V], u[kSpan][V], P[V], H[V];
#pragma unroll
      for (int j = 0; j < kSpan; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          a[j][v] = decay(rg.v[j][v]);
          u[j][v] = float(rx.v[j][v]);
        }
      if (!whole) {   // what lies behind the end changes nothing
#pragma unroll
        for (int j = 0; j < kSpan; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            a[j][v] = j < left ? a[j][v] : 1.f;
            u[j][v] = j < left ? u[j][v] : 0.f;
          }
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        P[v] = a[0][v];
        H[v] = u[0][v];
#pragma unroll
        for (int j = 1; j < kSpan; ++j) {
          H[v] = a[j][v] * H[v] + u[j][v];
          P[v] *= a[j][v];
        }
      }
      if (b + 1 < w.b1) {
        rx.load(fx, b + 1, w.len, me);
        rg.load(fg, b + 1, w.len, me);
      }
      join_slices<CL, V, true>(P, H, me.slice);
      if (me.slice == At::kSlices - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) agg[buf][me.wave][me.lane * V + v] = make_float2(P[v], H[v]);
      }
      shift_slices<CL, V, true>(P, H, me.slice);
      __syncthreads();
      if (kept && me.on && me.wave == 0 && me.slice == 0) {
#pragma unroll
        for (int v = 0; v < V; ++v) kept[(w.first + b) * s.channels + ch + v] = carry[v];
      }
      float state[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        state[v] = carry[v];
#pragma unroll
        for (int k = 0; k < WAVES; ++k) {
          if (k == me.wave) state[v] = carry[v];
          const float2 m = agg[buf][k][me.lane * V + v];
          carry[v] = m.x * carry[v] + m.y;
        }
        state[v] = P[v] * state[v] + H[v];
      }
      buf ^= 1;
      T* const to = fh.block(b, me.wave);
#pragma unroll
      for (int j = 0; j < kSpan; ++j) {
        typename VecOf<T, V>::type o;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          state[v] = a[j][v] * state[v] + u[j][v];
          o[v] = T(state[v]);
        }
        if (me.on && j < left) *fh.token(to, j) = o;
      }
    }
    if (last && me.on && w.b1 == w.blocks && me.wave == 0 && me.slice == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) last[w.seq * s.channels + ch + v] = carry[v];
    }
  }
}

template <typename T, typename G, int CL, int WAVES, int V>
__global__ __launch_bounds__(WAVES* kWave) void k_scan_grad(
    ScanShape s, const T* __restrict__ x, int64_t ldx, const G* __restrict__ g, int64_t ldg,
    const float* __restrict__ kept, const T* __restrict__ dh, int64_t lddh,
    const float* __restrict__ dlast, T* __restrict__ dx, G* __restrict__ dg,
    float* __restrict__ ds0, const float* __restrict__ ends) {
  typedef Place<CL, WAVES, V> At;
  constexpr int BT = At::kBlock;
  __shared__ float2 fwd[2][WAVES][CL * V];
  __shared__ float back[2][WAVES][CL * V];
  int buf = 0;
  for (int64_t id = item_id(s.items); id < s.items; id += gridDim.x) {
    const Item w = item_of<BT>(s, id);
    if (w.seq < 0) continue;
    if (w.seq >= s.nseq) {
      clear_rows<T, CL, WAVES, V>(s, w, dx);
      clear_rows<G, CL, WAVES, V>(s, w, dg);
      continue;
    }
    if (w.seg > 0 && w.b0 == w.b1) continue;
    const At me(w.tile, s.channels);
    const int64_t ch = me.channel();
    float carry[V];
#pragma unroll
    for (int v = 0; v < V; ++v) carry[v] = dlast ? dlast[w.seq * s.channels + ch + v] : 0.f;
    if (w.segs > 1)
      through<V, -1>(carry, ends + ((w.map - w.seg + w.segs - 1) * s.channels + ch) * 2,
                     s.channels * 2, w.segs - 1 - w.seg);
    const Lane<const T, V, At> fx(x + w.from * ldx + me.tile, ldx, me);
    const Lane<const G, V, At> fg(g + w.from * ldg + me.tile, ldg, me);
    const Lane<const T, V, At> fd(dh + w.from * lddh + me.tile, lddh, me);
    const int64_t out = w.from * s.channels + me.tile;
    const Lane<T, V, At> tx(dx + (dx ? out : 0), s.channels, me);
    const Lane<G, V, At> tg(dg + (dg ? out : 0), s.channels, me);
    Raw<T, V> rx, rd;
    Raw<G, V> rg;
    float next[V];   // the state in front of the block that is loaded
    auto load = [&](int64_t b) {
      rx.load(fx, b, w.len, me);
      rg.load(fg, b, w.len, me);
      rd.load(fd, b, w.len, me);
#pragma unroll
      for (int v = 0; v < V; ++v) next[v] = kept[(w.first + b) * s.channels + ch + v];
    };
    if (w.b0 < w.b1) load(w.b1 - 1);
    for (int64_t b = w.b1; b-- > w.b0;) {
      const bool whole = (b + 1) * BT <= w.len;
      const int left = whole ? kSpan : int(w.len - me.token(b) < kSpan ? w.len - me.token(b) : kSpan);
      float a[kSpan][V], u[kSpan][V], d[kSpan][V], P[V], H[V], Q[V], M[V], state[V], m[V];
#pragma unroll
      for (int v = 0; v < V; ++v) state[v] = next[v];
#pragma unroll
      for (int j = 0; j < kSpan; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          a[j][v] = decay(rg.v[j][v]);
          u[j][v] = float(rx.v[j][v]);
          d[j][v] = float(rd.v[j][v]);
        }
      if (!whole) {
#pragma unroll
        for (int j = 0; j < kSpan; ++j)
#pragma unroll
          for (int v = 0; v < V; ++v) {
            a[j][v] = j < left ? a[j][v] : 1.f;
            u[j][v] = j < left ? u[j][v] : 0.f;
            d[j][v] = j < left ? d[j][v] : 0.f;
          }
      }
      if (b > w.b0) load(b - 1);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        P[v] = a[0][v];
        H[v] = u[0][v];
#pragma unroll
        for (int j = 1; j < kSpan; ++j) {
          H[v] = a[j][v] * H[v] + u[j][v];
          P[v] *= a[j][v];
        }
        M[v] = a[kSpan - 1][v] * d[kSpan - 1][v];
#pragma unroll
        for (int j = kSpan - 2; j >= 0; --j) M[v] = a[j][v] * (d[j][v] + M[v]);
        Q[v] = P[v];
      }
      join_slices<CL, V, true>(P, H, me.slice);
      join_slices<CL, V, false>(Q, M, me.slice);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (me.slice == At::kSlices - 1)
          fwd[buf][me.wave][me.lane * V + v] = make_float2(P[v], H[v]);
        if (me.slice == 0) back[buf][me.wave][me.lane * V + v] = M[v];
      }
      shift_slices<CL, V, true>(P, H, me.slice);
      shift_slices<CL, V, false>(Q, M, me.slice);
      __syncthreads();
#pragma unroll
      for (int v = 0; v < V; ++v) {
        m[v] = carry[v];
        float2 f[WAVES];
#pragma unroll
        for (int k = 0; k < WAVES; ++k) {
          f[k] = fwd[buf][k][me.lane * V + v];
          if (k < me.wave) state[v] = f[k].x * state[v] + f[k].y;
        }
#pragma unroll
        for (int k = WAVES - 1; k >= 0; --k) {
          if (k == me.wave) m[v] = carry[v];
          carry[v] = f[k].x * carry[v] + back[buf][k][me.lane * V + v];
        }
        state[v] = P[v] * state[v] + H[v];
        m[v] = Q[v] * m[v] + M[v];
      }
      buf ^= 1;
#pragma unroll
      for (int j = 0; j < kSpan; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float after = a[j][v] * state[v] + u[j][v];
          u[j][v] = state[v];
          state[v] = after;
        }
      }
      T* const ox = tx.block(b, me.wave);
      G* const og = tg.block(b, me.wave);
#pragma unroll
      for (int j = kSpan - 1; j >= 0; --j) {
        typename VecOf<T, V>::type vx;
        typename VecOf<G, V>::type vg;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float l = d[j][v] + m[v];
          m[v] = a[j][v] * l;
          vx[v] = T(l);
          vg[v] = G(m[v] * u[j][v]);
        }
        if (me.on && j < left) {
          if (dx) *tx.token(ox, j) = vx;
          if (dg) *tg.token(og, j) = vg;
        }
      }
    }
    if (ds0 && me.on && w.seg == 0 && me.wave == 0 && me.slice == 0) {
#pragma unroll
      for (int v = 0; v < V; ++v) ds0[w.seq * s.channels + ch + v] = carry[v];
    }
  }
}

// Every segment's map, forwards (u = x: from its first token to its last) or
// backwards (u = dh).  Each span of threads walks a run of the segment's
// tokens; one join at the end.
template <typename T, typename G, int CL, int WAVES, int V, bool BACK>
__global__ __launch_bounds__(WAVES* kWave) void k_scan_ends(
    ScanShape s, const T* __restrict__ u, int64_t ldu, const G* __restrict__ g, int64_t ldg,
    float* __restrict__ ends) {
  typedef Place<CL, WAVES, V> At;
  constexpr int BT = At::kBlock, kRuns = WAVES * At::kSlices;
  __shared__ float2 agg[WAVES][CL * V];
  for (int64_t id = item_id(s.items); id < s.items; id += gridDim.x) {
    const Item w = item_of<BT>(s, id);
    if (w.seq < 0 || w.seq >= s.nseq || w.segs < 2) continue;
    const At me(w.tile, s.channels);
    const int64_t end = w.b1 * BT < w.len ? w.b1 * BT : w.len;
    const int64_t begin = w.b0 * BT < end ? w.b0 * BT : end;
    const int64_t each = (end - begin + kRuns - 1) / kRuns;
    const int run = me.wave * At::kSlices + me.slice;
    const int64_t lo = begin + run * each < end ? begin + run * each : end;
    const int64_t hi = lo + each < end ? lo + each : end;
    const T* pu = u + w.from * ldu + me.channel();
    const G* pg = g + w.from * ldg + me.channel();
    float P[V], H[V];
#pragma unroll
    for (int v = 0; v < V; ++v) P[v] = 1.f, H[v] = 0.f;
    for (int64_t k = 0; k < each; k += kSpan) {
      Raw<T, V> ru;
      Raw<G, V> rg;
      // backwards the walk begins at the end; tokens outside of the run change nothing
      const int64_t t = BACK ? hi - kSpan - k : lo + k;
#pragma unroll
      for (int j = 0; j < kSpan; ++j) {
        const int64_t q = t + j < 0 ? 0 : t + j < w.len ? t + j : w.len - 1;
        ru.v[j] = *reinterpret_cast<const typename VecOf<T, V>::type*>(pu + q * ldu);
        rg.v[j] = *reinterpret_cast<const typename VecOf<G, V>::type*>(pg + q * ldg);
      }
#pragma unroll
      for (int i = 0; i < kSpan; ++i) {
        const int j = BACK ? kSpan - 1 - i : i;
        const bool live = t + j >= lo && t + j < hi;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const float a = live ? decay(rg.v[j][v]) : 1.f;
          const float y = live ? float(ru.v[j][v]) : 0.f;
          H[v] = BACK ? a * (y + H[v]) : a * H[v] + y;
          P[v] *= a;
        }
      }
    }
    join_slices<CL, V, !BACK>(P, H, me.slice);
    __syncthreads();   // the item before has been read
    if (me.slice == (BACK ? 0 : At::kSlices - 1)) {
#pragma unroll
      for (int v = 0; v < V; ++v) agg[me.wave][me.lane * V + v] = make_float2(P[v], H[v]);
    }
    __syncthreads();
    if (me.on && me.wave == 0 && me.slice == 0) {
      float* e = ends + (w.map * s.channels + me.channel()) * 2;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float p = 1.f, q = 0.f;
#pragma unroll
        for (int i = 0; i < WAVES; ++i) {
          const float2 m = agg[BACK ? WAVES - 1 - i : i][me.lane * V + v];
          q = m.x * q + m.y;
          p *= m.x;
        }
        e[2 * v] = p;
        e[2 * v + 1] = q;
      }
    }
  }
}

// The sequences' first tokens from the caller's offsets: each is the largest
// of its predecessors and itself, clamped (they are on the device and cannot
// be refused here), so that no kernel leaves the arrays.
// With a table the segments of up to `each` blocks of BT tokens follow.
constexpr int kPlanBlock = 1024;
__global__ __launch_bounds__(kPlanBlock) void k_scan_plan(const int32_t* __restrict__ cu,
                                                          int64_t nseq, int64_t total,
                                                          int32_t* __restrict__ tok,
                                                          int64_t block_tokens, int64_t each,
                                                          int4* __restrict__ table,
                                                          int64_t parts) {
  constexpr int kWaves = kPlanBlock / kWave;
  __shared__ int tops[kWaves];
  __shared__ int2 sums[kWaves];
  const int lane = threadIdx.x % kWave, w = threadIdx.x / kWave;
  int carry = 0;          // the largest offset so far
  int64_t used = 0, maps = 0;   // entries so far, maps of cut sequences
  for (int64_t b = 0; b <= nseq; b += kPlanBlock) {
    const int64_t i = b + threadIdx.x;
    int v = i <= nseq ? cu[i] : 0;
    v = v < 0 ? 0 : (v > total ? int(total) : v);
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int u = __shfl_up(v, d, kWave);
      if (lane >= d && u > v) v = u;
    }
    if (lane == kWave - 1) tops[w] = v;
    __syncthreads();
    int before = carry;
    for (int k = 0; k < kWaves; ++k) {
      if (k < w && tops[k] > before) before = tops[k];
      if (tops[k] > carry) carry = tops[k];
    }
    v = v > before ? v : before;
    if (i <= nseq) tok[i] = v;
    if (table) {
      int prev = __shfl_up(v, 1, kWave);
      if (lane == 0) prev = before;
      const int64_t blocks = (int64_t(v) - prev + block_tokens - 1) / block_tokens;
      const int64_t cut = (blocks + each - 1) / each;
      const int mine = i >= 1 && i <= nseq ? int(cut < 1 ? 1 : cut) : 0;   // of sequence i - 1
      int2 at = make_int2(mine, mine > 1 ? mine : 0);
#pragma unroll
      for (int d = 1; d < kWave; d <<= 1) {
        const int p = __shfl_up(at.x, d, kWave), q = __shfl_up(at.y, d, kWave);
        if (lane >= d) at.x += p, at.y += q;
      }
      if (lane == kWave - 1) sums[w] = at;
      __syncthreads();
      int64_t first = used + at.x - mine, map = maps + at.y - mine;
      for (int k = 0; k < kWaves; ++k) {
        if (k < w) first += sums[k].x, map += sums[k].y;
        used += sums[k].x;
        maps += sums[k].y;
      }
      for (int k = 0; k < mine; ++k)
        if (first + k < parts) table[first + k] = make_int4(int(i - 1), k, int(map + k), 0);
    }
    __syncthreads();
  }
  if (table)
    for (int64_t k = used + threadIdx.x; k < parts; k += kPlanBlock) table[k] = make_int4(-1, 0, 0, 0);
}

// One token of every sequence; a thread has V channels of a row.
template <typename T, typename G, int V>
__global__ __launch_bounds__(256) void k_scan_step(const T* __restrict__ x, int64_t ldx,
                                                   const G* __restrict__ g, int64_t ldg,
                                                   int64_t rows, int64_t channels,
                                                   float* __restrict__ state, T* __restrict__ h) {
  const int64_t per = (channels + V - 1) / V, all = rows * per;
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < all;
       i += int64_t(gridDim.x) * 256) {
    const int64_t r = all < (int64_t(1) << 32) ? int64_t(uint32_t(i) / uint32_t(per)) : i / per;
    const int64_t c = (i - r * per) * V, have = channels - c;
    float xv[V], sv[V];
    load_f32<V>(x + r * ldx + c, have, xv);
    G gate[V];
#pragma unroll
    for (int v = 0; v < V; ++v) gate[v] = G(0.f);
    if (have >= V) {
      const auto q = *reinterpret_cast<const typename VecOf<G, V>::type*>(g + r * ldg + c);
#pragma unroll
      for (int v = 0; v < V; ++v) gate[v] = q[v];
    } else {
      for (int v = 0; v < have; ++v) gate[v] = g[r * ldg + c + v];
    }
    load_f32<V>(state + r * channels + c, have, sv);
#pragma unroll
    for (int v = 0; v < V; ++v) sv[v] = decay(gate[v]) * sv[v] + xv[v];
    store_f32<V>(state + r * channels + c, have, sv);
    store_f32<V>(h + r * channels + c, have, sv);
  }
}

// ---------------------------------------------------------------------------
// Host side
// ---------------------------------------------------------------------------

// Lanes along the channels and waves of a workgroup, and the segments of a
// sequence.  The sizes alone decide (what the forward pass keeps is laid out by
// them).
//
// Fewer lanes give more workgroups, down to rows of 64 bytes: 4 x 4096 x 2048 bf16
// in 256 workgroups of 64 bytes take 43 + 85 us, in 128 of 128 bytes and two segments
// 36 + 80 and 28 + 30 for the maps.  Groups of four waves overlap better where there
// are two or more on a CU (12345 x 999 fp32: 39 + 66 us against 47 + 84 with eight);
// one a CU has to be of eight (42 + 83 against 48 + 92).  More than 64 segments pay
// for their maps' loads (131072 x 256: 57 us instead of 53).  Spans of 16 tokens
// gain nothing, groups of 16 waves spill.
struct ScanPlan {
  int cl, waves, v, segments;
  int64_t tiles, blocks, block_tokens;   // blocks: of all sequences (packed: at most)
  int64_t each, parts, maps;   // packed, with a table: blocks of a segment, segments and
                               // segments of cut sequences at most
};
// Blocks of all packed sequences up to which the long ones are not cut, where there
// are kFill / 2 workgroups or more.  A workgroup walks a block in 1.5 us forward and 4
// in a training step, so 1024 blocks in one sequence are 1.5 and 4 ms.  16 in place of
// 1024 costs every other packed call the launch for the maps and gains little, since
// segments of less than 256 blocks are not made: 64 sequences of 2048 x 64 fp32 25.4 ->
// 28.8 us forward and 55 -> 61 training, 64 of 500 x 512 bf16 25.4 -> 29.0 and 57 -> 62;
// 64 of which one has 120000 tokens, x 64 fp32, 704 -> 750 and 1832 -> 1724.
constexpr int64_t kUncutBlocks = 1024;
ScanPlan scan_plan(const sla_scan_dims* d) {
  ScanPlan p{};
  p.v = d->type != SLA_F32 && d->channels % 2 == 0 ? 2 : 1;
  const int64_t lanes = d->channels / p.v, n = d->sequences ? d->sequences : 1;
  const int64_t mean = div_up(d->tokens, n);
  p.cl = 64;
  while (p.cl > 16 && (lanes <= p.cl / 2 || n * div_up(lanes, p.cl) < kFill)) p.cl /= 2;
  p.tiles = div_up(lanes, p.cl);
  const int64_t groups = n * p.tiles;
  const bool one_each = groups >= kFill / 2 && groups < kFill;   // a workgroup a CU: 8 waves
  p.waves = mean <= 4 * kSpan * (kWave / p.cl) ? 1 : one_each ? 8 : 4;
  p.block_tokens = int64_t(p.waves) * (kWave / p.cl) * kSpan;
  const int64_t blocks = div_up(mean, p.block_tokens);
  int64_t s = groups >= kFill / 2 ? 1 : div_up(kFill, groups);
  s = s < blocks / 2 ? s : blocks / 2;
  p.segments = int(s < 1 ? 1 : s < kMostSegments ? s : kMostSegments);
  p.blocks = d->packed ? d->tokens / p.block_tokens + n : n * blocks;
  if (d->packed) {
    p.segments = 1;
    const bool few = groups < kFill / 2;
    int64_t each = few ? div_up(p.blocks * p.tiles, kFill) : 4 * blocks;
    if (!few && each < 256) each = 256;
    each = (each < 2 ? 2 : each) | 1;
    if (p.blocks > (few ? 4 : kUncutBlocks) && each < p.blocks) {
      p.each = each;
      p.parts = n + p.blocks / each + 1;
      p.maps = 2 * (p.blocks / each + 1);   // a cut sequence is longer than `each`
    }
  }
  return p;
}

// Whether a thread's place in a wave's tokens fits 31 bits.
bool scan_stride(const ScanPlan& p, int64_t ld) {
  return p.cl == kWave || ld < (int64_t(1) << 24);
}

int64_t up256(int64_t n) { return div_up(n, 256) * 256; }

struct ScanSizes {
  ScanPlan plan;
  int64_t tok, kept, work;   // bytes: the offsets and the table, all that is kept, the workspace
  int64_t table;             // where the table begins
};
sla_status scan_sizes(const char* who, const sla_scan_dims* d, ScanSizes& z) {
  SLA_NET_REQUIRE(d, "%s: dims is NULL", who);
  SLA_NET_REQUIRE(valid_type(d->type) && (d->gate_type == d->type || d->gate_type == SLA_F32),
                  "%s: unknown or mixed types", who);
  SLA_NET_REQUIRE(d->sequences >= 0 && d->sequences < (int64_t(1) << 31) && d->tokens >= 0 &&
                      d->tokens < (int64_t(1) << 40), "%s: sequences or tokens out of range", who);
  SLA_NET_REQUIRE(d->channels >= 1 && d->channels < (int64_t(1) << 31),
                  "%s: channels out of range", who);
  if (d->packed) {
    SLA_NET_REQUIRE(d->tokens < (int64_t(1) << 31), "%s: too many tokens for 32-bit offsets", who);
    SLA_NET_REQUIRE(d->sequences > 0 || d->tokens == 0, "%s: tokens without a sequence", who);
  } else {
    SLA_NET_REQUIRE(d->sequences ? d->tokens % d->sequences == 0 : d->tokens == 0,
                    "%s: %lld tokens are not %lld equal sequences", who, (long long)d->tokens,
                    (long long)d->sequences);
  }
  z.plan = scan_plan(d);
  // no product of sizes below passes 63 bits: nothing larger fits a card
  const double all = double(z.plan.blocks + d->tokens + d->sequences * kMostSegments) *
                     double(d->channels);
  SLA_NET_REQUIRE(all < 1e15, "%s: too large", who);
  z.table = d->packed ? up256((d->sequences + 1) * 4) : 0;
  z.tok = z.table + up256(z.plan.parts * 16);
  z.kept = z.tok + up256(z.plan.blocks * d->channels * 4);
  const int64_t maps = z.plan.segments > 1 ? d->sequences * z.plan.segments : z.plan.maps;
  z.work = z.tok + up256(maps * d->channels * 8);
  return SLA_OK;
}

template <typename F>
sla_status with_scan(const sla_scan_dims* d, const ScanPlan& p, F&& f) {
  auto shape = [&](auto te, auto ge, auto v) -> sla_status {
    using std::integral_constant;
    auto waves = [&](auto cl) -> sla_status {
      if (p.waves == 1) return f(te, ge, cl, integral_constant<int, 1>(), v);
      // (eight waves: less than kFill workgroups, so the fewest lanes)
      if constexpr (cl.value == 16)
        if (p.waves == 8) return f(te, ge, cl, integral_constant<int, 8>(), v);
      return f(te, ge, cl, integral_constant<int, 4>(), v);
    };
    if (p.cl == 64) return waves(integral_constant<int, 64>());
    if (p.cl == 32) return waves(integral_constant<int, 32>());
    return waves(integral_constant<int, 16>());
  };
  auto width = [&](auto te, auto ge) -> sla_status {
    if constexpr (sizeof(te) == 2)
      if (p.v == 2) return shape(te, ge, std::integral_constant<int, 2>());
    return shape(te, ge, std::integral_constant<int, 1>());
  };
  const bool wide = d->gate_type == SLA_F32;
  if (d->type == SLA_F32) return width(float(), float());
  if (d->type == SLA_F16) return wide ? width(_Float16(), float()) : width(_Float16(), _Float16());
  return wide ? width(__bf16(), float()) : width(__bf16(), __bf16());
}

ScanShape scan_shape(const sla_scan_dims* d, const ScanSizes& z, const int32_t* tok) {
  const ScanPlan& p = z.plan;
  ScanShape s{};
  s.nseq = d->sequences;
  s.seqlen = d->sequences && !d->packed ? d->tokens / d->sequences : 0;
  s.total = d->tokens;
  s.channels = d->channels;
  s.tok = tok;
  s.tiles = int(p.tiles);
  s.segments = p.segments;
  if (p.parts) {
    s.table = (const int4*)((const char*)tok + z.table);
    s.parts = p.parts;
    s.each = p.each;
  }
  s.items = ((p.parts ? p.parts : s.nseq * p.segments) + (tok ? kGapItems : 0)) * p.tiles;
  return s;
}
int scan_grid(const ScanShape& s) { return int(s.items < kMostGroups ? s.items : kMostGroups); }

}  // namespace
}  // namespace net
}  // namespace sla

using namespace sla;
using namespace sla::net;

extern "C" {

sla_status sla_gated_scan_work(const sla_scan_dims* dims, int64_t* kept_bytes_host,
                               int64_t* work_bytes_host) {
  SLA_NET_BEGIN
  clear_error();
  ScanSizes z;
  SLA_TRY(scan_sizes("sla_gated_scan_work", dims, z));
  if (kept_bytes_host) *kept_bytes_host = z.kept;
  if (work_bytes_host) *work_bytes_host = z.work;
  return SLA_OK;
  SLA_NET_END
}

sla_status sla_gated_scan(const sla_scan_dims* dims, const void* x, int64_t ldx, const void* g,
                          int64_t ldg, const int32_t* offsets, const float* initial_state,
                          void* h, float* final_state, void* kept, int64_t kept_bytes, void* work,
                          int64_t work_bytes, hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  ScanSizes z;
  SLA_TRY(scan_sizes("sla_gated_scan", dims, z));
  if (dims->sequences == 0) return SLA_OK;
  SLA_NET_REQUIRE(dims->tokens == 0 || (x && g && h), "sla_gated_scan: an argument is NULL");
  SLA_NET_REQUIRE(!dims->packed || offsets, "sla_gated_scan: offsets is NULL");
  SLA_NET_REQUIRE(ldx >= dims->channels && ldg >= dims->channels,
                  "sla_gated_scan: a token stride is below channels");
  SLA_NET_REQUIRE(scan_stride(z.plan, ldx) && scan_stride(z.plan, ldg),
                  "sla_gated_scan: a token stride of 2^24 or more");
  SLA_NET_REQUIRE(!kept || kept_bytes >= z.kept,
                  "sla_gated_scan: kept block too small (sla_gated_scan_work)");
  SLA_NET_REQUIRE(z.work == 0 || (work && work_bytes >= z.work),
                  "sla_gated_scan: workspace too small (sla_gated_scan_work)");
  int32_t* tok = dims->packed ? (int32_t*)(kept ? kept : work) : nullptr;
  float* states = kept ? (float*)((char*)kept + z.tok) : nullptr;
  float* ends = (float*)((char*)work + z.tok);
  if (tok) {
    k_scan_plan<<<1, kPlanBlock, 0, stream>>>(
        offsets, dims->sequences, dims->tokens, tok, z.plan.block_tokens, z.plan.each,
        z.plan.parts ? (int4*)((char*)tok + z.table) : nullptr, z.plan.parts);
    LAUNCH_CHECK();
  }
  const ScanShape s = scan_shape(dims, z, tok);
  return with_scan(dims, z.plan, [&](auto te, auto ge, auto cl, auto waves, auto v) -> sla_status {
    using T = decltype(te);
    using G = decltype(ge);
    const int grid = scan_grid(s);
    if (s.segments > 1 || s.table) {
      k_scan_ends<T, G, cl.value, waves.value, v.value, false>
          <<<grid, waves.value * kWave, 0, stream>>>(s, (const T*)x, ldx, (const G*)g, ldg, ends);
      LAUNCH_CHECK();
    }
    k_scan<T, G, cl.value, waves.value, v.value><<<grid, waves.value * kWave, 0, stream>>>(
        s, (const T*)x, ldx, (const G*)g, ldg, initial_state, (T*)h, final_state, states, ends);
    LAUNCH_CHECK();
    return SLA_OK;
  });
  SLA_NET_END
}

sla_status sla_gated_scan_grad(const sla_scan_dims* dims, const void* x, int64_t ldx,
                               const void* g, int64_t ldg, const void* kept, int64_t kept_bytes,
                               const void* dh, int64_t lddh, const float* grad_final_state,
                               void* dx, void* dg, float* grad_initial_state, void* work,
                               int64_t work_bytes, hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  ScanSizes z;
  SLA_TRY(scan_sizes("sla_gated_scan_grad", dims, z));
  if (dims->sequences == 0) return SLA_OK;
  SLA_NET_REQUIRE(dims->tokens == 0 || (x && g && dh), "sla_gated_scan_grad: an argument is NULL");
  SLA_NET_REQUIRE(ldx >= dims->channels && ldg >= dims->channels && lddh >= dims->channels,
                  "sla_gated_scan_grad: a token stride is below channels");
  SLA_NET_REQUIRE(scan_stride(z.plan, ldx) && scan_stride(z.plan, ldg) &&
                      scan_stride(z.plan, lddh),
                  "sla_gated_scan_grad: a token stride of 2^24 or more");
  SLA_NET_REQUIRE(z.kept == 0 || (kept && kept_bytes >= z.kept),
                  "sla_gated_scan_grad: kept block too small (sla_gated_scan_work)");
  SLA_NET_REQUIRE(z.work == 0 || (work && work_bytes >= z.work),
                  "sla_gated_scan_grad: workspace too small (sla_gated_scan_work)");
  const int32_t* tok = dims->packed ? (const int32_t*)kept : nullptr;
  const float* states = (const float*)((const char*)kept + z.tok);
  float* ends = (float*)((char*)work + z.tok);
  const ScanShape s = scan_shape(dims, z, tok);
  return with_scan(dims, z.plan, [&](auto te, auto ge, auto cl, auto waves, auto v) -> sla_status {
    using T = decltype(te);
    using G = decltype(ge);
    const int grid = scan_grid(s);
    if (s.segments > 1 || s.table) {
      k_scan_ends<T, G, cl.value, waves.value, v.value, true>
          <<<grid, waves.value * kWave, 0, stream>>>(s, (const T*)dh, lddh, (const G*)g, ldg,
                                                     ends);
      LAUNCH_CHECK();
    }
    k_scan_grad<T, G, cl.value, waves.value, v.value><<<grid, waves.value * kWave, 0, stream>>>(
        s, (const T*)x, ldx, (const G*)g, ldg, states, (const T*)dh, lddh, grad_final_state,
        (T*)dx, (G*)dg, grad_initial_state, ends);
    LAUNCH_CHECK();
    return SLA_OK;
  });
  SLA_NET_END
}

sla_status sla_gated_scan_step(const sla_scan_dims* dims, const void* x, int64_t ldx,
                               const void* g, int64_t ldg, float* state, void* h,
                               hipStream_t stream) {
  SLA_NET_BEGIN
  clear_error();
  ScanSizes z;
  SLA_TRY(scan_sizes("sla_gated_scan_step", dims, z));
  SLA_NET_REQUIRE(!dims->packed && dims->tokens == dims->sequences,
                  "sla_gated_scan_step: one token of every sequence");
  if (dims->sequences == 0) return SLA_OK;
  SLA_NET_REQUIRE(x && g && state && h, "sla_gated_scan_step: an argument is NULL");
  SLA_NET_REQUIRE(ldx >= dims->channels && ldg >= dims->channels,
                  "sla_gated_scan_step: a token stride is below channels");
  const bool wide = dims->gate_type == SLA_F32;
  auto run = [&](auto te, auto ge) -> sla_status {
    using T = decltype(te);
    using G = decltype(ge);
    constexpr int V = 4;
    const int64_t groups = div_up(dims->sequences * div_up(dims->channels, V), 256);
    k_scan_step<T, G, V><<<int(groups < kMostGroups ? groups : kMostGroups), 256, 0, stream>>>(
        (const T*)x, ldx, (const G*)g, ldg, dims->sequences, dims->channels, state, (T*)h);
    LAUNCH_CHECK();
    return SLA_OK;
  };
  if (dims->type == SLA_F32) return run(float(), float());
  if (dims->type == SLA_F16) return wide ? run(_Float16(), float()) : run(_Float16(), _Float16());
  return wide ? run(__bf16(), float()) : run(__bf16(), __bf16());
  SLA_NET_END
}

}  // extern "C"
