// scan_kernels.hip -- the gated linear recurrence h_t = f_t h'_{t-1} +
// (1 - f_t) x_t with f = sigmoid(g), forward, backward and one step.
//
// A workgroup takes 64 C channels of one sequence (C per lane) and walks the
// time axis in tiles of a few steps per wave: each wave loads its steps,
// reduces them to one affine map h -> A h + B, the maps meet in LDS, every
// wave folds those before it into the state it starts from, and then runs its
// steps.  So the inputs are read once, with as many loads in flight as a wave
// has steps, and the time axis still has kWaves-fold parallelism inside a
// workgroup.  Where batch and channels alone do not fill the chip the time
// axis is cut into segments: a first kernel reduces each segment to its map,
// and each workgroup of the second folds the maps of the segments before it.
//
// 128 x 512 x 1024 bf16: forward 80 us (5.0 TB/s), backward 158 us (4.3 TB/s),
// bound by HBM with the vector units half busy.  2 x 16384 x 512, cut into 64
// segments: 16 + 21 us forward, 16 + 31 backward, the maps' reading of two tensors
// being what the cut costs.  Handing maps and states from tile to tile within one
// launch instead (tickets and polled words) reads everything once, but 512
// workgroups then load, wait and store in step: 44 and 69 us.
//
// A reset makes its map ignore the state, so an infinite or NaN state before it
// does not leak through 0 * Inf: such a map has A = -0, which no product of gates
// is, and which stays -0 under further gates.
//
// Rows of few channels are packed: the lanes of a wave then take neighbouring
// channels across sequences, and lengths and resets are each lane's own.

#include <type_traits>

#include "elem.h"
#include "train_internal.h"

namespace per {
namespace {

// Steps of a wave in one tile.  The backward pass keeps four values of a step
// (f, 1 - f, the packed inputs, the gate's weight), so that 16 steps of two
// channels would not leave two workgroups' registers to a CU.
constexpr int kForward = 16;
constexpr int kBackward = 8;
constexpr int kWaves = 8;                  // waves of a workgroup
constexpr int kMaxWaves = 16;              // where there is at most one to a CU
constexpr int kChunk = 64;                 // PER_SCAN_CHUNK
constexpr int kSegment = 128;              // segments are multiples of it
constexpr int kMaxSeg = 256;
constexpr float kLog2e = 1.44269504088896340736f;

// f = sigmoid(g) = 1 / (1 + e) and 1 - f = e / (1 + e), each within (1.5 |g| + 8)
// 2^-24 of itself: the exponent -log2(e) g is rounded once, and the exponential and
// the reciprocal are the hardware's, off by a step where correctly rounded ones would
// take several instructions more.  1 - f is not taken by subtraction, which would lose
// its digits next to f = 1.  e = exp(-g) is kept finite so that it does not become
// Inf * 0.
__device__ __forceinline__ void gate(float g, float& f, float& i) {
  const float e = __builtin_amdgcn_exp2f(__builtin_elementwise_minimum(-kLog2e * g, 126.0f));
  f = __builtin_amdgcn_rcpf(1.0f + e);
  i = e * f;
}

// Position of a lane: sequence, segment, first channel.
struct Place {
  int64_t b, d;
  int seg;
  bool in;                 // the lane has channels
  int64_t t_begin, t_end;  // steps of the segment
  int64_t live;            // steps before min(t_end, length)
};

template <int C, bool PACK>
__device__ __forceinline__ Place place(const ScanArgs& a) {
  static_assert(!PACK || C == 1, "packed lanes have one channel");
  const int lane = threadIdx.x & 63;
  const uint32_t id = blockIdx.x;
  Place p;
  if (PACK) {
    const uint64_t all = (uint64_t)a.B * (uint64_t)a.D;
    const uint32_t tiles = (uint32_t)((all + 63) / 64);
    p.seg = (int)(id / tiles);
    const uint64_t e = (uint64_t)(id % tiles) * 64 + lane;
    p.in = e < all;
    p.b = p.in ? (int64_t)(e / (uint64_t)a.D) : 0;
    p.d = p.in ? (int64_t)(e - (uint64_t)p.b * (uint64_t)a.D) : 0;
  } else {
    const uint32_t nct = (uint32_t)((a.D + 64 * C - 1) / (64 * C));
    const uint32_t r = id / nct;
    p.d = (int64_t)(id % nct) * (64 * C) + lane * C;
    p.in = p.d < a.D;
    // Where D is odd the last lane takes the channel before its own as well: it
    // loads, computes and stores the very values the lane before it does, in step
    // with it (plan() leaves out the D whose last lane has none before it).
    if (C > 1 && p.in && p.d > a.D - C) p.d = a.D - C;
    p.seg = (int)(r % (uint32_t)a.nseg);
    p.b = r / (uint32_t)a.nseg;
  }
  int64_t len = a.T;
  if (a.length) {
    len = a.length[p.b];
    len = len < 0 ? 0 : len > a.T ? a.T : len;
  }
  if (PACK && !p.in) len = 0;
  p.t_begin = (int64_t)p.seg * a.seg_steps;
  p.t_end = p.t_begin + a.seg_steps < a.T ? p.t_begin + a.seg_steps : a.T;
  p.live = len < p.t_end ? len : p.t_end;
  return p;
}

// Steps of [ts, ts + S) before `live`.
template <int S>
__device__ __forceinline__ int steps_at(int64_t ts, int64_t live) {
  const int64_t n = live - ts;
  return n < 0 ? 0 : n > S ? S : (int)n;
}

// Where episodes begin among the S steps from ts: bytes loaded a tile ahead (for
// the first tile beside the sequence's length), then bit s for step ts + s < ts +
// n.  One byte per lane where the lanes share a sequence, S where each has its own.
template <int S, bool PACK>
struct Begins {
  uint32_t w[PACK ? S / 4 : 1];
  __device__ __forceinline__ void load(const uint8_t* reset, int64_t ts, int64_t T) {
#pragma unroll
    for (int k = 0; k < (PACK ? S / 4 : 1); ++k) w[k] = 0;
    if (!reset || ts < 0) return;
    if constexpr (!PACK) {
      const int lane = threadIdx.x & 63;
      if (lane < S && ts + lane < T) w[0] = reset[ts + lane];
    } else if (ts + S <= T) {
      __builtin_memcpy(w, reset + ts, S);
    } else {
#pragma unroll
      for (int s = 0; s < S; ++s)
        if (ts + s < T) w[s / 4] |= (uint32_t)reset[ts + s] << (8 * (s & 3));
    }
  }
  __device__ __forceinline__ uint32_t mask(int n) const {
    uint32_t m = 0;
    if constexpr (!PACK) {
      m = (uint32_t)__ballot(w[0] != 0);
    } else {
#pragma unroll
      for (int k = 0; k < S / 4; ++k) {  // the top bit of each byte that is not 0, gathered
        const uint32_t t = (((w[k] & 0x7F7F7F7Fu) + 0x7F7F7F7Fu) | w[k]) & 0x80808080u;
        m |= (((t >> 7) * 0x10204080u) >> 28) << (4 * k);
      }
    }
    return m & ((1u << n) - 1);
  }
};

// Whether every lane has a whole tile without an episode's begin: nearly all of
// a long sequence, and it goes without the per-step conditions.
template <int S, bool PACK>
__device__ __forceinline__ bool whole(int n, uint32_t mask) {
  const bool w = n == S && mask == 0;
  return PACK ? __all(w) : w;
}

__device__ __forceinline__ bool ignores(float A) { return __float_as_uint(A) == 0x80000000u; }
// A product of gates that has come out as 0 stands for one that is not: an infinite
// state stays infinite through it (0 would make it NaN), a finite one vanishes.
__device__ __forceinline__ float gates(float A) {
  return __float_as_uint(A) == 0 ? 0x1p-149f : A;
}
// The map (A, B) on a state.
__device__ __forceinline__ float apply(float A, float B, float h) {
  return ignores(A) ? B : __builtin_fmaf(A, h, B);
}

// A [T x D] matrix of one sequence.  Where the lanes share the sequence a row's
// address is the same in all of them, the lane's channel an offset from it.
template <typename T>
struct Rows {
  T* p;
  int64_t st;
  uint32_t d;
  __device__ __forceinline__ T* at(int64_t t) const { return p + t * st + d; }
};

// S rows of C channels from row ts.  Without FULL only the first n are
// live: the others are loaded from the last of them (row 0 if there is none) and
// not used.
template <typename T, int C, bool FULL, int S>
__device__ __forceinline__ void load_steps(const Rows<const T>& r, int64_t ts, int n,
                                           Pack<T, C> (&v)[S]) {
#pragma unroll
  for (int s = 0; s < S; ++s)
    v[s] = load_pack<T, C>(r.at(FULL ? ts + s : n > 0 ? ts + (s < n ? s : n - 1) : 0));
}

template <typename T, int C, bool PACK>
__global__ __launch_bounds__(kMaxWaves * 64, 4) void scan_forward_kernel(ScanArgs a) {
  constexpr int S = kForward;
  __shared__ float sA[2][kMaxWaves][C][64], sB[2][kMaxWaves][C][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6;
  const Place p = place<C, PACK>(a);
  const bool in = p.in;
  const uint8_t* reset = a.reset ? a.reset + p.b * a.T : nullptr;
  Begins<S, PACK> begins;
  begins.load(reset, p.t_begin + wv * S, a.T);
  const uint32_t d32 = (uint32_t)p.d;
  const Rows<const T> x = {static_cast<const T*>(a.x) + p.b * a.x_sb, a.x_st, d32};
  const Rows<const T> g = {static_cast<const T*>(a.g) + p.b * a.g_sb, a.g_st, d32};
  const Rows<T> y = {static_cast<T*>(a.y) + p.b * a.y_sb, a.y_st, d32};
  float h[C];
#pragma unroll
  for (int c = 0; c < C; ++c) h[c] = a.h0 && in ? a.h0[p.b * a.D + p.d + c] : 0.0f;

  if (p.seg > 0) {  // fold the segments before this one: a run per wave, then the waves
    const int run = (p.seg + nw - 1) / nw;
    float A[C], B[C];
#pragma unroll
    for (int c = 0; c < C; ++c) A[c] = 1.0f, B[c] = 0.0f;
    for (int s = wv * run; s < (wv + 1) * run && s < p.seg; ++s) {
      const float* m = a.agg + (p.b * a.nseg + s) * 2 * a.D + p.d;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float sa = in ? m[c] : 0.0f, sb = in ? m[a.D + c] : 0.0f;
        B[c] = apply(sa, sb, B[c]);
        A[c] = ignores(sa) ? sa : gates(A[c] * sa);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) sA[1][wv][c][lane] = A[c], sB[1][wv][c][lane] = B[c];
    __syncthreads();
    for (int w = 0; w < nw; ++w) {
#pragma unroll
      for (int c = 0; c < C; ++c) h[c] = apply(sA[1][w][c][lane], sB[1][w][c][lane], h[c]);
    }
  }

  int buf = 0;
  for (int64_t t0 = p.t_begin; t0 < p.t_end; t0 += nw * S, buf ^= 1) {
    const int64_t ts = t0 + wv * S;
    const int n = steps_at<S>(ts, p.live);
    const uint32_t mask = begins.mask(n);
    begins.load(reset, ts + nw * S, a.T);
    float f[S][C], ix[S][C];
    float A[C], B[C];
#pragma unroll
    for (int c = 0; c < C; ++c) A[c] = 1.0f, B[c] = 0.0f;
    const bool full = whole<S, PACK>(n, mask);
    auto reduce = [&](auto is_full) {
      constexpr bool FULL = decltype(is_full)::value;
      Pack<T, C> px[S], pg[S];
      load_steps<T, C, FULL, S>(x, ts, n, px);
      load_steps<T, C, FULL, S>(g, ts, n, pg);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float xv[C], gv[C];
        unpack(px[s], xv);
        unpack(pg[s], gv);
        const bool r = !FULL && ((mask >> s) & 1u);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float i;
          gate(gv[c], f[s][c], i);
          ix[s][c] = i * xv[c];
          if (FULL || s < n) {
            B[c] = r ? ix[s][c] : __builtin_fmaf(f[s][c], B[c], ix[s][c]);
            A[c] = r ? -0.0f : A[c] * f[s][c];
          }
        }
      }
    };
    if ((PACK || in) && full) reduce(std::true_type{});
    else if (PACK ? __any(n > 0) : in && n > 0) reduce(std::false_type{});
#pragma unroll
    for (int c = 0; c < C; ++c) sA[buf][wv][c][lane] = gates(A[c]), sB[buf][wv][c][lane] = B[c];
    __syncthreads();
    float hs[C];
#pragma unroll
    for (int c = 0; c < C; ++c) hs[c] = h[c];
    for (int w = 0; w < nw; ++w) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (w == wv) hs[c] = h[c];
        h[c] = apply(sA[buf][w][c][lane], sB[buf][w][c][lane], h[c]);
      }
    }
    if (a.carries && in && ts % kChunk == 0 && ts < p.t_end) {
      float* c0 = a.carries + (p.b * ((a.T + kChunk - 1) / kChunk) + ts / kChunk) * a.D + p.d;
#pragma unroll
      for (int c = 0; c < C; ++c) c0[c] = hs[c];
    }
    if (in && full) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int c = 0; c < C; ++c) hs[c] = __builtin_fmaf(f[s][c], hs[c], ix[s][c]);
        store_vals<T, C>(y.at(ts + s), hs);
      }
    } else if (in) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (s < n) {
          const bool r = (mask >> s) & 1u;
#pragma unroll
          for (int c = 0; c < C; ++c)
            hs[c] = r ? ix[s][c] : __builtin_fmaf(f[s][c], hs[c], ix[s][c]);
          store_vals<T, C>(y.at(ts + s), hs);
        } else if (ts + s < p.t_end) {
          const float zero[C] = {};
          store_vals<T, C>(y.at(ts + s), zero);
        }
      }
    }
  }
  if (a.h_last && p.t_end == a.T && p.seg == a.nseg - 1 && wv == 0 && in) {
#pragma unroll
    for (int c = 0; c < C; ++c) a.h_last[p.b * a.D + p.d + c] = h[c];
  }
}

// The map of one segment: forward h -> A h + B, or (REV) of the gradient that
// flows back through it, E -> A E + B.  Waves take runs of whole tiles.
template <typename T, int C, bool PACK, bool REV>
__global__ __launch_bounds__(kWaves * 64, 4) void scan_segment_kernel(ScanArgs a) {
  constexpr int S = PACK ? kForward / 2 : kForward;  // packed lanes hold an address each
  __shared__ float sA[kWaves][C][64], sB[kWaves][C][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const Place p = place<C, PACK>(a);
  const bool in = p.in;
  const uint32_t d32 = (uint32_t)p.d;
  const Rows<const T> v =
      REV ? Rows<const T>{static_cast<const T*>(a.dy) + p.b * a.dy_sb, a.dy_st, d32}
          : Rows<const T>{static_cast<const T*>(a.x) + p.b * a.x_sb, a.x_st, d32};
  const Rows<const T> g = {static_cast<const T*>(a.g) + p.b * a.g_sb, a.g_st, d32};
  const uint8_t* reset = a.reset ? a.reset + p.b * a.T : nullptr;
  const int64_t run = a.seg_steps / kWaves;  // a multiple of S
  float A[C], B[C];
#pragma unroll
  for (int c = 0; c < C; ++c) A[c] = 1.0f, B[c] = 0.0f;
  for (int64_t k = 0; k < run; k += S) {
    const int64_t ts = p.t_begin + wv * run + (REV ? run - S - k : k);
    const int n = steps_at<S>(ts, p.live);
    if (PACK ? !__any(n > 0) : n == 0) continue;
    Begins<S, PACK> begins;
    begins.load(reset, ts, a.T);
    const uint32_t mask = begins.mask(n);
    if (!PACK && !in) continue;
    auto reduce = [&](auto is_full) {
      constexpr bool FULL = decltype(is_full)::value;
      Pack<T, C> pv[S], pg[S];
      load_steps<T, C, FULL, S>(v, ts, n, pv);
      load_steps<T, C, FULL, S>(g, ts, n, pg);
#pragma unroll
      for (int q = 0; q < S; ++q) {
        const int s = REV ? S - 1 - q : q;
        if (!FULL && s >= n) continue;
        const bool r = !FULL && ((mask >> s) & 1u);
        float vv[C], gf[C];
        unpack(pv[s], vv);
        unpack(pg[s], gf);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          float f, i;
          gate(gf[c], f, i);
          if (REV) {
            B[c] = r ? 0.0f : f * (B[c] + vv[c]);
          } else {
            const float b = i * vv[c];
            B[c] = r ? b : __builtin_fmaf(f, B[c], b);
          }
          A[c] = r ? -0.0f : A[c] * f;
        }
      }
    };
    if (whole<S, PACK>(n, mask)) reduce(std::true_type{});
    else reduce(std::false_type{});
  }
#pragma unroll
  for (int c = 0; c < C; ++c) sA[wv][c][lane] = gates(A[c]), sB[wv][c][lane] = B[c];
  __syncthreads();
  if (wv != 0) return;
#pragma unroll
  for (int c = 0; c < C; ++c) A[c] = 1.0f, B[c] = 0.0f;
#pragma unroll
  for (int q = 0; q < kWaves; ++q) {
    const int w = REV ? kWaves - 1 - q : q;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const float wa = sA[w][c][lane];
      B[c] = apply(wa, sB[w][c][lane], B[c]);
      A[c] = ignores(wa) ? wa : gates(A[c] * wa);
    }
  }
  if (in) {
    float* m = a.agg + (p.b * a.nseg + p.seg) * 2 * a.D + p.d;
#pragma unroll
    for (int c = 0; c < C; ++c) m[c] = A[c], m[a.D + c] = B[c];
  }
  if (!REV && a.h0 && p.seg == 0 && in) {
#pragma unroll
    for (int c = 0; c < C; ++c) a.h0_copy[p.b * a.D + p.d + c] = a.h0[p.b * a.D + p.d + c];
  }
}

// E_t = f_t (E_{t+1} + dy_t) is the gradient that reaches the state before
// step t (0 where an episode begins at t); full_t = E_{t+1} + dy_t that of h_t:
//   dx = full (1 - f),  dg = full (h' - x) f (1 - f).
// The states of a chunk are computed again from its carry.
template <typename T, int C, bool PACK>
__global__ __launch_bounds__(64 * kMaxWaves, 4) void scan_backward_kernel(ScanArgs a) {
  constexpr int S = kBackward;
  __shared__ float sA[2][kMaxWaves][C][64], sB[2][kMaxWaves][C][64], sQ[2][kMaxWaves][C][64];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nw = blockDim.x >> 6;
  const Place p = place<C, PACK>(a);
  const bool in = p.in;
  const uint32_t d32 = (uint32_t)p.d;
  const Rows<const T> x = {static_cast<const T*>(a.x) + p.b * a.x_sb, a.x_st, d32};
  const Rows<const T> g = {static_cast<const T*>(a.g) + p.b * a.g_sb, a.g_st, d32};
  const Rows<const T> dy = {static_cast<const T*>(a.dy) + p.b * a.dy_sb, a.dy_st, d32};
  const Rows<T> dx = {static_cast<T*>(a.dx) + p.b * a.dx_sb, a.dx_st, d32};
  const Rows<T> dg = {static_cast<T*>(a.dg) + p.b * a.dg_sb, a.dg_st, d32};
  const uint8_t* reset = a.reset ? a.reset + p.b * a.T : nullptr;
  float E[C];
#pragma unroll
  for (int c = 0; c < C; ++c) E[c] = a.dh_last && in ? a.dh_last[p.b * a.D + p.d + c] : 0.0f;

  if (p.seg < a.nseg - 1) {  // fold the segments after this one
    const int later = a.nseg - 1 - p.seg;
    const int run = (later + nw - 1) / nw;
    float A[C], B[C];
#pragma unroll
    for (int c = 0; c < C; ++c) A[c] = 1.0f, B[c] = 0.0f;
    // wave nw - 1 takes the last segments, each run from its end
    int hi = p.seg + 1 + (wv + 1) * run;
    if (hi > a.nseg) hi = a.nseg;
    for (int s = hi - 1; s >= p.seg + 1 + wv * run; --s) {
      const float* m = a.agg + (p.b * a.nseg + s) * 2 * a.D + p.d;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const float sa = in ? m[c] : 0.0f, sb = in ? m[a.D + c] : 0.0f;
        B[c] = apply(sa, sb, B[c]);
        A[c] = ignores(sa) ? sa : gates(A[c] * sa);
      }
    }
#pragma unroll
    for (int c = 0; c < C; ++c) sA[1][wv][c][lane] = A[c], sB[1][wv][c][lane] = B[c];
    __syncthreads();
    for (int w = nw - 1; w >= 0; --w) {
#pragma unroll
      for (int c = 0; c < C; ++c) E[c] = apply(sA[1][w][c][lane], sB[1][w][c][lane], E[c]);
    }
  }

  const int64_t tile = nw * S;
  const int64_t tiles = p.t_end > p.t_begin ? (p.t_end - p.t_begin + tile - 1) / tile : 0;
  Begins<S, PACK> begins;
  begins.load(reset, p.t_begin + (tiles - 1) * tile + wv * S, a.T);
  float Eo[C];  // what flows out of the wave's own steps, run one by one
#pragma unroll
  for (int c = 0; c < C; ++c) Eo[c] = E[c];
  int buf = 0;
  for (int64_t k = tiles - 1; k >= 0; --k, buf ^= 1) {
    const int64_t t0 = p.t_begin + k * tile;
    const int64_t ts = t0 + wv * S;
    const int n = steps_at<S>(ts, p.live);
    const uint32_t mask = begins.mask(n);
    begins.load(reset, ts - tile, a.T);
    float f[S][C], i[S][C];
    Pack<T, C> px[S], pd[S];
    float h[C], A[C], B[C], Q[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      A[c] = 1.0f;
      B[c] = Q[c] = 0.0f;
      h[c] = in ? a.carries[(p.b * ((a.T + kChunk - 1) / kChunk) + t0 / kChunk) * a.D + p.d + c]
                : 0.0f;
    }
    const bool full = whole<S, PACK>(n, mask);
    auto reduce = [&](auto is_full) {
      constexpr bool FULL = decltype(is_full)::value;
      Pack<T, C> pg[S];
      load_steps<T, C, FULL, S>(g, ts, n, pg);
      load_steps<T, C, FULL, S>(x, ts, n, px);
      load_steps<T, C, FULL, S>(dy, ts, n, pd);
#pragma unroll
      for (int s = 0; s < S; ++s) {
        float gv[C], xv[C];
        unpack(px[s], xv);
        unpack(pg[s], gv);
        const bool r = !FULL && ((mask >> s) & 1u);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          gate(gv[c], f[s][c], i[s][c]);
          if (FULL || s < n) {
            const float b = i[s][c] * xv[c];
            B[c] = r ? b : __builtin_fmaf(f[s][c], B[c], b);
            A[c] = r ? -0.0f : A[c] * f[s][c];
          }
        }
      }
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        if (!FULL && s >= n) continue;
        const bool r = !FULL && ((mask >> s) & 1u);
        float dv[C];
        unpack(pd[s], dv);
#pragma unroll
        for (int c = 0; c < C; ++c) Q[c] = r ? 0.0f : f[s][c] * (Q[c] + dv[c]);
      }
    };
    if ((PACK || in) && full) reduce(std::true_type{});
    else if (PACK ? __any(n > 0) : in && n > 0) reduce(std::false_type{});
#pragma unroll
    for (int c = 0; c < C; ++c) {
      sA[buf][wv][c][lane] = gates(A[c]);
      sB[buf][wv][c][lane] = B[c];
      sQ[buf][wv][c][lane] = Q[c];
    }
    __syncthreads();
    for (int w = 0; w < wv; ++w) {
#pragma unroll
      for (int c = 0; c < C; ++c) h[c] = apply(sA[buf][w][c][lane], sB[buf][w][c][lane], h[c]);
    }
    float Es[C];
#pragma unroll
    for (int c = 0; c < C; ++c) Es[c] = E[c];
    for (int w = nw - 1; w >= 0; --w) {
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (w == wv) Es[c] = E[c];
        E[c] = apply(sA[buf][w][c][lane], sQ[buf][w][c][lane], E[c]);
      }
    }
    auto finish = [&](auto is_full) {
      constexpr bool FULL = decltype(is_full)::value;
      float w[S][C];  // (h' - x) f (1 - f)
#pragma unroll
      for (int s = 0; s < S; ++s) {
        if (!FULL && s >= n) continue;
        const bool r = !FULL && ((mask >> s) & 1u);
        float xv[C];
        unpack(px[s], xv);
#pragma unroll
        for (int c = 0; c < C; ++c) {
          const float hp = r ? 0.0f : h[c];
          const float b = i[s][c] * xv[c];
          h[c] = r ? b : __builtin_fmaf(f[s][c], h[c], b);
          w[s][c] = (hp - xv[c]) * (f[s][c] * i[s][c]);
        }
      }
#pragma unroll
      for (int s = S - 1; s >= 0; --s) {
        if (FULL || s < n) {
          const bool r = !FULL && ((mask >> s) & 1u);
          float dv[C], ox[C], og[C];
          unpack(pd[s], dv);
#pragma unroll
          for (int c = 0; c < C; ++c) {
            const float full_t = Es[c] + dv[c];
            ox[c] = full_t * i[s][c];
            og[c] = full_t * w[s][c];
            Es[c] = r ? 0.0f : full_t * f[s][c];
          }
          store_once<T, C>(dx.at(ts + s), ox);
          store_once<T, C>(dg.at(ts + s), og);
        } else if (ts + s < p.t_end) {
          const float zero[C] = {};
          store_once<T, C>(dx.at(ts + s), zero);
          store_once<T, C>(dg.at(ts + s), zero);
        }
      }
    };
    if (in && full) finish(std::true_type{});
    else if (in) finish(std::false_type{});
#pragma unroll
    for (int c = 0; c < C; ++c) Eo[c] = Es[c];
  }
  if (a.dh0 && p.seg == 0 && wv == 0 && in) {
#pragma unroll
    for (int c = 0; c < C; ++c) a.dh0[p.b * a.D + p.d + c] = Eo[c];
  }
}

// One step of B sequences: 2^lg threads per row, C channels per thread and
// step of the loop.
template <typename T, int C>
__global__ __launch_bounds__(256) void scan_step_kernel(StepArgs a, int lg) {
  const int64_t b = (int64_t)blockIdx.x * (256 >> lg) + (threadIdx.x >> lg);
  if (b >= a.B) return;
  const bool r = a.reset && a.reset[b] != 0;
  const int64_t step = (int64_t)C << lg;
  for (int64_t d = blockIdx.y * step + (threadIdx.x & ((1 << lg) - 1)) * C; d < a.D;
       d += gridDim.y * step) {
    float x[C], g[C], h[C], o[C];
    unpack(load_pack<T, C>(static_cast<const T*>(a.x) + b * a.x_st + d), x);
    unpack(load_pack<T, C>(static_cast<const T*>(a.g) + b * a.g_st + d), g);
    unpack(load_pack<float, C>(a.h + b * a.D + d), h);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float f, i;
      gate(g[c], f, i);
      const float ix = i * x[c];
      o[c] = r ? ix : __builtin_fmaf(f, h[c], ix);
    }
    store_vals<float, C>(a.h_out + b * a.D + d, o);
    store_vals<T, C>(static_cast<T*>(a.y) + b * a.y_st + d, o);
  }
}

template <typename T, int C, bool PACK = false>
hipError_t forward_typed(ScanArgs a, uint32_t blocks, int waves, hipStream_t s) {
  if (a.nseg > 1) {
    const hipError_t e = enqueue(scan_segment_kernel<T, C, PACK, false>, dim3(blocks),
                                       dim3(kWaves * 64), 0, s, a);
    if (e != hipSuccess) return e;
    // The last segment's workgroup may write h_last = h0 before others start.
    if (a.h0) a.h0 = a.h0_copy;
  }
  return enqueue(scan_forward_kernel<T, C, PACK>, dim3(blocks), dim3(64 * waves), 0, s, a);
}

template <typename T, int C, bool PACK = false>
hipError_t backward_typed(const ScanArgs& a, uint32_t blocks, int waves, hipStream_t s) {
  if (a.nseg > 1) {
    const hipError_t e = enqueue(scan_segment_kernel<T, C, PACK, true>, dim3(blocks),
                                       dim3(kWaves * 64), 0, s, a);
    if (e != hipSuccess) return e;
  }
  return enqueue(scan_backward_kernel<T, C, PACK>, dim3(blocks), dim3(64 * waves), 0, s, a);
}

// Waves of a workgroup: as many as the sequence has steps for, up to 8, or 16 where
// there is at most one workgroup to a CU and the time axis is whole (forward and
// backward, 16 against 8: 8 x 512 x 256 bf16 29.7 and 36.1 us, 200 x 200 x 64 19.4
// and 23.9, 37 x 81 x 333 f32 15.1 and 17.1).  With more workgroups one of 16 waves
// on a CU leaves its loads and stores unoverlapped (128 x 256 x 333 bf16, 384
// workgroups: 60 us with 16, 52 with 8).
int waves_for(int64_t T, int steps, int64_t blocks, bool cut) {
  const int64_t w = (T + steps - 1) / steps;
  const int most = !cut && blocks <= 256 ? kMaxWaves : kWaves;
  return w < 1 ? 1 : w > most ? most : (int)w;
}

// How a batch is spread over the chip: channels per lane, packed lanes, segments
// of the time axis and their steps (a multiple of kSegment).  Times below are
// forward and backward together, bf16 unless said.
//
// The time axis is cut where fewer than 192 workgroups would walk it: a cut reads
// two of the tensors again, and without one a few workgroups cannot carry the load.
// With D = 1000, 16 workgroups to a sequence, cut and not: of 12 sequences (192) 600
// steps take 54 and 48 us, 1024 84 and 76, 4096 347 and 309; of 10 (160) 49 and 43,
// 78 and 64, 264 and 285; of 6 (96) 38 and 39, 49 and 56, 170 and 253.  So 192 is
// where no length gains from the cut any more; shorter sequences would do without it
// from 128 workgroups on.  Up to 512 steps the second launch of each pass costs what
// the cut saves, or more (1 x 186 x 164: 27 us cut, 16 not; 16 x 300 x 400: 35 and 26),
// with an exception the rule leaves on the slower side (4 x 512 x 1024: 29 and 31),
// and past it less (4 x 762 x 98 f16: 30 and 41).  Two channels per lane make
// better use of loads once the chip is full (128 x 512 x 1024: 234 against 241 us;
// 2 x 16384 x 512: 86 against 97), one below (4 x 512 x 256: 28 against 32; 32 x 80
// x 512: 12.7 against 14.6), or where it saves the cut (16 x 512 x 1024, when it was cut:
// 42 against 50).  So they do for odd D, whose rows are not aligned to a pair (128 x 256 x 333:
// 52 against 63; 32 x 388 x 1225: 87 against 97), unless the last tile would hold a
// lone channel: the lane before it would be another workgroup's.  Lanes are packed
// where several sequences share a wave evenly or at least four do (4096 x 128 x
// 8: 36 against 81 us, x 32: 79 against 97; x 40: 114 against 98, since a packed
// lane has its own addresses and row ends inside a wave).
struct Plan {
  bool two, packed;
  int64_t blocks;  // without the cut
  int n;
  int64_t steps;
};
constexpr int64_t kFull = 192;
constexpr int64_t kWhole = 512;

Plan plan_with(int64_t B, int64_t T, int64_t D, bool two) {
  const int64_t w = two ? 128 : 64;
  Plan p = {two, false, B * ((D + w - 1) / w), 1, T};
  p.packed = D <= 16 || D == 32;
  if (p.packed) p.blocks = (B * D + 63) / 64;
  const int64_t chunks = (T + kSegment - 1) / kSegment;
  if (p.blocks >= kFull || T <= kWhole) return p;
  int64_t n = (512 + p.blocks - 1) / p.blocks;
  if (n > kMaxSeg) n = kMaxSeg;
  if (n > chunks) n = chunks;
  p.steps = (chunks + n - 1) / n * kSegment;
  p.n = (int)((T + p.steps - 1) / p.steps);
  return p;
}

Plan plan(int64_t B, int64_t T, int64_t D) {
  if (D <= 64 || D % 128 == 1) return plan_with(B, T, D, false);
  const Plan two = plan_with(B, T, D, true), one = plan_with(B, T, D, false);
  if (two.blocks * two.n < kFull || (two.n > 1 && one.n == 1)) return one;
  return two;
}

template <typename T>
hipError_t forward_of(const Plan& p, const ScanArgs& a, uint32_t blocks, int waves, hipStream_t s) {
  return p.packed ? forward_typed<T, 1, true>(a, blocks, waves, s)
         : p.two  ? forward_typed<T, 2>(a, blocks, waves, s)
                  : forward_typed<T, 1>(a, blocks, waves, s);
}
template <typename T>
hipError_t backward_of(const Plan& p, const ScanArgs& a, uint32_t blocks, int waves,
                       hipStream_t s) {
  return p.packed ? backward_typed<T, 1, true>(a, blocks, waves, s)
         : p.two  ? backward_typed<T, 2>(a, blocks, waves, s)
                  : backward_typed<T, 1>(a, blocks, waves, s);
}

Plan set_plan(ScanArgs& a) {
  const Plan p = plan(a.B, a.T, a.D);
  a.nseg = p.n;
  a.seg_steps = p.steps;
  if (p.n > 1) a.h0_copy = a.agg + a.B * p.n * 2 * a.D;
  return p;
}

}  // namespace

int64_t scan_blocks(int64_t B, int64_t T, int64_t D) {
  const Plan p = plan(B, T, D);
  return p.blocks * p.n;
}

size_t scan_workspace(int64_t B, int64_t T, int64_t D) {
  const int n = plan(B, T, D).n;
  return n == 1 ? 0 : (size_t)(B * n * 2 * D + B * D) * 4;
}

hipError_t launch_scan_forward(ScanArgs a, int type, hipStream_t s) {
  const Plan p = set_plan(a);
  const uint32_t blocks = (uint32_t)(p.blocks * p.n);
  const int waves = waves_for(a.T, kForward, blocks, p.n > 1);
  if (type == 0)
    return forward_of<float>(p, a, blocks, waves, s);
  if (type == 1)
    return forward_of<bf16_t>(p, a, blocks, waves, s);
  return forward_of<f16_t>(p, a, blocks, waves, s);
}

hipError_t launch_scan_backward(ScanArgs a, int type, hipStream_t s) {
  const Plan p = set_plan(a);
  const uint32_t blocks = (uint32_t)(p.blocks * p.n);
  const int waves = waves_for(a.T, kBackward, blocks, p.n > 1);
  if (type == 0)
    return backward_of<float>(p, a, blocks, waves, s);
  if (type == 1)
    return backward_of<bf16_t>(p, a, blocks, waves, s);
  return backward_of<f16_t>(p, a, blocks, waves, s);
}

template <typename T, int C>
static hipError_t step_launch(const StepArgs& a, hipStream_t s) {
  const int64_t units = a.D / C;
  int lg = 0;
  while (lg < 8 && (int64_t(1) << lg) < units) ++lg;
  const int64_t cols = (units + (1 << lg) - 1) >> lg;
  const int64_t rows = (a.B + (256 >> lg) - 1) / (256 >> lg);
  return enqueue(scan_step_kernel<T, C>,
                       dim3((uint32_t)rows, (uint32_t)(cols < 65535 ? cols : 65535)), dim3(256), 0,
                       s, a, lg);
}

template <typename T>
static hipError_t step_typed(const StepArgs& a, hipStream_t s) {
  return a.D % 4 == 0 ? step_launch<T, 4>(a, s) : step_launch<T, 1>(a, s);
}

hipError_t launch_scan_step(const StepArgs& a, int type, hipStream_t s) {
  return type == 0 ? step_typed<float>(a, s) : type == 1 ? step_typed<bf16_t>(a, s)
                                                         : step_typed<f16_t>(a, s);
}

}  // namespace per
