// delta_kernels.hip -- the gated delta rule: forward, backward and one step.
//
// A chunk of 64 steps at a time.  With D_ij the product of the gates of steps j + 1 to i
// (0 across a reset), gamma_i that of the steps up to i, d_j that of the steps behind j,
// and A_ij = w_i D_ij k_i.k_j below the diagonal, what the state takes up is
//     U = (I + A)^-1 w (V - gamma K S),
// the outputs are scale (gamma Q S + (Q K^T . D) U), and the state goes on as
// gamma_63 S + (d K)^T U.  Backward, with P = scale (Q K^T . D) and dS the gradient of
// the state behind the chunk,
//     E = (I + A)^-T (P^T dO + d K dS),   G = w E = dV,
//     dS' = gamma_63 dS + scale (gamma Q)^T dO - (gamma K)^T G,
//     dQ = scale gamma dO S^T + (scale dO U^T . D) K,
//     dK = d U dS^T + (scale dO U^T . D)^T Q - gamma G S^T - (M + M^T) K,  M = G U^T . D,
//     the gradient by the logit of w is (1 - w) E.U, and that by log f_i the sum of
//     q_j.dq_j - v_j.dv_j over the steps j >= i of the chunk and dS.S behind it
// (all by rows; D is scale-free, a reset ends each sum).
//
// What does not depend on the state ((I + A)^-1, Q K^T . D, the decays) is prepared for
// all chunks at once; one pass then walks over the chunks of a sequence with a slice of
// the state's columns in each wave's registers (the columns are independent), forward
// in time, or backward for dS; and the rest of the backward pass takes all chunks at
// once again.
//
// Products run on the bf16 matrix units, f32 factors as sums of three bf16 values (24
// bits; products below 2^-24 of the largest are left out), 16-bit inputs as one or two:
// 16 times the f32 units' rate, for 3 to 6 products.  Where only an output in 16 bits
// depends on it, two values (16 bits) do.
//
// The layout of a 16 x 16 result (lane 16 g + n has rows 4 g .. 4 g + 3 of column n) is
// that of half an operand of the next product, if the 32 terms of a sum are taken in the
// order rows 4 g + e of the first 16, then of the second: results feed products without
// a move.  Operands are kept in that order as blocks of 16 bytes for each lane.
#include <algorithm>

#include "block_internal.h"
#include "elem.h"
#include "lanes.h"

namespace per {
namespace {

constexpr int kC = PER_DELTA_CHUNK;
typedef bf16_t bf8 __attribute__((ext_vector_type(8)));
typedef bf16_t bf4 __attribute__((ext_vector_type(4)));
typedef float f4 __attribute__((ext_vector_type(4)));

template <typename T>
struct Tag {
  using type = T;
};

// bf16 values that hold one of the type, and the weakest products that are taken of
// those behind an output of it: parts i and j where i + j <= kWeak.
template <typename T>
constexpr int kParts = 3;
template <>
constexpr int kParts<bf16_t> = 1;
template <>
constexpr int kParts<f16_t> = 2;
template <typename T>
constexpr int kOutParts = sizeof(T) == 4 ? 3 : 2;
template <typename T>
constexpr int kWeak = kOutParts<T> - 1;

// 8 values as N bf16 parts, each the rounding of what the ones before leave.
template <int N>
__device__ __forceinline__ void split(const f4& lo, const f4& hi, bf8 (&p)[N]) {
  typedef float f8 __attribute__((ext_vector_type(8)));
  f8 x = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = __builtin_convertvector(x, bf8);
    if (i + 1 < N) x = x - __builtin_convertvector(p[i], f8);
  }
}
template <int N>
__device__ __forceinline__ void split4(f4 x, bf4 (&p)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    p[i] = __builtin_convertvector(x, bf4);
    if (i + 1 < N) x = x - __builtin_convertvector(p[i], f4);
  }
}

// c + a b over 32 terms, from the parts of a and b, the weakest products first.
template <int WEAK, int NA, int NB>
__device__ __forceinline__ f4 mul(const bf8 (&a)[NA], const bf8 (&b)[NB], f4 c) {
#pragma unroll
  for (int s = WEAK; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB)
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[i], b[s - i], c, 0, 0, 0);
  return c;
}

// The same for several a: the products of one sum lie COUNT instructions apart.
template <int WEAK, int COUNT, int NA, int NB>
__device__ __forceinline__ void mul_each(const bf8 (&a)[COUNT][NA], const bf8 (&b)[NB], f4* c) {
#pragma unroll
  for (int s = WEAK; s >= 0; --s)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (s - i >= 0 && s - i < NB)
#pragma unroll
        for (int k = 0; k < COUNT; ++k)
          c[k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[k][i], b[s - i], c[k], 0, 0, 0);
}

// Operand blocks: N parts of 64 lanes of 16 bytes each.  As they are copied (what is
// prepared, in memory and LDS) lane l's lie at 16 l; where pieces of rows are put together
// in LDS at 16 (l ^ turn), with a turn for each block, or the pieces that a wave writes at
// once would meet in few of the banks.
template <int N>
__device__ __forceinline__ void load_block(const char* block, bf8 (&p)[N], uint32_t lane) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    p[i] = *reinterpret_cast<const bf8*>(block + i * 1024 + lane * 16);
}
// Rows 16 it.. of 32 KT terms; the 32 rows 32 jt.. as the terms of columns 16 dt..
__device__ __forceinline__ constexpr int row_turn(int kt) { return kt & 3; }
__device__ __forceinline__ constexpr int col_turn(int dt) { return dt & 7; }
template <int N, int KT>
__device__ __forceinline__ void load_rows(const char* rows, int it, int kt, bf8 (&p)[N], uint32_t lane) {
  load_block<N>(rows + (it * KT + kt) * N * 1024, p, lane ^ row_turn(kt));
}
template <int N>
__device__ __forceinline__ void load_cols(const char* cols, int dt, int jt, bf8 (&p)[N], uint32_t lane) {
  load_block<N>(cols + (dt * 2 + jt) * N * 1024, p, lane ^ col_turn(dt));
}
// The same at a constant place of an array, by the offset 16 lane of a buffer in it.
template <int N>
__device__ __forceinline__ void lds_block(const char* room, int place, int n, bf8 (&p)[N], uint32_t me) {
#pragma unroll
  for (int i = 0; i < N; ++i)
    p[i] = *reinterpret_cast<const bf8*>(room + me + (place + (n * N + i) * 1024));
}
template <int N, int KT>
__device__ __forceinline__ void lds_rows(const char* room, int place, int it, int kt, bf8 (&p)[N], uint32_t me) {
  lds_block<N>(room, place, it * KT + kt, p, me ^ (row_turn(kt) * 16));
}
template <int N>
__device__ __forceinline__ void lds_cols(const char* room, int place, int dt, int jt, bf8 (&p)[N], uint32_t me) {
  lds_block<N>(room, place, dt * 2 + jt, p, me ^ (col_turn(dt) * 16));
}
// Half of a block from a 16 x 16 result: its rows are the terms of the sum.
template <int N>
__device__ __forceinline__ void store_half(char* blocks, int n, int half, const f4& v, uint32_t lane) {
  bf4 p[N];
  split4<N>(v, p);
  char* at = blocks + n * N * 1024 + lane * 16 + half * 8;
#pragma unroll
  for (int i = 0; i < N; ++i) *reinterpret_cast<bf4*>(at + i * 1024) = p[i];
}

// 6 of the 8 blocks of 16 rows x 32 terms of a triangular 64 x 64 matrix: rows 16 it of
// a lower one meet terms 32 kt with kt <= it / 2, those of an upper one kt >= it / 2.
__device__ __forceinline__ constexpr int lower_block(int it, int kt) {
  return it < 2 ? it : 2 * (it - 1) + kt;
}
__device__ __forceinline__ constexpr int upper_block(int it, int kt) {
  return it < 2 ? 2 * it + kt : it + 2;
}

// A thread's 4 x 8 piece of a [64 x 32 KT] matrix, as it lies in memory: rows 4 a + r,
// columns 8 m + c; 0 from row `rows` and from column `width` on.
template <typename T>
struct Piece {
  typedef T row __attribute__((ext_vector_type(8)));
  row v[4];
};
template <typename T>
__device__ __forceinline__ void load_piece(const T* base, int64_t stride, int rows, int width,
                                           int a, int m, Piece<T>& v) {
  // a chunk's rows lie within 2^31 bytes
  const uint32_t at = (uint32_t)(4 * a) * (uint32_t)stride + 8 * m;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    typename Piece<T>::row x = {};
    const T* row = base + r * stride;
    if (4 * a + r < rows) {
      if (8 * m + 8 <= width) {
        x = load_pack<T, 8>(row + at).v;
      } else if (8 * m < width) {
        const int last = width - 1 - 8 * m;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          const T e = row[at + min(c, last)];
          x[c] = c <= last ? e : (T)0.0f;
        }
      }
    }
    v.v[r] = x;
  }
}
template <typename T>
__device__ __forceinline__ void unpack_piece(const Piece<T>& v, float (&x)[4][8]) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 8; ++c) x[r][c] = (float)v.v[r][c];
}
// Four of its values as N parts.
template <int N, typename V>
__device__ __forceinline__ void split_four(V x, bf4 (&p)[N]) {
  if constexpr (N == 1) {
    p[0] = __builtin_convertvector(x, bf4);
  } else {
    split4<N>(__builtin_convertvector(x, f4), p);
  }
}
// As rows: blocks it * KT + kt, the columns being the terms.  As columns: blocks dt * 2 +
// jt, the rows being the terms.
template <int N, int KT, typename T>
__device__ __forceinline__ void store_piece(const Piece<T>& v, int a, int m, char* rows, char* cols) {
  typedef T t4 __attribute__((ext_vector_type(4)));
  if (rows) {
    const int half = m % 4 / 2, g = m % 2 * 2;
    char* at = rows + (a / 4 * KT + m / 4) * N * 1024 + half * 8 + (16 * g + a % 4 * 4) * 16;
    const int turn = row_turn(m / 4);  // below 4, as r
#pragma unroll
    for (int r = 0; r < 4; ++r) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const t4 x = {v.v[r][4 * k], v.v[r][4 * k + 1], v.v[r][4 * k + 2], v.v[r][4 * k + 3]};
        bf4 p[N];
        split_four<N>(x, p);
#pragma unroll
        for (int q = 0; q < N; ++q)
          *reinterpret_cast<bf4*>(at + q * 1024 + (16 * k + (r ^ turn)) * 16) = p[q];
      }
    }
  }
  if (cols) {
    char* at = cols + (m / 2 * 2 + a / 8) * N * 1024 + a % 8 / 4 * 8 + (16 * (a % 4) + m % 2 * 8) * 16;
    const int turn = col_turn(m / 2);  // below 8, as c
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const t4 x = {v.v[0][c], v.v[1][c], v.v[2][c], v.v[3][c]};
      bf4 p[N];
      split_four<N>(x, p);
#pragma unroll
      for (int q = 0; q < N; ++q)
        *reinterpret_cast<bf4*>(at + q * 1024 + (c ^ turn) * 16) = p[q];
    }
  }
}
// The same of f32 values.
template <int N, int KT>
__device__ __forceinline__ void store_piece(const float (&x)[4][8], int a, int m, char* rows) {
  Piece<float> v;
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 8; ++c) v.v[r][c] = x[r][c];
  store_piece<N, KT, float>(v, a, m, rows, nullptr);
}
// A chunk's rows as operand blocks, by all of a workgroup's threads.
template <typename T, int KT>
__device__ __forceinline__ void stage(const T* base, int64_t stride, int rows, int width, char* as_rows,
                                      char* as_cols) {
  for (int id = threadIdx.x; id < 64 * KT; id += blockDim.x) {
    Piece<T> v;
    load_piece<T>(base, stride, rows, width, id / (4 * KT), id % (4 * KT), v);
    store_piece<kParts<T>, KT, T>(v, id / (4 * KT), id % (4 * KT), as_rows, as_cols);
  }
}

// What is prepared for each (sequence, chunk, head): the decays and writing strengths,
// then operand blocks: (I + A)^-1 and Q K^T . D (forward), or the transposes of both.
struct Decays {
  double log[kC];   // base 2, of the gates up to a step; 2^12 less behind each reset
  float first[kC];  // gamma; -1 behind a reset
  float last[kC];   // d
  float w[kC];
  int resets[kC];   // up to a step
};
constexpr int kInvParts = 3;
template <typename T>
constexpr int kScoreParts(bool backward) {
  return backward ? 3 : kOutParts<T>;
}
constexpr size_t prep_bytes(int score_parts) {
  return sizeof(Decays) + (size_t)6 * (kInvParts + score_parts) * 1024;
}
size_t prep_bytes_of(int type, bool backward) {
  return prep_bytes(backward || type == PER_F32 ? 3 : 2);
}

__device__ __forceinline__ int steps_of(const DeltaArgs& a, int64_t b) {
  return __builtin_amdgcn_readfirstlane(
      (int)(a.length ? min(max(a.length[b], (int64_t)0), a.T) : a.T));
}
template <typename T>
__device__ __forceinline__ const T* at(const Seq& s, int64_t b, int64_t t, int64_t h) {
  return static_cast<const T*>(s.p) + b * s.sb + t * s.st + h * s.sh;
}

// Quotient and rest of a workgroup's number, in scalar registers.
__device__ __forceinline__ void divide(uint32_t x, uint32_t by, int& quotient, int& rest) {
  quotient = __builtin_amdgcn_readfirstlane((int)(x / by));
  rest = (int)(x - (uint32_t)quotient * by);
}

// Of the gates of steps j + 1 to i, 0 across a reset.
__device__ __forceinline__ float decay(const Decays& d, int i, int j) {
  return __builtin_amdgcn_exp2f((float)(d.log[i] - d.log[j]));
}

// One workgroup of 4 waves for each (sequence, chunk, head).
template <typename T, int KT, bool BACKWARD>
__global__ __launch_bounds__(256) void delta_prepare_kernel(DeltaArgs a) {
  constexpr int N = kParts<T>, NS = kScoreParts<T>(BACKWARD), kPad = 68;
  __shared__ __attribute__((aligned(16))) char ks[4 * KT * N * 1024];
  __shared__ __attribute__((aligned(16))) char qs[4 * KT * N * 1024];
  __shared__ __attribute__((aligned(16))) float lower[kC][kPad];
  __shared__ __attribute__((aligned(16))) float inv[kC][kPad];
  __shared__ Decays dec;
  const int lane = threadIdx.x & 63, g = lane / 16, n = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  int b, c, h;
  divide(blockIdx.x, (uint32_t)a.H, b, h);
  divide((uint32_t)b, (uint32_t)a.chunks, b, c);
  const int64_t t0 = (int64_t)c * kC;
  const int rows = min(kC, steps_of(a, b) - (int)t0);
  if (rows <= 0) return;
  char* out = static_cast<char*>(a.prep) + (int64_t)blockIdx.x * prep_bytes(NS);
  const int hk = h / (a.H / a.HK);
  stage<T, KT>(at<T>(a.k, b, t0, hk), a.k.st, rows, a.DK, ks, nullptr);
  stage<T, KT>(at<T>(a.q, b, t0, hk), a.q.st, rows, a.DK, qs, nullptr);
  if (wave == 3) {
    const bool on = lane < rows;
    const float gate = on ? (float)*at<T>(a.g, b, t0 + lane, h) : 0.0f;
    const float wt = on ? (float)*at<T>(a.b, b, t0 + lane, h) : 0.0f;
    const bool reset = on && a.reset && a.reset[b * a.T + t0 + lane];
    // log f; a gate below 2^-256 is 0 in f32 whatever it is
    const float lf = fminf(gate, 0.0f) - log1pf(expf(-fabsf(gate)));
    double log = reset ? -4096.0 : on ? fmax((double)lf * 1.4426950408889634074, -256.0) : 0.0;
    if (lf != lf && !reset) log = (double)lf;
    int resets = reset;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const double l = __shfl_up(log, d);
      const int r = __shfl_up(resets, d);
      log += lane >= d ? l : 0.0;
      resets += lane >= d ? r : 0;
    }
    const double end = __shfl(log, 63);
    dec.log[lane] = log;
    dec.resets[lane] = resets;
    dec.first[lane] = resets == 0 ? __builtin_amdgcn_exp2f((float)log) : -1.0f;
    dec.last[lane] = __builtin_amdgcn_exp2f((float)(end - log));
    dec.w[lane] = on ? 1.0f / (1.0f + expf(-wt)) : 0.0f;
  }
  for (int i = threadIdx.x; i < kC * kPad; i += 256) (&inv[0][0])[i] = 0.0f;
  __syncthreads();
  for (int i = threadIdx.x; i < (int)sizeof(Decays) / 16; i += 256)
    reinterpret_cast<f4*>(out)[i] = reinterpret_cast<const f4*>(&dec)[i];

  // 12 pairs of 16 rows and 16 columns, 10 of them on or below the diagonal: A for the
  // inverse, and scores as halves of blocks, zeros above the diagonal
  char* scores = out + sizeof(Decays) + 6 * kInvParts * 1024;
  for (int id = wave; id < 12; id += 4) {
    const int it = id < 4 ? id / 2 : 2 + (id - 4) / 4, jt = id < 4 ? id % 2 : (id - 4) % 4;
    f4 kk = {}, qk = {};
    if (jt <= it) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        bf8 ki[N], kj[N], qi[N];
        load_rows<N, KT>(ks, it, kt, ki, lane);
        load_rows<N, KT>(ks, jt, kt, kj, lane);
        load_rows<N, KT>(qs, it, kt, qi, lane);
        if (BACKWARD) {  // rows of it, columns of jt
          kk = mul<2>(ki, kj, kk);
          qk = mul<2>(qi, kj, qk);
        } else {
          kk = mul<2>(kj, ki, kk);
          qk = mul<2>(kj, qi, qk);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int i = 16 * it + (BACKWARD ? 4 * g + r : n), j = 16 * jt + (BACKWARD ? n : 4 * g + r);
        const float d = decay(dec, i, j);
        lower[i][j] = j < i ? dec.w[i] * d * kk[r] : 0.0f;
        qk[r] = j <= i ? d * qk[r] : 0.0f;
      }
    }
    if (BACKWARD) {  // rows of it are the terms of a row of jt
      if (it / 2 >= jt / 2 && jt < 4) store_half<NS>(scores, upper_block(jt, it / 2), it % 2, qk, lane);
    } else {
      store_half<NS>(scores, lower_block(it, jt / 2), jt % 2, qk, lane);
    }
  }
  __syncthreads();

  // (I + A)^-1: the blocks of 16 on the diagonal by substitution, a column to a lane
  if (lane < 16) {
    const int o = 16 * wave;
    float x[16];
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      float s = r == lane ? 1.0f : 0.0f;
#pragma unroll
      for (int k = 0; k < r; ++k) s -= lower[o + r][o + k] * x[k];
      x[r] = s;
      inv[o + r][o + lane] = s;
    }
  }
  __syncthreads();
  // and below it X_ij = -X_ii sum_k A_ik X_kj, a column of blocks to a wave
  {
    const int j = wave;
    f4 x[3];
#pragma unroll
    for (int step = 0; step < 3; ++step) {
      const int i = j + 1 + step;
      if (i < 4) {
        f4 z = {};
#pragma unroll
        for (int s = 0; s <= step; ++s) {
          const int k = j + s;
          const f4 p = *reinterpret_cast<const f4*>(&lower[16 * i + n][16 * k + 4 * g]);
          f4 q;
          if (s == 0) {
#pragma unroll
            for (int r = 0; r < 4; ++r) q[r] = inv[16 * j + 4 * g + r][16 * j + n];
          } else {
            q = x[s - 1];
          }
#pragma unroll
          for (int r = 0; r < 4; ++r)
            z = __builtin_amdgcn_mfma_f32_16x16x4f32(p[r], q[r], z, 0, 0, 0);
        }
        const f4 p = *reinterpret_cast<const f4*>(&inv[16 * i + n][16 * i + 4 * g]);
        f4 y = {};
#pragma unroll
        for (int r = 0; r < 4; ++r)
          y = __builtin_amdgcn_mfma_f32_16x16x4f32(p[r], z[r], y, 0, 0, 0);
        x[step] = -y;
#pragma unroll
        for (int r = 0; r < 4; ++r) inv[16 * i + 4 * g + r][16 * j + n] = -y[r];
      }
    }
  }
  __syncthreads();
  char* blocks = out + sizeof(Decays);
  for (int id = wave; id < 6; id += 4) {
    f4 lo, hi;
    if (BACKWARD) {
      const int jt = id < 4 ? id / 2 : id - 2, kt = id < 4 ? id % 2 : 1;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        lo[r] = inv[32 * kt + 4 * g + r][16 * jt + n];
        hi[r] = inv[32 * kt + 16 + 4 * g + r][16 * jt + n];
      }
    } else {
      const int it = id < 2 ? id : id / 2 + 1, kt = id < 2 ? 0 : id % 2;
      lo = *reinterpret_cast<const f4*>(&inv[16 * it + n][32 * kt + 4 * g]);
      hi = *reinterpret_cast<const f4*>(&inv[16 * it + n][32 * kt + 16 + 4 * g]);
    }
    bf8 p[kInvParts];
    split<kInvParts>(lo, hi, p);
#pragma unroll
    for (int q = 0; q < kInvParts; ++q)
      *reinterpret_cast<bf8*>(blocks + (id * kInvParts + q) * 1024 + lane * 16) = p[q];
  }
}

// Copies whole 16 bytes from memory to LDS by a workgroup.
__device__ __forceinline__ void copy16(char* to, const char* from, int bytes) {
  for (int i = threadIdx.x * 16; i < bytes; i += blockDim.x * 16)
    *reinterpret_cast<f4*>(to + i) = *reinterpret_cast<const f4*>(from + i);
}

// W neighbouring values of a row, 0 past `width`.
template <typename T, int W>
__device__ __forceinline__ void load_few(const T* row, int col, int width, float (&v)[W]) {
  if (col + W <= width) {
    unpack<T, W>(load_pack<T, W>(row + col), v);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = col + i < width ? (float)row[col + i] : 0.0f;
  }
}
template <typename T, int W>
__device__ __forceinline__ void store_few(T* row, int col, int width, const float (&v)[W]) {
  if (col + W <= width) {
    store_vals<T, W>(row + col, v);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (col + i < width) row[col + i] = (T)v[i];
  }
}

// A wave's column of a matrix [rows x width] for each lane n, as 16 x 16 results: rows 16 t
// + 4 g + r of column col.  Through a buffer descriptor that ends with the last row: the
// unit checks every access against it, so rows past the end read 0 and write nothing
// without a branch, a row's place is one scalar for the whole wave, and a lane's part of it
// (its column, past all rows where it has none) one register for all rows.
template <typename T, int TILES>
struct Column {
  __amdgpu_buffer_rsrc_t buffer;
  uint32_t lane;  // the lane's part
  int step;       // bytes between rows
  __device__ __forceinline__ Column(const T* base, int64_t stride, int rows, int col, int width) {
    step = (int)stride * (int)sizeof(T);
    asm volatile("" : "+s"(step));  // else the places of all rows are kept from chunk to chunk
    const int bytes = (rows - 1) * step + width * (int)sizeof(T);
    buffer = __builtin_amdgcn_make_buffer_rsrc(const_cast<T*>(base), 0, rows > 0 ? bytes : 0, 0x00020000);
    lane = col < width ? (threadIdx.x & 63) / 16 * 4 * (uint32_t)step + (uint32_t)col * (uint32_t)sizeof(T)
                       : 0xFFFFFFFFu;
  }
  __device__ __forceinline__ void load(T (&v)[TILES][4]) const {
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (sizeof(T) == 4) {
          v[t][r] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b32(buffer, lane, (16 * t + r) * step, 0));
        } else {
          v[t][r] = __builtin_bit_cast(T, __builtin_amdgcn_raw_buffer_load_b16(buffer, lane, (16 * t + r) * step, 0));
        }
      }
  }
  __device__ __forceinline__ void store(const f4 (&v)[TILES]) const {
#pragma unroll
    for (int t = 0; t < TILES; ++t)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        if constexpr (sizeof(T) == 4) {
          __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, (T)v[t][r]), buffer, lane,
                                                (16 * t + r) * step, 0);
        } else {
          __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (T)v[t][r]), buffer, lane,
                                                (16 * t + r) * step, 0);
        }
      }
  }
};
template <typename T, int TILES>
__device__ __forceinline__ void load_column(const T* base, int64_t stride, int rows, int col, int width,
                                            T (&v)[TILES][4]) {
  if (stride >= width) {
    Column<T, TILES>(base, stride, rows, col, width).load(v);
    return;
  }
  // rows that overlap (an expanded array) do not end with the last
  asm volatile("" : "+s"(stride), "+s"(rows));
  const int g = (threadIdx.x & 63) / 16;
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * t + 4 * g + r;
      v[t][r] = (T)0.0f;
      if (row < rows && col < width) v[t][r] = base[row * stride + col];
    }
}
template <typename T, int TILES>
__device__ __forceinline__ void store_column(T* base, int64_t stride, int rows, int col, int width,
                                             const f4 (&v)[TILES]) {
  Column<T, TILES>(base, stride, rows, col, width).store(v);
}
template <int TILES>
__device__ __forceinline__ void load_state(const float* s, int DK, int DV, int col, f4 (&v)[TILES]) {
  float x[TILES][4] = {};
  if (s) load_column<float, TILES>(s, DV, DK, col, DV, x);
#pragma unroll
  for (int t = 0; t < TILES; ++t)
#pragma unroll
    for (int r = 0; r < 4; ++r) v[t][r] = x[t][r];
}
// The rows' values of a chunk, 4 neighbouring ones of each 16.
__device__ __forceinline__ f4 rows_of(const float (&v)[kC], int it) {
  return *reinterpret_cast<const f4*>(&v[16 * it + 4 * ((threadIdx.x & 63) / 16)]);
}

// A state that is not finite stays on its side of a reset: the rows of the chunk on
// that side (`with`) give 0 to the other rows' sums, where 0 times them would not be 0.
// Called where the chunk has a reset.
template <typename F>
__device__ __forceinline__ void keep_apart(f4 (&x)[4], F with) {
  const int g = (threadIdx.x & 63) / 16;
  float bad = 0.0f;
#pragma unroll
  for (int it = 0; it < 4; ++it)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (with(16 * it + 4 * g + r) && !__builtin_isfinite(x[it][r])) bad = 1.0f;
  bad = fmaxf(bad, xor_lanes(bad, 4));
  bad = fmaxf(bad, xor_lanes(bad, 5));
#pragma unroll
  for (int it = 0; it < 4; ++it)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (bad != 0.0f && with(16 * it + 4 * g + r)) x[it][r] = 0.0f;
}

constexpr int64_t carry_size(int DK, int DV) { return (int64_t)(DK + kC) * DV; }

// What a workgroup of THREADS takes from memory for a chunk, held in registers while
// the chunk before is computed: pieces of the keys and queries, and what is prepared.
template <typename T, int KT, int THREADS, int BYTES>
struct Ahead {
  static constexpr int kPieces = (128 * KT + THREADS - 1) / THREADS;
  static constexpr int kCopies = (BYTES / 16 + THREADS - 1) / THREADS;
  Piece<T> piece[kPieces];
  f4 copy[kCopies];

  // even: rows begin at whole 4 bytes, and hold whole pieces
  __device__ __forceinline__ void load(const T* ks, int64_t kst, const T* qs, int64_t qst, bool even, int DK,
                                       int rows, const char* prep) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int id = threadIdx.x + p * THREADS, at = id % (64 * KT), a = at / (4 * KT), m = at % (4 * KT);
      const int query = __builtin_amdgcn_readfirstlane(id / (64 * KT));
      if (query > 1) continue;
      const T* base = query ? qs : ks;
      const int64_t stride = query ? qst : kst;
      if (even) {
        int step = (int)stride * (int)sizeof(T);
        const __amdgpu_buffer_rsrc_t buffer = __builtin_amdgcn_make_buffer_rsrc(
            const_cast<T*>(base), 0, (rows - 1) * step + DK * (int)sizeof(T), 0x00020000);
        const uint32_t lane = 8 * m < DK ? 4 * a * (uint32_t)step + 8 * m * (uint32_t)sizeof(T) : 0xFFFFFFFFu;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if constexpr (sizeof(T) == 2) {
            piece[p].v[r] = __builtin_bit_cast(typename Piece<T>::row,
                                               __builtin_amdgcn_raw_buffer_load_b128(buffer, lane, r * step, 0));
          } else {
            typedef T t4 __attribute__((ext_vector_type(4)));
            const t4 lo = __builtin_bit_cast(t4, __builtin_amdgcn_raw_buffer_load_b128(buffer, lane, r * step, 0));
            const t4 hi = __builtin_bit_cast(
                t4, __builtin_amdgcn_raw_buffer_load_b128(buffer, lane, r * step + 16, 0));
            piece[p].v[r] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
          }
        }
      } else {
        int64_t step = stride;
        int width = DK;
        asm volatile("" : "+s"(step), "+s"(width));
        load_piece<T>(base, step, rows, width, a, m, piece[p]);
      }
    }
#pragma unroll
    for (int c = 0; c < kCopies; ++c) {
      const uint32_t at = (threadIdx.x + c * THREADS) * 16;
      if (at < BYTES) copy[c] = *reinterpret_cast<const f4*>(prep + at);
    }
  }
  // which: 1 keys, 2 queries, 3 both
  __device__ __forceinline__ void store(char* krows, char* kcols, char* qrows, char* qcols, char* prep,
                                        int which = 3) const {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int id = threadIdx.x + p * THREADS, at = id % (64 * KT);
      const int query = __builtin_amdgcn_readfirstlane(id / (64 * KT));
      if (query == 0) {
        if (which & 1)
          store_piece<kParts<T>, KT, T>(piece[p], at / (4 * KT), at % (4 * KT), krows, kcols);
      } else if (query == 1 && (which & 2)) {
        store_piece<kParts<T>, KT, T>(piece[p], at / (4 * KT), at % (4 * KT), qrows, qcols);
      }
    }
    if (which & 1) {
#pragma unroll
      for (int c = 0; c < kCopies; ++c) {
        const uint32_t at = (threadIdx.x + c * THREADS) * 16;
        if (at < BYTES) *reinterpret_cast<f4*>(prep + at) = copy[c];
      }
    }
  }
};
// Whether rows of an array begin at whole 4 bytes, are whole pieces, and do not overlap.
template <typename T>
__device__ __forceinline__ bool even_rows(const T* p, int64_t stride, int D) {
  return D % 8 == 0 && stride >= D && (((uint32_t)(uintptr_t)p | (uint32_t)stride * (uint32_t)sizeof(T)) & 3) == 0;
}

// A workgroup has a head of a sequence and 16 columns of its state for each of its waves.
// While a chunk is computed the next one's operands are on their way in registers; they
// go to a second place in LDS where there is room for one, so a chunk needs one barrier.
template <typename T, int KT, int WAVES>
__global__ __launch_bounds__(64 * WAVES)
__attribute__((amdgpu_waves_per_eu(WAVES / 4, WAVES == 4 ? 1 : 4))) void delta_forward_kernel(DeltaArgs a, int slices) {
  constexpr int N = kParts<T>, NO = kOutParts<T>, WEAK = kWeak<T>;
  constexpr int kTile = 4 * KT * N * 1024, kPrep = (int)prep_bytes(NO);
  constexpr bool kApart = N < 3;  // queries have a place of their own in LDS
  constexpr int kRoom = (kApart ? 3 : 2) * kTile + kPrep;
  constexpr int kSome = 2;  // blocks that are held at a time
  constexpr bool kTwice = 2 * kRoom <= 160 * 1024;
  __shared__ __attribute__((aligned(16))) char room[(kTwice ? 2 : 1) * kRoom];
  constexpr int kCols = kTile, kQueries = kApart ? 2 * kTile : 0, kReady = kRoom - kPrep;
  constexpr int kInvs = kReady + (int)sizeof(Decays), kScores = kInvs + 6 * kInvParts * 1024;

  const int lane = threadIdx.x & 63, g = lane / 16, n = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  int bh, b, h, hk, slice, rest;
  divide(blockIdx.x, (uint32_t)slices, bh, slice);
  divide((uint32_t)bh, (uint32_t)a.H, b, h);
  divide((uint32_t)h, (uint32_t)(a.H / a.HK), hk, rest);
  const int col = (slice * WAVES + wave) * 16 + n;
  const int steps = steps_of(a, b);
  const int64_t unit0 = (int64_t)b * a.chunks * a.H + h;  // the head's first chunk; others lie H apart
  const T *ks = at<T>(a.k, b, 0, hk), *qs = at<T>(a.q, b, 0, hk), *vs = at<T>(a.v, b, 0, h);
  const bool even = even_rows(ks, a.k.st, a.DK) && even_rows(qs, a.q.st, a.DK);
  T* os = const_cast<T*>(at<T>(a.o, b, 0, h));

  f4 s[2 * KT];
  load_state<2 * KT>(a.s0 ? a.s0 + (int64_t)bh * a.DK * a.DV : nullptr, a.DK, a.DV, col, s);
  Ahead<T, KT, 64 * WAVES, kPrep> ahead;
  T v[4][4];
  if (steps > 0) {
    ahead.load(ks, a.k.st, qs, a.q.st, even, a.DK, min(kC, steps),
               static_cast<const char*>(a.prep) + unit0 * kPrep);
    load_column<T, 4>(vs, a.v.st, min(kC, steps), col, a.DV, v);
    ahead.store(room, room + kCols, room + kQueries, nullptr, room + kReady, kApart ? 3 : 1);
  }
  __syncthreads();
  for (int t0 = 0, flip = 0; t0 < steps; t0 += kC) {
    const int rows = min(kC, steps - t0), more = min(kC, steps - t0 - kC);
    const int64_t unit = unit0 + t0 / kC * a.H;
    char* now = room + (kTwice ? flip * kRoom : 0);
    const Decays& dec = *reinterpret_cast<const Decays*>(now + kReady);
    const bool resets = __builtin_amdgcn_readfirstlane(dec.resets[kC - 1]) != 0;
    // one register for all places in LDS
    uint32_t me = (uint32_t)(now - room) + (uint32_t)lane * 16;
    asm volatile("" : "+v"(me));
    f4 r[4];  // V
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int i = 0; i < 4; ++i) r[it][i] = (float)v[it][i];
    Ahead<T, KT, 64 * WAVES, kPrep> queries;
    if constexpr (!kApart) queries = ahead;
    if (more > 0) {
      ahead.load(ks + (int64_t)(t0 + kC) * a.k.st, a.k.st, qs + (int64_t)(t0 + kC) * a.q.st, a.q.st, even,
                 a.DK, more, static_cast<const char*>(a.prep) + (unit + a.H) * kPrep);
      load_column<T, 4>(vs + (int64_t)(t0 + kC) * a.v.st, a.v.st, more, col, a.DV, v);
    }
    float* carry = a.carries ? a.carries + unit * carry_size(a.DK, a.DV) : nullptr;
    if (carry) store_column<float, 2 * KT>(carry, a.DV, a.DK, col, a.DV, s);

    // K S and Q S
    f4 x[4] = {}, y[4] = {};
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      bf8 sp[3], kp[4][N], qp[4][N];
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        lds_rows<N, KT>(room, 0, it, kt, kp[it], me);
        if constexpr (kApart) lds_rows<N, KT>(room, kQueries, it, kt, qp[it], me);
      }
      split<3>(s[2 * kt], s[2 * kt + 1], sp);
      mul_each<2>(kp, sp, x);
      if constexpr (kApart) mul_each<WEAK>(qp, sp, y);
    }
    if constexpr (!kApart) {
      __syncthreads();
      queries.store(nullptr, nullptr, now + kQueries, nullptr, nullptr, 2);
      __syncthreads();
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        bf8 sp[3], qp[4][N];
#pragma unroll
        for (int it = 0; it < 4; ++it) lds_rows<N, KT>(room, kQueries, it, kt, qp[it], me);
        split<3>(s[2 * kt], s[2 * kt + 1], sp);
        mul_each<WEAK>(qp, sp, y);
      }
    }
    // w (V - gamma K S)
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const f4 first = rows_of(dec.first, it), w = rows_of(dec.w, it);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[it][i] *= first[i];
        y[it][i] *= first[i];
        if (resets && first[i] < 0.0f) x[it][i] = y[it][i] = 0.0f;
        x[it][i] = w[i] * (r[it][i] - x[it][i]);
      }
    }
    if (resets) keep_apart(x, [&](int i) { return dec.first[i] >= 0.0f; });
    // U
    f4 u[4] = {};
    {
      bf8 xp[3], p[kSome][kInvParts], q[2][kInvParts];
      split<3>(x[0], x[1], xp);
#pragma unroll
      for (int i0 = 0; i0 < 4; i0 += kSome) {
#pragma unroll
        for (int i = 0; i < kSome; ++i) lds_block<kInvParts>(room, kInvs, lower_block(i0 + i, 0), p[i], me);
        mul_each<2>(p, xp, u + i0);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) lds_block<kInvParts>(room, kInvs, lower_block(i + 2, 1), q[i], me);
      split<3>(x[2], x[3], xp);
      mul_each<2>(q, xp, u + 2);
    }
    if (carry) store_column<float, 4>(carry + (int64_t)a.DK * a.DV, a.DV, kC, col, a.DV, u);
    // the outputs
    {
      bf8 p[4][NO], up[NO];
#pragma unroll
      for (int it = 0; it < 4; ++it) lds_block<NO>(room, kScores, lower_block(it, 0), p[it], me);
      split<NO>(u[0], u[1], up);
      mul_each<WEAK>(p, up, y);
      bf8 q[2][NO];
#pragma unroll
      for (int it = 0; it < 2; ++it) lds_block<NO>(room, kScores, lower_block(it + 2, 1), q[it], me);
      split<NO>(u[2], u[3], up);
      mul_each<WEAK>(q, up, y + 2);
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      y[it] = y[it] * a.scale;
      u[it] = u[it] * rows_of(dec.last, it);
    }
    store_column<T, 4>(os + (int64_t)t0 * a.o.st, a.o.st, rows, col, a.DV, y);
    // the state behind the chunk
    const float kept = dec.first[kC - 1];
#pragma unroll
    for (int dt = 0; dt < 2 * KT; ++dt) s[dt] = resets ? f4{} : s[dt] * kept;
#pragma unroll
    for (int jt = 0; jt < 2; ++jt) {
      bf8 up[3];
      split<3>(u[2 * jt], u[2 * jt + 1], up);
#pragma unroll
      for (int d0 = 0; d0 < 2 * KT; d0 += kSome) {
        bf8 p[kSome][N];
#pragma unroll
        for (int i = 0; i < kSome; ++i) lds_cols<N>(room, kCols, d0 + i, jt, p[i], me);
        mul_each<2>(p, up, s + d0);
      }
    }
    if (more > 0) {
      if (kTwice) {
        flip ^= 1;
      } else {
        __syncthreads();
      }
      char* next = room + (kTwice ? flip * kRoom : 0);
      ahead.store(next, next + kCols, next + kQueries, nullptr, next + kReady, kApart ? 3 : 1);
    }
    __syncthreads();
  }
  if (a.s_last) store_column<float, 2 * KT>(a.s_last + (int64_t)bh * a.DK * a.DV, a.DV, a.DK, col, a.DV, s);
  for (int64_t t = steps + g; t < a.T; t += 4)
    if (col < a.DV) os[t * a.o.st + col] = (T)0.0f;
}

// Backward in time: dS behind each chunk, E, and dV.
template <typename T, int KT, int WAVES>
__global__ __launch_bounds__(64 * WAVES)
__attribute__((amdgpu_waves_per_eu(WAVES / 4, WAVES == 4 ? 1 : 4))) void delta_reverse_kernel(DeltaArgs a, int slices) {
  constexpr int N = kParts<T>;
  constexpr int kTile = 4 * KT * N * 1024, kPrep = (int)prep_bytes(3);
  constexpr bool kApart = N < 3;
  constexpr int kRoom = (kApart ? 3 : 2) * kTile + kPrep;
  constexpr int kSome = 2;  // blocks that are held at a time
  constexpr bool kTwice = 2 * kRoom <= 160 * 1024;
  __shared__ __attribute__((aligned(16))) char room[(kTwice ? 2 : 1) * kRoom];
  constexpr int kCols = kTile, kQueries = kApart ? 2 * kTile : 0, kReady = kRoom - kPrep;
  constexpr int kInvs = kReady + (int)sizeof(Decays), kScores = kInvs + 6 * kInvParts * 1024;

  const int lane = threadIdx.x & 63, g = lane / 16, n = lane % 16;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  int bh, b, h, hk, slice, rest;
  divide(blockIdx.x, (uint32_t)slices, bh, slice);
  divide((uint32_t)bh, (uint32_t)a.H, b, h);
  divide((uint32_t)h, (uint32_t)(a.H / a.HK), hk, rest);
  const int col = (slice * WAVES + wave) * 16 + n;
  const int steps = steps_of(a, b);
  const int64_t unit0 = (int64_t)b * a.chunks * a.H + h;
  const T *ks = at<T>(a.k, b, 0, hk), *qs = at<T>(a.q, b, 0, hk), *os = at<T>(a.o, b, 0, h);
  const bool even = even_rows(ks, a.k.st, a.DK) && even_rows(qs, a.q.st, a.DK);
  T* dvs = const_cast<T*>(at<T>(a.dv, b, 0, h));

  f4 s[2 * KT];
  load_state<2 * KT>(a.s0 ? a.s0 + (int64_t)bh * a.DK * a.DV : nullptr, a.DK, a.DV, col, s);
  Ahead<T, KT, 64 * WAVES, kPrep> ahead;
  T d[4][4];  // dO
  const int tail = steps > 0 ? (steps - 1) / kC * kC : -kC;  // the last chunk
  if (steps > 0) {
    ahead.load(ks + (int64_t)tail * a.k.st, a.k.st, qs + (int64_t)tail * a.q.st, a.q.st, even, a.DK,
               steps - tail, static_cast<const char*>(a.prep) + (unit0 + tail / kC * a.H) * kPrep);
    load_column<T, 4>(os + (int64_t)tail * a.o.st, a.o.st, steps - tail, col, a.DV, d);
    ahead.store(room, room + kCols, nullptr, room + kQueries, room + kReady, kApart ? 3 : 1);
  }
  __syncthreads();
  for (int t0 = tail, flip = 0; t0 >= 0; t0 -= kC) {
    const int rows = min(kC, steps - t0);
    const int64_t unit = unit0 + t0 / kC * a.H;
    char* now = room + (kTwice ? flip * kRoom : 0);
    const Decays& dec = *reinterpret_cast<const Decays*>(now + kReady);
    const bool resets = __builtin_amdgcn_readfirstlane(dec.resets[kC - 1]) != 0;
    uint32_t me = (uint32_t)(now - room) + (uint32_t)lane * 16;
    asm volatile("" : "+v"(me));
    f4 o[4];
#pragma unroll
    for (int it = 0; it < 4; ++it)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[it][i] = (float)d[it][i];
    Ahead<T, KT, 64 * WAVES, kPrep> queries;
    if constexpr (!kApart) queries = ahead;
    if (t0 > 0) {
      ahead.load(ks + (int64_t)(t0 - kC) * a.k.st, a.k.st, qs + (int64_t)(t0 - kC) * a.q.st, a.q.st, even,
                 a.DK, kC, static_cast<const char*>(a.prep) + (unit - a.H) * kPrep);
      load_column<T, 4>(os + (int64_t)(t0 - kC) * a.o.st, a.o.st, kC, col, a.DV, d);
    }
    store_column<float, 2 * KT>(a.dstate + unit * a.DK * a.DV, a.DV, a.DK, col, a.DV, s);

    // d K dS + scale P^T dO
    f4 x[4] = {}, y[4] = {};
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      bf8 sp[3], kp[4][N];
#pragma unroll
      for (int it = 0; it < 4; ++it) lds_rows<N, KT>(room, 0, it, kt, kp[it], me);
      split<3>(s[2 * kt], s[2 * kt + 1], sp);
      mul_each<2>(kp, sp, x);
    }
    {
      bf8 p[2][3], q[kSome][3], op[N];
#pragma unroll
      for (int jt = 0; jt < 2; ++jt) lds_block<3>(room, kScores, upper_block(jt, 0), p[jt], me);
      split<N>(o[0], o[1], op);
      mul_each<2>(p, op, y);
      split<N>(o[2], o[3], op);
#pragma unroll
      for (int j0 = 0; j0 < 4; j0 += kSome) {
#pragma unroll
        for (int i = 0; i < kSome; ++i) lds_block<3>(room, kScores, upper_block(j0 + i, 1), q[i], me);
        mul_each<2>(q, op, y + j0);
      }
    }
    if constexpr (!kApart) {
      __syncthreads();  // the keys' rows make room for the queries
      queries.store(nullptr, nullptr, nullptr, now + kQueries, nullptr, 2);
    }
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const f4 last = rows_of(dec.last, it);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[it][i] = (resets && last[i] == 0.0f ? 0.0f : last[i] * x[it][i]) + a.scale * y[it][i];
    }
    if (resets)
      keep_apart(x, [&](int i) { return dec.resets[i] == dec.resets[kC - 1]; });
    // E
    f4 e[4] = {};
    {
      bf8 p[2][kInvParts], q[kSome][kInvParts], xp[3];
#pragma unroll
      for (int jt = 0; jt < 2; ++jt) lds_block<kInvParts>(room, kInvs, upper_block(jt, 0), p[jt], me);
      split<3>(x[0], x[1], xp);
      mul_each<2>(p, xp, e);
      split<3>(x[2], x[3], xp);
#pragma unroll
      for (int j0 = 0; j0 < 4; j0 += kSome) {
#pragma unroll
        for (int i = 0; i < kSome; ++i) lds_block<kInvParts>(room, kInvs, upper_block(j0 + i, 1), q[i], me);
        mul_each<2>(q, xp, e + j0);
      }
    }
    store_column<float, 4>(a.e + unit * kC * a.DV, a.DV, kC, col, a.DV, e);
    // dV, then what goes back to the state before the chunk
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const f4 first = rows_of(dec.first, it);
      e[it] = e[it] * rows_of(dec.w, it);
      y[it] = e[it];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[it][i] *= -first[i];
        o[it][i] *= a.scale * first[i];
        if (resets && first[i] < 0.0f) e[it][i] = o[it][i] = 0.0f;
      }
    }
    store_column<T, 4>(dvs + (int64_t)t0 * a.dv.st, a.dv.st, rows, col, a.DV, y);
    if constexpr (!kApart) __syncthreads();
    const float kept = dec.first[kC - 1];
#pragma unroll
    for (int dt = 0; dt < 2 * KT; ++dt) s[dt] = resets ? f4{} : s[dt] * kept;
#pragma unroll
    for (int jt = 0; jt < 2; ++jt) {
      bf8 ep[3], op[3];
      split<3>(e[2 * jt], e[2 * jt + 1], ep);
      split<3>(o[2 * jt], o[2 * jt + 1], op);
#pragma unroll
      for (int d0 = 0; d0 < 2 * KT; d0 += kSome) {
        bf8 p[kSome][N], q[kSome][N];
#pragma unroll
        for (int i = 0; i < kSome; ++i) {
          lds_cols<N>(room, kCols, d0 + i, jt, p[i], me);
          lds_cols<N>(room, kQueries, d0 + i, jt, q[i], me);
        }
        mul_each<2>(p, ep, s + d0);
        mul_each<2>(q, op, s + d0);
      }
    }
    if (t0 > 0) {
      if (kTwice) {
        flip ^= 1;
      } else {
        __syncthreads();
      }
      char* next = room + (kTwice ? flip * kRoom : 0);
      ahead.store(next, next + kCols, nullptr, next + kQueries, next + kReady, kApart ? 3 : 1);
    }
    __syncthreads();
  }
  if (a.s_last) store_column<float, 2 * KT>(a.s_last + (int64_t)bh * a.DK * a.DV, a.DV, a.DK, col, a.DV, s);
  for (int64_t t = steps + g; t < a.T; t += 4)
    if (col < a.DV) dvs[t * a.dv.st + col] = (T)0.0f;
}

// dQ, dK and the gradients of gates and strengths, for each (sequence, chunk, head of
// keys): 8 waves.  What sums over the state's columns takes 64 of them at a time; a wave
// has 16 columns of dQ and dK (dt) and NI of the chunk's 4 groups of rows.
template <typename T, int KT>
__global__ __launch_bounds__(512) void delta_gradient_kernel(DeltaArgs a) {
  constexpr int N = kParts<T>, NO = kOutParts<T>, WEAK = kWeak<T>;
  constexpr int kDt = 2 * KT, NI = kDt / 2;
  constexpr int kTile = 4 * KT * N * 1024;
  constexpr int kStage = (8 * N + 16 * NO) * 1024, kPairs = 20 * NO * 1024;
  constexpr bool kApart = N < 3;
  __shared__ __attribute__((aligned(16))) char space[kStage > kPairs ? kStage : kPairs];
  __shared__ __attribute__((aligned(16))) char kcols_[kTile], qcols_[kApart ? kTile : 16];
  __shared__ __attribute__((aligned(16))) Decays dec;
  __shared__ float eu[kC], gv[kC], qd[kDt][kC], ends[8][2];
  char *dos = space, *us = dos + 8 * N * 1024, *gs = us + 8 * NO * 1024;
  char *da = space, *dt_ = da + 6 * NO * 1024, *mm = dt_ + 6 * NO * 1024;
  char *kcols = kcols_, *qcols = kApart ? qcols_ : kcols_;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  int b, c, hk;
  divide(blockIdx.x, (uint32_t)a.HK, b, hk);
  divide((uint32_t)b, (uint32_t)a.chunks, b, c);
  const int shared = a.H / a.HK;
  const int64_t t0 = (int64_t)c * kC;
  const int steps = steps_of(a, b), rows = min(kC, steps - (int)t0);
  const int here = (int)min((int64_t)kC, a.T - t0);  // rows that are written
  const int dt = wave % kDt, i0 = wave / kDt * NI;
  f4 dq[NI] = {}, dk[NI] = {};

  if (rows > 0) {
    for (int gi = 0; gi < shared; ++gi) {
      // else every place in LDS is computed before this loop, and registers run out
      int lane = threadIdx.x & 63;
      asm volatile("" : "+v"(lane));
      const int g = lane / 16, n = lane % 16, dcol = 16 * dt + n;
      const int h = hk * shared + gi;
      const int64_t unit = ((int64_t)b * a.chunks + c) * a.H + h;
      const float* s0 = a.carries + unit * carry_size(a.DK, a.DV);
      const float* u = s0 + (int64_t)a.DK * a.DV;
      const float* ds = a.dstate + unit * a.DK * a.DV;
      const float* e = a.e + unit * kC * a.DV;
      f4 qs[NI] = {}, k1[NI] = {}, k2[NI] = {}, pair[5] = {};
      float ss = 0.0f;
      __syncthreads();
      copy16(reinterpret_cast<char*>(&dec), static_cast<const char*>(a.prep) + unit * prep_bytes(3),
             sizeof(Decays));
      if (threadIdx.x < kC) eu[threadIdx.x] = gv[threadIdx.x] = 0.0f;
      if (kApart && gi == 0) {
        stage<T, KT>(at<T>(a.k, b, t0, hk), a.k.st, rows, a.DK, nullptr, kcols);
        stage<T, KT>(at<T>(a.q, b, t0, hk), a.q.st, rows, a.DK, nullptr, qcols);
      }
      for (int v0 = 0; v0 < a.DV; v0 += 64) {
        __syncthreads();
        const int width = a.DV - v0;
        {
          // 128 threads each: U; dO; G and the sums E.U; the sums G.V
          const int pa = wave % 2 * 8 + lane / 8, pm = lane % 8, job = wave / 2;
          if (job == 0) {
            Piece<float> x;
            load_piece<float>(u + v0, a.DV, kC, width, pa, pm, x);
            store_piece<NO, 2, float>(x, pa, pm, us, nullptr);
          } else if (job == 1) {
            Piece<T> x;
            load_piece<T>(at<T>(a.o, b, t0, h) + v0, a.o.st, rows, width, pa, pm, x);
            store_piece<N, 2, T>(x, pa, pm, dos, nullptr);
          } else {
            Piece<float> p;
            float x[4][8], y[4][8];
            load_piece<float>(e + v0, a.DV, kC, width, pa, pm, p);
            unpack_piece<float>(p, x);
            if (job == 2) {
              load_piece<float>(u + v0, a.DV, kC, width, pa, pm, p);
              unpack_piece<float>(p, y);
            } else {
              Piece<T> q;
              load_piece<T>(at<T>(a.v, b, t0, h) + v0, a.v.st, rows, width, pa, pm, q);
              unpack_piece<T>(q, y);
            }
            float sum[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const float w = dec.w[4 * pa + r];
              sum[r] = 0.0f;
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                sum[r] += x[r][k] * y[r][k];
                x[r][k] *= w;
              }
              if (job == 3) sum[r] *= w;
#pragma unroll
              for (int q = 0; q < 3; ++q) sum[r] += xor_lanes(sum[r], q);
              if (pm == 0) (job == 2 ? eu : gv)[4 * pa + r] += sum[r];
            }
            if (job == 2) store_piece<NO, 2>(x, pa, pm, gs);
          }
        }
        __syncthreads();
        // 64 x 64 products: waves 0 to 3 G U^T, twice for the 16 x 16 on the diagonal (once
        // for each side of it), waves 4 to 7 dO U^T and its transpose
#pragma unroll 1
        for (int kt = 0; kt < 2; ++kt) {
#pragma unroll
          for (int p = 0; p < 5; ++p) {
            __builtin_amdgcn_sched_barrier(0);  // else all loads come first, and registers run out
            if (wave < 4) {
              // rows j, columns i: U_j G_i above the diagonal of this result, G_j U_i below
              const int it = wave, jt = p < 2 ? wave : (wave + p - 1) & 3;
              const bool up = p < 2 ? p == 0 : jt < it;
              bf8 x[NO], y[NO];
              load_rows<NO, 2>(up ? us : gs, jt, kt, x, lane);
              load_rows<NO, 2>(up ? gs : us, it, kt, y, lane);
              pair[p] = mul<WEAK>(x, y, pair[p]);
            } else {
              const int id = (wave - 4) * 5 + p, k = id % 10;
              const int it = k < 1 ? 0 : k < 3 ? 1 : k < 6 ? 2 : 3, jt = k - it * (it + 1) / 2;
              bf8 x[NO], y[N];
              load_rows<NO, 2>(us, jt, kt, x, lane);
              load_rows<N, 2>(dos, it, kt, y, lane);
              pair[p] = id < 10 ? mul<WEAK>(x, y, pair[p]) : mul<WEAK>(y, x, pair[p]);
            }
          }
        }
        // dO S^T, U dS^T, G S^T
#pragma unroll 1
        for (int kt = 0; kt < 2; ++kt) {
          const int v = v0 + 32 * kt + 4 * g;
          f4 x[2], y[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float p[4] = {}, q[4] = {};
            if (dcol < a.DK) {
              load_few<float, 4>(s0 + (int64_t)dcol * a.DV, v + 16 * k, a.DV, p);
              load_few<float, 4>(ds + (int64_t)dcol * a.DV, v + 16 * k, a.DV, q);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              x[k][r] = p[r];
              y[k][r] = q[r];
              ss += p[r] * q[r];
            }
          }
          bf8 xp[NO], yp[NO];
          split<NO>(x[0], x[1], xp);
          split<NO>(y[0], y[1], yp);
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            bf8 od[N], ou[NO], og[NO];
            load_rows<N, 2>(dos, i0 + i, kt, od, lane);
            load_rows<NO, 2>(us, i0 + i, kt, ou, lane);
            load_rows<NO, 2>(gs, i0 + i, kt, og, lane);
            qs[i] = mul<WEAK>(od, xp, qs[i]);
            k1[i] = mul<WEAK>(ou, yp, k1[i]);
            k2[i] = mul<WEAK>(og, xp, k2[i]);
          }
        }
      }
      __syncthreads();
      // the 64 x 64 matrices with their decays, as operands
      if (wave < 4) {
        const int it = wave;
#pragma unroll
        for (int p = 0; p < 5; ++p) {
          if (p == 1) continue;
          __builtin_amdgcn_sched_barrier(0);
          const int jt = p < 2 ? wave : (wave + p - 1) & 3;
          f4 v;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = 16 * it + n, j = 16 * jt + 4 * g + r;
            const float x = p == 0 && j > i ? pair[1][r] : pair[p][r];
            v[r] = i == j ? 0.0f : -x * decay(dec, max(i, j), min(i, j));
          }
          store_half<NO>(mm, it * 2 + jt / 2, jt % 2, v, lane);
        }
        const f4 zero = {};
        if (wave == 0) store_half<NO>(da, lower_block(0, 0), 1, zero, lane);
        if (wave == 1) store_half<NO>(da, lower_block(2, 1), 1, zero, lane);
        if (wave == 2) store_half<NO>(dt_, upper_block(1, 0), 0, zero, lane);
        if (wave == 3) store_half<NO>(dt_, upper_block(3, 1), 0, zero, lane);
      } else {
#pragma unroll
        for (int p = 0; p < 5; ++p) {
          const int id = (wave - 4) * 5 + p, k = id % 10;
          const int it = k < 1 ? 0 : k < 3 ? 1 : k < 6 ? 2 : 3, jt = k - it * (it + 1) / 2;
          __builtin_amdgcn_sched_barrier(0);
          f4 v;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int i = 16 * it + (id < 10 ? n : 4 * g + r);
            const int j = 16 * jt + (id < 10 ? 4 * g + r : n);
            v[r] = j <= i ? a.scale * pair[p][r] * decay(dec, i, j) : 0.0f;
          }
          if (id < 10) {
            store_half<NO>(da, lower_block(it, jt / 2), jt % 2, v, lane);
          } else {
            store_half<NO>(dt_, upper_block(jt, it / 2), it % 2, v, lane);
          }
        }
      }
      if (!kApart) stage<T, KT>(at<T>(a.k, b, t0, hk), a.k.st, rows, a.DK, nullptr, kcols);
      __syncthreads();
      float end = 0.0f;
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        const int it = i0 + i;
        bf4 kp[N];
#pragma unroll
        for (int q = 0; q < N; ++q)
          kp[q] = *reinterpret_cast<const bf4*>(kcols + ((dt * 2 + it / 2) * N + q) * 1024 +
                                                (lane ^ col_turn(dt)) * 16 + it % 2 * 8);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * it + 4 * g + r;
          const float first = dec.first[row], last = dec.last[row];
          float kx = 0.0f;
#pragma unroll
          for (int q = N - 1; q >= 0; --q) kx += (float)kp[q][r];
          qs[i][r] = first >= 0.0f ? qs[i][r] * (a.scale * first) : 0.0f;
          k1[i][r] = last != 0.0f ? k1[i][r] * last : 0.0f;
          end += kx * k1[i][r];
          if (first >= 0.0f) k1[i][r] -= first * k2[i][r];
        }
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          bf8 y[N], x[NO];
          load_cols<N>(kcols, dt, kt, y, lane);
          if (kt <= it / 2) {
            load_block<NO>(da + lower_block(it, kt) * NO * 1024, x, lane);
            qs[i] = mul<WEAK>(x, y, qs[i]);
          }
          load_block<NO>(mm + (it * 2 + kt) * NO * 1024, x, lane);
          k1[i] = mul<WEAK>(x, y, k1[i]);
        }
      }
      if (!kApart) {
        __syncthreads();
        stage<T, KT>(at<T>(a.q, b, t0, hk), a.q.st, rows, a.DK, nullptr, qcols);
        __syncthreads();
      }
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        __builtin_amdgcn_sched_barrier(0);
        const int it = i0 + i;
#pragma unroll
        for (int kt = 0; kt < 2; ++kt) {
          if (kt < it / 2) continue;
          bf8 y[N], x[NO];
          load_cols<N>(qcols, dt, kt, y, lane);
          load_block<NO>(dt_ + upper_block(it, kt) * NO * 1024, x, lane);
          k1[i] = mul<WEAK>(x, y, k1[i]);
        }
        bf4 qp[N];
#pragma unroll
        for (int q = 0; q < N; ++q)
          qp[q] = *reinterpret_cast<const bf4*>(qcols + ((dt * 2 + it / 2) * N + q) * 1024 +
                                                (lane ^ col_turn(dt)) * 16 + it % 2 * 8);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float x = 0.0f;
#pragma unroll
          for (int q = N - 1; q >= 0; --q) x += (float)qp[q][r];
          x *= qs[i][r];
#pragma unroll
          for (int q = 0; q < 4; ++q) x += xor_lanes(x, q);
          if (n == 0) qd[dt][16 * it + 4 * g + r] = x;
        }
        dq[i] += qs[i];
        dk[i] += k1[i];
      }
      // dS . S behind the chunk
      if (i0 > 0) ss = 0.0f;
#pragma unroll
      for (int q = 0; q < 6; ++q) {
        end += xor_lanes(end, q);
        ss += xor_lanes(ss, q);
      }
      if (lane == 0) {
        ends[wave][0] = end;
        ends[wave][1] = ss;
      }
      __syncthreads();
      if (wave == 0) {
        double z = 0.0, last = 0.0, across = 0.0;
#pragma unroll
        for (int k = 0; k < kDt; ++k) z += qd[k][lane];
        z -= gv[lane];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          last += ends[k][0];
          across += ends[k][1];
        }
        const float kept = dec.first[kC - 1];
        if (kept >= 0.0f) last += (double)kept * across;
        if (lane == kC - 1) z += last;
        const int mine = dec.resets[lane];
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
          const double o = __shfl_down(z, d);
          const int theirs = __shfl_down(mine, d);
          if (lane + d < 64 && theirs == mine) z += o;
        }
        const int before = __shfl_up(mine, 1);
        const bool reset = lane == 0 ? mine != 0 : mine != before;
        if (lane < here) {
          const bool on = lane < rows;
          const float gate = on ? (float)*at<T>(a.g, b, t0 + lane, h) : 0.0f;
          const float wt = on ? (float)*at<T>(a.b, b, t0 + lane, h) : 0.0f;
          *const_cast<T*>(at<T>(a.dg, b, t0 + lane, h)) =
              (T)(on && !reset ? (float)z / (1.0f + expf(gate)) : 0.0f);
          *const_cast<T*>(at<T>(a.db, b, t0 + lane, h)) =
              (T)(on ? eu[lane] / (1.0f + expf(wt)) : 0.0f);
        }
      }
    }
  } else {
    for (int i = threadIdx.x; i < here * shared; i += 512) {
      const int64_t t = t0 + i / shared;
      const int h = hk * shared + i % shared;
      *const_cast<T*>(at<T>(a.dg, b, t, h)) = (T)0.0f;
      *const_cast<T*>(at<T>(a.db, b, t, h)) = (T)0.0f;
    }
  }
  int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));  // the places of dQ and dK are computed here, not before the loop
  const int g = lane / 16, dcol = 16 * dt + lane % 16;
#pragma unroll
  for (int i = 0; i < NI; ++i)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = 16 * (i0 + i) + 4 * g + r;
      if (row < here && dcol < a.DK) {
        const_cast<T*>(at<T>(a.dq, b, t0 + row, hk))[dcol] = (T)(row < rows ? dq[i][r] : 0.0f);
        const_cast<T*>(at<T>(a.dk, b, t0 + row, hk))[dcol] = (T)(row < rows ? dk[i][r] : 0.0f);
      }
    }
}

// One step: a workgroup has a head's state, 32 groups of 4 columns by PARTS groups of 16
// rows, so all of it is asked for at once.  The state is read and written once.
template <typename T, int PARTS>
__global__ __launch_bounds__(32 * PARTS) void delta_step_kernel(DeltaArgs a, int slices) {
  __shared__ float sum[2][PARTS][128];
  __shared__ float ks[16 * PARTS], qs[16 * PARTS];
  int bh, b, h, hk, slice, rest;
  divide(blockIdx.x, (uint32_t)slices, bh, slice);
  divide((uint32_t)bh, (uint32_t)a.H, b, h);
  divide((uint32_t)h, (uint32_t)(a.H / a.HK), hk, rest);
  const int part = threadIdx.x / 32, cl = threadIdx.x % 32 * 4, col = slice * 128 + cl;
  const float* s = a.s0 + (int64_t)bh * a.DK * a.DV;
  float v[16][4];
  const bool reset = a.reset && a.reset[b];
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int row = part * 16 + r;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[r][i] = 0.0f;
    if (row < a.DK && !reset) load_few<float, 4>(s + (int64_t)row * a.DV, col, a.DV, v[r]);
  }
  {
    const int i = threadIdx.x;
    const int c = i % (16 * PARTS);
    const T* from = i < 16 * PARTS ? at<T>(a.k, b, 0, hk) : at<T>(a.q, b, 0, hk);
    (i < 16 * PARTS ? ks : qs)[c] = c < a.DK ? (float)from[c] : 0.0f;
  }
  float vs[4];
  load_few<T, 4>(at<T>(a.v, b, 0, h), col, a.DV, vs);
  const float gate = (float)*at<T>(a.g, b, 0, h), wt = (float)*at<T>(a.b, b, 0, h);
  const float f = 1.0f / (1.0f + expf(-gate)), w = 1.0f / (1.0f + expf(-wt));
  __syncthreads();
  float k[4] = {}, q[4] = {};
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const float kr = ks[part * 16 + r];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[r][i] *= f;
      k[i] += kr * v[r][i];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[0][part][cl + i] = k[i];
  __syncthreads();
  float u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x = 0.0f;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) x += sum[0][p][cl + i];
    u[i] = col + i < a.DV ? w * (vs[i] - x) : 0.0f;
  }
  float* to = a.s_last + (int64_t)bh * a.DK * a.DV;
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    const int row = part * 16 + r;
    const float kr = ks[row], qr = qs[row];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[r][i] += kr * u[i];
      q[i] += qr * v[r][i];
    }
    if (row < a.DK) store_few<float, 4>(to + (int64_t)row * a.DV, col, a.DV, v[r]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sum[1][part][cl + i] = q[i];
  __syncthreads();
  for (int i = threadIdx.x; i < 128; i += 32 * PARTS) {
    const int c = slice * 128 + i;
    if (c >= a.DV) break;
    float x = 0.0f;
#pragma unroll
    for (int p = 0; p < PARTS; ++p) x += sum[1][p][i];
    const_cast<T*>(at<T>(a.o, b, 0, h))[c] = (T)(a.scale * x);
  }
}

template <typename F>
hipError_t by_type(int type, F f) {
  switch (type) {
    case PER_F32: return f(Tag<float>{});
    case PER_BF16: return f(Tag<bf16_t>{});
    default: return f(Tag<f16_t>{});
  }
}
template <int K>
struct Size {
  static constexpr int value = K;
};
template <typename F>
hipError_t by_keys(int DK, F f) {
  if (DK <= 32) return f(Size<1>{});
  if (DK <= 64) return f(Size<2>{});
  return f(Size<4>{});
}

hipError_t launch_prepare(const DeltaArgs& a, int type, bool backward, hipStream_t s) {
  return by_type(type, [&](auto tag) {
    return by_keys(a.DK, [&](auto keys) {
      using T = typename decltype(tag)::type;
      constexpr int KT = decltype(keys)::value;
      return enqueue(backward ? delta_prepare_kernel<T, KT, true> : delta_prepare_kernel<T, KT, false>,
                     dim3((uint32_t)(a.B * a.chunks * a.H)), dim3(256), 0, s, a);
    });
  });
}

}  // namespace

size_t delta_workspace(int64_t B, int64_t T, int64_t H, int64_t DK, int64_t DV, int type,
                       bool backward, DeltaArgs* a, void* ws) {
  const int64_t units = B * ((T + kC - 1) / kC) * H;
  const size_t prep = (size_t)units * prep_bytes_of(type, backward);
  const size_t state = backward ? ((size_t)(units * DK * DV) * 4 + 15) / 16 * 16 : 0;
  const size_t rows = backward ? (size_t)(units * kC * DV) * 4 : 0;
  if (a) {
    char* p = static_cast<char*>(ws);
    a->prep = p;
    a->dstate = reinterpret_cast<float*>(p + prep);
    a->e = reinterpret_cast<float*>(p + prep + state);
  }
  return prep + state + rows;
}

// Waves of a workgroup, 16 columns of the state each: up to 128 columns, or 64 where the
// states are few and twice as many workgroups find a place, or where 8 waves' registers
// do not hold what a chunk takes (f32, and 128 keys of f16).
static int column_waves(const DeltaArgs& a, int type) {
  if (type == PER_F32 || (type == PER_F16 && a.DK > 64)) return 4;
  return a.DV <= 64 || a.B * a.H * ((a.DV + 127) / 128) <= 128 ? 4 : 8;
}
template <typename T, int KT>
struct Columns {
  static constexpr int most = kParts<T> == 3 || (kParts<T> == 2 && KT == 4) ? 4 : 8;
  static constexpr auto forward4 = delta_forward_kernel<T, KT, 4>;
  static constexpr auto forward8 = delta_forward_kernel<T, KT, most>;
  static constexpr auto reverse4 = delta_reverse_kernel<T, KT, 4>;
  static constexpr auto reverse8 = delta_reverse_kernel<T, KT, most>;
};

hipError_t launch_delta_forward(const DeltaArgs& a, int type, hipStream_t s) {
  hipError_t e = a.chunks > 0 ? launch_prepare(a, type, false, s) : hipSuccess;
  if (e != hipSuccess) return e;
  const int waves = column_waves(a, type), slices = (a.DV + 16 * waves - 1) / (16 * waves);
  return by_type(type, [&](auto tag) {
    return by_keys(a.DK, [&](auto keys) {
      using K = Columns<typename decltype(tag)::type, decltype(keys)::value>;
      return enqueue(waves == 4 ? K::forward4 : K::forward8, dim3((uint32_t)(a.B * a.H * slices)),
                     dim3(64 * waves), 0, s, a, slices);
    });
  });
}

hipError_t launch_delta_backward(const DeltaArgs& a, int type, hipStream_t s) {
  hipError_t e = a.chunks > 0 ? launch_prepare(a, type, true, s) : hipSuccess;
  if (e != hipSuccess) return e;
  const int waves = column_waves(a, type), slices = (a.DV + 16 * waves - 1) / (16 * waves);
  return by_type(type, [&](auto tag) {
    return by_keys(a.DK, [&](auto keys) {
      using T = typename decltype(tag)::type;
      constexpr int KT = decltype(keys)::value;
      using K = Columns<T, KT>;
      const hipError_t e = enqueue(waves == 4 ? K::reverse4 : K::reverse8,
                                   dim3((uint32_t)(a.B * a.H * slices)), dim3(64 * waves), 0, s, a,
                                   slices);
      if (e != hipSuccess || a.chunks == 0) return e;
      return enqueue(delta_gradient_kernel<T, KT>, dim3((uint32_t)(a.B * a.chunks * a.HK)), dim3(512),
                     0, s, a);
    });
  });
}

hipError_t launch_delta_step(const DeltaArgs& a, int type, hipStream_t s) {
  const int slices = (a.DV + 127) / 128;
  return by_type(type, [&](auto tag) {
    return by_keys(a.DK, [&](auto keys) {
      constexpr int parts = 2 * decltype(keys)::value;
      return enqueue(delta_step_kernel<typename decltype(tag)::type, parts>,
                     dim3((uint32_t)(a.B * a.H * slices)), dim3(32 * parts), 0, s, a, slices);
    });
  });
}

}  // namespace per
