// distill_kernels.hip -- distillation from a teacher's top logits: per-row loss
// and its gradient by the student's logits.
//
// With m the row's largest logit and S = sum exp((z - m) / tau) over all tokens,
// m_r and S_r the same over the tokens of the rest, the gradient by z_j is
//   w tau (exp((z_j - m) / tau) / S - p_j)   at a token of the teacher's top,
//   w tau C exp((z_j - m_r) / tau)           at the others,
//   C = exp((m_r - m) / tau) / S - p_r / S_r,
// so one coefficient serves the whole row and K places are put right after.
// Without a rest m_r = m and C = 1 / S.  The rest has its own largest logit
// because the row's may be a top token so far above it that every exp((z - m) /
// tau) of the rest is 0 in f32, where log q_r is an ordinary number.
//
// A thread's sums are f32, chunk by chunk; what threads join is f64.  The loss is
// tau^2 times a difference of logarithms of S and S_r, in which the roundings of
// joins in f32 stood out: of a student near its teacher (V = 120000, tau = 32) they
// left an error of 8e-5 in a loss of 8e-7, and leave 3e-9 now.
//
// A row is read in 16-byte chunks aligned in memory; chunk j holds the tokens
// [j * kVec - mis, (j + 1) * kVec - mis).  The tokens of the top are marked in
// a bitmap in LDS, so sums over the rest leave them out instead of
// subtracting them, and repeated entries are found.

#include "elem.h"
#include "lanes.h"
#include "train_internal.h"

namespace per {
namespace {

constexpr float kNegInf = -__builtin_inff();

template <typename T>
constexpr int kVec = 16 / (int)sizeof(T);

__device__ __forceinline__ float ex2(float v) { return __builtin_amdgcn_exp2f(v); }

// Over a wave, or over its groups of 2^lg lanes (lg the same in every lane).
__device__ __forceinline__ float wave_max(float v, int lg = 6) {
#pragma unroll
  for (int s = 0; s < 6; ++s) {
    if (s >= lg) break;
    v = fmaxf(v, xor_lanes(v, s));
  }
  return v;
}
__device__ __forceinline__ bool wave_any(bool b, int lg) {
  return wave_max(b ? 1.0f : 0.0f, lg) != 0.0f;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int s = 0; s < 6; ++s) v += xor_lanes(v, s);
  return v;
}
__device__ __forceinline__ double wave_sum(double v, int lg = 6) {
#pragma unroll
  for (int s = 0; s < 6; ++s) {
    if (s >= lg) break;
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __float_as_uint(xor_lanes(__uint_as_float((uint32_t)u), s));
    const uint32_t hi = __float_as_uint(xor_lanes(__uint_as_float((uint32_t)(u >> 32)), s));
    v += __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
  }
  return v;
}

// A row of logits as aligned chunks.
template <typename T>
struct Row {
  const T* z;
  int mis;        // tokens between the aligned address before the row and the row
  uint32_t V;
  uint32_t chunks;
};
template <typename T>
__device__ __forceinline__ Row<T> row_of(const DistillArgs& a, int64_t n) {
  Row<T> r;
  r.z = static_cast<const T*>(a.z) + n * a.stride;
  r.mis = (int)((reinterpret_cast<uintptr_t>(r.z) & 15) / sizeof(T));
  r.V = (uint32_t)a.V;
  r.chunks = (r.V + r.mis + kVec<T> - 1) / kVec<T>;
  return r;
}

template <typename T>
using Chunk = Pack<T, kVec<T>>;

// Chunk j; -Inf where it reaches outside the row.  ONCE: past the caches.
template <typename T, bool ONCE = false>
__device__ __forceinline__ Chunk<T> load_chunk(const Row<T>& r, uint32_t j) {
  const int64_t i0 = (int64_t)j * kVec<T> - r.mis;
  Chunk<T> v;
  if (i0 >= 0 && i0 + kVec<T> <= r.V) {
    if (ONCE) {
      v = load_once<Chunk<T>>(r.z + i0);
    } else {
      const T* p = static_cast<const T*>(__builtin_assume_aligned(r.z + i0, 16));
      __builtin_memcpy(&v, p, 16);
    }
  } else {
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e)
      v.v[e] = i0 + e >= 0 && i0 + e < r.V ? r.z[i0 + e] : (T)kNegInf;
  }
  return v;
}

// Hides where a chunk came from, so that the compiler keeps it packed between
// two passes over it instead of holding its values as f32 (a row of 17 chunks
// per thread would not fit the registers).
template <typename T>
__device__ __forceinline__ void keep_packed(Chunk<T>& v) {
  uint4 u;
  __builtin_memcpy(&u, &v, 16);
  asm volatile("" : "+v"(u.x), "+v"(u.y), "+v"(u.z), "+v"(u.w));
  __builtin_memcpy(&v, &u, 16);
}

// Stores kVec gradients at chunk j of a row of V tokens.
template <typename T>
__device__ __forceinline__ void store_chunk(T* grad, const Row<T>& r, uint32_t j,
                                            const float (&g)[kVec<T>]) {
  const int64_t i0 = (int64_t)j * kVec<T> - r.mis;
  if (i0 >= 0 && i0 + kVec<T> <= r.V) {
    store_once<T, kVec<T>>(grad + i0, g);
  } else {
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e)
      if (i0 + e >= 0 && i0 + e < r.V) grad[i0 + e] = (T)g[e];
  }
}

// ------------------------------------------------------------------ the teacher
//
// LDS of a workgroup: a bitmap, then the K entries.  With a rest the bitmap
// marks the tokens of chunks [c0, c1) of the row; without one it only has to
// find repeated entries, and marks them modulo its size.  Tokens that merely meet
// there cost patch_top a second look, K^2 of LDS reads (10 us of a row with K = 239),
// so the size grows with K: at most one row in four has such a pair up to K = 256,
// and past that no two tokens meet, 2^18 bits being a whole part's (1024 rows of 139000
// with K = 1024: 180 us, 380 where 2^17 bits let one pair of each row meet).
__host__ __device__ inline uint32_t hash_words(int K) {
  return K <= 128 ? 1024 : K <= 181 ? 2048 : K <= 256 ? 4096 : 8192;
}
__host__ __device__ inline uint32_t mark_words(bool tail, int64_t tokens, int K) {
  const uint32_t w = (uint32_t)((tokens + 127) / 128 * 4), h = hash_words(K);
  return !tail && w > h ? h : w;
}

struct Lds {
  uint32_t* bits;  // bit i - c0 * kVec + mis of token i
  int* idx;        // token, -1 where absent
  float* p;        // teacher's probability
  float* z;        // student's logit
};
__device__ __forceinline__ Lds lds_of(char* mem, int K, uint32_t words) {
  Lds l;
  l.bits = reinterpret_cast<uint32_t*>(mem);
  l.idx = reinterpret_cast<int*>(l.bits + words);
  l.p = reinterpret_cast<float*>(l.idx + K);
  l.z = l.p + K;
  return l;
}

// An entry of the lane: token and teacher's logit, whose bits are converted where
// it is used, since that waits for the load.  The first one is loaded ahead of the
// row.
struct Entry {
  int i;
  uint32_t bits;
};
__device__ __forceinline__ uint32_t teacher_bits(const DistillArgs& a, int64_t at) {
  return a.t_type == 0 ? static_cast<const uint32_t*>(a.t)[at]
                       : (uint32_t) static_cast<const uint16_t*>(a.t)[at];
}
__device__ __forceinline__ float teacher_logit(const DistillArgs& a, uint32_t bits) {
  if (a.t_type == 0) return __uint_as_float(bits);
  if (a.t_type == 1) return __uint_as_float(bits << 16);
  return (float)__builtin_bit_cast(f16_t, (uint16_t)bits);
}
__device__ __forceinline__ Entry entry_at(const DistillArgs& a, int64_t n, int k) {
  Entry e = {-1, 0};
  if (k < a.K && n < a.N) {
    e.i = a.tidx[n * a.K + k];
    e.bits = teacher_bits(a, n * a.K + k);
  }
  return e;
}

// Clears the bitmap, by one whole wave.
__device__ __forceinline__ void clear_marks(uint32_t* bits, uint32_t words) {
  for (uint32_t w = 4 * (threadIdx.x & 63); w < words; w += 256)
    *reinterpret_cast<uint4*>(bits + w) = make_uint4(0, 0, 0, 0);
}
// Marks token i if it lies in [lo, hi); whether it was marked before.
template <bool TAIL>
__device__ __forceinline__ bool mark(uint32_t* bits, int K, int i, int64_t lo, int64_t hi) {
  if (i < lo || i >= hi) return false;
  uint32_t bit = (uint32_t)(i - lo);
  if (!TAIL) bit &= 32 * hash_words(K) - 1;
  return (atomicOr(&bits[bit >> 5], 1u << (bit & 31)) >> (bit & 31)) & 1u;
}

// 2^lg lanes of a wave: the entries of a row to LDS, marked in its bitmap
// (cleared before) over chunks [c0, c1).  What comes back is the lane's own share.
struct Entries {
  float tm, z0;  // largest teacher's and student's logits of the entries present
  bool any, dup;
  uint32_t own;  // bit r: the entry of the lane's round r is the first of its token in the span
};
template <typename T, bool TAIL>
__device__ __forceinline__ Entries read_entries(const DistillArgs& a, const Row<T>& r, int64_t n,
                                                const Lds& l, bool marks, uint32_t c0, uint32_t c1,
                                                Entry e, int lg = 6) {
  const int first = threadIdx.x & ((1 << lg) - 1);
  const int64_t lo = (int64_t)c0 * kVec<T> - r.mis;
  const int64_t hi = (int64_t)c1 * kVec<T> - r.mis;
  Entries o = {kNegInf, kNegInf, false, false, 0};
  if (n >= a.N) return o;
  uint32_t round = 1;
  for (int k = first; k < a.K; k += 1 << lg, round <<= 1) {
    if (k != first) e = entry_at(a, n, k);
    const int i = e.i < 0 || e.i >= (int64_t)r.V ? -1 : e.i;
    const float z = i >= 0 ? (float)r.z[i] : kNegInf;
    const float t = teacher_logit(a, e.bits);
    if (i >= 0) {
      o.any = true;
      o.tm = fmaxf(o.tm, t);
      if (marks) {
        const bool again = mark<TAIL>(l.bits, a.K, i, lo, hi);
        o.dup |= again;
        if (!again && i >= lo && i < hi) o.own |= round;
      }
    }
    l.idx[k] = i;
    l.p[k] = t;
    l.z[k] = z;
    o.z0 = fmaxf(o.z0, z);
  }
  return o;
}

// The same lanes: the probabilities to LDS, and the sums over the entries.  The
// K exponentials are taken in f64: the rest 1 - sum p would lose its digits in
// f32 where the top holds nearly everything.
template <bool TAIL>
__device__ __forceinline__ Teacher sum_entries(const DistillArgs& a, int64_t n, const Lds& l,
                                               const Entries& e, int lg = 6) {
  const int first = threadIdx.x & ((1 << lg) - 1);
  const int K = n < a.N ? a.K : 0;
  const float tm = wave_max(e.tm, lg);
  float z0 = wave_max(e.z0, lg);
  if (z0 == kNegInf) z0 = 0.0f;
  // Without a rest: e = exp((t - largest) / tau), p = e / sum e.
  const double ref = TAIL || tm == kNegInf ? 0.0 : (double)tm;
  const double norm = TAIL && n < a.N ? (double)a.tlse[n] : 0.0;
  Teacher o = {0.0, 0.0, 0.0, 0.0, 1.0, z0, false, false};
  for (int k = first; k < K; k += 1 << lg) {
    double p = 0.0;
    if (l.idx[k] >= 0) {
      const double lp = ((double)l.p[k] - ref) * a.inv_tau - norm;
      p = exp(lp);
      if (!(p == 0.0)) {
        o.h += p * lp;
        o.ps += p;
        // the difference first: logits at the type's lowest value cancel
        o.pz += p * ((double)l.z[k] - (double)z0);
      }
    }
    l.p[k] = (float)p;
  }
  o.h = wave_sum(o.h, lg);
  o.ps = wave_sum(o.ps, lg);
  o.pz = wave_sum(o.pz, lg);
  o.any = wave_any(e.any, lg) && o.ps != 0.0;  // entries at -Inf are none
  o.dup = wave_any(e.dup, lg);
  if (TAIL) {
    o.rest = 1.0 - o.ps;
    if (o.rest < 0.0) o.rest = 0.0;
  } else if (o.any) {
    const double inv = 1.0 / o.ps;
    const float scale = (float)inv;
    for (int k = first; k < K; k += 1 << lg) l.p[k] *= scale;
    o.h *= inv;
    o.pz *= inv;
    o.norm = o.ps;
    o.ps = 1.0;
  }
  return o;
}

// The student's side of a row: m and S, m_r and S_r (S_r = 0, m_r = m where no
// token of the rest has mass, or without a rest).
struct Student {
  float m, mr;
  double S, Sr;
};

// The row's loss from the teacher's sums and the student's statistics:
//   sum p (log p - log q) = h - log norm + ps log S - sum p (z - m) / tau
// (norm = 1 with a rest, ps = 1 without one), and the rest's term.
__device__ __forceinline__ float row_loss(const DistillArgs& a, const Teacher& t, const Student& s,
                                          bool tail) {
  const double logS = log(s.S / t.norm);
  double v = t.h + t.ps * logS;
  if (t.ps != 0.0) v -= (t.pz + t.ps * ((double)t.z0 - (double)s.m)) * a.inv_tau;
  if (tail && t.rest > 0.0 && s.Sr != 0.0)
    v += t.rest * (log(t.rest * s.S / s.Sr) - ((double)s.mr - (double)s.m) * a.inv_tau);
  return (float)(v * (double)a.tau * (double)a.tau);
}

// C in f32, by every thread.  With one maximum it is (S_r - p_r S) / (S S_r), the
// difference taken as (1 - p_r) S_r - p_r S_t with S_t = S - S_r: S_r and p_r S agree
// in most of their digits where the top holds little or tau is large.
template <bool TAIL>
__device__ __forceinline__ float rest_coef(const DistillArgs& a, float m, float S, float mr,
                                           float Sr, float St, double p_rest) {
  if (!TAIL) return 1.0f / S;
  if (Sr == 0.0f) return 0.0f;
  const float pr = (float)p_rest, pt = (float)(1.0 - p_rest);
  if (mr == m) return (pt * Sr - pr * St) / (S * Sr);
  return ex2((mr - m) * a.c) / S - pr / Sr;
}

// What a row's gradient needs from the forward pass: m, S (0: the row has no
// loss), m_r, C, behind which its probabilities p_k stand.
template <bool TAIL>
__device__ __forceinline__ void save_row(const DistillArgs& a, int64_t n, bool dead,
                                         const Student& s, double p_rest) {
  float C = 0.0f;
  if (!TAIL) {
    C = 1.0f / (float)s.S;
  } else if (s.Sr != 0.0) {
    const double e = s.mr == s.m ? 1.0 : exp(((double)s.mr - (double)s.m) * a.inv_tau);
    C = (float)(e * s.Sr - p_rest * s.S) / (float)(s.S * s.Sr);
  }
  float* to = a.saved + n * (4 + a.K);
  to[0] = s.m;
  to[1] = dead ? 0.0f : (float)s.S;
  to[2] = s.mr;
  to[3] = dead ? 0.0f : C;
}

// Where the rest's sum against the row's largest logit is below this, it is taken
// again against its own: above, what its smallest terms lose to underflow is less
// than 2^-42 of it (2^24 terms below 2^-126).
// Rows without such a distance pay nothing for it (8192 x 65536 bf16: 403 us), rows
// with it two more passes over their registers (583).
constexpr float kFar = 0x1p-60f;

// Puts right the gradient at the teacher's tokens within [lo, hi).
template <typename T>
__device__ __forceinline__ void patch_top(const DistillArgs& a, const Lds& l, T* grad, float m,
                                          float S, float scale, bool dup, int64_t lo, int64_t hi,
                                          int first, int step) {
  for (int k = first; k < a.K; k += step) {
    const int i = l.idx[k];
    if (i < 0 || i < lo || i >= hi) continue;
    float p = l.p[k];
    if (dup) {  // every entry of the token writes the same sum
      p = 0.0f;
      for (int q = 0; q < a.K; ++q)
        if (l.idx[q] == i) p += l.p[q];
    }
    grad[i] = (T)(scale * (ex2((l.z[k] - m) * a.c) / S - p));
  }
}

// Marks of chunk j (bit e: its token e is in the top), j counted from c0.
template <typename T>
__device__ __forceinline__ uint32_t chunk_bits(const uint32_t* bits, uint32_t j) {
  const uint32_t at = j * kVec<T>;
  return (bits[at >> 5] >> (at & 31)) & ((1u << kVec<T>) - 1);
}

// Adds exp((z - m) / tau) of a chunk to the rest's sum, or to the top's.
template <typename T, bool TAIL>
__device__ __forceinline__ void add_chunk(const Chunk<T>& v, float m, float c, uint32_t marks,
                                          float& rest, float& top) {
  float z[kVec<T>], sum = 0.0f;
  unpack(v, z);
  if (!TAIL || marks == 0) {
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) sum += ex2((z[e] - m) * c);
  } else {
#pragma unroll
    for (int e = 0; e < kVec<T>; ++e) {
      const float x = ex2((z[e] - m) * c);
      if ((marks >> e) & 1u) top += x;
      else sum += x;
    }
  }
  rest += sum;
}

// A chunk's largest logit and m, and its sum against m, without its marked tokens.
template <typename T>
__device__ __forceinline__ float rest_max(const Chunk<T>& v, uint32_t marks, float m) {
  float z[kVec<T>];
  unpack(v, z);
#pragma unroll
  for (int e = 0; e < kVec<T>; ++e) m = (marks >> e) & 1u ? m : fmaxf(m, z[e]);
  return m;
}
template <typename T>
__device__ __forceinline__ float rest_sum(const Chunk<T>& v, uint32_t marks, float m, float c) {
  float z[kVec<T>], s = 0.0f;
  unpack(v, z);
#pragma unroll
  for (int e = 0; e < kVec<T>; ++e) s += (marks >> e) & 1u ? 0.0f : ex2((z[e] - m) * c);
  return s;
}

// ------------------------------------------------- one workgroup holds the row
//
// NT threads hold the row, R chunks each, so it is read once: the largest logit,
// the sum and the gradient are three passes over registers.  512 threads of 17
// chunks leave room for two rows to a CU, one loading while the other stores (8192
// x 65536 bf16, fused: 388-412 us, 5.4 TB/s; with one row of 1024 threads to a CU
// 637 us).  With SIDE one more wave reads the teacher beside them (its chain of loads
// and f64 exponentials is as long as the row's own), else the first wave does.
// Gradients are stored past the caches: 64 MB 42.8 -> 34.6 us, and the products
// that read them next take no longer (1 GB with both products of the head: 2915
// us stored through, 2909 past).
template <typename T, int NT, int R, bool TAIL, bool SIDE>
__global__ __launch_bounds__(SIDE ? NT + 64 : NT, NT < 512 ? 1 : 4)
void distill_row_kernel(DistillArgs a) {
  extern __shared__ __attribute__((aligned(16))) char mem[];
  __shared__ float red[3][NT / 64];
  __shared__ double wide[2][NT / 64];  // the waves' sums over the rest and over all tokens
  __shared__ Teacher t;  // kept here, not in registers across the passes
  const int64_t n = blockIdx.x;
  const int tid = threadIdx.x, wv = tid >> 6;
  const bool row_wave = !SIDE || wv < NT / 64;
  const bool teacher_wave = wv == (SIDE ? NT / 64 : 0);
  const Row<T> r = row_of<T>(a, n);
  T* grad = static_cast<T*>(a.grad) + n * a.grad_stride;
  Entry first = {-1, 0};
  if (SIDE && teacher_wave) first = entry_at(a, n, tid & 63);
  const float w = a.weight ? a.weight[n] : 1.0f;
  if (w == 0.0f) {
    const float zero[kVec<T>] = {};
    for (uint32_t j = tid; j < r.chunks; j += blockDim.x) store_chunk(grad, r, j, zero);
    if (tid == 0) a.loss[n] = 0.0f;
    return;
  }
  const uint32_t words = mark_words(TAIL, (int64_t)r.chunks * kVec<T>, a.K);
  const Lds l = lds_of(mem, a.K, words);
  Entries entries;
  auto sums = [&] {
    const Teacher o = sum_entries<TAIL>(a, n, l, entries);
    if ((tid & 63) == 0) t = o;
  };
  auto read_teacher = [&] {
    if (!teacher_wave) return;
    clear_marks(l.bits, words);
    if (!SIDE) first = entry_at(a, n, tid & 63);
    entries = read_entries<T, TAIL>(a, r, n, l, true, 0, r.chunks, first);
    if (!SIDE) sums();
  };
  // With SIDE the row's loads go out first.  Without it they would take registers
  // that the first wave's f64 exponentials need: with the teacher first, three rows
  // of 9 chunks a thread are on a CU, and two the other way (4096 x 32768 bf16: 105
  // and 128 us; four and three of 7 chunks, 4096 x 26000 with a rest: 91 and 100).
  if (!SIDE) read_teacher();
  Chunk<T> v[R];
  if (row_wave) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const uint32_t j = tid + q * NT;
      if (j < r.chunks) {
        // Never with SIDE.  The branch stays in those variants for the code it
        // makes, with the same traffic: 8192 x 10000 bf16 77 us, 84 without, 4096 x
        // 10000 38 and 43, but 512 x 24000 15.9 and 13.7.
        v[q] = a.once ? load_chunk<T, true>(r, j) : load_chunk(r, j);
      } else {
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e) v[q].v[e] = (T)kNegInf;
      }
    }
  }
  if (SIDE) read_teacher();
  float m = kNegInf;
  if (row_wave) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float z[kVec<T>];
      unpack(v[q], z);
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e) m = fmaxf(m, z[e]);
      keep_packed<T>(v[q]);
    }
    m = wave_max(m);
    if ((tid & 63) == 0) red[0][wv] = m;
  }
  __syncthreads();
  if (SIDE && teacher_wave) sums();  // beside the row's own
  m = red[0][0];
#pragma unroll
  for (int q = 1; q < NT / 64; ++q) m = fmaxf(m, red[0][q]);
  if (m == kNegInf) m = 0.0f;
  float rest = 0.0f, top = 0.0f;
  if (row_wave) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const uint32_t j = tid + q * NT;
      if (j < r.chunks)
        add_chunk<T, TAIL>(v[q], m, a.c, TAIL ? chunk_bits<T>(l.bits, j) : 0u, rest, top);
      keep_packed<T>(v[q]);
    }
    const double wr = wave_sum((double)rest), wt = TAIL ? wave_sum((double)top) : 0.0;
    if ((tid & 63) == 0) {
      red[1][wv] = (float)wr;
      red[2][wv] = (float)wt;
      wide[0][wv] = wr;
      wide[1][wv] = wr + wt;
    }
  }
  __syncthreads();
  rest = top = 0.0f;
#pragma unroll
  for (int q = 0; q < NT / 64; ++q) {
    rest += red[1][q];
    if (TAIL) top += red[2][q];
  }
  const float S = rest + top;
  float mr = m;
  if (TAIL && rest < kFar) {  // the same in every thread
    if (row_wave) {
      mr = kNegInf;
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const uint32_t j = tid + q * NT;
        if (j < r.chunks) mr = rest_max<T>(v[q], chunk_bits<T>(l.bits, j), mr);
        keep_packed<T>(v[q]);
      }
      mr = wave_max(mr);
      if ((tid & 63) == 0) red[0][wv] = mr;
    }
    __syncthreads();
    mr = red[0][0];
#pragma unroll
    for (int q = 1; q < NT / 64; ++q) mr = fmaxf(mr, red[0][q]);
    rest = 0.0f;
    if (mr == kNegInf) {
      mr = m;
    } else {
      if (row_wave) {
#pragma unroll
        for (int q = 0; q < R; ++q) {
          const uint32_t j = tid + q * NT;
          if (j < r.chunks) rest += rest_sum<T>(v[q], chunk_bits<T>(l.bits, j), mr, a.c);
          keep_packed<T>(v[q]);
        }
        const double wr = wave_sum((double)rest);
        if ((tid & 63) == 0) {
          red[1][wv] = (float)wr;
          wide[0][wv] = wr;
        }
      }
      __syncthreads();
      rest = 0.0f;
#pragma unroll
      for (int q = 0; q < NT / 64; ++q) rest += red[1][q];
    }
  }
  const bool dead = S == 0.0f || (!TAIL && !t.any);
  const float scale = dead ? 0.0f : w * a.tau;
  const float coef = dead ? 0.0f : scale * rest_coef<TAIL>(a, m, S, mr, rest, top, t.rest);
  if (row_wave) {
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const uint32_t j = tid + q * NT;
      if (j < r.chunks) {
        float z[kVec<T>], g[kVec<T>];
        unpack(v[q], z);
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e) g[e] = dead ? 0.0f : coef * ex2((z[e] - mr) * a.c);
        store_chunk(grad, r, j, g);
      }
    }
  }
  if (teacher_wave) {
    Student st = {m, mr, 0.0, 0.0};
    for (int q = 0; q < NT / 64; ++q) {
      st.S += wide[1][q];
      st.Sr += rest == 0.0f ? 0.0 : wide[0][q];
    }
    const float loss = dead ? 0.0f : row_loss(a, t, st, TAIL);
    if ((tid & 63) == 0) a.loss[n] = loss;
  }
  __syncthreads();
  if (!dead) patch_top(a, l, grad, m, S, scale, t.dup, 0, (int64_t)r.V, tid, blockDim.x);
}

// ------------------------------------------------------ rows taken in parts
//
// Rows longer than a workgroup's registers, few rows, and the two calls apart: 256
// threads go over a part's chunks, one more wave takes the entries.  A row's parts
// meet in a second launch of one wave per row (16 x 131071 bf16 with a rest: 5.8 +
// 3.6 us, and 5.2 for the gradient; 4096 x 32768, forward and backward: 154 us, 5.2
// TB/s over three readings and writings).  With a rest the row's waves see only its
// tokens, and the extra wave sums the top's, each once (4096 x 32768: 165 us; with the
// top in the row's waves 201).
constexpr int kPartThreads = 256;
constexpr int kBatch = 2;  // chunks a thread loads at once

// Chunks [c0, c1) of the workgroup's part.
struct Span {
  uint32_t c0, c1;
};
template <typename T>
__device__ __forceinline__ Span span_of(const DistillArgs& a, const Row<T>& r, int split) {
  const uint32_t per = (r.chunks + a.splits - 1) / a.splits;
  Span s;
  s.c0 = (uint32_t)split * per < r.chunks ? (uint32_t)split * per : r.chunks;
  s.c1 = s.c0 + per < r.chunks ? s.c0 + per : r.chunks;
  return s;
}

template <typename T>
__device__ __forceinline__ void load_batch(const Row<T>& r, uint32_t j0, uint32_t c1,
                                           Chunk<T> (&v)[kBatch]) {
#pragma unroll
  for (int q = 0; q < kBatch; ++q) {
    const uint32_t j = j0 + q * kPartThreads;
    if (j < c1) {
      v[q] = load_chunk(r, j);
    } else {
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e) v[q].v[e] = (T)kNegInf;
    }
  }
}

// Statistics of a part: largest logit and sum of exp((z - largest) / tau) over the
// tokens of the rest (of all tokens without one), and over the top's.
struct Part {
  float mr, mt;
  double rest, top;
};
static_assert(sizeof(Part) == 24, "the workspace counts 24 bytes");
constexpr Part kNoPart = {kNegInf, kNegInf, 0.0, 0.0};

// Factor that takes a sum against `from` to one against `to`, where `to` is not
// smaller.  -Inf comes with a sum of 0, or NaN where nothing but NaN was seen.  A
// thread's sum is moved in f32, one of many whose errors average; a part's in f64.
__device__ __forceinline__ float shift(float from, float to, float sum, float c) {
  return from == kNegInf ? (sum == sum ? 0.0f : 1.0f) : ex2((from - to) * c);
}
__device__ __forceinline__ double moved(float from, float to, double sum, double inv_tau) {
  if (from == kNegInf) return sum == sum ? 0.0 : sum;
  return from == to ? sum : sum * exp(((double)from - (double)to) * inv_tau);
}

// A row's loss and what its gradient needs, by one wave.
template <bool TAIL>
__device__ __forceinline__ void finish_row(const DistillArgs& a, int64_t n, bool off,
                                           const Teacher& t, const Part& p) {
  Student s;
  s.m = TAIL ? fmaxf(p.mr, p.mt) : p.mr;
  s.S = moved(p.mr, s.m, p.rest, a.inv_tau);
  if (TAIL) s.S += moved(p.mt, s.m, p.top, a.inv_tau);
  if (s.m == kNegInf) s.m = 0.0f;
  s.mr = p.mr == kNegInf ? s.m : p.mr;
  s.Sr = p.rest;
  const bool dead = off || s.S == 0.0 || (!TAIL && !t.any);
  const float loss = dead ? 0.0f : row_loss(a, t, s, TAIL);
  if ((threadIdx.x & 63) == 0) {
    a.loss[n] = loss;
    if (a.saved) save_row<TAIL>(a, n, dead, s, t.rest);
  }
}

// Takes the marked tokens out of a chunk: -Inf has no mass.  Once per chunk here;
// where a row stays in registers, the selects of rest_max and rest_sum take fewer.
template <typename T>
__device__ __forceinline__ void drop_top(Chunk<T>& v, uint32_t marks) {
  if (marks == 0) return;
#pragma unroll
  for (int e = 0; e < kVec<T>; ++e) v.v[e] = (marks >> e) & 1u ? (T)kNegInf : v.v[e];
}

// Largest logit and sums of one part of a row; the first part's extra wave
// reads the teacher.
template <typename T, bool TAIL>
__global__ __launch_bounds__(kPartThreads + 64) void distill_part_kernel(DistillArgs a) {
  extern __shared__ __attribute__((aligned(16))) char mem[];
  __shared__ float red[kPartThreads / 64];
  __shared__ double sums_of[kPartThreads / 64];
  __shared__ float top_mt;
  __shared__ double top_sum;
  __shared__ Teacher whole;  // where the part is the row
  const int64_t n = blockIdx.x / (uint32_t)a.splits;
  const int split = (int)(blockIdx.x % (uint32_t)a.splits);
  const int tid = threadIdx.x, wv = tid >> 6;
  const bool row_wave = wv < kPartThreads / 64;
  Part* part = static_cast<Part*>(a.part) + blockIdx.x;
  if (a.weight && a.weight[n] == 0.0f) {
    if (tid == 0) *part = kNoPart;
    if (a.splits == 1 && !row_wave) finish_row<TAIL>(a, n, true, Teacher{}, kNoPart);
    return;
  }
  const Row<T> r = row_of<T>(a, n);
  const Span s = span_of(a, r, split);
  const uint32_t words = TAIL ? mark_words(true, (int64_t)(s.c1 - s.c0) * kVec<T>, a.K) : 0;
  const Lds l = lds_of(mem, a.K, words);
  Chunk<T> v[kBatch];
  Entries entries;
  if (row_wave) {
    load_batch(r, s.c0 + tid, s.c1, v);
  } else {
    if (split == 0) {
      const Entry first = entry_at(a, n, tid & 63);
      clear_marks(l.bits, words);
      entries = read_entries<T, TAIL>(a, r, n, l, TAIL, s.c0, s.c1, first);
    } else if (TAIL) {
      const int64_t lo = (int64_t)s.c0 * kVec<T> - r.mis, hi = (int64_t)s.c1 * kVec<T> - r.mis;
      clear_marks(l.bits, words);
      entries.own = 0;
      uint32_t round = 1;
      for (int k = tid & 63; k < a.K; k += 64, round <<= 1) {
        const int i = a.tidx[n * a.K + k];
        if (i < 0 || i >= (int64_t)r.V || i < lo || i >= hi) continue;
        l.z[k] = (float)r.z[i];
        if (!mark<true>(l.bits, a.K, i, lo, hi)) entries.own |= round;
      }
    }
  }
  if (TAIL) __syncthreads();
  if (!row_wave && split == 0) {
    const Teacher t = sum_entries<TAIL>(a, n, l, entries);
    if ((tid & 63) == 0) (a.splits == 1 ? whole : a.teacher[n]) = t;
    if (a.saved)
      for (int k = tid & 63; k < a.K; k += 64) a.saved[n * (4 + a.K) + 4 + k] = l.p[k];
  }
  if (TAIL && !row_wave) {  // the top's tokens of the part, each once
    float mt = kNegInf, top = 0.0f;
    uint32_t own = entries.own;
    for (int k = tid & 63; k < a.K; k += 64, own >>= 1)
      if (own & 1u) mt = fmaxf(mt, l.z[k]);
    mt = wave_max(mt);
    own = entries.own;
    for (int k = tid & 63; k < a.K; k += 64, own >>= 1)
      if (own & 1u) top += ex2((l.z[k] - (mt == kNegInf ? 0.0f : mt)) * a.c);
    const double sum = wave_sum((double)top);
    if ((tid & 63) == 0) top_mt = mt, top_sum = sum;
  }
  float m = kNegInf, rest = 0.0f;
  if (row_wave) {
    for (uint32_t j0 = s.c0 + tid; j0 < s.c1; j0 += kBatch * kPartThreads) {
      float mb = m;
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const uint32_t j = j0 + q * kPartThreads;
        if (TAIL && j < s.c1) drop_top<T>(v[q], chunk_bits<T>(l.bits, j - s.c0));
        mb = rest_max<T>(v[q], 0, mb);
      }
      if (mb > m) {
        rest *= shift(m, mb, rest, a.c);
        m = mb;
      }
      const float ms = m == kNegInf ? 0.0f : m;
      float sum = 0.0f;  // so a thread adds at most 128 of these, of a part's 2^18 tokens
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const uint32_t j = j0 + q * kPartThreads;
        if (j < s.c1) sum += rest_sum<T>(v[q], 0, ms, a.c);
      }
      rest += sum;
      if (j0 + kBatch * kPartThreads < s.c1) load_batch(r, j0 + kBatch * kPartThreads, s.c1, v);
    }
    const float mw = wave_max(m);
    if ((tid & 63) == 0) red[wv] = mw;
  }
  __syncthreads();
  Part all = kNoPart;
#pragma unroll
  for (int q = 0; q < kPartThreads / 64; ++q) all.mr = fmaxf(all.mr, red[q]);
  if (TAIL) all.mt = top_mt, all.top = top_sum;
  if (row_wave) {
    const double sum = wave_sum((double)rest * (double)shift(m, all.mr, rest, a.c));
    if ((tid & 63) == 0) sums_of[wv] = sum;
  }
  __syncthreads();
  if (a.splits == 1 ? row_wave : tid != 0) return;
#pragma unroll
  for (int q = 0; q < kPartThreads / 64; ++q) all.rest += sums_of[q];
  if (a.splits == 1) finish_row<TAIL>(a, n, false, whole, all);
  else *part = all;
}

// Joins a row's parts; one wave per row.
template <bool TAIL>
__global__ __launch_bounds__(64) void distill_join_kernel(DistillArgs a) {
  const int64_t n = blockIdx.x;
  const int lane = threadIdx.x;
  const Part* part = static_cast<const Part*>(a.part) + n * a.splits;
  const bool off = a.weight && a.weight[n] == 0.0f;
  Teacher t = {0.0, 0.0, 0.0, 0.0, 1.0, 0.0f, false, false};
  if (!off) t = a.teacher[n];
  Part all = kNoPart;
  for (int q = lane; q < a.splits; q += 64) {
    all.mr = fmaxf(all.mr, part[q].mr);
    if (TAIL) all.mt = fmaxf(all.mt, part[q].mt);
  }
  all.mr = wave_max(all.mr);
  if (TAIL) all.mt = wave_max(all.mt);
  for (int q = lane; q < a.splits; q += 64) {
    const Part p = part[q];
    all.rest += moved(p.mr, all.mr, p.rest, a.inv_tau);
    if (TAIL) all.top += moved(p.mt, all.mt, p.top, a.inv_tau);
  }
  all.rest = wave_sum(all.rest);
  if (TAIL) all.top = wave_sum(all.top);
  finish_row<TAIL>(a, n, off, t, all);
}

constexpr int kAhead = 4;  // entries a lane loads at once

// Gradient of one part of a row from its saved statistics and probabilities.
template <typename T, bool TAIL>
__global__ __launch_bounds__(kPartThreads + 64) void distill_grad_kernel(DistillArgs a) {
  extern __shared__ __attribute__((aligned(16))) char mem[];
  __shared__ uint32_t sh_dup;
  const int64_t n = blockIdx.x / (uint32_t)a.splits;
  const int tid = threadIdx.x, wv = tid >> 6;
  const bool row_wave = wv < kPartThreads / 64;
  const Row<T> r = row_of<T>(a, n);
  const Span s = span_of(a, r, (int)(blockIdx.x % (uint32_t)a.splits));
  const int64_t lo = (int64_t)s.c0 * kVec<T> - r.mis, hi = (int64_t)s.c1 * kVec<T> - r.mis;
  T* grad = static_cast<T*>(a.grad) + n * a.grad_stride;
  const float* saved = a.saved + n * (4 + a.K);
  const float w = a.weight ? a.weight[n] : 1.0f;
  const float m = saved[0], S = saved[1], mr = saved[2];
  if (w == 0.0f || S == 0.0f) {
    const float zero[kVec<T>] = {};
    for (uint32_t j = s.c0 + tid; j < s.c1; j += kPartThreads + 64) store_chunk(grad, r, j, zero);
    return;
  }
  const uint32_t words = mark_words(false, (int64_t)(s.c1 - s.c0) * kVec<T>, a.K);
  const Lds l = lds_of(mem, a.K, words);
  Chunk<T> v[kBatch];
  if (row_wave) {
    load_batch(r, s.c0 + tid, s.c1, v);
  } else {
    bool dup = false;
    clear_marks(l.bits, words);
    for (int k0 = tid & 63; k0 < a.K; k0 += 64 * kAhead) {
      int i[kAhead];
      float p[kAhead], z[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + 64 * u;
        i[u] = k < a.K ? a.tidx[n * a.K + k] : -1;
        p[u] = k < a.K ? saved[4 + k] : 0.0f;
        if (i[u] >= (int64_t)r.V || i[u] < lo || i[u] >= hi) i[u] = -1;
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) z[u] = i[u] >= 0 ? (float)r.z[i[u]] : 0.0f;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int k = k0 + 64 * u;
        if (k >= a.K) break;
        l.idx[k] = i[u];
        l.p[k] = p[u];
        l.z[k] = z[u];
        if (i[u] >= 0) dup |= mark<false>(l.bits, a.K, i[u], lo, hi);
      }
    }
    const bool any = __any(dup);
    if ((tid & 63) == 0) sh_dup = any;
  }
  __syncthreads();  // the top's logits are read before they may be overwritten
  const float scale = w * a.tau;
  if (row_wave) {
    const float coef = scale * saved[3];
    for (uint32_t j0 = s.c0 + tid; j0 < s.c1; j0 += kBatch * kPartThreads) {
#pragma unroll
      for (int q = 0; q < kBatch; ++q) {
        const uint32_t j = j0 + q * kPartThreads;
        if (j < s.c1) {
          float z[kVec<T>], g[kVec<T>];
          unpack(v[q], z);
#pragma unroll
          for (int e = 0; e < kVec<T>; ++e) g[e] = coef * ex2((z[e] - mr) * a.c);
          store_chunk(grad, r, j, g);
        }
      }
      if (j0 + kBatch * kPartThreads < s.c1) load_batch(r, j0 + kBatch * kPartThreads, s.c1, v);
    }
  }
  __syncthreads();
  patch_top(a, l, grad, m, S, scale, sh_dup != 0, lo, hi, tid, blockDim.x);
}

// ---------------------------------------------------------- one wave per row
//
// Rows of up to 256 chunks, or more where there are many, four to a workgroup, each
// within one wave, which needs no barrier for its maximum and sums.  One more wave
// reads the four teachers at once, K entries of a row on the next power of two of
// lanes: the f64 arithmetic of a row, spent by a whole wave on each, took longer
// than the row itself (16384 x 500 bf16, K = 16: 27.6 -> 18-20 us).  Where K leaves it
// fewer than four rows, two or four waves do (610 x 457 f16, K = 102: 13.9 -> 6.4 us,
// 16384 x 500 bf16 with a rest, K = 64: 55 -> 29).
enum Pass { kFused, kLoss, kGradient };
constexpr int kWaveRows = 4;

// Lanes for the K entries of a row (log2), and the waves that take four rows'.
__host__ __device__ inline int entry_lanes(int K) {
  int lg = 0;
  while (lg < 6 && (1 << lg) < K) ++lg;
  return lg;
}
int teacher_waves(int K) {
  const int per = 64 >> entry_lanes(K);
  return per >= kWaveRows ? 1 : kWaveRows / per;
}

template <typename T, int R, bool TAIL, int PASS>
__global__ __launch_bounds__(PASS == kGradient ? 64 * kWaveRows : 128 * kWaveRows, R == 12 ? 4 : 1)
void distill_wave_kernel(DistillArgs a, uint32_t words) {
  extern __shared__ __attribute__((aligned(16))) char mem[];
  __shared__ Student stat[kWaveRows];
  __shared__ Teacher teachers[kWaveRows];
  const int lane = threadIdx.x & 63;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * kWaveRows;
  auto lds_row = [&](int q) {
    return lds_of(mem + (size_t)q * 4 * (words + 3 * (size_t)((a.K + 3) / 4 * 4)), a.K, words);
  };
  if (PASS != kGradient && wv >= kWaveRows) {  // the teachers
    const int lg = entry_lanes(a.K), k0 = lane & ((1 << lg) - 1);
    const int q = ((wv - kWaveRows) << (6 - lg)) + (lane >> lg);
    const int64_t n = q < kWaveRows ? n0 + q : a.N;
    const Entry first = entry_at(a, n, k0);
    const int own = kWaveRows / ((int)(blockDim.x >> 6) - kWaveRows);  // rows of the wave
    for (int b = 0; b < own; ++b) clear_marks(lds_row((wv - kWaveRows) * own + b).bits, words);
    const Row<T> r = row_of<T>(a, n < a.N ? n : n0);
    const Lds l = lds_row(q < kWaveRows ? q : 0);
    const Entries e = read_entries<T, TAIL>(a, r, n, l, true, 0, r.chunks, first, lg);
    if (TAIL) __syncthreads();
    const Teacher t = sum_entries<TAIL>(a, n, l, e, lg);
    if (q < kWaveRows && k0 == 0) teachers[q] = t;
    if (PASS == kLoss && a.saved && n < a.N)
      for (int k = k0; k < a.K; k += 1 << lg) a.saved[n * (4 + a.K) + 4 + k] = l.p[k];
    __syncthreads();
    if (q < kWaveRows && k0 == 0 && n < a.N) {
      const float w = PASS == kFused && a.weight ? a.weight[n] : 1.0f;
      const Student s = stat[q];
      const bool dead = w == 0.0f || s.S == 0.0 || (!TAIL && !t.any);
      a.loss[n] = dead ? 0.0f : row_loss(a, t, s, TAIL);
      if (PASS == kLoss && a.saved) save_row<TAIL>(a, n, dead, s, t.rest);
    }
    return;
  }

  const int64_t n = n0 + wv;
  const bool here = n < a.N;
  const Row<T> r = row_of<T>(a, here ? n : n0);
  const Lds l = lds_row(wv);
  T* grad = static_cast<T*>(a.grad) + n * a.grad_stride;
  const float w = !here ? 0.0f : PASS != kLoss && a.weight ? a.weight[n] : 1.0f;
  Chunk<T> v[R];
#pragma unroll
  for (int q = 0; q < R; ++q) {
    const uint32_t j = lane + q * 64;
    if (w != 0.0f && j < r.chunks) {
      v[q] = load_chunk(r, j);
    } else {
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e) v[q].v[e] = (T)kNegInf;
    }
  }
  float m, S, mr, coef = 0.0f;
  bool dead, dup;
  if (PASS == kGradient) {
    const float* saved = a.saved + (here ? n : 0) * (4 + a.K);
    m = saved[0];
    S = saved[1];
    mr = saved[2];
    coef = saved[3];
    dead = w == 0.0f || S == 0.0f;
    dup = false;
    clear_marks(l.bits, words);
    for (int k = lane; k < a.K && !dead; k += 64) {
      const int i = a.tidx[n * a.K + k];
      const bool ok = i >= 0 && i < (int64_t)r.V;
      l.idx[k] = ok ? i : -1;
      l.p[k] = saved[4 + k];
      if (ok) {
        l.z[k] = (float)r.z[i];
        dup |= mark<false>(l.bits, a.K, i, 0, (int64_t)r.V);
      }
    }
    dup = __any(dup);
  } else {
    m = kNegInf;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      float z[kVec<T>];
      unpack(v[q], z);
#pragma unroll
      for (int e = 0; e < kVec<T>; ++e) m = fmaxf(m, z[e]);
    }
    m = wave_max(m);
    if (m == kNegInf) m = 0.0f;
    if (TAIL) __syncthreads();  // the marks
    float rest = 0.0f, top = 0.0f;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const uint32_t j = lane + q * 64;
      if (w != 0.0f && j < r.chunks)
        add_chunk<T, TAIL>(v[q], m, a.c, TAIL ? chunk_bits<T>(l.bits, j) : 0u, rest, top);
    }
    mr = m;
    double wr = wave_sum((double)rest);
    const double wt = TAIL ? wave_sum((double)top) : 0.0, ws = wr + wt;
    if (TAIL && w != 0.0f && wr < kFar) {  // the same in every lane
      mr = kNegInf;
#pragma unroll
      for (int q = 0; q < R; ++q) {
        const uint32_t j = lane + q * 64;
        if (j < r.chunks) mr = rest_max<T>(v[q], chunk_bits<T>(l.bits, j), mr);
      }
      mr = wave_max(mr);
      rest = 0.0f;
      if (mr == kNegInf) {
        mr = m;
      } else {
#pragma unroll
        for (int q = 0; q < R; ++q) {
          const uint32_t j = lane + q * 64;
          if (j < r.chunks) rest += rest_sum<T>(v[q], chunk_bits<T>(l.bits, j), mr, a.c);
        }
      }
      wr = wave_sum((double)rest);
    }
    S = (float)ws;
    if (lane == 0) stat[wv] = {m, mr, ws, wr};
    __syncthreads();  // the teachers, whose logits are read before they may be overwritten
    const Teacher t = teachers[wv];
    dead = w == 0.0f || S == 0.0f || (!TAIL && !t.any);
    dup = t.dup;
    if (PASS == kFused) coef = rest_coef<TAIL>(a, m, S, mr, (float)wr, (float)wt, t.rest);
  }
  if (PASS != kLoss && here) {
    const float scale = dead ? 0.0f : w * a.tau;
    coef = dead ? 0.0f : scale * coef;
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const uint32_t j = lane + q * 64;
      if (j < r.chunks) {
        float z[kVec<T>], g[kVec<T>];
        unpack(v[q], z);
#pragma unroll
        for (int e = 0; e < kVec<T>; ++e) g[e] = dead ? 0.0f : coef * ex2((z[e] - mr) * a.c);
        store_chunk(grad, r, j, g);
      }
    }
    if (!dead) patch_top(a, l, grad, m, S, scale, dup, 0, (int64_t)r.V, lane, 64);
  }
}

size_t lds_bytes(int K, bool tail, int64_t tokens) {
  return (size_t)K * 12 + (size_t)mark_words(tail, tokens, K) * 4;
}

int elem_size(int type) { return type == 0 ? 4 : 2; }

// Tokens of the largest part, whole chunks.
int64_t part_tokens(const DistillArgs& a, int type) {
  const int vec = 16 / elem_size(type);
  const int64_t chunks = (a.V + vec - 1 + vec - 1) / vec;
  return (chunks + a.splits - 1) / a.splits * vec;
}

template <typename T, int NT, int R, bool SIDE>
hipError_t row_launch(const DistillArgs& a, hipStream_t s) {
  const size_t lds = lds_bytes(a.K, a.tlse != nullptr, a.V + 2 * kVec<T>);
  const dim3 grid((uint32_t)a.N), block(SIDE ? NT + 64 : NT);
  return a.tlse ? enqueue(distill_row_kernel<T, NT, R, true, SIDE>, grid, block, lds, s, a)
                : enqueue(distill_row_kernel<T, NT, R, false, SIDE>, grid, block, lds, s, a);
}

// Whether the wave kernel takes rows of so many chunks.  From 1024 rows on there are
// enough waves to hide its loads: 16384 x 4000 bf16 75 us, 80 by workgroups; 64 x 4000
// 8 and 6.  The two calls apart gain more, since a row has no parts to join (1500 x
// 5900 bf16 with a rest 22 us, 30 in parts; 6000 x 5900 69 and 67; fused 46 and 41).
bool by_waves(int64_t N, int64_t chunks, bool fused) {
  return chunks <= (N < 1024 ? 256 : fused ? 512 : 768);
}

template <typename T, int PASS, bool TAIL>
hipError_t wave_launch(const DistillArgs& a, hipStream_t s) {
  const int64_t chunks = (a.V + 2 * kVec<T> - 2) / kVec<T>;  // at most, for any alignment
  const uint32_t words = mark_words(TAIL, chunks * kVec<T>, a.K);
  const size_t lds = (size_t)kWaveRows * 4 * (words + 3 * (size_t)((a.K + 3) / 4 * 4));
  const dim3 grid((uint32_t)((a.N + kWaveRows - 1) / kWaveRows));
  const dim3 block(64 * (PASS == kGradient ? kWaveRows : kWaveRows + teacher_waves(a.K)));
  if (chunks <= 64)
    return enqueue(distill_wave_kernel<T, 1, TAIL, PASS>, grid, block, lds, s, a, words);
  if constexpr (PASS != kFused)
    if (chunks > 512)
      return enqueue(distill_wave_kernel<T, 12, TAIL, PASS>, grid, block, lds, s, a, words);
  if (chunks > 256)
    return enqueue(distill_wave_kernel<T, 8, TAIL, PASS>, grid, block, lds, s, a, words);
  return enqueue(distill_wave_kernel<T, 4, TAIL, PASS>, grid, block, lds, s, a, words);
}
template <typename T, int PASS>
hipError_t wave_typed(const DistillArgs& a, hipStream_t s) {
  return a.tlse ? wave_launch<T, PASS, true>(a, s) : wave_launch<T, PASS, false>(a, s);
}

template <typename T>
hipError_t row_typed(DistillArgs a, hipStream_t s) {
  const int64_t chunks = (a.V + 2 * kVec<T> - 2) / kVec<T>;
  if (by_waves(a.N, chunks, true)) return wave_typed<T, kFused>(a, s);
  // Few chunks to a thread and few threads leave room for more rows on a CU (4096 x
  // 10000 bf16: 512 x 9 64 us, 512 x 4 48, 256 x 6 43; 4096 x 20000: 512 x 9 93 us,
  // 512 x 7 75), more threads are faster where each CU has two rows or fewer (512 x
  // 10000 with a rest: 256 x 8 10.3 us, 512 x 4 9.5).  The teacher's extra wave pays
  // in the small workgroups (512 x 11000 with a rest: 10.4 us, 11.8 without; 4096 x
  // 11000 40 and 42) and where there are few rows (256 x 32000: 12.3 us, 14.1
  // without); otherwise it takes the next row's place on the CU (1024 x 23000: 32.4
  // us, 27.6 without).
  if (chunks <= 256 * 4) return row_launch<T, 256, 4, true>(a, s);
  if (chunks <= 256 * 6 && a.N > 512) return row_launch<T, 256, 6, true>(a, s);
  if (chunks <= 512 * 4) return row_launch<T, 512, 4, true>(a, s);
  // Long rows that fill half of the 256 MB Infinity Cache are loaded past it (2048 x
  // 32768 bf16, 128 MB: 61 -> 56 us, 4096: 111 -> 101, 8192 x 65536 403 -> 399), not
  // fewer (1024 x 32768: 29 -> 32) nor short ones (8192 x 10000: 73 -> 81).
  a.once = a.N * a.V * (int64_t)sizeof(T) >= (int64_t(1) << 27);
  if (chunks <= 512 * 7)
    return a.N <= 512 ? row_launch<T, 512, 7, true>(a, s) : row_launch<T, 512, 7, false>(a, s);
  if (chunks <= 512 * 9)
    return a.N <= 256 ? row_launch<T, 512, 9, true>(a, s) : row_launch<T, 512, 9, false>(a, s);
  return chunks <= 512 * 17 ? row_launch<T, 512, 17, false>(a, s)
                            : row_launch<T, 1024, 17, false>(a, s);
}

template <typename T>
hipError_t stats_typed(const DistillArgs& a, int type, hipStream_t s) {
  if (distill_small(a.N, a.V, type)) return wave_typed<T, kLoss>(a, s);
  const dim3 grid((uint32_t)(a.N * a.splits)), block(kPartThreads + 64);
  if (a.tlse) {
    const hipError_t e = enqueue(distill_part_kernel<T, true>, grid, block,
                                       lds_bytes(a.K, true, part_tokens(a, type)), s, a);
    if (e != hipSuccess || a.splits == 1) return e;
    return enqueue(distill_join_kernel<true>, dim3((uint32_t)a.N), dim3(64), 0, s, a);
  }
  const hipError_t e = enqueue(distill_part_kernel<T, false>, grid, block,
                                     lds_bytes(a.K, true, 0), s, a);
  if (e != hipSuccess || a.splits == 1) return e;
  return enqueue(distill_join_kernel<false>, dim3((uint32_t)a.N), dim3(64), 0, s, a);
}

template <typename T>
hipError_t grad_typed(const DistillArgs& a, int type, hipStream_t s) {
  if (distill_small(a.N, a.V, type)) return wave_typed<T, kGradient>(a, s);
  const dim3 grid((uint32_t)(a.N * a.splits)), block(kPartThreads + 64);
  const size_t lds = lds_bytes(a.K, false, part_tokens(a, type));
  return a.tlse ? enqueue(distill_grad_kernel<T, true>, grid, block, lds, s, a)
                : enqueue(distill_grad_kernel<T, false>, grid, block, lds, s, a);
}

}  // namespace

bool distill_small(int64_t N, int64_t V, int type) {
  const int vec = 16 / elem_size(type);
  return by_waves(N, (V + 2 * vec - 2) / vec, false);
}

// A workgroup takes the whole row where it fits the registers: from 128 rows on, and
// below where 512 threads of 9 chunks do (5 x 11692 f32 with a rest 5.8 us, 11.6 in
// parts; 60 x 32000 bf16 9.0 and 13.5; of longer rows, 5 x 60000 16.7 and 11.3).
bool distill_resident(int64_t N, int64_t V, int type) {
  const int vec = 16 / elem_size(type);
  const int64_t chunks = (V + 2 * vec - 2) / vec;
  return chunks <= 1024 * 17 && (N >= 128 || chunks <= 512 * 9);
}

// Up to five workgroups to a CU: with more, the last of them start when the others
// are done (147 x 120926 bf16 with a rest, both calls: 34.0 us, 35.7 of up to 2048
// workgroups, 45 of 4096; 300 x 131071 51.6, 53.5 of 1024), and a row in one part
// needs no join (700 x 8000: 20.1 -> 15.0 us).
constexpr int64_t kPartGroups = 1280;

int distill_splits(int64_t N, int64_t V, int type) {
  const int vec = 16 / elem_size(type);
  const int64_t chunks = (V + 2 * vec - 2) / vec;
  const int64_t most = (chunks + kPartThreads * kBatch - 1) / (kPartThreads * kBatch);
  int64_t n = N ? kPartGroups / N : 1;
  if (n > most) n = most;
  // the bitmap of a part lies in LDS
  const int64_t least = (V + (1 << 18) - 1) >> 18;
  if (n < least) n = least;
  return (int)(n < 1 ? 1 : n);
}

hipError_t launch_distill_fused(const DistillArgs& a, int type, hipStream_t s) {
  return type == 0 ? row_typed<float>(a, s) : type == 1 ? row_typed<bf16_t>(a, s)
                                                        : row_typed<f16_t>(a, s);
}

hipError_t launch_distill_forward(const DistillArgs& a, int type, hipStream_t s) {
  return type == 0 ? stats_typed<float>(a, type, s)
                   : type == 1 ? stats_typed<bf16_t>(a, type, s) : stats_typed<f16_t>(a, type, s);
}

hipError_t launch_distill_backward(const DistillArgs& a, int type, hipStream_t s) {
  return type == 0 ? grad_typed<float>(a, type, s)
                   : type == 1 ? grad_typed<bf16_t>(a, type, s) : grad_typed<f16_t>(a, type, s);
}

}  // namespace per
