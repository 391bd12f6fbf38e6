// rows_kernels.hip -- the 8-bit row store: quantising rows as they are written
// to the ring and reading them back as sequences.
//
// A lane holds 8 neighbouring columns (a unit: one 16-byte load of a 16-bit
// type, 8 bytes of codes); a group of 32, 64 or 128 columns is 4, 8 or 16
// neighbouring lanes, so its largest magnitude is found by lane exchanges.  Each
// row is read and written once; what bounds the large calls is HBM, the small
// ones (400 rows of 64: 2.9 us) the launch.

#include "elem.h"
#include "lanes.h"
#include "train_internal.h"

namespace per {
namespace {

constexpr int kThreads = 256;
constexpr float kTinyMax = 0x1p-100f;  // smallest magnitude a scale is made for

template <int FMT>
constexpr float kTop = FMT == 0 ? 448.0f : 127.0f;

__device__ __forceinline__ uint32_t max_xor(uint32_t v, int s) {
  const float f = __uint_as_float(v);
  return max(v, __float_as_uint(xor_lanes(f, s)));
}

// The codes of 8 values times inv, as two words.  `special`: some value of
// the wave is not finite.
template <int FMT>
__device__ __forceinline__ uint2 quantise(const float (&x)[8], float inv, bool special) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = x[i] * inv;
  if (special) {  // infinities saturate; NaN passes both selects
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = q[i] > kTop<FMT> ? kTop<FMT> : q[i];
      q[i] = q[i] < -kTop<FMT> ? -kTop<FMT> : q[i];
      if (FMT == 1) q[i] = q[i] != q[i] ? 0.0f : q[i];
    }
  }
  // |x| <= a gives |q| <= M (1 + 2^-22), which rounds to M in both formats.
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (FMT == 0) {
      int v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h], q[4 * h + 1], 0, false);
      v = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * h + 2], q[4 * h + 3], v, true);
      w[h] = (uint32_t)v;
    } else {
      uint32_t v = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v |= ((uint32_t)(int)__builtin_rintf(q[4 * h + i]) & 0xFFu) << (8 * i);
      w[h] = v;
    }
  }
  return make_uint2(w[0], w[1]);
}

// Bits of the largest magnitude among the finite values of x.
__device__ __forceinline__ uint32_t finite_max(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t b = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    m = max(m, b < 0x7F800000u ? b : 0u);
  }
  return m;
}

__device__ __forceinline__ uint32_t any_max(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  return m;
}

// Columns [8u, 8u + 8) of a row of dim columns, 0 past its end.
template <typename T>
__device__ __forceinline__ void load_unit(const T* row, uint32_t u, uint32_t dim, float (&x)[8]) {
  if (8 * u + 8 <= dim) {
    unpack(load_pack<T, 8>(row + 8 * u), x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 8 * u + i < dim ? (float)row[8 * u + i] : 0.0f;
  }
}

__device__ __forceinline__ void store_codes(uint8_t* row, uint32_t u, uint32_t dim, uint2 w) {
  if (8 * u + 8 <= dim) {
    __builtin_memcpy(row + 8 * u, &w, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * u + i < dim) row[8 * u + i] = (uint8_t)((i < 4 ? w.x : w.y) >> (8 * (i & 3)));
  }
}

struct Scale {
  float scale, inv;
};
template <int FMT>
__device__ __forceinline__ Scale make_scale(uint32_t max_bits) {
  const float a = fmaxf(__uint_as_float(max_bits), kTinyMax);
  Scale s;
  s.scale = a * (1.0f / kTop<FMT>);
  s.inv = 1.0f / s.scale;
  return s;
}

// The slot row j is written to, or -1.  Of the rows that name one slot only
// the one whose claim stands writes it, and takes the claim back: a row that
// reads the slot's claim later finds 0, which is no row's claim either.
__device__ __forceinline__ int64_t slot_of(const RowsArgs& a, uint32_t j, bool* claimed) {
  *claimed = false;
  if (!a.slots) {
    const int64_t s = a.first + j;
    return s >= a.capacity ? s - a.capacity : s;
  }
  const int64_t s = a.slots[j];
  if (s < 0 || s >= a.capacity) return -1;
  *claimed = a.claims[s] == j + 1;
  return *claimed ? s : -1;
}

// 2^lg lanes per row, U units per lane and step.  ROW: one scale for the row,
// whose units all lie in one step; else groups of 2^lg_group lanes.  Steps
// beyond the first are taken by blockIdx.y (ring writes) or by a loop.
//
// x / scale is taken as x * (1 / scale), one division per group instead of one
// per value: at 3 bytes moved a value, ten more instructions would show.
// 65536 rows of 2048 bf16, groups of 128: 75 us, 5.4 TB/s (a large copy: 4.8).
template <typename T, int FMT, int U, bool ROW>
__global__ __launch_bounds__(kThreads) void rows_write_kernel(RowsArgs a, int lg) {
  const uint32_t lane = threadIdx.x & ((1u << lg) - 1);
  const uint32_t j = blockIdx.x * (uint32_t)(kThreads >> lg) + (threadIdx.x >> lg);
  const bool row = j < a.rows;
  const T* src = static_cast<const T*>(a.src) + (int64_t)j * a.stride;
  const uint32_t step = (uint32_t)U << lg;
  int64_t slot = -1;
  bool known = false;
  for (uint32_t u0 = blockIdx.y * step; 8 * u0 < a.dim; u0 += gridDim.y * step) {
    // The row is loaded, and reduced, before its slot and claim are known: most
    // rows are written, and three dependent loads would cost their latencies.
    float x[U][8];
    uint32_t m[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = u0 + ((uint32_t)i << lg) + lane;
      if (row && 8 * u < a.dim) {
        load_unit(src, u, a.dim, x[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
      }
    }
    if (!known && row) {
      bool claimed;
      slot = slot_of(a, j, &claimed);
      if (claimed && lane == 0) a.claims[slot] = 0;
    }
    known = true;
    const bool live = slot >= 0;
    uint8_t* codes = a.codes + slot * a.cs;
    float* scales = a.scales + slot * a.ss;
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      m[i] = any_max(x[i]);
      all = max(all, m[i]);
    }
    const bool special = __any(all >= 0x7F800000u);
    if (special) {
#pragma unroll
      for (int i = 0; i < U; ++i) m[i] = finite_max(x[i]);
    }
    if (ROW) {
      uint32_t r = 0;
#pragma unroll
      for (int i = 0; i < U; ++i) r = max(r, m[i]);
#pragma unroll
      for (int s = 0; s < 6; ++s)
        if (s < lg) r = max_xor(r, s);
#pragma unroll
      for (int i = 0; i < U; ++i) m[i] = r;
    } else {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        m[i] = max_xor(max_xor(m[i], 0), 1);
        if (a.lg_group > 2) m[i] = max_xor(m[i], 2);
        if (a.lg_group > 3) m[i] = max_xor(m[i], 3);
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const uint32_t u = u0 + ((uint32_t)i << lg) + lane;
      const Scale sc = make_scale<FMT>(m[i]);
      const uint2 w = quantise<FMT>(x[i], sc.inv, special);
      if (live && 8 * u < a.dim) {
        store_codes(codes, u, a.dim, w);
        if (ROW) {
          if (u == 0) scales[0] = sc.scale;
        } else if ((u & ((1u << a.lg_group) - 1)) == 0) {
          scales[u >> a.lg_group] = sc.scale;
        }
      }
    }
  }
}

// One scale for a row too long for one wave's registers: a workgroup of NT threads
// per row, U units per thread at a time.  HOLD: the row is one such step and stays
// in registers; else it is read again (from the L2) to quantise it.  256 rows of
// 65536 bf16, 1024 threads of four units: 13.7 us (256 of one: 28.5).
template <typename T, int FMT, int NT, int U, bool HOLD>
__global__ __launch_bounds__(NT) void rows_write_long_kernel(RowsArgs a) {
  __shared__ uint32_t wave_max[NT / 64];
  __shared__ int wave_special[NT / 64];
  const uint32_t j = blockIdx.x;
  bool claimed;
  const int64_t slot = slot_of(a, j, &claimed);
  const T* src = static_cast<const T*>(a.src) + (int64_t)j * a.stride;
  float x[U][8];
  auto load = [&](uint32_t u0) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (8 * (u0 + i * NT) < a.dim) {
        load_unit(src, u0 + i * NT, a.dim, x[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
      }
    }
  };
  uint32_t all = 0, fin = 0;
  auto reduce = [&] {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      all = max(all, any_max(x[i]));
      fin = max(fin, finite_max(x[i]));
    }
  };
  if (slot >= 0) {
    if (HOLD) {
      load(threadIdx.x);
      reduce();
    } else {
      for (uint32_t u0 = threadIdx.x; 8 * u0 < a.dim; u0 += NT * U) {
        load(u0);
        reduce();
      }
    }
  }
  fin = wave_max_u32(fin);
  const bool odd = __any(all >= 0x7F800000u);
  if ((threadIdx.x & 63) == 0) {
    wave_max[threadIdx.x >> 6] = fin;
    wave_special[threadIdx.x >> 6] = odd;
  }
  __syncthreads();  // every thread has read the claim
  if (slot < 0) return;
  if (claimed && threadIdx.x == 0) a.claims[slot] = 0;
  bool special = false;
  uint32_t m = 0;
#pragma unroll
  for (int w = 0; w < NT / 64; ++w) {
    m = max(m, wave_max[w]);
    special |= wave_special[w] != 0;
  }
  const Scale sc = make_scale<FMT>(m);
  if (threadIdx.x == 0) a.scales[slot * a.ss] = sc.scale;
  uint8_t* codes = a.codes + slot * a.cs;
  for (uint32_t u0 = threadIdx.x; 8 * u0 < a.dim; u0 += NT * U) {
    if (!HOLD) load(u0);
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (8 * (u0 + i * NT) < a.dim)
        store_codes(codes, u0 + i * NT, a.dim, quantise<FMT>(x[i], sc.inv, special));
  }
}

// Each row claims its slot with its batch position; the largest stands.
__global__ __launch_bounds__(kThreads) void rows_claim_kernel(RowsArgs a) {
  const uint32_t j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= a.rows) return;
  const int64_t s = a.slots[j];
  if (s >= 0 && s < a.capacity) atomicMax(&a.claims[s], j + 1);
}

template <int FMT>
__device__ __forceinline__ void decode(uint2 w, float scale, float (&x)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t v = h ? w.y : w.x;
    if (FMT == 0) {
      const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, false);
      const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)v, true);
      x[4 * h] = lo[0] * scale;
      x[4 * h + 1] = lo[1] * scale;
      x[4 * h + 2] = hi[0] * scale;
      x[4 * h + 3] = hi[1] * scale;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[4 * h + i] = (float)(int)(int8_t)(v >> (8 * i)) * scale;
    }
  }
}

// 2^lg lanes per output row, U units per lane, blockIdx.y over column steps.
//
// 512 sequences of 80 rows of 1024 to bf16: 26.5 us, 4.8 TB/s, the rate of a large
// copy.  Stores past the caches take 16.5 us alone, but what reads the rows next
// then finds none of them: with the recurrence behind it 42.4 us become 44.9, and
// at twice the sequences 77 become 93.
template <typename T, int FMT, int U>
__global__ __launch_bounds__(kThreads) void rows_read_kernel(RowsArgs a, int lg) {
  const uint32_t lane = threadIdx.x & ((1u << lg) - 1);
  const uint32_t r = blockIdx.x * (uint32_t)(kThreads >> lg) + (threadIdx.x >> lg);
  if (r >= a.rows) return;
  const uint32_t b = a.window == 1 ? r : r / a.window;
  int64_t slot = a.slots[b];
  const bool live = slot >= 0 && slot < a.capacity;
  slot += r - b * a.window;
  if (live && slot >= a.capacity) slot %= a.capacity;
  const uint8_t* codes = a.codes + slot * a.cs;
  const float* scales = a.scales + slot * a.ss;
  T* out = static_cast<T*>(a.out) + (int64_t)r * a.stride;
  const uint32_t u0 = ((blockIdx.y * (uint32_t)U) << lg) + lane;
  uint2 w[U];
  float sc[U];
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t u = u0 + ((uint32_t)i << lg);
    w[i] = make_uint2(0, 0);
    sc[i] = 0.0f;
    if (live && 8 * u < a.dim) {
      if (8 * u + 8 <= a.dim) {
        __builtin_memcpy(&w[i], codes + 8 * u, 8);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t c = 8 * u + e < a.dim ? codes[8 * u + e] : 0u;
          if (e < 4) w[i].x |= c << (8 * e);
          else w[i].y |= c << (8 * (e - 4));
        }
      }
      sc[i] = scales[a.lg_group < 0 ? 0 : u >> a.lg_group];
    }
  }
#pragma unroll
  for (int i = 0; i < U; ++i) {
    const uint32_t u = u0 + ((uint32_t)i << lg);
    if (8 * u >= a.dim) continue;
    float x[8];
    decode<FMT>(w[i], sc[i], x);
    if (8 * u + 8 <= a.dim) {
      store_vals<T, 8>(out + 8 * u, x);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (8 * u + e < a.dim) out[8 * u + e] = (T)x[e];
    }
  }
}

int ceil_log2(uint32_t v) {
  int l = 0;
  while ((1u << l) < v) ++l;
  return l;
}

template <typename T, int FMT>
hipError_t write_typed(const RowsArgs& a, hipStream_t s) {
  if (a.slots) {
    const hipError_t e = enqueue(rows_claim_kernel, dim3((a.rows + kThreads - 1) / kThreads),
                                       dim3(kThreads), 0, s, a);
    if (e != hipSuccess) return e;
  }
  const uint32_t units = (a.dim + 7) / 8;
  int lg = ceil_log2(units);
  if (lg > 6) lg = 6;
  const bool row = a.lg_group < 0;
  if (!row && lg < a.lg_group) lg = a.lg_group;
  const uint32_t per_lane = (units + (1u << lg) - 1) >> lg;
  if (row && per_lane > 4) {
    const dim3 grid(a.rows);
    if (units <= kThreads * 2)
      return enqueue(rows_write_long_kernel<T, FMT, kThreads, 2, true>, grid, dim3(kThreads),
                           0, s, a);
    if (units <= kThreads * 4)
      return enqueue(rows_write_long_kernel<T, FMT, kThreads, 4, true>, grid, dim3(kThreads),
                           0, s, a);
    if (units <= 1024 * 4)
      return enqueue(rows_write_long_kernel<T, FMT, 1024, 4, true>, grid, dim3(1024), 0, s, a);
    return enqueue(rows_write_long_kernel<T, FMT, 1024, 4, false>, grid, dim3(1024), 0, s, a);
  }
  const uint32_t rpb = kThreads >> lg;
  const int U = per_lane <= 1 ? 1 : per_lane <= 2 ? 2 : 4;
  // Rows that name their slots are not split: the first part to run would
  // take the claim back before the others read it.  So one wave walks a whole row:
  // 2048 x 8192 bf16 17 us, 13 in ring order; 256 x 65536 80 and 11; 16 x 2^20 1190
  // and 15.
  const uint32_t steps = a.slots ? 1 : (per_lane + U - 1) / U;
  const dim3 grid((a.rows + rpb - 1) / rpb, steps);
  if (row) {
    if (U == 1) return enqueue(rows_write_kernel<T, FMT, 1, true>, grid, dim3(kThreads), 0, s, a, lg);
    if (U == 2) return enqueue(rows_write_kernel<T, FMT, 2, true>, grid, dim3(kThreads), 0, s, a, lg);
    return enqueue(rows_write_kernel<T, FMT, 4, true>, grid, dim3(kThreads), 0, s, a, lg);
  }
  if (U == 1) return enqueue(rows_write_kernel<T, FMT, 1, false>, grid, dim3(kThreads), 0, s, a, lg);
  if (U == 2) return enqueue(rows_write_kernel<T, FMT, 2, false>, grid, dim3(kThreads), 0, s, a, lg);
  return enqueue(rows_write_kernel<T, FMT, 4, false>, grid, dim3(kThreads), 0, s, a, lg);
}

template <typename T, int FMT>
hipError_t read_typed(const RowsArgs& a, hipStream_t s) {
  const uint32_t units = (a.dim + 7) / 8;
  int lg = ceil_log2(units);
  if (lg > 6) lg = 6;
  const uint32_t per_lane = (units + (1u << lg) - 1) >> lg;
  const uint32_t rpb = kThreads >> lg;
  const uint32_t nx = (a.rows + rpb - 1) / rpb;
  if (per_lane <= 1)
    return enqueue(rows_read_kernel<T, FMT, 1>, dim3(nx), dim3(kThreads), 0, s, a, lg);
  if (per_lane <= 2)
    return enqueue(rows_read_kernel<T, FMT, 2>, dim3(nx), dim3(kThreads), 0, s, a, lg);
  return enqueue(rows_read_kernel<T, FMT, 4>, dim3(nx, (per_lane + 3) / 4), dim3(kThreads), 0,
                       s, a, lg);
}

}  // namespace

hipError_t launch_rows_write(const RowsArgs& a, int type, int format, hipStream_t s) {
  if (format == 0)
    return type == 0 ? write_typed<float, 0>(a, s)
                     : type == 1 ? write_typed<bf16_t, 0>(a, s) : write_typed<f16_t, 0>(a, s);
  return type == 0 ? write_typed<float, 1>(a, s)
                   : type == 1 ? write_typed<bf16_t, 1>(a, s) : write_typed<f16_t, 1>(a, s);
}

hipError_t launch_rows_read(const RowsArgs& a, int type, int format, hipStream_t s) {
  if (format == 0)
    return type == 0 ? read_typed<float, 0>(a, s)
                     : type == 1 ? read_typed<bf16_t, 0>(a, s) : read_typed<f16_t, 0>(a, s);
  return type == 0 ? read_typed<float, 1>(a, s)
                   : type == 1 ? read_typed<bf16_t, 1>(a, s) : read_typed<f16_t, 1>(a, s);
}

}  // namespace per
