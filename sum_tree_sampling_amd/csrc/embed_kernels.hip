// embed_kernels.hip -- the embedding of tokens, and its gradient.
//
// Forward, a group of lanes copies a row of the table, scaled.  Backward, the tokens
// are sorted with their positions (stable, by digits of up to 9 bits), the sorted rows
// are cut into chunks of equal length, a wave to a chunk and a slice of the columns, and
// each token's rows are added in the order of their positions.  A token whose rows lie
// inside one chunk is written at once; what chunks share goes to the workspace, and a
// second launch adds a token's parts in order, so a token that is half of all rows is
// summed by as many waves as the others.  No sum is made with atomics.
//
// Memory bounds the large calls: 65536 tokens of 65536 x 1024 (f32 table and gradient,
// bf16 rows) take 50 us forward (293 MB, 5.9 TB/s) and 94 us for the sums (402 MB, 4.3
// TB/s, rows in the tokens' order), beside 22 us of sorting (four launches, each 2 to 7)
// and 9 us of joins.  20001 x 333 f32 of 501 tokens, 40 % of them one, take 10 us forward
// and 12 + 10 + 16: five launches in order, each a chain of dependent loads.
#include <algorithm>

#include "block_internal.h"
#include "elem.h"
#include "lanes.h"

namespace per {
namespace {

template <typename T>
struct Tag {
  using type = T;
};

// Token n, or V where it is absent.
__device__ __forceinline__ uint32_t token_at(const EmbedArgs& a, int64_t n) {
  const int64_t t = a.token_bytes == 4 ? (int64_t)static_cast<const int32_t*>(a.tokens)[n]
                                       : static_cast<const int64_t*>(a.tokens)[n];
  return t >= 0 && t < a.V ? (uint32_t)t : (uint32_t)a.V;
}

// ---------------------------------------------------------------------- forward

// 2^lg lanes to a row and kRows rows one after the other, W columns to a lane at a time;
// the rows' loads are all on their way before the first is stored (20001 x 333 f32: 9.8
// us, and 10.5 with one row at a time).
constexpr int kRows = 4;
template <typename F, typename T, int W>
__global__ __launch_bounds__(256) void embed_forward_kernel(EmbedArgs a, int lg) {
  const uint32_t lane = threadIdx.x & ((1u << lg) - 1);
  const int64_t step = (int64_t)256 >> lg;  // rows of the workgroup at a time
  const int64_t n0 = (int64_t)blockIdx.x * kRows * step + (threadIdx.x >> lg);
  const uint32_t D = (uint32_t)a.D;
  uint32_t token[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) token[r] = n0 + r * step < a.N ? token_at(a, n0 + r * step) : (uint32_t)a.V;
  for (uint32_t col = lane * W; col < D; col += (uint32_t)W << lg) {
    Pack<F, W> v[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const bool there = token[r] < (uint32_t)a.V;
      const F* from = static_cast<const F*>(a.src) + (there ? (int64_t)token[r] * a.src_stride : 0);
      if (col + W <= D) {
        v[r] = load_pack<F, W>(from + col);
      } else {
        const uint32_t last = D - 1 - col;
#pragma unroll
        for (uint32_t i = 0; i < W; ++i) v[r].v[i] = from[col + min(i, last)];
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (n0 + r * step >= a.N) break;
      const bool there = token[r] < (uint32_t)a.V;
      T* to = static_cast<T*>(a.dst) + (n0 + r * step) * a.dst_stride + col;
      float x[W];
      unpack<F, W>(v[r], x);
#pragma unroll
      for (int i = 0; i < W; ++i) x[i] = there ? x[i] * a.scale : 0.0f;
      if (col + W <= D) {
        store_vals<T, W>(to, x);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i)
          if (col + i < D) to[i] = (T)x[i];
      }
    }
  }
}

// ---------------------------------------------------------------------- sorting

// Ranks of a wave's items among the wave's earlier ones with the same digit, item by
// item: cnt holds the wave's count of each digit so far (in LDS, its own).  Lanes of
// the same digit find each other by one ballot for each of its bits.
__device__ __forceinline__ uint32_t wave_rank(uint32_t digit, bool valid, int bits,
                                              volatile uint32_t* cnt) {
  uint64_t same = __ballot(valid);
  for (int b = 0; b < bits; ++b) {
    const uint64_t set = __ballot(digit >> b & 1u);
    same &= digit >> b & 1u ? set : ~set;
  }
  const int lane = threadIdx.x & 63;
  const uint64_t below = same & ((1ull << lane) - 1);
  const uint32_t before = valid ? cnt[digit] : 0;
  __builtin_amdgcn_wave_barrier();
  if (valid && below == 0) cnt[digit] = before + (uint32_t)__popcll(same);
  __builtin_amdgcn_wave_barrier();
  return before + (uint32_t)__popcll(below);
}

constexpr int kBins = 512;

// Exclusive sum over the threads of a workgroup of WAVES waves.
template <int WAVES>
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* space) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  uint32_t s = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_up(s, d);
    if (lane >= d) s += o;
  }
  if (lane == 63) space[wave] = s;
  __syncthreads();
  uint32_t base = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) base += w < wave ? space[w] : 0;
  __syncthreads();
  return base + s - v;
}

// Up to kSmall tokens by one workgroup, all passes in LDS, a token to a thread.
constexpr int64_t kSmall = 1024;
__global__ __launch_bounds__(1024) void embed_sort_small_kernel(EmbedArgs a, int bits, int passes) {
  __shared__ uint32_t cnt[16][kBins];
  __shared__ uint32_t keys[kSmall], pos[kSmall];
  __shared__ uint32_t space[16];
  const int wave = threadIdx.x / 64;
  const bool valid = threadIdx.x < (uint32_t)a.N;
  uint32_t p = threadIdx.x, k = valid ? token_at(a, p) : 0;
  const uint32_t mask = (1u << bits) - 1;
  for (int pass = 0; pass < passes; ++pass) {
    const int shift = pass * bits;
    for (int j = threadIdx.x; j < 16 * kBins; j += 1024) (&cnt[0][0])[j] = 0;
    __syncthreads();
    const uint32_t rank = wave_rank(k >> shift & mask, valid, bits, cnt[wave]);
    __syncthreads();
    uint32_t total = 0;
    if (threadIdx.x < kBins) {
#pragma unroll
      for (int w = 0; w < 16; ++w) {
        const uint32_t c = cnt[w][threadIdx.x];
        cnt[w][threadIdx.x] = total;
        total += c;
      }
    }
    const uint32_t base = block_exclusive<16>(total, space);
    if (threadIdx.x < kBins) {
#pragma unroll
      for (int w = 0; w < 16; ++w) cnt[w][threadIdx.x] += base;
    }
    __syncthreads();
    if (valid) {
      const uint32_t to = cnt[wave][k >> shift & mask] + rank;
      keys[to] = k;
      pos[to] = p;
    }
    __syncthreads();
    if (valid) {
      k = keys[threadIdx.x];
      p = pos[threadIdx.x];
    }
  }
  if (valid) {
    a.keys[threadIdx.x] = k;
    a.pos[threadIdx.x] = p;
  }
}

// More of them: a block has `per` consecutive items, and each pass is two launches, the
// digits' counts of each block and the scatter.  With 8 tokens to a thread one workgroup
// could sort 8192, but takes longer than these four launches (the whole gradient of 50000 x
// 64 f32: 2049 tokens 24.4 and 23.1 us, 8192 tokens 28.7 and 25.4).
constexpr int kSortThreads = 1024, kSortTile = 1024;  // a wave has 64 items of a tile

__device__ __forceinline__ uint32_t sort_key(const EmbedArgs& a, const uint32_t* keys, int64_t n) {
  return keys ? keys[n] : token_at(a, n);
}

__global__ __launch_bounds__(kSortThreads) void embed_count_kernel(EmbedArgs a,
                                                                   const uint32_t* keys, int shift,
                                                                   int bits, int64_t per) {
  __shared__ uint32_t cnt[kBins];
  for (int j = threadIdx.x; j < kBins; j += kSortThreads) cnt[j] = 0;
  __syncthreads();
  const int64_t lo = blockIdx.x * per, hi = min(a.N, lo + per);
  const uint32_t mask = (1u << bits) - 1;
  for (int64_t n = lo + threadIdx.x; n < hi; n += kSortThreads)
    atomicAdd(&cnt[sort_key(a, keys, n) >> shift & mask], 1u);
  __syncthreads();
  for (int j = threadIdx.x; j < kBins; j += kSortThreads)
    a.counts[(int64_t)blockIdx.x * kBins + j] = cnt[j];
}

__global__ __launch_bounds__(kSortThreads) void embed_scatter_kernel(
    EmbedArgs a, const uint32_t* keys, const uint32_t* pos, uint32_t* keys_to, uint32_t* pos_to,
    int shift, int bits, int64_t per) {
  constexpr int kWaves = kSortThreads / 64, kRounds = kSortTile / kSortThreads;
  __shared__ uint32_t cnt[kWaves][kBins];
  __shared__ uint32_t base[kBins];
  __shared__ uint32_t space[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x / 64;
  const uint32_t mask = (1u << bits) - 1;
  // where this block's items of each digit begin: the blocks' counts are added by 8
  // groups of threads, 4 neighbouring digits to a thread
  {
    static_assert(kSortThreads == 8 * kBins / 4 && 2 * 8 * kBins <= kWaves * kBins, "groups");
    uint32_t before[4] = {0, 0, 0, 0}, total[4] = {0, 0, 0, 0};
    const uint32_t group = threadIdx.x / (kBins / 4), at = threadIdx.x % (kBins / 4);
    const uint4* counts = reinterpret_cast<const uint4*>(a.counts) + at;
#pragma unroll 8
    for (uint32_t b = group; b < gridDim.x; b += 8) {
      const uint4 c = counts[(int64_t)b * (kBins / 4)];
      const bool mine = b < blockIdx.x;
      total[0] += c.x;
      total[1] += c.y;
      total[2] += c.z;
      total[3] += c.w;
      before[0] += mine ? c.x : 0;
      before[1] += mine ? c.y : 0;
      before[2] += mine ? c.z : 0;
      before[3] += mine ? c.w : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cnt[group][4 * at + i] = total[i];
      cnt[8 + group][4 * at + i] = before[i];
    }
    __syncthreads();
    uint32_t all = 0, mine = 0;
    if (threadIdx.x < kBins) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        all += cnt[k][threadIdx.x];
        mine += cnt[8 + k][threadIdx.x];
      }
    }
    const uint32_t begin = block_exclusive<kWaves>(all, space);
    if (threadIdx.x < kBins) base[threadIdx.x] = begin + mine;
    __syncthreads();
  }
  const int64_t lo = blockIdx.x * per, hi = min(a.N, lo + per);
  for (int64_t tile = lo; tile < hi; tile += kSortTile) {
    for (int j = threadIdx.x; j < kWaves * kBins; j += kSortThreads) (&cnt[0][0])[j] = 0;
    __syncthreads();
    uint32_t k[kRounds], p[kRounds], r[kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
      const int64_t n = tile + (wave * kRounds + i) * 64 + lane;
      k[i] = n < hi ? sort_key(a, keys, n) : 0;
      p[i] = n < hi ? (pos ? pos[n] : (uint32_t)n) : 0;
    }
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      r[i] = wave_rank(k[i] >> shift & mask, tile + (wave * kRounds + i) * 64 + lane < hi, bits,
                       cnt[wave]);
    __syncthreads();
    for (int j = threadIdx.x; j < kBins; j += kSortThreads) {
      uint32_t run = base[j];
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const uint32_t c = cnt[w][j];
        cnt[w][j] = run;
        run += c;
      }
      base[j] = run;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kRounds; ++i)
      if (tile + (wave * kRounds + i) * 64 + lane < hi) {
        const uint32_t to = cnt[wave][k[i] >> shift & mask] + r[i];
        keys_to[to] = k[i];
        pos_to[to] = p[i];
      }
    __syncthreads();
  }
}

// ---------------------------------------------------------------------- sums

// Adds nothing past D; v holds W columns from col on.
template <typename G, int W>
__device__ __forceinline__ void write_sum(const EmbedArgs& a, uint32_t token, uint32_t col,
                                          const float (&v)[W]) {
  G* to = static_cast<G*>(a.dst) + (int64_t)token * a.dst_stride + col;
  const uint32_t D = (uint32_t)a.D;
  if (col + W <= D) {
    float out[W];
#pragma unroll
    for (int i = 0; i < W; ++i) out[i] = v[i] * a.scale;
    if (a.accumulate) {
      float old[W];
      unpack<G, W>(load_pack<G, W>(to), old);
#pragma unroll
      for (int i = 0; i < W; ++i) out[i] += old[i];
    }
    store_vals<G, W>(to, out);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (col + i < D) to[i] = (G)(v[i] * a.scale + (a.accumulate ? (float)to[i] : 0.0f));
  }
}
template <int W>
__device__ __forceinline__ void write_part(const EmbedArgs& a, int64_t chunk, int which,
                                           uint32_t col, const float (&v)[W]) {
  float* to = a.part + (chunk * 2 + which) * a.D + col;
  if (col + W <= (uint32_t)a.D) {
    store_vals<float, W>(to, v);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (col + i < (uint32_t)a.D) to[i] = v[i];
  }
}

constexpr int kZeroRows = 16;  // rows of the gradient that a wave looks over

// The first of the sorted keys that is not below `key`.
__device__ __forceinline__ int64_t lower_bound(const uint32_t* keys, int64_t n, uint32_t key) {
  int64_t lo = 0;
  while (n > 0) {
    const int64_t half = n / 2;
    const bool right = keys[lo + half] < key;
    lo = right ? lo + half + 1 : lo;
    n = right ? n - half - 1 : half;
  }
  return lo;
}

// A wave to a chunk of sorted rows and a slice of 64 * W columns; the waves behind
// `units` write zeros to rows whose token does not occur.
template <typename T, typename G>
__global__ __launch_bounds__(256) void embed_sum_kernel(EmbedArgs a, uint32_t slices,
                                                        int64_t units) {
  constexpr int W = 16 / (int)sizeof(T), kBatch = 8;
  const int lane = threadIdx.x & 63;
  const int64_t unit = (int64_t)blockIdx.x * 4 + threadIdx.x / 64;
  const uint32_t D = (uint32_t)a.D;
  if (unit >= units) {
    if (a.accumulate) return;
    const int64_t first = (unit - units) * kZeroRows;
    if (first >= a.V) return;
    const int64_t row = first + (lane & (kZeroRows - 1));
    bool absent = false;
    if (row < a.V) {
      const int64_t at = lower_bound(a.keys, a.N, (uint32_t)row);
      absent = at >= a.N || a.keys[at] != (uint32_t)row;
    }
    uint32_t todo = (uint32_t)__ballot(absent) & ((1u << kZeroRows) - 1);
    constexpr int Z = 16 / (int)sizeof(G);
    float zero[Z] = {};
    while (todo) {
      const int r = __builtin_ctz(todo);
      todo &= todo - 1;
      G* to = static_cast<G*>(a.dst) + (first + r) * a.dst_stride;
      for (uint32_t col = lane * Z; col < D; col += 64 * Z) {
        if (col + Z <= D) {
          store_vals<G, Z>(to + col, zero);
        } else {
          for (uint32_t c = col; c < D; ++c) to[c] = (G)0.0f;
        }
      }
    }
    return;
  }
  const int64_t chunk = unit / slices;
  const uint32_t col = ((uint32_t)(unit % slices) * 64 + lane) * W;
  const int64_t i0 = chunk << a.lg_rows;
  const int rows = (int)min((int64_t)1 << a.lg_rows, a.N - i0);
  // lane l holds the chunk's key and position l (at most 64 rows)
  const uint32_t mine = lane < rows ? a.keys[i0 + lane] : (uint32_t)a.V;
  const uint32_t where = lane < rows ? a.pos[i0 + lane] : 0;
  const uint32_t past = i0 > 0 ? a.keys[i0 - 1] : 0xFFFFFFFFu;
  const uint32_t next = i0 + rows < a.N ? a.keys[i0 + rows] : 0xFFFFFFFFu;
  const int live = __popcll(__ballot(mine < (uint32_t)a.V));  // absent tokens come last
  if (live == 0) return;
  const T* src = static_cast<const T*>(a.src) + col;
  const bool full = col + W <= D;
  float acc[W] = {};
  uint32_t cur = (uint32_t)__builtin_amdgcn_readlane((int)mine, 0);
  bool joins = cur == past;  // the token's first rows lie in chunks before
  for (int b = 0; b < live; b += kBatch) {
    float v[kBatch][W];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int at = b + i < live ? b + i : live - 1;
      const int64_t off = (int64_t)(uint32_t)__builtin_amdgcn_readlane((int)where, at) * a.src_stride;
      if (full) {
        unpack<T, W>(load_pack<T, W>(src + off), v[i]);
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) v[i][j] = col + j < D ? (float)src[off + j] : 0.0f;
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (b + i < live) {
        const uint32_t key = (uint32_t)__builtin_amdgcn_readlane((int)mine, b + i);
        if (key != cur) {
          if (col < D) {
            if (joins) {
              write_part<W>(a, chunk, 0, col, acc);
            } else {
              write_sum<G, W>(a, cur, col, acc);
            }
          }
#pragma unroll
          for (int j = 0; j < W; ++j) acc[j] = 0.0f;
          cur = key;
          joins = false;
        }
#pragma unroll
        for (int j = 0; j < W; ++j) acc[j] += v[i][j];
      }
    }
  }
  if (col >= D) return;
  if (joins) {
    write_part<W>(a, chunk, 0, col, acc);
  } else if (next == cur) {
    write_part<W>(a, chunk, 1, col, acc);
  } else {
    write_sum<G, W>(a, cur, col, acc);
  }
}

// A token that begins in a chunk and goes on in others: a workgroup adds its parts in the
// chunks' order, a run of them to each of its waves.  Most find nothing to do.  16 waves
// where there are more chunks than tokens, so that a token has many parts (1251 chunks of
// 501 tokens: 16.2 us, 21 with 4 waves that add 8 parts at a time), else 4, which come and go faster
// (1024 chunks of 65536 tokens: 8.8 us, 23.5 with 16).
template <typename G, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void embed_join_kernel(EmbedArgs a, uint32_t slices, int64_t chunks) {
  constexpr int W = 4;
  __shared__ float sum[WAVES][64][W];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int64_t first = blockIdx.x / slices;
  const uint32_t col = ((uint32_t)(blockIdx.x % slices) * 64 + lane) * W;
  const uint32_t D = (uint32_t)a.D;
  const int64_t i0 = first << a.lg_rows, i1 = (first + 1) << a.lg_rows;
  const uint32_t key = a.keys[i1], last = a.keys[i1 - 1], head = a.keys[i0];
  const uint32_t past = first > 0 ? a.keys[i0 - 1] : 0xFFFFFFFFu;
  if (key >= (uint32_t)a.V || last != key || (head == key && past == key)) return;
  // chunks behind the first that begin with the token: they follow each other
  int64_t more = 1;
  for (;;) {
    const int64_t c = first + 1 + more + threadIdx.x;
    const int n = __syncthreads_count(c < chunks && a.keys[min(c, chunks - 1) << a.lg_rows] == key);
    more += n;
    if (n < 64 * WAVES) break;
  }
  // part 1 of the first chunk, then part 0 of the others
  const int64_t per = (more + WAVES) / WAVES;  // of more + 1 parts
  const int64_t lo = wave * per, hi = min(more + 1, lo + per);
  float acc[W] = {};
  if (col < D) {
    const float* part = a.part + first * 2 * a.D + col;
    auto add = [&](const float* p) {
      float v[W];
      if (col + W <= D) {
        unpack<float, W>(load_pack<float, W>(p), v);
      } else {
#pragma unroll
        for (int i = 0; i < W; ++i) v[i] = col + i < D ? p[i] : 0.0f;
      }
#pragma unroll
      for (int i = 0; i < W; ++i) acc[i] += v[i];
    };
    int64_t j = lo;
    if (j == 0) {
      add(part + a.D);
      j = 1;
    }
#pragma unroll 16
    for (; j < hi; ++j) add(part + j * 2 * a.D);
  }
#pragma unroll
  for (int i = 0; i < W; ++i) sum[wave][lane][i] = acc[i];
  __syncthreads();
  if (wave == 0 && col < D) {
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
#pragma unroll
      for (int i = 0; i < W; ++i) acc[i] += sum[w][lane][i];
    write_sum<G, W>(a, key, col, acc);
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

// Blocks of a sorting pass.
int64_t sort_blocks(int64_t N) { return std::min<int64_t>(256, (N + kSortTile - 1) / kSortTile); }

// Rows of a chunk: at least 1024 waves where the rows allow it, 8 to 64 rows each.
int chunk_rows(int64_t N, int64_t D) {
  const int64_t slices = (D + 511) / 512;
  int lg = 3;
  while (lg < 6 && (N * slices >> (lg + 1)) >= 1024) ++lg;
  return lg;
}

}  // namespace

size_t embed_workspace(int64_t N, int64_t V, int64_t D, EmbedArgs* a, void* ws) {
  (void)V;
  const int lg = chunk_rows(N, D);
  const int64_t chunks = (N + (1 << lg) - 1) >> lg;
  const size_t list = ((size_t)N * 4 + 15) / 16 * 16;
  const size_t counts = N > kSmall ? (size_t)sort_blocks(N) * kBins * 4 : 0;
  const size_t lists = N > kSmall ? 4 : 2;
  if (a) {
    char* p = static_cast<char*>(ws);
    a->keys = reinterpret_cast<uint32_t*>(p);
    a->pos = reinterpret_cast<uint32_t*>(p + list);
    a->keys2 = reinterpret_cast<uint32_t*>(p + 2 * list);
    a->pos2 = reinterpret_cast<uint32_t*>(p + 3 * list);
    a->counts = reinterpret_cast<uint32_t*>(p + lists * list);
    a->part = reinterpret_cast<float*>(p + lists * list + counts);
    a->lg_rows = lg;
  }
  return lists * list + counts + (size_t)chunks * 2 * (size_t)D * 4;
}

hipError_t launch_embed_forward(const EmbedArgs& a, int table_type, int out_type, hipStream_t s) {
  return by_type(table_type, [&](auto from) {
    return by_type(out_type, [&](auto to) {
      using F = typename decltype(from)::type;
      using T = typename decltype(to)::type;
      constexpr int W = sizeof(F) == 4 && sizeof(T) == 4 ? 4 : 8;
      int lg = 0;
      while (lg < 8 && ((int64_t)W << lg) < a.D) ++lg;
      const int64_t rows = kRows * (256 >> lg);
      return enqueue(embed_forward_kernel<F, T, W>, dim3((uint32_t)((a.N + rows - 1) / rows)),
                     dim3(256), 0, s, a, lg);
    });
  });
}

hipError_t launch_embed_backward(EmbedArgs a, int dout_type, int grad_type, hipStream_t s) {
  int all = 1;  // bits of a key, V among them
  while (a.V >> all) ++all;
  const int passes = (all + 8) / 9, bits = (all + passes - 1) / passes;
  hipError_t e = hipSuccess;
  if (a.N > 0 && a.N <= kSmall) {
    e = enqueue(embed_sort_small_kernel, dim3(1), dim3(1024), 0, s, a, bits, passes);
  } else if (a.N > 0) {
    const int64_t blocks = sort_blocks(a.N);
    const int64_t per = ((a.N + blocks - 1) / blocks + kSortTile - 1) / kSortTile * kSortTile;
    uint32_t *k0 = nullptr, *p0 = nullptr;
    for (int pass = 0; pass < passes && e == hipSuccess; ++pass) {
      // the last pass ends in keys, pos
      const bool here = (passes - pass) % 2 == 1;
      uint32_t *k1 = here ? a.keys : a.keys2, *p1 = here ? a.pos : a.pos2;
      e = enqueue(embed_count_kernel, dim3((uint32_t)blocks), dim3(kSortThreads), 0, s, a, k0,
                  pass * bits, bits, per);
      if (e == hipSuccess)
        e = enqueue(embed_scatter_kernel, dim3((uint32_t)blocks), dim3(kSortThreads), 0, s, a, k0,
                    p0, k1, p1, pass * bits, bits, per);
      k0 = k1;
      p0 = p1;
    }
  }
  if (e != hipSuccess) return e;
  const int64_t chunks = (a.N + (1 << a.lg_rows) - 1) >> a.lg_rows;
  const int64_t zeros = a.accumulate ? 0 : (a.V + kZeroRows - 1) / kZeroRows;
  return by_type(grad_type, [&](auto to) {
    using G = typename decltype(to)::type;
    hipError_t e = by_type(dout_type, [&](auto from) {
      using T = typename decltype(from)::type;
      const uint32_t slices = (uint32_t)((a.D * (int64_t)sizeof(T) + 1023) / 1024);
      const int64_t units = chunks * slices;
      const int64_t blocks = (units + zeros + 3) / 4;
      if (blocks == 0) return hipSuccess;
      return enqueue(embed_sum_kernel<T, G>, dim3((uint32_t)blocks), dim3(256), 0, s, a, slices,
                     units);
    });
    if (e != hipSuccess || chunks < 2) return e;
    const uint32_t slices = (uint32_t)((a.D + 255) / 256);
    const int waves = chunks > a.V ? 16 : 4;
    return enqueue(waves == 16 ? embed_join_kernel<G, 16> : embed_join_kernel<G, 4>,
                   dim3((uint32_t)((chunks - 1) * slices)), dim3(64 * waves), 0, s, a, slices, chunks);
  });
}

}  // namespace per
