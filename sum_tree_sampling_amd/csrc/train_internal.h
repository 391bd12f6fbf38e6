// train_internal.h -- shared definitions of the sequence operators (the public
// ABI is include/per_train.h).
#pragma once

#include "per_internal.h"

namespace per {

// Every launch of these operators goes through here.  An entry point runs its
// launches twice: first `counting`, which only takes the work-items of the
// largest (a dispatch holds fewer than 2^32), so that a call too large for one
// of them is refused before any of them has run.
struct Launches {
  bool counting = false;
  uint64_t items = 0;
};
Launches& launches();  // the calling thread's

template <typename... KArgs, typename... Args>
hipError_t enqueue(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t lds, hipStream_t s,
                   Args... args) {
  Launches& l = launches();
  if (l.counting) {
    const uint64_t n = (uint64_t)grid.x * block.x;
    if (n > l.items) l.items = n;
    return hipSuccess;
  }
  return launch_kernel(kern, grid, block, lds, s, args...);
}

// ------------------------------------------------------------ 8-bit row store
struct RowsArgs {
  uint8_t* codes;
  float* scales;
  int64_t cs, ss;         // strides of a row: bytes, floats
  int64_t capacity;
  int64_t first;          // ring write: slot of row 0
  const int64_t* slots;   // write_at: the slot of each row; read: d_idx
  uint32_t* claims;       // write_at: last batch position + 1 by slot
  const void* src;
  void* out;
  int64_t stride;         // elements between rows of src / out
  uint32_t dim;
  uint32_t rows;          // rows to write, or output rows to read
  uint32_t window;        // read: output rows per index
  int lg_group;           // log2 of the lanes that share a scale (8 columns each); < 0: the row
};
hipError_t launch_rows_write(const RowsArgs& a, int type, int format, hipStream_t s);
hipError_t launch_rows_read(const RowsArgs& a, int type, int format, hipStream_t s);

// --------------------------------------------------- gated linear recurrence
struct ScanArgs {
  int64_t B, T, D;
  const void* x;
  const void* g;
  const void* dy;
  void* y;
  void* dx;
  void* dg;
  int64_t x_sb, x_st, g_sb, g_st, y_sb, y_st, dy_sb, dy_st, dx_sb, dx_st, dg_sb, dg_st;
  const uint8_t* reset;
  const int64_t* length;
  const float* h0;
  float* h_last;
  float* carries;
  const float* dh_last;
  float* dh0;
  float* agg;             // [B x nseg x 2 x D] maps (A, B) of the segments
  float* h0_copy;         // [B x D] h0 as the first kernel found it (h_last may be h0)
  int64_t seg_steps;      // steps of a segment (a multiple of the chunk; T if nseg == 1)
  int nseg;
};
// Workspace and workgroups for this size.
size_t scan_workspace(int64_t B, int64_t T, int64_t D);
int64_t scan_blocks(int64_t B, int64_t T, int64_t D);
hipError_t launch_scan_forward(ScanArgs a, int type, hipStream_t s);
hipError_t launch_scan_backward(ScanArgs a, int type, hipStream_t s);

struct StepArgs {
  int64_t B, D;
  const void* x;
  const void* g;
  void* y;
  int64_t x_st, g_st, y_st;
  const uint8_t* reset;
  const float* h;
  float* h_out;
};
hipError_t launch_scan_step(const StepArgs& a, int type, hipStream_t s);

// --------------------------------------------------------------- distillation
// What a row's teacher entries sum to.
struct Teacher {
  double h;     // sum p log p
  double ps;    // sum p
  double pz;    // sum p (z - z0)
  double rest;  // p_r
  double norm;  // sum of exp((t - largest) / tau) without a rest, else 1
  float z0;     // largest student's logit at an entry
  bool any;     // an entry is present
  bool dup;     // two entries may name one token of the part
};
struct DistillArgs {
  int64_t N, V;
  int K;
  const void* z;
  int64_t stride;
  const int32_t* tidx;
  const void* t;
  int t_type;
  const float* tlse;
  double inv_tau;
  float c;                // log2(e) / tau
  float tau;
  const float* weight;    // NULL: 1
  float* loss;
  float* saved;           // [N x (4 + K)]
  void* grad;
  int64_t grad_stride;
  void* part;             // [N x splits] statistics of 24 bytes
  Teacher* teacher;       // [N]
  int splits;
  bool once;              // logits are loaded past the caches
};
// Whether one wave holds a whole row (then no call needs a workspace), whether
// one workgroup does in per_distill, and if not, how many parts each row is
// split into.
bool distill_small(int64_t N, int64_t V, int type);
bool distill_resident(int64_t N, int64_t V, int type);
int distill_splits(int64_t N, int64_t V, int type);
hipError_t launch_distill_fused(const DistillArgs& a, int type, hipStream_t s);
hipError_t launch_distill_forward(const DistillArgs& a, int type, hipStream_t s);
hipError_t launch_distill_backward(const DistillArgs& a, int type, hipStream_t s);

}  // namespace per
