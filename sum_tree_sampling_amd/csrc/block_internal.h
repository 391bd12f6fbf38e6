// block_internal.h -- shared definitions of the operators of a student that reads
// tokens (the public ABI is include/per_block.h).
#pragma once

#include "../../include/per_block.h"
#include "train_internal.h"

namespace per {

// ------------------------------------------------------------------ embedding
struct EmbedArgs {
  int64_t N, V, D;
  const void* tokens;
  int token_bytes;
  const void* src;        // table, or dout
  void* dst;              // out, or grad
  int64_t src_stride, dst_stride;
  float scale;
  bool accumulate;
  uint32_t *keys, *pos;   // sorted tokens and their positions
  uint32_t *keys2, *pos2; // the other side of each sorting pass
  uint32_t* counts;       // [blocks x bins] of a sorting pass
  float* part;            // [chunks x 2 x D] sums of tokens that chunks share
  int lg_rows;            // log2 of the rows of a chunk
};
size_t embed_workspace(int64_t N, int64_t V, int64_t D, EmbedArgs* a, void* ws);
hipError_t launch_embed_forward(const EmbedArgs& a, int table_type, int out_type, hipStream_t s);
hipError_t launch_embed_backward(EmbedArgs a, int dout_type, int grad_type, hipStream_t s);

// ----------------------------------------------------------------- layer norm
struct NormArgs {
  int64_t N;
  uint32_t D;
  const void* x;
  const void* dy;
  const void* weight;
  const void* bias;
  bool affine_f32;
  float eps;
  void* y;                // y, or dx
  int64_t xs, dys, ys;
  float* stats;           // [N x 2] mean, 1 / deviation
  float* dweight;
  float* dbias;
  float* part;            // [blocks x 2 x D] sums over a block's rows
  float* means;           // [N x 2] mean(e), mean(e xhat) of rows too long for registers
  int blocks;
};
size_t norm_workspace(int64_t N, int64_t D, int type, NormArgs* a, void* ws);
hipError_t launch_norm_forward(const NormArgs& a, int type, hipStream_t s);
hipError_t launch_norm_backward(const NormArgs& a, int type, hipStream_t s);

// ----------------------------------------------------------- gated delta rule
struct Seq {
  void* p;
  int64_t sb, st, sh;
};
struct DeltaArgs {
  int64_t B, T;
  int H, HK, DK, DV;
  int64_t chunks;         // of 64 steps
  Seq q, k, v, g, b, o;   // o: the outputs, or their gradient
  Seq dq, dk, dv, dg, db;
  const uint8_t* reset;
  const int64_t* length;
  const float* s0;        // state before the sequence; backward: gradient of the last state
  float* s_last;          // last state; backward: gradient of s0
  float* carries;
  float scale;
  void* prep;             // per (sequence, chunk, head): what prepare_kernel leaves
  float* dstate;          // backward: gradient of the state behind each chunk
  float* e;               // backward: [B x chunks x H x 64 x DV] E
  int segments;           // of the time axis, 1: not cut
  int segment_chunks;
  float* states;          // [B x H x segments x DK x DV] that segments begin with
  float* locals;          // [..] what a segment makes of a state of 0
  float* maps;            // [B x H x segments x DK x 32, 64 or 128] what it makes of the unit columns
  int* flags;             // [B x H x segments] whether it has a reset
};
size_t delta_workspace(int64_t B, int64_t T, int64_t H, int64_t DK, int64_t DV, int type,
                       bool backward, DeltaArgs* a, void* ws);
hipError_t launch_delta_forward(const DeltaArgs& a, int type, hipStream_t s);
hipError_t launch_delta_backward(const DeltaArgs& a, int type, hipStream_t s);
hipError_t launch_delta_step(const DeltaArgs& a, int type, hipStream_t s);

}  // namespace per
