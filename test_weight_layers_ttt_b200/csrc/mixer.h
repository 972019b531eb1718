// Launch wrappers of the token-mixer operators around the layer: the short causal
// convolution (short_conv.cu), the selective scan (selective_scan.cu) and the head norm with
// position rotation (head_norm.cu). All of them enqueue on `s` and return the launch status;
// the arguments were checked by mixer_api.cu.
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace ttt {

// out[c] = sum over r of part[r, c], rows in a fixed order, for the n0 + n1 + n2 columns of three
// outputs side by side (each may be null).
struct SumOuts {
  float* p[3];
  long long n[3];
};
cudaError_t column_sums(const float* part, long long R, const SumOuts& outs, cudaStream_t s);

// ------------------------------------------------------------------ short convolution
struct ConvArgs {
  int B, N, D, width, act;
  long long x_row;          // elements between tokens of x; sequences are N * x_row apart
  const void* x;
  const float* w;           // [width, D]
  const float* bias;        // [D] or null
  const void* state_in;     // [B, width - 1, D] or null
  const int* lens;          // [B] or null
  void* y;                  // forward, step
  void* state_out;          // forward: [B, width - 1, D] or null; step: in and out
  const void* dy;           // backward
  const void* dstate_out;   // [B, width - 1, D] or null
  void* dx;
  void* dstate_in;          // or null
  float* partials;          // backward: conv_bwd_rows() rows of [width + 1, D]
};

cudaError_t conv_fwd(int dt, const ConvArgs& a, cudaStream_t s);
cudaError_t conv_step(int dt, const ConvArgs& a, cudaStream_t s);
// Rows of the backward's partial sums, each [width + 1, D] (tap gradients, then the bias's).
long long conv_bwd_rows(int B, int N, int D);
cudaError_t conv_bwd(int dt, const ConvArgs& a, cudaStream_t s);

// ------------------------------------------------------------------ head norm and rotation
struct HeadArgs {
  int B, N, h, norm, rot, pairs;
  float eps;
  int H[3];                 // heads of q, k, v (0: absent)
  long long row[3];         // elements between tokens of x[i]; heads are h apart
  const void* x[3];         // token-major
  const float* w[2];        // norm weights [h] of q and k, or null
  const float* inv_freq;    // [rot / 2]
  const int* positions;     // [B, N] or null: pos0 + t
  long long pos0;
  void* out[3];             // forward: [B, H, N, h]
  const void* dout[3];      // backward: [B, H, N, h]
  void* dx[3];              // backward: [B, N, H, h]
  float* partials;          // backward with weights: rows of [2, h], one per block
};

cudaError_t head_fwd(int dt, const HeadArgs& a, cudaStream_t s);
// *rows: the rows of partials that the launch writes, at most head_bwd_max_rows().
cudaError_t head_bwd(int dt, const HeadArgs& a, long long* rows, cudaStream_t s);
long long head_bwd_max_rows(int B, int N);

// ------------------------------------------------------------------ selective scan
struct ScanArgs {
  int B, N, D, S, G, softplus;
  long long u_row, dt_row, z_row, b_row, c_row;   // elements between tokens
  const void *u, *dt, *z;                         // [B, N, D]; z may be null
  const void *Bm, *Cm;                            // [B, N, G, S]
  const float* A;                                 // [D, S]
  const float* Dskip;                             // [D] or null
  const float* dt_bias;                           // [D] or null
  const float* state_in;                          // [B, D, S] or null (zeros)
  const int* lens;                                // [B] or null
  void* y;                                        // forward, step: [B, N, D]
  float* state_out;                               // forward: or null; step: in and out
  // The sequence in `chunks` pieces of `chunk` tokens (scan_chunks).
  int chunk, chunks;
  float* ends;    // [B, chunks, D, SP]: chunk end states from zero, then chunk start states
  float* dsum;    // [B, chunks, D]: sum of delta over a chunk
  // backward
  const void* dy;
  const float* dstate_out;                        // [B, D, S] or null
  void *du, *ddt, *dz, *dB, *dC;
  float *dA, *dD, *ddt_bias, *dstate_in;          // dD, ddt_bias, dstate_in may be null
  float* marks;   // [B, subs, D, SP]: state (from the chunk's zero) before each 8 tokens
  float* msum;    // [B, subs, D]: sum of delta from the chunk's start to the mark
  float* back;    // [B, chunks, D, SP]: a chunk's share of the state gradient before it, then
                  // the state gradient behind each chunk
  float* bcpart;  // [channel blocks of a group, B, N, G, 2, SP]: partial dB and dC
  float* part;    // [B, chunks, D S + 2 D]: partial dA, dD and ddt_bias
};

constexpr int kScanSub = 8;            // tokens between two marks of the backward
constexpr int kScanMaxState = 64;
int scan_padded_state(int S);          // SP: 8, 16, 32 or 64
int scan_channel_blocks(int D, int G, int S);   // blocks of one group's channels
// Pieces a sequence is cut into so that the GPU is filled; the piece length goes to *chunk.
int scan_chunks(int B, int N, int D, int G, int S, bool backward, int* chunk);
// The launches of a pass in order; those for chunks == 1 may be skipped (see mixer_api.cu).
cudaError_t scan_fwd_ends(int dt, const ScanArgs& a, cudaStream_t s);
cudaError_t scan_join(const ScanArgs& a, bool backward, cudaStream_t s);
cudaError_t scan_fwd_outputs(int dt, const ScanArgs& a, cudaStream_t s);
cudaError_t scan_step(int dt, const ScanArgs& a, cudaStream_t s);
cudaError_t scan_bwd_marks(int dt, const ScanArgs& a, cudaStream_t s);
cudaError_t scan_bwd_main(int dt, const ScanArgs& a, cudaStream_t s);
cudaError_t scan_bwd_sum_bc(int dt, const ScanArgs& a, cudaStream_t s);

}  // namespace ttt
