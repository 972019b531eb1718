// The short causal depthwise convolution: pre[t] = bias + sum_j w[j] x[t - j] for width 2..8
// taps, y = pre or silu(pre), with the last width - 1 inputs as the state of a sequence.
//
// HBM bound: a token costs one read and one write of its channels forward, two reads and one
// write backward. A thread owns V consecutive channels over a run of tokens and slides the
// window through registers, so a row is read once per run (plus width - 1 halo rows) and every
// access of the vector form is 8 or 16 bytes. kRing rows are on their way while one is used
// (when the ring came 2 rows took 74 us, 4 rows 58 us, 8 rows 56 us forward, and 4 rows 70 us, 8
// rows 74 us backward); the arithmetic is two-wide. 2 x 32768 tokens of 1024 channels, width 4,
// silu, bf16: 59 us forward, 4.5 TB/s, the exponential unit (two results per silu) busy 60 % of it
// and the issue slots 51 %; 4 x 4096 tokens of 2048 channels backward: 59 us with the column sums,
// 63 % of the issue slots. Neither is full: both launch 1024 blocks, of which the registers (96 and
// 95) let 5 run on an SM, 1.38 rounds of them. Few channels leave the column sums to few blocks: 16
// x 32768 tokens of 8 channels backward take 248 us, 100 us of it the sums.
#include "mixer.h"
#include "mixer_common.cuh"

namespace ttt {
namespace {

constexpr int kConvThreads = 128;

__device__ __forceinline__ int sequence_length(const int* lens, int b, int N) {
  return lens ? min(max(lens[b], 0), N) : N;
}

// Row `i` of the inputs with the state in front of them (row width - 1 is token 0).
template <typename T, int V, int K>
__device__ __forceinline__ void history_row(const ConvArgs& a, int b, int c, long long i,
                                            float (&f)[V]) {
  if (i >= K - 1) {
    load_vec<T, V>(static_cast<const T*>(a.x) +
                       ((long long)b * a.N + i - (K - 1)) * a.x_row + c, f);
  } else if (a.state_in) {
    load_vec<T, V>(static_cast<const T*>(a.state_in) + ((long long)b * (K - 1) + i) * a.D + c, f);
  } else {
#pragma unroll
    for (int q = 0; q < V; ++q) f[q] = 0.0f;
  }
}

// The rows of up to two tensors on their way to a thread: kRing of them in shared memory by
// asynchronous copies, each thread's own, where a row's access has the 4 bytes that such a copy
// takes at least; else kRing in registers.
constexpr int kRing = 4;
template <typename T, int V, int TENSORS>
struct Rows {
  using U = typename Pack<T, V>::U;
  static constexpr bool shared = V * sizeof(T) >= 4;
  U held[shared ? 1 : TENSORS][shared ? 1 : kRing];
  U* ring;
  __device__ __forceinline__ Rows(U* base) : ring(base + threadIdx.x) {}
  // Entry i (a compile-time number below kRing) of tensor k from p, or zeros.
  __device__ __forceinline__ void load(int k, int i, const T* p, bool on) {
    if constexpr (shared) copy_async<sizeof(U)>(ring + (k * kRing + i) * kConvThreads, p, on);
    else load_here(p, on, held[k][i]);
  }
  __device__ __forceinline__ void loaded() {   // the loads of one row of every tensor
    if constexpr (shared) copies_commit();
  }
  __device__ __forceinline__ void wait_oldest() {
    if constexpr (shared) copies_wait_but<kRing - 1>();
  }
  __device__ __forceinline__ void drain() {    // no copy outlives its thread
    if constexpr (shared) copies_wait();
  }
  __device__ __forceinline__ void take(int k, int i, float (&f)[V]) {
    if constexpr (shared) unpack<T, V>(ring[(k * kRing + i) * kConvThreads], f);
    else unpack<T, V>(held[k][i], f);
  }
};

// V fp32 parameters, aligned or not.
template <int V>
__device__ __forceinline__ void load_params(const float* p, float (&f)[V]) {
#pragma unroll
  for (int q = 0; q < V; ++q) f[q] = p[q];
}

// grid (channel blocks * runs, B): the channel blocks of one run are neighbours.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) conv_fwd_kernel(ConvArgs a, int cblocks, int run) {
  __shared__ __align__(16) typename Pack<T, V>::U ring[V * sizeof(T) >= 4 ? kRing * kConvThreads : 1];
  const int c = ((blockIdx.x % cblocks) * kConvThreads + threadIdx.x) * V;
  if (c >= a.D) return;
  const int b = blockIdx.y;
  const int t0 = (int)(blockIdx.x / cblocks) * run;
  const int t1 = min(a.N, t0 + run);
  const int n = sequence_length(a.lens, b, a.N);
  T* y = static_cast<T*>(a.y) + (long long)b * a.N * a.D + c;
  const T* x = static_cast<const T*>(a.x) + (long long)b * a.N * a.x_row + c;
  float w[K][V], bias[V];
#pragma unroll
  for (int j = 0; j < K; ++j) load_params<V>(a.w + (long long)j * a.D + c, w[j]);
#pragma unroll
  for (int q = 0; q < V; ++q) bias[q] = a.bias ? a.bias[c + q] : 0.0f;

  if (t0 < n) {
    float win[K - 1][V];   // win[j - 1] = x[t - j]
#pragma unroll
    for (int j = 1; j < K; ++j) history_row<T, V, K>(a, b, c, (long long)t0 - j + K - 1, win[j - 1]);
    const int te = min(t1, n);
    Rows<T, V, 1> rows(ring);
    const T* ahead = x + (long long)t0 * a.x_row;
    const auto fetch = [&](int i, int t) {
      rows.load(0, i, ahead, t < te);
      rows.loaded();
      ahead += a.x_row;
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) fetch(i, t0 + i);
    for (int t = t0; t < te; t += kRing) {
#pragma unroll
      for (int i = 0; i < kRing; ++i) {
        float cur[V], o[V];
        rows.wait_oldest();
        rows.take(0, i, cur);
        fetch(i, t + i + kRing);
        fma_v<V>(o, w[0], cur, bias);
#pragma unroll
        for (int j = 1; j < K; ++j) fma_v<V>(o, w[j], win[j - 1], o);
        if (a.act) {
#pragma unroll
          for (int q = 0; q < V; ++q) o[q] *= fast_sigmoid(o[q]);
        }
        if (t + i < te) store_vec<T, V>(y + (long long)(t + i) * a.D, o);
#pragma unroll
        for (int q = 0; q < V; ++q) {
#pragma unroll
          for (int j = K - 2; j > 0; --j) win[j][q] = win[j - 1][q];
          win[0][q] = cur[q];
        }
      }
    }
    rows.drain();
  }
  // rows behind the sequence's end
  const float zero[V] = {};
  for (int t = max(t0, n); t < t1; ++t) store_vec<T, V>(y + (long long)t * a.D, zero);
  // the state: rows n .. n + K - 2 of the history. This thread is the only one that reads
  // its channels' state, and row i is written after row n + i was read, so state_out may be
  // state_in.
  if (a.state_out && t0 == 0) {
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
      float f[V];
      history_row<T, V, K>(a, b, c, (long long)n + i, f);
      store_vec<T, V>(static_cast<T*>(a.state_out) + ((long long)b * (K - 1) + i) * a.D + c, f);
    }
  }
}

// One token per sequence, the state shifted in place. grid (channel blocks, B).
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) conv_step_kernel(ConvArgs a) {
  const int c = (blockIdx.x * kConvThreads + threadIdx.x) * V;
  if (c >= a.D) return;
  const int b = blockIdx.y;
  T* st = static_cast<T*>(a.state_out) + (long long)b * (K - 1) * a.D + c;
  typename Pack<T, V>::U raw[K];   // oldest first
#pragma unroll
  for (int i = 0; i < K - 1; ++i) raw[i] = load_raw<T, V>(st + (long long)i * a.D);
  raw[K - 1] = load_raw<T, V>(static_cast<const T*>(a.x) + (long long)b * a.x_row + c);
  float acc[V];
#pragma unroll
  for (int q = 0; q < V; ++q) acc[q] = a.bias ? a.bias[c + q] : 0.0f;
#pragma unroll
  for (int j = 0; j < K; ++j) {
    float w[V], f[V];
    load_params<V>(a.w + (long long)j * a.D + c, w);
    unpack<T, V>(raw[K - 1 - j], f);
#pragma unroll
    for (int q = 0; q < V; ++q) acc[q] = fmaf(w[q], f[q], acc[q]);
  }
#pragma unroll
  for (int q = 0; q < V; ++q) acc[q] = a.act ? acc[q] * fast_sigmoid(acc[q]) : acc[q];
  store_vec<T, V>(static_cast<T*>(a.y) + (long long)b * a.D + c, acc);
#pragma unroll
  for (int i = 0; i < K - 1; ++i)
    *reinterpret_cast<typename Pack<T, V>::U*>(st + (long long)i * a.D) = raw[i + 1];
}

// With g[t] = dy[t] act'(pre[t]):  dx[t] = sum_j w[j] g[t + j],  dw[j] = sum_t g[t] x[t - j],
// dbias = sum_t g[t]; row i of dstate_out adds to dx of history row n + i. A thread walks its
// run and the width - 1 tokens behind it (their g enters its last dx), and adds dw and dbias
// of its own tokens into one row of partials, which column_sums joins in a fixed order.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kConvThreads) conv_bwd_kernel(ConvArgs a, int cblocks, int run) {
  __shared__ __align__(16) typename Pack<T, V>::U ring[V * sizeof(T) >= 4 ? 2 * kRing * kConvThreads : 1];
  const int c = ((blockIdx.x % cblocks) * kConvThreads + threadIdx.x) * V;
  if (c >= a.D) return;
  const int b = blockIdx.y;
  const int r = blockIdx.x / cblocks, runs = gridDim.x / cblocks;
  const int t0 = r * run, t1 = min(a.N, t0 + run);
  const int n = sequence_length(a.lens, b, a.N);
  const T* x = static_cast<const T*>(a.x) + (long long)b * a.N * a.x_row + c;
  const T* dy = static_cast<const T*>(a.dy) + (long long)b * a.N * a.D + c;
  T* dx = static_cast<T*>(a.dx) + (long long)b * a.N * a.D + c;
  float w[K][V], bias[V], dw[K][V], db[V];
#pragma unroll
  for (int j = 0; j < K; ++j) {
    load_params<V>(a.w + (long long)j * a.D + c, w[j]);
#pragma unroll
    for (int q = 0; q < V; ++q) dw[j][q] = 0.0f;
  }
#pragma unroll
  for (int q = 0; q < V; ++q) {
    bias[q] = a.bias ? a.bias[c + q] : 0.0f;
    db[q] = 0.0f;
  }
  float win[K - 1][V], g[K][V];   // win[j - 1] = x[s - j], g[j] = g[s - j]
#pragma unroll
  for (int j = 0; j < K; ++j)
#pragma unroll
    for (int q = 0; q < V; ++q) g[j][q] = 0.0f;
  if (t0 < n) {
#pragma unroll
    for (int j = 1; j < K; ++j) history_row<T, V, K>(a, b, c, (long long)t0 - j + K - 1, win[j - 1]);
  } else {
#pragma unroll
    for (int j = 1; j < K; ++j)
#pragma unroll
      for (int q = 0; q < V; ++q) win[j - 1][q] = 0.0f;
  }
  const int s1 = t1 + K - 1, se = min(s1, n);
  Rows<T, V, 2> rows(ring);
  const T* ahead_x = x + (long long)t0 * a.x_row;
  const T* ahead_g = dy + (long long)t0 * a.D;
  const auto fetch = [&](int i, int s) {
    rows.load(0, i, ahead_x, s < se);
    rows.load(1, i, ahead_g, s < se);
    rows.loaded();
    ahead_x += a.x_row;
    ahead_g += a.D;
  };
#pragma unroll
  for (int i = 0; i < kRing; ++i) fetch(i, t0 + i);
  for (int s0 = t0; s0 < s1; s0 += kRing) {
#pragma unroll
    for (int i = 0; i < kRing; ++i) {
      const int s = s0 + i;
      float cur[V];
#pragma unroll
      for (int q = 0; q < V; ++q)
#pragma unroll
        for (int j = K - 1; j > 0; --j) g[j][q] = g[j - 1][q];
      rows.wait_oldest();
      rows.take(0, i, cur);           // zeros behind the sequence's end
      rows.take(1, i, g[0]);
      fetch(i, s + kRing);
      if (a.act && s < se) {          // behind the end g is 0, and stays it for an infinite window
        float pre[V];
        fma_v<V>(pre, w[0], cur, bias);
#pragma unroll
        for (int j = 1; j < K; ++j) fma_v<V>(pre, w[j], win[j - 1], pre);
#pragma unroll
        for (int q = 0; q < V; ++q) {
          const float sg = fast_sigmoid(pre[q]);
          g[0][q] *= sg * fmaf(pre[q], 1.0f - sg, 1.0f);
        }
      }
      if (s < se && s < t1) {         // this run's own tokens
        fma_v<V>(dw[0], g[0], cur, dw[0]);
#pragma unroll
        for (int j = 1; j < K; ++j) fma_v<V>(dw[j], g[0], win[j - 1], dw[j]);
#pragma unroll
        for (int q = 0; q < V; ++q) db[q] += g[0][q];
      }
#pragma unroll
      for (int q = 0; q < V; ++q) {
#pragma unroll
        for (int j = K - 2; j > 0; --j) win[j][q] = win[j - 1][q];
        win[0][q] = cur[q];
      }
      const int t = s - (K - 1);      // the row of dx that g[s] completes
      if (s < s1 && (t >= t0 || r == 0)) {
        float o[V] = {};              // rows behind the sequence's end
        if (t < n) {
          mul_v<V>(o, w[0], g[K - 1]);
#pragma unroll
          for (int j = 1; j < K; ++j) fma_v<V>(o, w[j], g[K - 1 - j], o);
        }
        const int i_out = t + K - 1 - n;   // the row of dstate_out that this row became
        if (a.dstate_out && i_out >= 0 && i_out < K - 1) {
          float f[V];
          load_vec<T, V>(static_cast<const T*>(a.dstate_out) +
                             ((long long)b * (K - 1) + i_out) * a.D + c, f);
#pragma unroll
          for (int q = 0; q < V; ++q) o[q] += f[q];
        }
        if (t >= 0)
          store_vec<T, V>(dx + (long long)t * a.D, o);
        else if (a.dstate_in)
          store_vec<T, V>(static_cast<T*>(a.dstate_in) +
                              ((long long)b * (K - 1) + t + K - 1) * a.D + c, o);
      }
    }
  }
  rows.drain();
  float* part = a.partials + ((long long)b * runs + r) * (K + 1) * a.D + c;
#pragma unroll
  for (int q = 0; q < V; ++q) {
#pragma unroll
    for (int j = 0; j < K; ++j) part[(long long)j * a.D + q] = dw[j][q];
    part[(long long)K * a.D + q] = db[q];
  }
}

// 32 columns x 16 row groups per block; row group g adds rows g, g + 16, ... in order.
constexpr int kSumRows = 16;
__global__ void __launch_bounds__(32 * kSumRows) column_sums_kernel(const float* part, long long R, long long C,
                                                                    SumOuts outs) {
  __shared__ float acc[kSumRows][33];
  long long c = (long long)blockIdx.x * 32 + threadIdx.x;
  float v = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (long long r = threadIdx.y; r < R; r += kSumRows) v += part[r * C + c];
  }
  acc[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0 && c < C) {
#pragma unroll
    for (int g = 1; g < kSumRows; ++g) v += acc[g][threadIdx.x];
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      if (c >= 0 && c < outs.n[k] && outs.p[k]) outs.p[k][c] = v;
      c -= outs.n[k];
    }
  }
}

// Tokens of one thread's run. Long runs re-read less halo (width - 1 rows per run); short
// ones give small problems enough threads: `enough` per SM while the run is over 8. 512 forward
// and 256 backward, whose runs re-read at both ends (2 x 8192 tokens of 1024 channels in bf16:
// 19 us against 24 us forward and 37 us against 48 us backward with 1024).
constexpr int kFwdEnough = 512, kBwdEnough = 256;
int conv_run(int B, int N, int D, int V, int enough) {
  const long long groups = (long long)B * ((D + V - 1) / V);
  int run = 64;
  while (run > 8 && groups * ((N + run - 1) / run) < 148LL * enough) run /= 2;
  return run;
}

enum Pass { FWD, BWD, STEP };

// Channels of a vector thread: 16 bytes, 4 elements where a thread holds more rows in
// registers than that leaves room for (the backward's 4 * width + 2, wide forward windows).
constexpr int kBwdVec = 4;
template <typename T>
constexpr int conv_vec(Pass pass, int width) {
  return pass == BWD || (pass == FWD && width > 5) ? 4 : 16 / (int)sizeof(T);
}

template <typename T, Pass P, int V, int K>
cudaError_t launch_width(const ConvArgs& a, cudaStream_t s) {
  const int cblocks = ((a.D + V - 1) / V + kConvThreads - 1) / kConvThreads;
  if constexpr (P == STEP) {
    conv_step_kernel<T, V, K><<<dim3(cblocks, a.B), kConvThreads, 0, s>>>(a);
  } else {
    const int run = P == BWD ? conv_run(a.B, a.N, a.D, kBwdVec, kBwdEnough) : conv_run(a.B, a.N, a.D, V, kFwdEnough);
    const int runs = a.N > 0 ? (a.N + run - 1) / run : 1;
    const dim3 grid((unsigned)((long long)cblocks * runs), a.B);
    if constexpr (P == FWD)
      conv_fwd_kernel<T, V, K><<<grid, kConvThreads, 0, s>>>(a, cblocks, run);
    else
      conv_bwd_kernel<T, V, K><<<grid, kConvThreads, 0, s>>>(a, cblocks, run);
  }
  return cudaGetLastError();
}

// Vector accesses when the channels, the row stride and every buffer allow them, else one
// element at a time.
template <typename T, Pass P, int K>
cudaError_t launch_vec(const ConvArgs& a, cudaStream_t s) {
  constexpr int V = conv_vec<T>(P, K);
  bool vec = a.D % V == 0 && a.x_row % V == 0;
  for (const void* p : {a.x, a.state_in, (const void*)a.y, (const void*)a.state_out, a.dy,
                        a.dstate_out, (const void*)a.dx, (const void*)a.dstate_in})
    vec = vec && reinterpret_cast<uintptr_t>(p) % (V * sizeof(T)) == 0;
  return vec ? launch_width<T, P, V, K>(a, s) : launch_width<T, P, 1, K>(a, s);
}

template <typename T, Pass P>
cudaError_t launch_typed(const ConvArgs& a, cudaStream_t s) {
  switch (a.width) {
    case 2: return launch_vec<T, P, 2>(a, s);
    case 3: return launch_vec<T, P, 3>(a, s);
    case 4: return launch_vec<T, P, 4>(a, s);
    case 5: return launch_vec<T, P, 5>(a, s);
    case 6: return launch_vec<T, P, 6>(a, s);
    case 7: return launch_vec<T, P, 7>(a, s);
    case 8: return launch_vec<T, P, 8>(a, s);
  }
  return cudaErrorInvalidValue;
}

template <Pass P>
cudaError_t launch(int dt, const ConvArgs& a, cudaStream_t s) {
  return dt == DT_BF16 ? launch_typed<bf16, P>(a, s) : launch_typed<float, P>(a, s);
}

}  // namespace

cudaError_t column_sums(const float* part, long long R, const SumOuts& outs, cudaStream_t s) {
  const long long C = outs.n[0] + outs.n[1] + outs.n[2];
  column_sums_kernel<<<(unsigned)((C + 31) / 32), dim3(32, kSumRows), 0, s>>>(part, R, C, outs);
  return cudaGetLastError();
}

cudaError_t conv_fwd(int dt, const ConvArgs& a, cudaStream_t s) { return launch<FWD>(dt, a, s); }
cudaError_t conv_step(int dt, const ConvArgs& a, cudaStream_t s) { return launch<STEP>(dt, a, s); }
cudaError_t conv_bwd(int dt, const ConvArgs& a, cudaStream_t s) { return launch<BWD>(dt, a, s); }

long long conv_bwd_rows(int B, int N, int D) {
  const int run = conv_run(B, N, D, kBwdVec, kBwdEnough);
  return (long long)B * (N > 0 ? (N + run - 1) / run : 1);
}

}  // namespace ttt
