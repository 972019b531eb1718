// The selective state space scan. Per sequence, channel d and state element s
//     delta_t = softplus(dt_t + dt_bias),  a_t = exp(delta_t A[d, s]),
//     h_t = a_t h_{t-1} + delta_t u_t B_t[s],
//     y_t = sum_s C_t[s] h_t + D[d] u_t,  times silu(z_t) when gated.
//
// What bounds it: one exponential per (token, channel, state) - 16 per token and channel at
// the usual S = 16 - against 16 exponentials per clock and SM (measured; the fp32 pipe does 125
// operations, two-wide or not). That is 231 us for 8 x 2048 tokens of 4096 channels, where HBM
// needs 82 us. The kernel takes 447 us: the exponential unit is busy 62 % of it, the shared
// memory pipe 71 %, the schedulers 60 %, so what is left is their overlap.
//
// Layout: a lane keeps 4 states of one channel (2 channels in the backward) in registers, packed
// in pairs for the two-wide fp32 instructions, which halves the issue slots; SL lanes share a
// channel's states; tiles of tokens are staged in shared memory as fp32 with softplus already
// applied, the next tile's operands on their way meanwhile. Larger register tiles have fewer
// instructions and less shared memory traffic, but too few warps: 8 states a lane took 568 us
// against 519 us at the time, 2 channels x 4 states 523 us against 447 us. Each
// lane's part of a sum over states goes through shared memory to the threads that write the
// results (a transposing shuffle took 6 more instructions per token).
//
// The time axis is cut into chunks when batch x channels alone would leave SMs idle: a first
// pass takes each chunk's end state from zero (its decay is exp(A sum delta), one number per
// state), scan_join carries the states over the chunks, and the outputs pass starts every chunk
// from its state. That doubles the exponentials, so it is done only for few channels.
#include <algorithm>
#include <cfloat>

#include "mixer.h"
#include "mixer_common.cuh"

namespace ttt {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- exponentials
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// A for exp2, kept finite: a padded token's step of 0 times it is 0, and its decay 1.
__device__ __forceinline__ float log2_rate(float A) {
  const float a = A * kLog2e;
  return a < -FLT_MAX ? -FLT_MAX : a;
}
// exp2(d a) for the recurrences. Just below 0, where slow decays live, the hardware's result is
// low by 0.6e-8 to 2.7e-8 in the mean (measured), which a recurrence with a memory of 1000
// steps would add up a thousandfold: half of that goes back in with the exponent, whose product
// becomes a fused one at no cost (exp2(0) stays 1).
constexpr float kExpBias = 1.5e-8f;
__device__ __forceinline__ f2 ex2_2(f2 v);
__device__ __forceinline__ f2 decay2(f2 d, f2 a) { return ex2_2(fma2(d, a, both(kExpBias))); }
__device__ __forceinline__ f2 ex2_2(f2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack2(ex2(lo), ex2(hi));
}

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1], for two values. log1p(e) / e is
// a polynomial of degree 9, interpolated at the Chebyshev nodes of [0, 1] (relative error 1.2e-7
// in fp32): it keeps the relative accuracy of small steps, which a logarithm of 1 + e loses, and
// leaves the exponential unit alone.
__device__ __forceinline__ f2 softplus2(f2 x) {
  float lo, hi;
  unpack2(x, lo, hi);
  const f2 e = ex2_2(pack2(-fabsf(lo) * kLog2e, -fabsf(hi) * kLog2e));
  f2 p = both(-0.0031760570127516985f);
  p = fma2(p, e, both(0.019542526453733444f));
  p = fma2(p, e, both(-0.056373611092567444f));
  p = fma2(p, e, both(0.10543623566627502f));
  p = fma2(p, e, both(-0.1526966691017151f));
  p = fma2(p, e, both(0.1966327428817749f));
  p = fma2(p, e, both(-0.24951615929603577f));
  p = fma2(p, e, both(0.33329710364341736f));
  p = fma2(p, e, both(-0.49999892711639404f));
  p = fma2(p, e, both(1.0f));
  return fma2(e, p, pack2(fmaxf(lo, 0.0f), fmaxf(hi, 0.0f)));
}
__device__ __forceinline__ float softplus(float x) {
  float lo, hi;
  unpack2(softplus2(pack2(x, 0.0f)), lo, hi);
  return lo;
}

// ---------------------------------------------------------------- tiles
// N consecutive elements of a row; VEC: in accesses of up to 16 bytes (all N or none valid).
template <typename T, int N, bool VEC> struct Raw {
  static constexpr int W = N * sizeof(T) > 16 ? 16 / (int)sizeof(T) : N;
  union {
    T t[N];
    typename Pack<T, W>::U u[N / W];
    typename Pack<T, 1>::U e[N];
    unsigned w[(N * sizeof(T) + 3) / 4];
  };
  __device__ __forceinline__ void load(const T* p, int valid) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < N / W; ++i) {
        load_here(p + i * W, valid > 0, u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) load_here(p + i, i < valid, e[i]);
    }
  }
  __device__ __forceinline__ void store(T* p, int valid) const {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < N / W; ++i)
        if (valid > 0) reinterpret_cast<typename Pack<T, W>::U*>(p)[i] = u[i];
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i < valid) p[i] = t[i];
    }
  }
  __device__ __forceinline__ float get(int i) const { return to_f32(t[i]); }
  __device__ __forceinline__ void set(int i, float v) { t[i] = from_f32<T>(v); }
  __device__ __forceinline__ void set_pair(int i, float lo, float hi) {   // i even
    if constexpr (VEC && sizeof(T) == 2 && N > 1) {
      w[i / 2] = bf16_pair(lo, hi);
    } else {
      t[i] = from_f32<T>(lo);
      if constexpr (N > 1) t[i + 1] = from_f32<T>(hi);
    }
  }
};

// A block's channels: block cb of group g covers c0 .. c1 - 1.
struct Range {
  int g, c0, c1;
};
__device__ __forceinline__ Range block_channels(int block, int blocks_per_group, int D, int G, int CB) {
  Range r;
  const int per = D / G;
  r.g = block / blocks_per_group;
  r.c0 = r.g * per + (block % blocks_per_group) * CB;
  r.c1 = min(r.c0 + CB, (r.g + 1) * per);
  return r;
}

__device__ __forceinline__ int sequence_length(const int* lens, int b, int N) {
  return lens ? min(max(lens[b], 0), N) : N;
}

// Sums `n` values of each lane over the LANES lanes that differ in the lane bits
// [SHIFT, SHIFT + log2 LANES): afterwards v[0 .. max(1, n / LANES)) of a lane are the sums
// whose index starts with that lane's bits (lanes share a sum where n < LANES).
template <int LANES, int SHIFT, int n, int NV>
__device__ __forceinline__ void butterfly(float (&v)[NV], int lane) {
  if constexpr (LANES > 1) {
    constexpr int mask = (LANES / 2) << SHIFT;
    if constexpr (n > 1) {
      const bool up = lane & mask;
#pragma unroll
      for (int i = 0; i < n / 2; ++i) {
        const float keep = up ? v[i + n / 2] : v[i], send = up ? v[i] : v[i + n / 2];
        v[i] = keep + __shfl_xor_sync(0xffffffffu, send, mask);
      }
      butterfly<LANES / 2, SHIFT, n / 2>(v, lane);
    } else {
      v[0] += __shfl_xor_sync(0xffffffffu, v[0], mask);
      butterfly<LANES / 2, SHIFT, 1>(v, lane);
    }
  }
}

// ---------------------------------------------------------------- forward
// A lane holds M states of one channel, packed in pairs; SL lanes share a channel (lane =
// state group * CH + channel: groups in the high lane bits, so that a 16-byte read of B or C,
// the same for all channels, takes 2 cycles of the shared memory pipe instead of 4).
constexpr int kFwdWarps = 4, kFwdThreads = 32 * kFwdWarps;

template <int SL> struct FwdTile {
  static constexpr int M = 4;
  static constexpr int SP = M * SL;                        // padded states
  static constexpr int CH = 32 / SL;                       // channels of a warp
  static constexpr int CB = kFwdWarps * CH;                // channels of a block
  static constexpr int TT = SL == 2 ? 8 : SL == 4 ? 16 : 32;   // tokens of a staged tile
  static constexpr int EPT = TT * CB / kFwdThreads;        // channels a thread stages (one token)
  static constexpr int TPR = CB / EPT;                     // threads of a token's row
  static constexpr int BCN = TT * SP / 4 / kFwdThreads > 0 ? TT * SP / 4 / kFwdThreads : 1;
};

// TT rows of B or C of one group, four states at a time: held in registers between the load
// and the store so that the next tile's loads run under this one's arithmetic.
template <typename T, int SL>
struct RowsBC {
  using L = FwdTile<SL>;
  Raw<T, 4, true> v[L::BCN];
  __device__ __forceinline__ void load(const T* p, long long row, int S, bool vec, int live) {
#pragma unroll
    for (int j = 0; j < L::BCN; ++j) {
      const int i = threadIdx.x + j * kFwdThreads, k = i / (L::SP / 4), s = i % (L::SP / 4) * 4;
      const int on = k < min(live, L::TT) ? S - s : 0;
      if (vec) {
        v[j].load(p + k * row + s, on);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) load_here(p + k * row + s + q, q < on, v[j].e[q]);
      }
    }
  }
  __device__ __forceinline__ void store(float* dst) const {
#pragma unroll
    for (int j = 0; j < L::BCN; ++j) {
      const int i = threadIdx.x + j * kFwdThreads;
      const float f[4] = {v[j].get(0), v[j].get(1), v[j].get(2), v[j].get(3)};
      if (i < L::TT * L::SP / 4) store_vec<float, 4>(dst + i * 4, f);
    }
  }
};

// One chunk of one sequence for CB channels. OUT: from the chunk's start state, writing y (and
// the state behind the last chunk); else from zero, writing the end state and the sum of delta.
// grid (channel blocks, chunks, B).
template <typename T, int SL, bool VEC, bool OUT>
__global__ void __launch_bounds__(kFwdThreads) scan_fwd_kernel(ScanArgs a, int blocks_per_group,
                                                               bool vec_b, bool vec_c) {
  using L = FwdTile<SL>;
  constexpr int TT = L::TT, CB = L::CB, SP = L::SP, EPT = L::EPT, M = L::M;
  constexpr bool AHEAD = L::BCN <= 2;   // B and C of the next tile are loaded a tile ahead
  constexpr int UN = 4;                 // tokens in one basic block (2: 456 us, 8: 467 us, 4: 447 us
                                        // at 8 x 2048 tokens of 4096 channels)
  __shared__ __align__(16) float2 sDU[TT * CB];            // delta; delta u
  __shared__ __align__(16) float sY[OUT ? SL * TT * CB : 4];   // each state group's sum of C h
  __shared__ __align__(16) float sB[TT * SP], sC[OUT ? TT * SP : 4];
  __shared__ __align__(16) float sBias[CB], sSkip[CB];
  const Range r = block_channels(blockIdx.x, blocks_per_group, a.D, a.G, CB);
  const int chunk = blockIdx.y, b = blockIdx.z;
  const int len = sequence_length(a.lens, b, a.N);
  const int t0 = chunk * a.chunk, t1 = min(a.N, t0 + a.chunk), te = min(t1, len);
  const int lane = threadIdx.x % 32, sl = lane / L::CH;
  const int cw = threadIdx.x / 32 * L::CH + lane % L::CH, c = r.c0 + cw;   // channel in block; channel
  const bool mine = c < r.c1;
  // staging: EPT channels of one token per thread
  const int row = threadIdx.x / L::TPR, col = threadIdx.x % L::TPR * EPT;
  const int sc = r.c0 + col, valid = min(EPT, r.c1 - sc);
  const long long seq = (long long)b * a.N;
  for (int i = threadIdx.x; i < CB; i += kFwdThreads) {
    const bool in = r.c0 + i < r.c1;
    sBias[i] = a.dt_bias && in ? a.dt_bias[r.c0 + i] : 0.0f;
    sSkip[i] = OUT && a.Dskip && in ? a.Dskip[r.c0 + i] : 0.0f;
  }
  __syncthreads();
  f2 A2[M / 2], h[M / 2];
  float dsum = 0.0f;
  const long long at = (((long long)b * a.chunks + chunk) * a.D + c) * SP + sl * M;
  {
    float v[M], w[M] = {};
    const long long io = ((long long)b * a.D + c) * a.S;
#pragma unroll
    for (int i = 0; i < M; ++i) {
      const int s = sl * M + i;
      const bool on = mine && s < a.S;
      v[i] = on ? log2_rate(a.A[(long long)c * a.S + s]) : 0.0f;
      if (OUT && a.chunks > 1) w[i] = mine ? a.ends[at + i] : 0.0f;
      else if (OUT && a.state_in) w[i] = on ? a.state_in[io + s] : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < M / 2; ++i) {
      A2[i] = pack2(v[2 * i], v[2 * i + 1]);
      h[i] = pack2(w[2 * i], w[2 * i + 1]);
    }
  }
  Raw<T, EPT, VEC> ru, rd, rz;
  RowsBC<T, SL> rb, rc;
  // the next tile's rows
  const T* pB = static_cast<const T*>(a.Bm) + (seq + t0) * a.b_row + (long long)r.g * a.S;
  const T* pC = static_cast<const T*>(a.Cm) + (seq + t0) * a.c_row + (long long)r.g * a.S;
  const T* pu = static_cast<const T*>(a.u) + (seq + t0 + row) * a.u_row + sc;
  const T* pd = static_cast<const T*>(a.dt) + (seq + t0 + row) * a.dt_row + sc;
  const T* pz = static_cast<const T*>(a.z) + (seq + t0 + row) * a.z_row + sc;
  T* py = static_cast<T*>(a.y) + (seq + t0 + row) * a.D + sc;
  auto fetch_bc = [&](int t) {
    rb.load(pB, a.b_row, a.S, vec_b, te - t);
    if (OUT) rc.load(pC, a.c_row, a.S, vec_c, te - t);
    pB += TT * a.b_row;
    pC += TT * a.c_row;
  };
  auto fetch = [&](int t) {
    const int ok = t + row < te ? valid : 0;
    ru.load(pu, ok);
    rd.load(pd, ok);
    if (OUT && a.z) rz.load(pz, ok);
    if (AHEAD) fetch_bc(t);
    pu += TT * a.u_row;
    pd += TT * a.dt_row;
    if (OUT) pz += TT * a.z_row;
  };
  fetch(t0);
  for (int t = t0; t < te; t += TT) {
    const bool on = t + row < te;
    if (!AHEAD) fetch_bc(t);
    rb.store(sB);
    if (OUT) rc.store(sC);
#pragma unroll
    for (int i = 0; i < EPT; i += 2) {   // (columns behind c1 are staged and not used)
      f2 d = add2(pack2(rd.get(i), rd.get(i + 1)), *reinterpret_cast<const f2*>(&sBias[col + i]));
      if (a.softplus) d = softplus2(d);
      if (!on) d = 0;
      float d0, d1;
      unpack2(d, d0, d1);
      store_vec<float, 4>(&sDU[row * CB + col + i].x, {d0, d0 * ru.get(i), d1, d1 * ru.get(i + 1)});
    }
    __syncthreads();
    const Raw<T, EPT, VEC> uu = ru, zz = rz;
    fetch(t + TT);   // nothing behind te; unconditional, for a branch would wait for its loads

#pragma unroll 1
    for (int k0 = 0; k0 < TT; k0 += UN) {
      float sum[UN];   // stored behind the last read: a store would hold back the reads after it
#pragma unroll
      for (int j = 0; j < UN; ++j) {
        const int k = k0 + j;
        const float2 du = sDU[k * CB + cw];
        const f2 d2 = pack2(du.x, du.x), x2 = pack2(du.y, du.y);
        if (!OUT) dsum += du.x;
        f2 y = 0;
#pragma unroll
        for (int i = 0; i < M / 2; ++i) {
          const f2 e = decay2(d2, A2[i]);
          h[i] = fma2(e, h[i], mul2(x2, *reinterpret_cast<const f2*>(&sB[k * SP + sl * M + 2 * i])));
          if (OUT) y = fma2(h[i], *reinterpret_cast<const f2*>(&sC[k * SP + sl * M + 2 * i]), y);
        }
        if (OUT) {
          float lo, hi;
          unpack2(y, lo, hi);
          sum[j] = lo + hi;
        }
      }
      if (OUT) {
#pragma unroll
        for (int j = 0; j < UN; ++j) sY[((k0 + j) * kFwdWarps + threadIdx.x / 32) * 32 + lane] = sum[j];
      }
    }
    __syncthreads();
    if (OUT && on) {
      Raw<T, EPT, VEC> out;
#pragma unroll
      for (int i = 0; i < EPT; i += 2) {
        // the groups' sums from another one on in each warp's channels: no bank is read twice
        f2 y = mul2(*reinterpret_cast<const f2*>(&sSkip[col + i]), pack2(uu.get(i), uu.get(i + 1)));
#pragma unroll
        for (int q = 0; q < SL; ++q)
          y = add2(y, *reinterpret_cast<const f2*>(&sY[(row * kFwdWarps + col / L::CH) * 32 +
                                                      (q + col / L::CH) % SL * L::CH + col % L::CH + i]));
        if (a.z) {
          const float z0 = zz.get(i), z1 = zz.get(i + 1);
          y = mul2(y, mul2(pack2(z0, z1), pack2(fast_sigmoid(z0), fast_sigmoid(z1))));
        }
        float y0, y1;
        unpack2(y, y0, y1);
        out.set_pair(i, y0, y1);
      }
      out.store(py, valid);
    }
    py += TT * (long long)a.D;
  }
  if (OUT) {
    Raw<T, EPT, VEC> zero;   // rows behind the sequence's end
#pragma unroll
    for (int i = 0; i < EPT; ++i) zero.set(i, 0.0f);
    for (int t = max(t0, len) + row; t < t1; t += TT)
      zero.store(static_cast<T*>(a.y) + (seq + t) * a.D + sc, valid);
  }
  float w[M];
#pragma unroll
  for (int i = 0; i < M / 2; ++i) unpack2(h[i], w[2 * i], w[2 * i + 1]);
  if (OUT) {
    if (a.state_out && chunk == a.chunks - 1 && mine) {
#pragma unroll
      for (int i = 0; i < M; ++i)
        if (sl * M + i < a.S) a.state_out[((long long)b * a.D + c) * a.S + sl * M + i] = w[i];
    }
  } else if (mine) {
#pragma unroll
    for (int i = 0; i < M; ++i) a.ends[at + i] = w[i];
    if (sl == 0) a.dsum[((long long)b * a.chunks + chunk) * a.D + c] = dsum;
  }
}

// Carries states over the chunks, in place: ends[k] becomes the state chunk k starts from, and
// in the backward back[k] the state gradient behind chunk k. One thread per (b, d, s) and
// direction; eight chunks' loads at a time, for the recurrence itself is short, its loads are not.
template <bool BWD>
__global__ void __launch_bounds__(256) scan_join_kernel(ScanArgs a, int SP) {
  constexpr int U = 8;
  const long long n = (long long)a.B * a.D * SP;
  TTT_GRID_LOOP(item, BWD ? 2 * n : n) {
    const bool back = BWD && item >= n;
    const long long i = back ? item - n : item;
    const int s = (int)(i % SP);
    const long long bd = i / SP;
    const int d = (int)(bd % a.D), b = (int)(bd / a.D);
    const bool on = s < a.S;
    const float A2 = on ? log2_rate(a.A[(long long)d * a.S + s]) : 0.0f;
    const float* first = back ? a.dstate_out : a.state_in;
    float* io = back ? a.back : a.ends;
    float h = on && first ? first[bd * a.S + s] : 0.0f;
    const int last = a.chunks - 1;
    const long long bk = (long long)b * a.chunks;
    // step j of the walk is chunk j forward, chunk last - j backward
    const auto chunk = [&](int j) { return bk + (back ? last - j : j); };
    for (int j0 = 0; j0 <= last; j0 += U) {
      float end[U], sum[U];
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const bool in = j0 + j < last;   // the walk's last chunk passes nothing on
        end[j] = in ? io[(chunk(j0 + j) * a.D + d) * SP + s] : 0.0f;
        sum[j] = in ? a.dsum[chunk(j0 + j) * a.D + d] : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (j0 + j > last) break;
        io[(chunk(j0 + j) * a.D + d) * SP + s] = h;
        h = fmaf(ex2(A2 * sum[j]), h, end[j]);
      }
    }
  }
}

// ---------------------------------------------------------------- one token
// SL lanes per channel, 4 states each, for NB sequences: the state is read and written once (HBM
// bound for many sequences, one launch's latency for few). With NB > 1 a lane has that many
// state loads in flight and reads A once for them. VEC: whole aligned runs of four states
// everywhere. grid (channels, B / NB).
template <typename T, int SL, bool VEC, int NB>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanArgs a) {
  const int i = blockIdx.x * (kThreads / SL) + threadIdx.x / SL, b0 = blockIdx.y * NB;
  const int s0 = threadIdx.x % SL * 4;
  const bool on = i < a.D;
  const int d = on ? i : a.D - 1, g = d / (a.D / a.G);
  const float* A = a.A + (long long)d * a.S;
  float h[NB][4] = {}, A4[4] = {}, B4[NB][4] = {}, C4[NB][4] = {}, u[NB], z[NB], delta[NB];
  const auto state = [&](int j) { return a.state_out + ((long long)(b0 + j) * a.D + d) * a.S + s0; };
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    const int b = min(b0 + j, a.B - 1);
    const T* Bm = static_cast<const T*>(a.Bm) + b * a.b_row + (long long)g * a.S + s0;
    const T* Cm = static_cast<const T*>(a.Cm) + b * a.c_row + (long long)g * a.S + s0;
    const bool live = b0 + j < a.B;
    if constexpr (VEC) {
      if (s0 < a.S && live) load_vec<float, 4>(state(j), h[j]);
      if (s0 < a.S) {
        load_input<T, 4>(Bm, B4[j]);
        load_input<T, 4>(Cm, C4[j]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (s0 + k < a.S) {
          if (live) h[j][k] = state(j)[k];
          B4[j][k] = to_f32(Bm[k]);
          C4[j][k] = to_f32(Cm[k]);
        }
    }
    u[j] = to_f32(static_cast<const T*>(a.u)[b * a.u_row + d]);
    z[j] = a.z ? to_f32(static_cast<const T*>(a.z)[b * a.z_row + d]) : 0.0f;
    delta[j] = to_f32(static_cast<const T*>(a.dt)[b * a.dt_row + d]);
  }
  const float bias = a.dt_bias ? a.dt_bias[d] : 0.0f, skip = a.Dskip ? a.Dskip[d] : 0.0f;
  if constexpr (VEC) {
    if (s0 < a.S) load_input<float, 4>(A + s0, A4);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s0 + k < a.S) A4[k] = A[s0 + k];
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) A4[k] = log2_rate(A4[k]);
#pragma unroll
  for (int j = 0; j < NB; ++j) {
    delta[j] += bias;
    if (a.softplus) delta[j] = softplus(delta[j]);
    float y = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      h[j][k] = fmaf(ex2(fmaf(delta[j], A4[k], kExpBias)), h[j][k], delta[j] * u[j] * B4[j][k]);
      y = fmaf(h[j][k], C4[j][k], y);
    }
    const bool live = on && b0 + j < a.B;
    if (live) {
      if constexpr (VEC) {
        if (s0 < a.S) store_vec<float, 4>(state(j), h[j]);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (s0 + k < a.S) state(j)[k] = h[j][k];
      }
    }
#pragma unroll
    for (int m = SL / 2; m > 0; m /= 2) y += __shfl_xor_sync(0xffffffffu, y, m);
    if (live && s0 == 0) {
      y = fmaf(skip, u[j], y);
      if (a.z) y *= z[j] * fast_sigmoid(z[j]);
      static_cast<T*>(a.y)[(long long)(b0 + j) * a.D + d] = from_f32<T>(y);
    }
  }
}

// ---------------------------------------------------------------- backward
// With g_t = dy_t silu(z_t) and dh_t = C_t g_t + a_{t+1} dh_{t+1}:
//     p_t = dh_t a_t h_{t-1},  x_t = sum_s dh_t B_t,
//     dA += delta_t p_t,  dB_t = sum_d dh_t delta_t u_t,  dC_t = sum_d g_t h_t,
//     du_t = D g_t + delta_t x_t,  ddelta_t = sum_s A p_t + u_t x_t,
//     dz_t = dy_t silu'(z_t) (sum_s C_t h_t + D u_t).
// The states are recomputed, not saved: the first pass leaves a mark (the state from the
// chunk's zero) every 8 tokens and the main pass walks the marks backwards. Marks of 8 tokens
// cost S / 8 * 4 bytes per token and channel (8 at S = 16, less than the operands), and their
// states recomputed are as many as registers hold. Some 25 fp32 operations and 2.5 exponentials
// per state, 7 shuffles per token of a lane (8 states), shared memory and scheduler cycles around
// them: at 4 x 4096 tokens of 2048 channels 980 us (258 us marks, 690 us main pass, 32 us joins and
// sums) against 115 us of exponentials and some 290 us of fp32 operations; the main pass issues 53 %
// of the time with the 12 warps per SM that its registers leave.

// Marks, chunk end states, and with more than one chunk the chunk's share of the state gradient
// in front of it, sum_t (prod_{t' <= t} a_t') C_t g_t. Same tiling as the forward.
template <typename T, int SL, bool VEC, bool SPLIT>
__global__ void __launch_bounds__(kFwdThreads) scan_marks_kernel(ScanArgs a, int blocks_per_group,
                                                                 bool vec_b, bool vec_c) {
  using L = FwdTile<SL>;
  constexpr int TT = L::TT, CB = L::CB, SP = L::SP, EPT = L::EPT, M = L::M;
  constexpr bool AHEAD = L::BCN <= 2;
  __shared__ __align__(16) float2 sDU[TT * CB];   // delta; delta u
  __shared__ __align__(16) float sG[SPLIT ? TT * CB : 4];
  __shared__ __align__(16) float sB[TT * SP], sC[SPLIT ? TT * SP : 4];
  const Range r = block_channels(blockIdx.x, blocks_per_group, a.D, a.G, CB);
  const int chunk = blockIdx.y, b = blockIdx.z;
  const int len = sequence_length(a.lens, b, a.N);
  const int t0 = chunk * a.chunk, te = min(min(a.N, t0 + a.chunk), len);
  const int lane = threadIdx.x % 32, sl = lane / L::CH;
  const int cw = threadIdx.x / 32 * L::CH + lane % L::CH, c = r.c0 + cw;
  const bool mine = c < r.c1;
  const int row = threadIdx.x / L::TPR, col = threadIdx.x % L::TPR * EPT;
  const int sc = r.c0 + col, valid = min(EPT, r.c1 - sc);
  const long long seq = (long long)b * a.N;
  const int subs = (a.N + kScanSub - 1) / kScanSub;
  float bias[EPT];
#pragma unroll
  for (int i = 0; i < EPT; ++i) bias[i] = a.dt_bias && i < valid ? a.dt_bias[sc + i] : 0.0f;
  f2 A2[M / 2], h[M / 2], prod[M / 2], share[M / 2];
  float dsum = 0.0f;
#pragma unroll
  for (int i = 0; i < M / 2; ++i) {
    const int s = sl * M + 2 * i;
    const float lo = mine && s < a.S ? a.A[(long long)c * a.S + s] : 0.0f;
    const float hi = mine && s + 1 < a.S ? a.A[(long long)c * a.S + s + 1] : 0.0f;
    A2[i] = pack2(log2_rate(lo), log2_rate(hi));
    h[i] = share[i] = 0;
    prod[i] = both(1.0f);
  }
  Raw<T, EPT, VEC> ru, rd, rz, rg;
  RowsBC<T, SL> rb, rc;
  // the next tile's rows
  const T* pB = static_cast<const T*>(a.Bm) + (seq + t0) * a.b_row + (long long)r.g * a.S;
  const T* pC = static_cast<const T*>(a.Cm) + (seq + t0) * a.c_row + (long long)r.g * a.S;
  const T* pu = static_cast<const T*>(a.u) + (seq + t0 + row) * a.u_row + sc;
  const T* pd = static_cast<const T*>(a.dt) + (seq + t0 + row) * a.dt_row + sc;
  const T* pz = static_cast<const T*>(a.z) + (seq + t0 + row) * a.z_row + sc;
  const T* pg = static_cast<const T*>(a.dy) + (seq + t0 + row) * a.D + sc;
  auto fetch_bc = [&](int t) {
    rb.load(pB, a.b_row, a.S, vec_b, te - t);
    if (SPLIT) rc.load(pC, a.c_row, a.S, vec_c, te - t);
    pB += TT * a.b_row;
    pC += TT * a.c_row;
  };
  auto fetch = [&](int t) {
    const int ok = t + row < te ? valid : 0;
    ru.load(pu, ok);
    rd.load(pd, ok);
    if (SPLIT) rg.load(pg, ok);
    if (SPLIT && a.z) rz.load(pz, ok);
    if (AHEAD) fetch_bc(t);
    pu += TT * a.u_row;
    pd += TT * a.dt_row;
    if (SPLIT) pz += TT * a.z_row;
    if (SPLIT) pg += TT * (long long)a.D;
  };
  const auto store_states = [&](float* p, const f2 (&v)[M / 2]) {   // p: the channel's row
    float w[M];
#pragma unroll
    for (int i = 0; i < M / 2; ++i) unpack2(v[i], w[2 * i], w[2 * i + 1]);
    if (mine) store_vec<float, M>(p + sl * M, w);
  };
  fetch(t0);
  for (int t = t0; t < te; t += TT) {
    const bool on = t + row < te;
    if (!AHEAD) fetch_bc(t);
    rb.store(sB);
    if (SPLIT) rc.store(sC);
#pragma unroll
    for (int i = 0; i < EPT; i += 2) {
      f2 d = add2(pack2(rd.get(i), rd.get(i + 1)), pack2(bias[i], bias[i + 1]));
      if (a.softplus) d = softplus2(d);
      if (!on) d = 0;
      float d0, d1;
      unpack2(d, d0, d1);
      store_vec<float, 4>(&sDU[row * CB + col + i].x, {d0, d0 * ru.get(i), d1, d1 * ru.get(i + 1)});
      if (SPLIT) {
        float g0 = rg.get(i), g1 = rg.get(i + 1);
        if (a.z) {
          const float z0 = rz.get(i), z1 = rz.get(i + 1);
          g0 *= z0 * fast_sigmoid(z0);
          g1 *= z1 * fast_sigmoid(z1);
        }
        store_vec<float, 2>(&sG[row * CB + col + i], {g0, g1});
      }
    }
    __syncthreads();
    fetch(t + TT);
#pragma unroll 1
    for (int k0 = 0; k0 < TT && t + k0 < te; k0 += kScanSub) {
      const long long mark = (long long)b * subs + (t + k0) / kScanSub;
      store_states(a.marks + (mark * a.D + c) * SP, h);
      if (sl == 0 && mine) a.msum[mark * a.D + c] = dsum;
#pragma unroll
      for (int j = 0; j < kScanSub; ++j) {
        const int k = k0 + j;
        const float2 du = sDU[k * CB + cw];
        const f2 d2 = both(du.x), x2 = both(du.y), g2 = both(SPLIT ? sG[k * CB + cw] : 0.0f);
        dsum += du.x;
#pragma unroll
        for (int i = 0; i < M / 2; ++i) {
          const f2 e = decay2(d2, A2[i]);
          h[i] = fma2(e, h[i], mul2(x2, *reinterpret_cast<const f2*>(&sB[k * SP + sl * M + 2 * i])));
          if (SPLIT) {
            prod[i] = mul2(prod[i], e);
            share[i] = fma2(prod[i], mul2(g2, *reinterpret_cast<const f2*>(&sC[k * SP + sl * M + 2 * i])), share[i]);
          }
        }
      }
    }
    __syncthreads();
  }
  const long long at = ((long long)b * a.chunks + chunk) * a.D + c;
  if (SPLIT) {
    store_states(a.ends + at * SP, h);
    store_states(a.back + at * SP, share);
    if (sl == 0 && mine) a.dsum[at] = dsum;
  }
}

// The main pass's tile: a lane holds 2 channels x 4 states (8 recurrences, so that the sums
// over the channels, whose shuffles cost most, run over fewer lanes), lane = state group * CL +
// channel pair.
template <int SL> struct BwdTile {
  static constexpr int SP = 4 * SL;
  static constexpr int CL = 32 / SL;                       // channel pairs of a warp
  static constexpr int WC = 2 * CL;                        // channels of a warp
  static constexpr int CB = kWarps * WC;                   // channels of a block
  static constexpr int EPT = kScanSub * CB / kThreads;     // channels a thread stages (one token)
  static constexpr int TPR = CB / EPT;                     // threads of a token's row
};

// Shared memory of a main-pass block. `raw` holds the operands of the 8 tokens as they are in
// memory (u, dt, z, dy), for the staging and again for the per-channel results: registers are
// what the recurrences need.
template <typename T, int SL> struct BwdShared {
  using L = BwdTile<SL>;
  static constexpr int K = kScanSub, CB = L::CB, SP = L::SP;
  float4 du[K * CB / 2];            // channel pair: delta, delta, delta u, delta u
  float4 px[K * kThreads];          // sums over a lane's 4 states: p and x of both channels
  float2 y[K * kThreads];           // C h of both channels
  float4 start[2 * kThreads];       // the chunk's start state, lane by lane
  float4 marks[2][CB * SL];         // states before the 8 tokens, 4 per entry, see mark_slot
  alignas(16) float g[K * CB];
  float B[K * SP], C[K * SP];
  float w[kWarps][K][2 * SP];       // sums over a warp's channels
  float acc[2][K * CB];             // dD and ddt_bias of each staging slot
  float bias[CB], skip[CB];         // dt_bias and D, zeros where absent
  float msum[2][CB];
  alignas(16) T raw[2][4][K * CB];
  alignas(16) T rawbc[2][2][K * SP];
};

// Shared memory read before is read again after this, not kept in registers: the passes over the
// 8 tokens read the same operands, and the compiler would hold them (and the exponentials of
// the first 4 tokens) at the price of spilling the states.
__device__ __forceinline__ void read_again() { asm volatile("" ::: "memory"); }

// Where a lane's sums lie among its warp's 32 in BwdShared::px and y: even channel pairs first,
// odd ones first in odd warps, so that the threads which add them up (two pairs of two warps
// in a quarter warp) read different banks.
template <int CL>
__device__ __forceinline__ int sum_slot(int warp, int sl, int cl) {
  return warp * 32 + sl * CL + cl / 2 + (((cl ^ warp) & 1) ? CL / 2 : 0);
}

// Where 4 states (group sl) of channel ch lie in BwdShared::marks: rotated by the channel pair,
// for the lanes of a quarter warp read one group of different pairs.
template <int SL>
__device__ __forceinline__ int mark_slot(int ch, int sl) {
  return ch * SL + ((sl + ch / 2) & (SL - 1));
}

// The main pass of one chunk, 8 tokens at a time from its end. grid (channel blocks, chunks, B).
// Of the 8 tokens only 4 at a time hold their a_t and h_t in registers: the first 4 are run
// through once for the state in front of the last 4, and again when their turn comes. That is
// half an exponential more per state, and three blocks per SM instead of two (1251 us against
// 1322 us at the time, both sides without spills; not for S <= 8, whose shared memory of 79 KB in
// bf16 and 96 KB in fp32 leaves room for two, and which spill 12 bytes; 2 tokens at a time, four blocks and 1.75
// exponentials 702 to 753 us against 700 us). A token's operands are read, and its channel
// sums shuffled, a token apart from their use (756 -> 698 us). VEC: the next 8 tokens' operands
// come by asynchronous copies under this one's arithmetic; else through registers, two blocks.
template <typename T, int SL, bool VEC>
__global__ void __launch_bounds__(kThreads, VEC ? 3 : 2) scan_bwd_kernel(ScanArgs a, int blocks_per_group,
                                                                         bool vec_b, bool vec_c) {
  using L = BwdTile<SL>;
  constexpr int K = kScanSub, H = K / 2, CB = L::CB, SP = L::SP, EPT = L::EPT, CL = L::CL;
  extern __shared__ __align__(16) unsigned char smem[];
  BwdShared<T, SL>& sm = *reinterpret_cast<BwdShared<T, SL>*>(smem);
  const Range r = block_channels(blockIdx.x, blocks_per_group, a.D, a.G, CB);
  const int chunk = blockIdx.y, b = blockIdx.z;
  const int len = sequence_length(a.lens, b, a.N);
  const int t0 = chunk * a.chunk, t1 = min(a.N, t0 + a.chunk), te = min(t1, len);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int sl = lane / CL, cl = lane % CL, pair = warp * CL + cl;   // state group; channel pair
  const int c = r.c0 + 2 * pair;
  const int row = threadIdx.x / L::TPR, col = threadIdx.x % L::TPR * EPT, slot = row * CB + col;
  const int sc = r.c0 + col, valid = min(EPT, r.c1 - sc);
  const long long seq = (long long)b * a.N;
  const int subs = (a.N + K - 1) / K;
  const int cb = blockIdx.x % blocks_per_group;
  float* bcpart = a.bcpart + (((long long)cb * a.B + b) * a.N * a.G + r.g) * 2 * SP;
  f2 A2[2][2], carry[2][2], dA[2][2];   // [channel][state pair]
  const long long bk = (long long)b * a.chunks + chunk;
#pragma unroll
  for (int z = 0; z < 2; ++z) {
    float w[4] = {}, g[4] = {}, v[4];
    if (c + z < r.c1 && a.chunks > 1) {
      load_vec<float, 4>(a.ends + (bk * a.D + c + z) * SP + sl * 4, w);
      load_vec<float, 4>(a.back + (bk * a.D + c + z) * SP + sl * 4, g);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = sl * 4 + i;
      const bool on = c + z < r.c1 && s < a.S;
      const long long io = ((long long)b * a.D + c + z) * a.S + s;
      v[i] = on ? log2_rate(a.A[(long long)(c + z) * a.S + s]) : 0.0f;
      if (on && a.chunks == 1) {        // one piece: nothing was joined
        w[i] = a.state_in ? a.state_in[io] : 0.0f;
        g[i] = a.dstate_out ? a.dstate_out[io] : 0.0f;
      }
    }
    sm.start[z * kThreads + threadIdx.x] = make_float4(w[0], w[1], w[2], w[3]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      carry[z][i] = pack2(g[2 * i], g[2 * i + 1]);
      A2[z][i] = pack2(v[2 * i], v[2 * i + 1]);
      dA[z][i] = 0;
    }
  }
#pragma unroll
  for (int i = 0; i < EPT; ++i) sm.acc[0][slot + i] = sm.acc[1][slot + i] = 0.0f;
  for (int i = threadIdx.x; i < CB; i += kThreads) {
    const bool in = r.c0 + i < r.c1;
    sm.bias[i] = a.dt_bias && in ? a.dt_bias[r.c0 + i] : 0.0f;
    sm.skip[i] = a.Dskip && in ? a.Dskip[r.c0 + i] : 0.0f;
  }
  const int lane_sum = sum_slot<CL>(warp, sl, cl);

  const int last = te > t0 ? (te - 1 - t0) / K * K + t0 : t0 - K;   // first token of the last 8
  // the next 8 tokens' rows, walked backwards
  const T* src[4];
  long long stride[4] = {a.u_row, a.dt_row, a.z_row, a.D};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const void* p = i == 0 ? a.u : i == 1 ? a.dt : i == 2 ? a.z : a.dy;
    src[i] = static_cast<const T*>(p) + (seq + last + row) * stride[i] + sc;
    stride[i] *= K;
  }
  Raw<T, EPT, false> regs[VEC ? 1 : 4];
  // the operands of the 8 tokens from t on (none in front of t0 or behind te) into buffer `buf`
  const auto fetch = [&](int t, int buf) {
    const int k = t + row, ok = t >= t0 && k < te ? valid : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i == 2 && !a.z) continue;
      if constexpr (VEC) {
        constexpr int BYTES = EPT * sizeof(T) > 16 ? 16 : EPT * (int)sizeof(T);
#pragma unroll
        for (int q = 0; q < EPT * (int)sizeof(T) / BYTES; ++q)
          copy_async<BYTES>(&sm.raw[buf][i][slot + q * BYTES / sizeof(T)], src[i] + q * BYTES / sizeof(T), ok > 0);
      } else {
        regs[i].load(src[i], ok);
      }
      src[i] -= stride[i];
    }
    const long long mark = ((long long)b * subs + t / K) * a.D + r.c0;
    const bool in = t >= t0 && t < te;
    for (int i = threadIdx.x; i < CB * SL; i += kThreads) {
      const int ch = i / SL;
      copy_async<16>(&sm.marks[buf][mark_slot<SL>(ch, i % SL)], a.marks + mark * SP + i * 4,
                     in && r.c0 + ch < r.c1);
    }
    if (threadIdx.x < CB)
      copy_async<4>(&sm.msum[buf][threadIdx.x], a.msum + mark + threadIdx.x, in && r.c0 + threadIdx.x < r.c1);
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const long long stride = w ? a.c_row : a.b_row;
      const T* p = static_cast<const T*>(w ? a.Cm : a.Bm) + (seq + t) * stride + (long long)r.g * a.S;
      if (w ? vec_c : vec_b) {
        for (int i = threadIdx.x; i < K * SL; i += kThreads) {
          const int q = i / SL, s = i % SL * 4;
          copy_async<4 * sizeof(T)>(&sm.rawbc[buf][w][i * 4], p + q * stride + s, t >= t0 && t + q < te && s < a.S);
        }
      } else {
        for (int i = threadIdx.x; i < K * SP; i += kThreads) {
          const int q = i / SP, s = i % SP;
          sm.rawbc[buf][w][i] = t >= t0 && t + q < te && s < a.S ? p[q * stride + s] : from_f32<T>(0.0f);
        }
      }
    }
  };
  int buf = 0;
  if (last >= t0) fetch(last, 0);
  for (int t = last; t >= t0; t -= K, buf ^= 1) {
    const bool on = t + row < te;
    if constexpr (!VEC) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < EPT; ++e) sm.raw[buf][i][slot + e] = regs[i].t[e];
    }
    copies_wait();
    __syncthreads();   // also: everybody is done with the tile before
    fetch(t - K, buf ^ 1);
    // stage: delta, delta u and the gated dy in fp32, B and C in fp32
    {
      float u[EPT], raw[EPT], g[EPT], z[EPT], bias[EPT];
      load_vec<float, EPT>(&sm.bias[col], bias);
      load_vec<T, EPT>(&sm.raw[buf][0][slot], u);
      load_vec<T, EPT>(&sm.raw[buf][1][slot], raw);
      load_vec<T, EPT>(&sm.raw[buf][3][slot], g);
      if (a.z) load_vec<T, EPT>(&sm.raw[buf][2][slot], z);
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        raw[i] += bias[i];
        if (a.z) g[i] *= z[i] * fast_sigmoid(z[i]);
      }
      if constexpr (EPT == 1) {
        const float d = on ? (a.softplus ? softplus(raw[0]) : raw[0]) : 0.0f;
        float* p = reinterpret_cast<float*>(&sm.du[slot / 2]) + slot % 2;
        p[0] = d;
        p[2] = d * u[0];
      } else {
#pragma unroll
        for (int i = 0; i < EPT; i += 2) {
          f2 d = pack2(raw[i], raw[i + 1]);
          if (a.softplus) d = softplus2(d);
          if (!on) d = 0;
          float d0, d1;
          unpack2(d, d0, d1);
          sm.du[(slot + i) / 2] = make_float4(d0, d1, d0 * u[i], d1 * u[i + 1]);
        }
      }
      store_vec<float, EPT>(&sm.g[slot], g);
      for (int i = threadIdx.x; i < 2 * K * SL; i += kThreads) {
        const int w = i / (K * SL), at = i % (K * SL) * 4;
        float f[4];
        load_vec<T, 4>(&sm.rawbc[buf][w][at], f);
        store_vec<float, 4>(w ? &sm.C[at] : &sm.B[at], f);
      }
    }
    __syncthreads();

    // the state in front of the 8 tokens: the mark plus the chunk's decayed start state
    f2 h0[2][2], h4[2][2];
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const float4 S4 = sm.start[z * kThreads + threadIdx.x];
      const float4 M4 = sm.marks[buf][mark_slot<SL>(2 * pair + z, sl)];
      const f2 m2 = both(sm.msum[buf][2 * pair + z]);
      h4[z][0] = h0[z][0] = fma2(ex2_2(mul2(m2, A2[z][0])), pack2(S4.x, S4.y), pack2(M4.x, M4.y));
      h4[z][1] = h0[z][1] = fma2(ex2_2(mul2(m2, A2[z][1])), pack2(S4.z, S4.w), pack2(M4.z, M4.w));
    }
    // Operands of a token, read one token ahead of their use.
    struct Operands {
      float4 du, B, C;
      float2 g;
    };
    const auto read = [&](int k, Operands& o, bool with_c, bool with_g) {
      read_again();
      o.du = sm.du[k * (CB / 2) + pair];
      o.B = *reinterpret_cast<const float4*>(&sm.B[k * SP + sl * 4]);
      if (with_c) o.C = *reinterpret_cast<const float4*>(&sm.C[k * SP + sl * 4]);
      if (with_g) o.g = *reinterpret_cast<const float2*>(&sm.g[k * CB + 2 * pair]);
    };
    // one token forward: its a_t, and the state behind it in place
    const auto advance = [&](const Operands& o, f2 (&e)[2][2], f2 (&h)[2][2]) {
      const f2 B2[2] = {pack2(o.B.x, o.B.y), pack2(o.B.z, o.B.w)};
      const f2 d2[2] = {both(o.du.x), both(o.du.y)}, x2[2] = {both(o.du.z), both(o.du.w)};
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          e[z][i] = decay2(d2[z], A2[z][i]);
          h[z][i] = fma2(e[z][i], h[z][i], mul2(x2[z], B2[i]));
        }
    };
    const auto read_out = [&](int k, const Operands& o, const f2 (&h)[2][2]) {
      const f2 C2[2] = {pack2(o.C.x, o.C.y), pack2(o.C.z, o.C.w)};
      float y[2];
#pragma unroll
      for (int z = 0; z < 2; ++z) {
        float lo, hi;
        unpack2(fma2(h[z][1], C2[1], mul2(h[z][0], C2[0])), lo, hi);
        y[z] = lo + hi;
      }
      sm.y[k * kThreads + lane_sum] = make_float2(y[0], y[1]);
    };
    // the sums over the warp's channels of token k: lane cl gets those from index cl * 8 / CL on
    const auto sum_channels = [&](int k, float (&v)[8]) {
      butterfly<CL, 0, 8>(v, lane);
      constexpr int SHARE = CL > 8 ? CL / 8 : 1, OV = CL > 8 ? 1 : 8 / CL;
      if (cl % SHARE == 0) {
#pragma unroll
        for (int q = 0; q < OV; ++q) {
          const int id = cl / SHARE * OV + q;
          sm.w[warp][k][(id / 4) * SP + sl * 4 + id % 4] = v[q];
        }
      }
    };
    Operands now, next;
    read(0, now, a.z, false);
#pragma unroll
    for (int k = 0; k < H; ++k) {
      f2 e[2][2];
      read(k + 1, next, a.z, false);
      advance(now, e, h4);
      if (a.z) read_out(k, now, h4);
      now = next;
    }
    float before[8];                    // dB, dC of the token behind, summed a token later
#pragma unroll
    for (int half = 1; half >= 0; --half) {
      f2 e[H][2][2], h[H][2][2];
#pragma unroll
      for (int k = 0; k < H; ++k) {
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int i = 0; i < 2; ++i) h[k][z][i] = k ? h[k - 1][z][i] : half ? h4[z][i] : h0[z][i];
        if (k + 1 < H) read(half * H + k + 1, next, half && a.z, false);
        else read(half * H + k, next, true, true);
        advance(now, e[k], h[k]);
        if (half && a.z) read_out(half * H + k, now, h[k]);
        now = next;
      }
#pragma unroll
      for (int j = H - 1; j >= 0; --j) {
        const int k = half * H + j;
        if (j > 0) read(k - 1, next, true, true);
        else if (half) read(0, next, false, false);
        const f2 B2[2] = {pack2(now.B.x, now.B.y), pack2(now.B.z, now.B.w)};
        const f2 C2[2] = {pack2(now.C.x, now.C.y), pack2(now.C.z, now.C.w)};
        const f2 d2[2] = {both(now.du.x), both(now.du.y)}, x2[2] = {both(now.du.z), both(now.du.w)};
        const f2 g2[2] = {both(now.g.x), both(now.g.y)};
        f2 sp[2], sx[2], sb[2], sc2[2];
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const f2 dh = fma2(g2[z], C2[i], carry[z][i]);
            carry[z][i] = mul2(e[j][z][i], dh);
            const f2 p = mul2(carry[z][i], j ? h[j - 1][z][i] : half ? h4[z][i] : h0[z][i]);
            dA[z][i] = fma2(d2[z], p, dA[z][i]);
            sp[z] = i ? fma2(A2[z][i], p, sp[z]) : mul2(A2[z][i], p);
            sx[z] = i ? fma2(dh, B2[i], sx[z]) : mul2(dh, B2[i]);
            sb[i] = z ? fma2(dh, x2[z], sb[i]) : mul2(dh, x2[z]);
            sc2[i] = z ? fma2(g2[z], h[j][z][i], sc2[i]) : mul2(g2[z], h[j][z][i]);
          }
        if (k + 1 < K) sum_channels(k + 1, before);
        // over the states: left to the per-channel pass below
        float4 px;
        float lo, hi;
        unpack2(sp[0], lo, hi);
        px.x = lo + hi;
        unpack2(sp[1], lo, hi);
        px.y = lo + hi;
        unpack2(sx[0], lo, hi);
        px.z = lo + hi;
        unpack2(sx[1], lo, hi);
        px.w = lo + hi;
        sm.px[k * kThreads + lane_sum] = px;
        unpack2(sb[0], before[0], before[1]);
        unpack2(sb[1], before[2], before[3]);
        unpack2(sc2[0], before[4], before[5]);
        unpack2(sc2[1], before[6], before[7]);
        now = next;
      }
    }
    sum_channels(0, before);
    __syncthreads();
    // per (token, channel)
    if (on) {
      float u[EPT], raw[EPT], dy[EPT], z[EPT], p[EPT], x[EPT], y[EPT], delta[EPT];
#pragma unroll
      for (int i = 0; i < EPT; i += 2) {
        const int ch = col + i;
        f2 p2 = 0, x2 = 0, y2 = 0;
#pragma unroll
        for (int q = 0; q < SL; ++q) {
          const int at = row * kThreads + sum_slot<CL>(ch / L::WC, q, ch % L::WC / 2);
          const float4 v = sm.px[at];
          p2 = add2(p2, pack2(v.x, v.y));
          x2 = add2(x2, pack2(v.z, v.w));
          if (a.z) y2 = add2(y2, *reinterpret_cast<const f2*>(&sm.y[at]));
        }
        const float4 du = sm.du[(slot + i) / 2];
        float lo[4], hi[4] = {0.0f, 0.0f, 0.0f, du.y};
        unpack2(p2, lo[0], hi[0]);
        unpack2(x2, lo[1], hi[1]);
        unpack2(y2, lo[2], hi[2]);
        lo[3] = du.x;
        if constexpr (EPT == 1) {
          p[0] = ch % 2 ? hi[0] : lo[0];
          x[0] = ch % 2 ? hi[1] : lo[1];
          y[0] = ch % 2 ? hi[2] : lo[2];
          delta[0] = ch % 2 ? hi[3] : lo[3];
        } else {
          p[i] = lo[0];
          p[i + 1] = hi[0];
          x[i] = lo[1];
          x[i + 1] = hi[1];
          y[i] = lo[2];
          y[i + 1] = hi[2];
          delta[i] = lo[3];
          delta[i + 1] = hi[3];
        }
      }
      float g[EPT], skip[EPT], bias[EPT], acc[2][EPT], o1[EPT], o2[EPT], o3[EPT];
      load_vec<T, EPT>(&sm.raw[buf][0][slot], u);
      load_vec<T, EPT>(&sm.raw[buf][1][slot], raw);
      load_vec<float, EPT>(&sm.g[slot], g);
      load_vec<float, EPT>(&sm.bias[col], bias);
      load_vec<float, EPT>(&sm.skip[col], skip);
      load_vec<float, EPT>(&sm.acc[0][slot], acc[0]);
      load_vec<float, EPT>(&sm.acc[1][slot], acc[1]);
      mul_v<EPT>(o1, delta, x);
      fma_v<EPT>(o1, skip, g, o1);               // du
      mul_v<EPT>(o2, p, kLn2);
      fma_v<EPT>(o2, u, x, o2);                  // the gradient of delta
      if (a.softplus) {
        float sg[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) sg[i] = fast_sigmoid(raw[i] + bias[i]);
        mul_v<EPT>(o2, o2, sg);
      }
      fma_v<EPT>(acc[0], g, u, acc[0]);
      fma_v<EPT>(acc[1], o2, 1.0f, acc[1]);
      Raw<T, EPT, VEC> odu, odt, odz;
#pragma unroll
      for (int i = 0; i < EPT; i += 2) {
        odu.set_pair(i, o1[i], o1[EPT > 1 ? i + 1 : i]);
        odt.set_pair(i, o2[i], o2[EPT > 1 ? i + 1 : i]);
      }
      if (a.z) {                                 // dz = dy y silu'(z), silu' = s (1 + z (1 - s))
        load_vec<T, EPT>(&sm.raw[buf][3][slot], dy);
        load_vec<T, EPT>(&sm.raw[buf][2][slot], z);
        float sg[EPT], ns[EPT], one[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          sg[i] = fast_sigmoid(z[i]);
          ns[i] = 1.0f - sg[i];
          one[i] = 1.0f;
        }
        fma_v<EPT>(y, skip, u, y);
        fma_v<EPT>(o3, z, ns, one);
        mul_v<EPT>(o3, o3, sg);
        mul_v<EPT>(y, y, dy);
        mul_v<EPT>(o3, o3, y);
#pragma unroll
        for (int i = 0; i < EPT; i += 2) odz.set_pair(i, o3[i], o3[EPT > 1 ? i + 1 : i]);
      }
      store_vec<float, EPT>(&sm.acc[0][slot], acc[0]);
      store_vec<float, EPT>(&sm.acc[1][slot], acc[1]);
      const long long o = (seq + t + row) * a.D + sc;
      odu.store(static_cast<T*>(a.du) + o, valid);
      odt.store(static_cast<T*>(a.ddt) + o, valid);
      if (a.z) odz.store(static_cast<T*>(a.dz) + o, valid);
    }
    // per (token, state): the block's channels
    for (int i = threadIdx.x; i < K * 2 * SL; i += kThreads) {
      const int k = i / (2 * SL), q = i % (2 * SL) * 4;
      if (t + k < te) {
        float v[4];
        load_vec<float, 4>(&sm.w[0][k][q], v);
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          float f[4];
          load_vec<float, 4>(&sm.w[w][k][q], f);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] += f[e];
        }
        store_vec<float, 4>(&bcpart[(long long)(t + k) * a.G * 2 * SP + q], v);
      }
    }
  }
  copies_wait();   // the copies in front of t0 are empty, but in flight
  // rows behind the sequence's end
  Raw<T, EPT, VEC> zero;
#pragma unroll
  for (int i = 0; i < EPT; ++i) zero.set(i, 0.0f);
  for (int t = max(t0, len) + row; t < t1; t += K) {
    const long long o = (seq + t) * a.D + sc;
    zero.store(static_cast<T*>(a.du) + o, valid);
    zero.store(static_cast<T*>(a.ddt) + o, valid);
    if (a.z) zero.store(static_cast<T*>(a.dz) + o, valid);
  }
  for (int i = threadIdx.x; i < (t1 - max(t0, len)) * 2 * SP; i += kThreads)
    bcpart[(long long)(max(t0, len) + i / (2 * SP)) * a.G * 2 * SP + i % (2 * SP)] = 0.0f;
#pragma unroll
  for (int z = 0; z < 2; ++z)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float w[2], g[2];
      unpack2(dA[z][i], w[0], w[1]);
      unpack2(carry[z][i], g[0], g[1]);
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int s = sl * 4 + 2 * i + q;
        if (c + z >= r.c1 || s >= a.S) continue;
        a.part[bk * a.D * (a.S + 2) + (long long)(c + z) * a.S + s] = w[q];
        if (a.dstate_in && chunk == 0) a.dstate_in[((long long)b * a.D + c + z) * a.S + s] = g[q];
      }
    }
  // dD and ddt_bias: the 8 token rows of a channel in a fixed order
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * CB; i += kThreads) {
    const int ch = i % CB, which = i / CB;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) v += sm.acc[which][k * CB + ch];
    if (r.c0 + ch < r.c1) a.part[bk * a.D * (a.S + 2) + (long long)a.D * (a.S + which) + r.c0 + ch] = v;
  }
}

// dB and dC: the sum over the channel blocks of a group, rounded once. Four states a thread.
template <typename T>
__global__ void __launch_bounds__(256) scan_sum_bc_kernel(ScanArgs a, int blocks_per_group, int SP) {
  const long long n = (long long)a.B * a.N * a.G * 2 * SP;   // of one channel block
  TTT_GRID_LOOP(i, n / 4) {
    const int q = (int)(i * 4 % (2 * SP)), s = q % SP;
    const long long row = i * 4 / (2 * SP);
    float v[4] = {};
#pragma unroll 8
    for (int k = 0; k < blocks_per_group; ++k) {
      float f[4];
      load_vec<float, 4>(a.bcpart + k * n + i * 4, f);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += f[e];
    }
    T* out = static_cast<T*>(q < SP ? a.dB : a.dC) + row * a.S;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (s + e < a.S) out[s + e] = from_f32<T>(v[e]);
  }
}

// ---------------------------------------------------------------- launches
int state_lanes(int S) { return S <= 8 ? 2 : S <= 16 ? 4 : S <= 32 ? 8 : 16; }

// Whether every run of `ept` channels that a thread stages is whole and aligned for the
// accesses of Raw<T, ept, true>.
bool fits(const ScanArgs& a, int ept, int size) {
  const int w = ept * size > 16 ? 16 : ept * size;
  if (a.D / a.G % ept) return false;
  for (long long row : {a.u_row, a.dt_row, a.z ? a.z_row : 0LL, (long long)a.D})
    if (row * size % w) return false;
  for (const void* p : {a.u, a.dt, a.z, (const void*)a.y, a.dy, (const void*)a.du,
                        (const void*)a.ddt, (const void*)a.dz})
    if (reinterpret_cast<uintptr_t>(p) % w) return false;
  return true;
}

enum Kernel { ENDS, OUTPUTS, MARKS, MAIN };

// Whether the S states of every row of B or C are whole aligned runs of four.
bool fits_four(const ScanArgs& a, const void* p, long long row, int size) {
  return a.S % 4 == 0 && row % 4 == 0 && reinterpret_cast<uintptr_t>(p) % (4 * size) == 0;
}

template <typename T, int SL, bool VEC, Kernel K>
cudaError_t launch_kernel(const ScanArgs& a, cudaStream_t s) {
  constexpr int CB = K == MAIN ? BwdTile<SL>::CB : FwdTile<SL>::CB;
  const int bpg = (a.D / a.G + CB - 1) / CB;
  const bool vb = fits_four(a, a.Bm, a.b_row, sizeof(T)), vc = fits_four(a, a.Cm, a.c_row, sizeof(T));
  const dim3 grid(bpg * a.G, K == ENDS ? a.chunks - 1 : a.chunks, a.B);
  if constexpr (K == ENDS || K == OUTPUTS)
    scan_fwd_kernel<T, SL, VEC, K == OUTPUTS><<<grid, kFwdThreads, 0, s>>>(a, bpg, vb, vc);
  if constexpr (K == MARKS) {
    if (a.chunks > 1) scan_marks_kernel<T, SL, VEC, true><<<grid, kFwdThreads, 0, s>>>(a, bpg, vb, vc);
    else scan_marks_kernel<T, SL, VEC, false><<<grid, kFwdThreads, 0, s>>>(a, bpg, vb, vc);
  }
  if constexpr (K == MAIN) {
    constexpr size_t bytes = sizeof(BwdShared<T, SL>);
    const cudaError_t e = cudaFuncSetAttribute(scan_bwd_kernel<T, SL, VEC>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
    scan_bwd_kernel<T, SL, VEC><<<grid, kThreads, bytes, s>>>(a, bpg, vb, vc);
  }
  return cudaGetLastError();
}

template <typename T, int SL, Kernel K>
cudaError_t launch_vec(const ScanArgs& a, cudaStream_t s) {
  constexpr int ept = K == MAIN ? BwdTile<SL>::EPT : FwdTile<SL>::EPT;
  if constexpr (K != MAIN || ept * sizeof(T) >= 4)   // an asynchronous copy has 4 bytes at least
    if (fits(a, ept, sizeof(T))) return launch_kernel<T, SL, true, K>(a, s);
  return launch_kernel<T, SL, false, K>(a, s);
}

template <typename T, Kernel K>
cudaError_t launch_state(const ScanArgs& a, cudaStream_t s) {
  switch (state_lanes(a.S)) {
    case 2: return launch_vec<T, 2, K>(a, s);
    case 4: return launch_vec<T, 4, K>(a, s);
    case 8: return launch_vec<T, 8, K>(a, s);
    default: return launch_vec<T, 16, K>(a, s);
  }
}

template <Kernel K>
cudaError_t launch(int dt, const ScanArgs& a, cudaStream_t s) {
  return dt == DT_BF16 ? launch_state<bf16, K>(a, s) : launch_state<float, K>(a, s);
}

template <typename T, int SL, bool VEC>
cudaError_t launch_step_vec(const ScanArgs& a, cudaStream_t s) {
  // Four sequences a lane once that still gives every SM 1024 threads.
  const unsigned blocks = (a.D + kThreads / SL - 1) / (kThreads / SL);
  if ((long long)blocks * (a.B / 4) >= 148 * 8)
    scan_step_kernel<T, SL, VEC, 4><<<dim3(blocks, (a.B + 3) / 4), kThreads, 0, s>>>(a);
  else
    scan_step_kernel<T, SL, VEC, 1><<<dim3(blocks, a.B), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <typename T, int SL>
cudaError_t launch_step(const ScanArgs& a, cudaStream_t s) {
  const bool vec = fits_four(a, a.Bm, a.b_row, sizeof(T)) && fits_four(a, a.Cm, a.c_row, sizeof(T)) &&
                   (reinterpret_cast<uintptr_t>(a.state_out) | reinterpret_cast<uintptr_t>(a.A)) % 16 == 0;
  return vec ? launch_step_vec<T, SL, true>(a, s) : launch_step_vec<T, SL, false>(a, s);
}

template <typename T>
cudaError_t launch_step_state(const ScanArgs& a, cudaStream_t s) {
  switch (state_lanes(a.S)) {
    case 2: return launch_step<T, 2>(a, s);
    case 4: return launch_step<T, 4>(a, s);
    case 8: return launch_step<T, 8>(a, s);
    default: return launch_step<T, 16>(a, s);
  }
}

}  // namespace

int scan_padded_state(int S) { return 4 * state_lanes(S); }

int scan_channel_blocks(int D, int G, int S) {
  const int CB = kWarps * 64 / state_lanes(S);
  return (D / G + CB - 1) / CB;
}

// Blocks to fill the card with: two rounds of those that run at a time (148 SMs x 7 forward, x 3
// backward, counted for bf16, aligned, S <= 16 and used for all: fp32 and more states have 4 or 5
// forward, odd channels 2 backward; one round: 400 us against 387 us forward for 32768 tokens of 1024 channels, 990 us
// against 980 us backward for the sizes above, three rounds 394 us and 990 us), and the tokens'
// worth of work that starting and joining a chunk costs (8, 24 and 40 gave the same times; 64
// fewer and worse balanced chunks, 1203 us against 1100 us backward at the time). The forward's
// first pass doubles its exponentials, so a sequence is cut for it only where whole sequences
// would leave most SMs idle.
constexpr long long kFwdSlots = 148 * 14, kBwdSlots = 148 * 6, kChunkCost = 24;

int scan_chunks(int B, int N, int D, int G, int S, bool backward, int* chunk) {
  const int CB = backward ? kWarps * 64 / state_lanes(S) : kFwdWarps * 32 / state_lanes(S);
  const long long blocks = (long long)B * G * ((D / G + CB - 1) / CB);
  const long long slots = backward ? kBwdSlots : kFwdSlots;
  const long long most = std::min<long long>(std::max(1, (N + 31) / 32), 1024);
  // rounds of blocks x (tokens of a chunk + cost of a chunk), the least over the counts
  long long best = 1, least = 0;
  for (long long n = 1; n <= most; ++n) {
    const long long len = ((N + n - 1) / n + 31) / 32 * 32;
    long long time = (std::max<long long>(blocks * n, 1) + slots - 1) / slots * (len + kChunkCost);
    if (!backward && n > 1) time *= 2;
    if (n == 1 || time < least) {
      least = time;
      best = n;
    }
    if (n > 1 && blocks * n > 8 * slots) break;   // balanced to an eighth
  }
  long long len = (N + best - 1) / best;
  len = std::max<long long>((len + 31) / 32 * 32, 32);   // whole staged tiles
  *chunk = (int)len;
  return N > 0 ? (int)((N + len - 1) / len) : 1;
}

cudaError_t scan_fwd_ends(int dt, const ScanArgs& a, cudaStream_t s) { return launch<ENDS>(dt, a, s); }
cudaError_t scan_fwd_outputs(int dt, const ScanArgs& a, cudaStream_t s) { return launch<OUTPUTS>(dt, a, s); }
cudaError_t scan_bwd_marks(int dt, const ScanArgs& a, cudaStream_t s) { return launch<MARKS>(dt, a, s); }
cudaError_t scan_bwd_main(int dt, const ScanArgs& a, cudaStream_t s) { return launch<MAIN>(dt, a, s); }

cudaError_t scan_join(const ScanArgs& a, bool backward, cudaStream_t s) {
  const int SP = scan_padded_state(a.S);
  const unsigned grid = grid_for((long long)a.B * a.D * SP * (backward ? 2 : 1), 256);
  if (backward) scan_join_kernel<true><<<grid, 256, 0, s>>>(a, SP);
  else scan_join_kernel<false><<<grid, 256, 0, s>>>(a, SP);
  return cudaGetLastError();
}

cudaError_t scan_step(int dt, const ScanArgs& a, cudaStream_t s) {
  return dt == DT_BF16 ? launch_step_state<bf16>(a, s) : launch_step_state<float>(a, s);
}

cudaError_t scan_bwd_sum_bc(int dt, const ScanArgs& a, cudaStream_t s) {
  const int SP = scan_padded_state(a.S), bpg = scan_channel_blocks(a.D, a.G, a.S);
  const unsigned grid = grid_for((long long)a.B * a.N * a.G * 2 * SP / 4, 256);
  if (dt == DT_BF16) scan_sum_bc_kernel<bf16><<<grid, 256, 0, s>>>(a, bpg, SP);
  else scan_sum_bc_kernel<float><<<grid, 256, 0, s>>>(a, bpg, SP);
  return cudaGetLastError();
}

}  // namespace ttt
