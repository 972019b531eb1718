// The selective state space scan. Per sequence, channel d and state element s
//     delta_t = softplus(dt_t + dt_bias),  a_t = exp(delta_t A[d, s]),
//     h_t = a_t h_{t-1} + delta_t u_t B_t[s],
//     y_t = sum_s C_t[s] h_t + D[d] u_t,  times silu(z_t) when gated.
//
// What bounds it: one exponential per (token, channel, state) - 16 per token and channel at
// the usual S = 16 - against 16 exponentials per clock and SM; the four fp32 operations
// around it need half that time and HBM less than that. So the work is laid out for the
// exponential unit to run without a pause: a lane keeps a register tile of 2 channels x 4
// states (8 independent recurrences, the channel pair packed for the two-wide fp32
// instructions, which halves the issue slots), SL lanes share a channel's states, and tiles of
// tokens are staged in shared memory as fp32 with softplus already applied. The sums over the
// states leave a warp by transposing butterflies (SL values over SL lanes in SL - 1 shuffles).
//
// The time axis is cut into chunks when batch x channels alone would leave SMs idle: a first
// pass takes each chunk's end state from zero (its decay is exp(A sum delta), one number per
// state), scan_join carries the states over the chunks, and the outputs pass starts every chunk
// from its state. That doubles the exponentials, so it is done only for few channels.
#include "mixer.h"
#include "mixer_common.cuh"

namespace ttt {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// ---------------------------------------------------------------- two-wide fp32
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(f2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ f2 ex2_2(f2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  return pack2(ex2(lo), ex2(hi));
}

// softplus(x) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1]. log1p(e) / e is a polynomial of
// degree 9, interpolated at the Chebyshev nodes of [0, 1] (relative error 1.2e-7 in fp32): it
// keeps the relative accuracy of small steps, which a logarithm of 1 + e loses, without a
// second special-function result.
__device__ __forceinline__ float softplus(float x) {
  const float e = ex2(-fabsf(x) * kLog2e);
  float p = -0.0031760570127516985f;
  p = fmaf(p, e, 0.019542526453733444f);
  p = fmaf(p, e, -0.056373611092567444f);
  p = fmaf(p, e, 0.10543623566627502f);
  p = fmaf(p, e, -0.1526966691017151f);
  p = fmaf(p, e, 0.1966327428817749f);
  p = fmaf(p, e, -0.24951615929603577f);
  p = fmaf(p, e, 0.33329710364341736f);
  p = fmaf(p, e, -0.49999892711639404f);
  p = fmaf(p, e, 1.0f);
  return fmaxf(x, 0.0f) + e * p;
}

// ---------------------------------------------------------------- tiles
// SL lanes share a channel: lane = channel pair * SL + state group, 4 states per lane.
template <int SL> struct Tile {
  static constexpr int SP = 4 * SL;                        // padded states
  static constexpr int CL = 32 / SL;                       // channel pairs of a warp
  static constexpr int WC = 2 * CL;                        // channels of a warp
  static constexpr int CB = kWarps * WC;                   // channels of a block
  static constexpr int TT = SL == 16 ? 32 : 4 * SL;        // tokens of a staged tile
  static constexpr int EPT = TT * CB / kThreads;           // channels a thread stages (one token)
  static constexpr int TPR = CB / EPT;                     // threads of a token's row
};

// N consecutive elements of a row; VEC: in accesses of up to 16 bytes (all N or none valid).
template <typename T, int N, bool VEC> struct Raw {
  static constexpr int W = N * sizeof(T) > 16 ? 16 / (int)sizeof(T) : N;
  union {
    T t[N];
    typename Pack<T, W>::U u[N / W];
  };
  __device__ __forceinline__ void load(const T* p, int valid) {
    if constexpr (VEC) {
#pragma unroll
      for (int i = 0; i < N / W; ++i) {
        if (valid > 0) u[i] = load_raw<T, W>(p + i * W);
        else u[i] = typename Pack<T, W>::U{};
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) t[i] = i < valid ? p[i] : from_f32<T>(0.0f);
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

// A lane's 4 states of its 2 channels, scaled; zero outside the channels and states.
template <int SL>
__device__ __forceinline__ void load_A(const ScanArgs& a, int c, int c1, int s0, f2 (&A2)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool on = s0 + i < a.S;
    const float lo = on && c < c1 ? a.A[(long long)c * a.S + s0 + i] : 0.0f;
    const float hi = on && c + 1 < c1 ? a.A[(long long)(c + 1) * a.S + s0 + i] : 0.0f;
    A2[i] = pack2(lo * kLog2e, hi * kLog2e);
  }
}

// Element s of the lane's channel pair in a [D, S] array.
__device__ __forceinline__ f2 load_pair(const float* p, int c, int c1, int s, int S) {
  const float lo = c < c1 && s < S ? p[(long long)c * S + s] : 0.0f;
  const float hi = c + 1 < c1 && s < S ? p[(long long)(c + 1) * S + s] : 0.0f;
  return pack2(lo, hi);
}
__device__ __forceinline__ void store_pair(float* p, int c, int c1, int s, int S, f2 v) {
  float lo, hi;
  unpack2(v, lo, hi);
  if (s < S) {
    if (c < c1) p[(long long)c * S + s] = lo;
    if (c + 1 < c1) p[(long long)(c + 1) * S + s] = hi;
  }
}

// The lane's 4 states of both channels in a [D, SP] array of the workspace (16-byte rows).
template <int SL>
__device__ __forceinline__ void load_tile(const float* p, int c, int c1, int s0, f2 (&v)[4]) {
  float lo[4] = {}, hi[4] = {};
  if (c < c1) load_vec<float, 4>(p + (long long)c * 4 * SL + s0, lo);
  if (c + 1 < c1) load_vec<float, 4>(p + (long long)(c + 1) * 4 * SL + s0, hi);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pack2(lo[i], hi[i]);
}
template <int SL>
__device__ __forceinline__ void store_tile(float* p, int c, int c1, int s0, const f2 (&v)[4]) {
  float lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2(v[i], lo[i], hi[i]);
  if (c < c1) store_vec<float, 4>(p + (long long)c * 4 * SL + s0, lo);
  if (c + 1 < c1) store_vec<float, 4>(p + (long long)(c + 1) * 4 * SL + s0, hi);
}

// TOKENS rows of B or C for one group from token t on, each value twice (both channels of a
// pair multiply by it), zero behind `live` tokens and S states.
template <typename T, int SL, int TOKENS>
__device__ __forceinline__ void stage_bc(f2* dst, const void* src, long long row, const ScanArgs& a,
                                         int b, int g, int t, int live) {
  constexpr int SP = 4 * SL;
  const T* p = static_cast<const T*>(src) + ((long long)b * a.N + t) * row + (long long)g * a.S;
  for (int i = threadIdx.x; i < TOKENS * SP; i += kThreads) {
    const int k = i / SP, s = i % SP;
    const float v = k < live && s < a.S ? to_f32(p[k * row + s]) : 0.0f;
    dst[i] = pack2(v, v);
  }
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
// One chunk of one sequence for CB channels. OUT: from the chunk's start state, writing y (and
// the state behind the last chunk); else from zero, writing the end state and the sum of delta.
// grid (channel blocks, chunks, B).
template <typename T, int SL, bool VEC, bool OUT>
__global__ void __launch_bounds__(kThreads) scan_fwd_kernel(ScanArgs a, int blocks_per_group) {
  using L = Tile<SL>;
  constexpr int TT = L::TT, CB = L::CB, SP = L::SP, EPT = L::EPT;
  __shared__ __align__(16) float sD[TT * CB], sU[TT * CB];   // delta; u, then y
  __shared__ __align__(16) f2 sB[TT * SP], sC[OUT ? TT * SP : 2];
  const Range r = block_channels(blockIdx.x, blocks_per_group, a.D, a.G, CB);
  const int chunk = blockIdx.y, b = blockIdx.z;
  const int len = sequence_length(a.lens, b, a.N);
  const int t0 = chunk * a.chunk, t1 = min(a.N, t0 + a.chunk), te = min(t1, len);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int sl = lane % SL, cw = warp * L::WC + lane / SL * 2;   // state group; channel in block
  const int c = r.c0 + cw;
  // staging: EPT channels of one token per thread
  const int row = threadIdx.x / L::TPR, col = threadIdx.x % L::TPR * EPT;
  const int sc = r.c0 + col, valid = min(EPT, r.c1 - sc);
  const long long seq = (long long)b * a.N;
  float bias[EPT];
#pragma unroll
  for (int i = 0; i < EPT; ++i) bias[i] = a.dt_bias && i < valid ? a.dt_bias[sc + i] : 0.0f;

  f2 A2[4], h[4], dsum = 0;
  load_A<SL>(a, c, r.c1, sl * 4, A2);
  const long long at = ((long long)b * a.chunks + chunk) * a.D * SP;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = 0;
    if (OUT && a.chunks == 1 && a.state_in)
      h[i] = load_pair(a.state_in + (long long)b * a.D * a.S, c, r.c1, sl * 4 + i, a.S);
  }
  if (OUT && a.chunks > 1) load_tile<SL>(a.ends + at, c, r.c1, sl * 4, h);
  // D of the channel whose y this lane writes
  const int cy = c + (sl & 1);
  float skip[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) skip[i] = a.Dskip && c + i < r.c1 ? a.Dskip[c + i] : 0.0f;
  const float skip_y = cy == c ? skip[0] : skip[1];

  Raw<T, EPT, VEC> ru, rd, rz;
  auto fetch = [&](int t) {
    const int k = t + row, ok = k < te ? valid : 0;
    ru.load(static_cast<const T*>(a.u) + (seq + k) * a.u_row + sc, ok);
    rd.load(static_cast<const T*>(a.dt) + (seq + k) * a.dt_row + sc, ok);
    if (OUT && a.z) rz.load(static_cast<const T*>(a.z) + (seq + k) * a.z_row + sc, ok);
  };
  if (t0 < te) fetch(t0);
  for (int t = t0; t < te; t += TT) {
    const bool on = t + row < te;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const float raw = rd.get(i) + bias[i];
      sD[row * CB + col + i] = on && i < valid ? (a.softplus ? softplus(raw) : raw) : 0.0f;
      sU[row * CB + col + i] = ru.get(i);
    }
    stage_bc<T, SL, TT>(sB, a.Bm, a.b_row, a, b, r.g, t, te - t);
    if (OUT) stage_bc<T, SL, TT>(sC, a.Cm, a.c_row, a, b, r.g, t, te - t);
    __syncthreads();
    const Raw<T, EPT, VEC> gate = rz;
    if (t + TT < te) fetch(t + TT);

    constexpr int TB = OUT ? SL / 2 : 1;   // tokens whose sums leave together: SL values
#pragma unroll 1
    for (int k0 = 0; k0 < TT; k0 += TB) {
      float v[SL];
#pragma unroll
      for (int j = 0; j < TB; ++j) {
        const int k = k0 + j;
        const f2 d2 = *reinterpret_cast<const f2*>(&sD[k * CB + cw]);
        const f2 du = mul2(d2, *reinterpret_cast<const f2*>(&sU[k * CB + cw]));
        if (!OUT) dsum = add2(dsum, d2);
        f2 y = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 e = ex2_2(mul2(d2, A2[i]));
          h[i] = fma2(e, h[i], mul2(du, sB[k * SP + sl * 4 + i]));
          if (OUT) y = fma2(h[i], sC[k * SP + sl * 4 + i], y);
        }
        if (OUT) unpack2(y, v[2 * j], v[2 * j + 1]);
      }
      if (OUT) {
        // lane sl gets token k0 + sl / 2, channel sl & 1; all lanes have read this u
        butterfly<SL, 0, SL>(v, lane);
        float* p = &sU[(k0 + sl / 2) * CB + cw + (sl & 1)];
        *p = fmaf(skip_y, *p, v[0]);
      }
    }
    __syncthreads();
    if (OUT && on) {
      Raw<T, EPT, VEC> out;
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        float y = sU[row * CB + col + i];
        if (a.z) {
          const float z = gate.get(i);
          y *= z * fast_sigmoid(z);
        }
        out.set(i, y);
      }
      out.store(static_cast<T*>(a.y) + (seq + t + row) * a.D + sc, valid);
    }
  }
  if (OUT) {
    Raw<T, EPT, VEC> zero;   // rows behind the sequence's end
#pragma unroll
    for (int i = 0; i < EPT; ++i) zero.set(i, 0.0f);
    for (int t = max(t0, len) + row; t < t1; t += TT)
      zero.store(static_cast<T*>(a.y) + (seq + t) * a.D + sc, valid);
    if (a.state_out && chunk == a.chunks - 1)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        store_pair(a.state_out + (long long)b * a.D * a.S, c, r.c1, sl * 4 + i, a.S, h[i]);
  } else {
    store_tile<SL>(a.ends + at, c, r.c1, sl * 4, h);
    if (sl == 0) store_pair(a.dsum + ((long long)b * a.chunks + chunk) * a.D, c, r.c1, 0, 1, dsum);
  }
}

// Carries states over the chunks, in place: ends[k] becomes the state chunk k starts from, and
// in the backward back[k] the state gradient behind chunk k. One thread per (b, d, s).
template <bool BWD>
__global__ void __launch_bounds__(256) scan_join_kernel(ScanArgs a, int SP) {
  TTT_GRID_LOOP(i, (long long)a.B * a.D * SP) {
    const int s = (int)(i % SP);
    const long long bd = i / SP;
    const int d = (int)(bd % a.D), b = (int)(bd / a.D);
    const bool on = s < a.S;
    const float A2 = on ? a.A[(long long)d * a.S + s] * kLog2e : 0.0f;
    const long long io = bd * a.S + s;
    float h = on && a.state_in ? a.state_in[io] : 0.0f;
    for (int k = 0; k < a.chunks; ++k) {
      const long long bk = (long long)b * a.chunks + k, at = (bk * a.D + d) * SP + s;
      const float end = k + 1 < a.chunks ? a.ends[at] : 0.0f;
      const float e = k + 1 < a.chunks ? ex2(A2 * a.dsum[bk * a.D + d]) : 0.0f;
      a.ends[at] = h;
      h = fmaf(e, h, end);
    }
    if (!BWD) continue;
    float g = on && a.dstate_out ? a.dstate_out[io] : 0.0f;
    for (int k = a.chunks - 1; k >= 0; --k) {
      const long long bk = (long long)b * a.chunks + k, at = (bk * a.D + d) * SP + s;
      const float share = k > 0 ? a.back[at] : 0.0f;
      const float e = k > 0 ? ex2(A2 * a.dsum[bk * a.D + d]) : 0.0f;
      a.back[at] = g;
      g = fmaf(e, g, share);
    }
  }
}

// ---------------------------------------------------------------- one token
// SL lanes per channel, 4 states each; the state is read and written once (HBM bound for many
// sequences, one launch's latency for few).
template <typename T, int SL, bool VEC>
__global__ void __launch_bounds__(kThreads) scan_step_kernel(ScanArgs a) {
  const long long i = ((long long)blockIdx.x * kThreads + threadIdx.x) / SL;
  const int sl = threadIdx.x % SL;
  const bool on = i < (long long)a.B * a.D;
  const int b = on ? (int)(i / a.D) : 0, d = on ? (int)(i % a.D) : 0;
  const int g = d / (a.D / a.G), s0 = sl * 4;
  const float u = to_f32(static_cast<const T*>(a.u)[b * a.u_row + d]);
  float delta = to_f32(static_cast<const T*>(a.dt)[b * a.dt_row + d]) + (a.dt_bias ? a.dt_bias[d] : 0.0f);
  if (a.softplus) delta = softplus(delta);
  const T* Bm = static_cast<const T*>(a.Bm) + b * a.b_row + (long long)g * a.S;
  const T* Cm = static_cast<const T*>(a.Cm) + b * a.c_row + (long long)g * a.S;
  const float* A = a.A + (long long)d * a.S;
  float* st = a.state_out + ((long long)b * a.D + d) * a.S;
  float y = 0.0f, h[4];
  if (VEC) {
    if (s0 < a.S) {
      float A4[4], b4[4], c4[4];
      load_vec<float, 4>(st + s0, h);
      load_vec<float, 4>(A + s0, A4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        b4[k] = to_f32(Bm[s0 + k]);
        c4[k] = to_f32(Cm[s0 + k]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h[k] = fmaf(ex2(delta * (A4[k] * kLog2e)), h[k], delta * u * b4[k]);
        y = fmaf(h[k], c4[k], y);
      }
      if (on) store_vec<float, 4>(st + s0, h);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s0 + k < a.S) {
        h[k] = fmaf(ex2(delta * (A[s0 + k] * kLog2e)), st[s0 + k], delta * u * to_f32(Bm[s0 + k]));
        y = fmaf(h[k], to_f32(Cm[s0 + k]), y);
        if (on) st[s0 + k] = h[k];
      }
  }
#pragma unroll
  for (int m = SL / 2; m > 0; m /= 2) y += __shfl_xor_sync(0xffffffffu, y, m);
  if (on && sl == 0) {
    if (a.Dskip) y = fmaf(a.Dskip[d], u, y);
    if (a.z) {
      const float z = to_f32(static_cast<const T*>(a.z)[b * a.z_row + d]);
      y *= z * fast_sigmoid(z);
    }
    static_cast<T*>(a.y)[(long long)b * a.D + d] = from_f32<T>(y);
  }
}

// ---------------------------------------------------------------- backward
// With g_t = dy_t silu(z_t) and dh_t = C_t g_t + a_{t+1} dh_{t+1}:
//     p_t = dh_t a_t h_{t-1},  x_t = sum_s dh_t B_t,
//     dA += delta_t p_t,  dB_t = sum_d dh_t delta_t u_t,  dC_t = sum_d g_t h_t,
//     du_t = D g_t + delta_t x_t,  ddelta_t = sum_s A p_t + u_t x_t,
//     dz_t = dy_t silu'(z_t) (sum_s C_t h_t + D u_t).
// The states are recomputed, not saved: the first pass leaves a mark (the state from the
// chunk's zero) every 8 tokens, the main pass walks the marks backwards and holds 8 tokens of
// a_t and h_t in registers, so each a_t is computed twice in all. 8 tokens: the marks then cost
// S / 8 * 4 bytes per token and channel (8 at S = 16, less than the operands), and 8 tokens of
// (a, h) fill the 128 registers that two blocks per SM leave.

// Marks, chunk end states, and with more than one chunk the chunk's share of the state gradient
// in front of it, sum_t (prod_{t' <= t} a_t') C_t g_t. Same tiling as the forward.
template <typename T, int SL, bool VEC, bool SPLIT>
__global__ void __launch_bounds__(kThreads) scan_marks_kernel(ScanArgs a, int blocks_per_group) {
  using L = Tile<SL>;
  constexpr int TT = L::TT, CB = L::CB, SP = L::SP, EPT = L::EPT;
  __shared__ __align__(16) float sD[TT * CB], sU[TT * CB], sG[SPLIT ? TT * CB : 4];
  __shared__ __align__(16) f2 sB[TT * SP], sC[SPLIT ? TT * SP : 2];
  const Range r = block_channels(blockIdx.x, blocks_per_group, a.D, a.G, CB);
  const int chunk = blockIdx.y, b = blockIdx.z;
  const int len = sequence_length(a.lens, b, a.N);
  const int t0 = chunk * a.chunk, te = min(min(a.N, t0 + a.chunk), len);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int sl = lane % SL, cw = warp * L::WC + lane / SL * 2;
  const int c = r.c0 + cw;
  const int row = threadIdx.x / L::TPR, col = threadIdx.x % L::TPR * EPT;
  const int sc = r.c0 + col, valid = min(EPT, r.c1 - sc);
  const long long seq = (long long)b * a.N;
  const int subs = (a.N + kScanSub - 1) / kScanSub;
  float bias[EPT];
#pragma unroll
  for (int i = 0; i < EPT; ++i) bias[i] = a.dt_bias && i < valid ? a.dt_bias[sc + i] : 0.0f;
  f2 A2[4], h[4], prod[4], share[4], dsum = 0;
  load_A<SL>(a, c, r.c1, sl * 4, A2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h[i] = share[i] = 0;
    prod[i] = pack2(1.0f, 1.0f);
  }
  Raw<T, EPT, VEC> ru, rd, rz, rg;
  auto fetch = [&](int t) {
    const int k = t + row, ok = k < te ? valid : 0;
    ru.load(static_cast<const T*>(a.u) + (seq + k) * a.u_row + sc, ok);
    rd.load(static_cast<const T*>(a.dt) + (seq + k) * a.dt_row + sc, ok);
    if (SPLIT) rg.load(static_cast<const T*>(a.dy) + (seq + k) * a.D + sc, ok);
    if (SPLIT && a.z) rz.load(static_cast<const T*>(a.z) + (seq + k) * a.z_row + sc, ok);
  };
  if (t0 < te) fetch(t0);
  for (int t = t0; t < te; t += TT) {
    const bool on = t + row < te;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const float raw = rd.get(i) + bias[i];
      sD[row * CB + col + i] = on && i < valid ? (a.softplus ? softplus(raw) : raw) : 0.0f;
      sU[row * CB + col + i] = ru.get(i);
      if (SPLIT) {
        float g = rg.get(i);
        if (a.z) {
          const float z = rz.get(i);
          g *= z * fast_sigmoid(z);
        }
        sG[row * CB + col + i] = g;
      }
    }
    stage_bc<T, SL, TT>(sB, a.Bm, a.b_row, a, b, r.g, t, te - t);
    if (SPLIT) stage_bc<T, SL, TT>(sC, a.Cm, a.c_row, a, b, r.g, t, te - t);
    __syncthreads();
    if (t + TT < te) fetch(t + TT);
#pragma unroll 1
    for (int k0 = 0; k0 < TT && t + k0 < te; k0 += kScanSub) {
      const long long mark = (long long)b * subs + (t + k0) / kScanSub;
      store_tile<SL>(a.marks + mark * a.D * SP, c, r.c1, sl * 4, h);
      if (sl == 0) store_pair(a.msum + mark * a.D, c, r.c1, 0, 1, dsum);
#pragma unroll
      for (int j = 0; j < kScanSub; ++j) {
        const int k = k0 + j;
        const f2 d2 = *reinterpret_cast<const f2*>(&sD[k * CB + cw]);
        const f2 du = mul2(d2, *reinterpret_cast<const f2*>(&sU[k * CB + cw]));
        dsum = add2(dsum, d2);
        f2 g2 = 0;
        if (SPLIT) g2 = *reinterpret_cast<const f2*>(&sG[k * CB + cw]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f2 e = ex2_2(mul2(d2, A2[i]));
          h[i] = fma2(e, h[i], mul2(du, sB[k * SP + sl * 4 + i]));
          if (SPLIT) {
            prod[i] = mul2(prod[i], e);
            share[i] = fma2(prod[i], mul2(g2, sC[k * SP + sl * 4 + i]), share[i]);
          }
        }
      }
    }
    __syncthreads();
  }
  const long long bk = (long long)b * a.chunks + chunk, at = bk * a.D * SP;
  store_tile<SL>(a.ends + at, c, r.c1, sl * 4, h);
  if (SPLIT) store_tile<SL>(a.back + at, c, r.c1, sl * 4, share);
  if (sl == 0) store_pair(a.dsum + bk * a.D, c, r.c1, 0, 1, dsum);
}

template <int SL> struct BwdTile : Tile<SL> {
  static constexpr int EPT = kScanSub * Tile<SL>::CB / kThreads;   // 16 / SL
  static constexpr int TPR = Tile<SL>::CB / EPT;
};

// The main pass of one chunk, 8 tokens at a time from its end. grid (channel blocks, chunks, B).
template <typename T, int SL, bool VEC>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_kernel(ScanArgs a, int blocks_per_group) {
  using L = BwdTile<SL>;
  constexpr int K = kScanSub, CB = L::CB, SP = L::SP, EPT = L::EPT, CL = L::CL;
  __shared__ __align__(16) float sD[K * CB], sU[K * CB], sG[K * CB];
  __shared__ __align__(16) float sP[K * CB], sX[K * CB], sY[K * CB];   // sums over the states
  __shared__ __align__(16) f2 sB[K * SP], sC[K * SP];
  __shared__ float sW[kWarps][K][2 * SP];                               // sums over the channels
  const Range r = block_channels(blockIdx.x, blocks_per_group, a.D, a.G, CB);
  const int chunk = blockIdx.y, b = blockIdx.z;
  const int len = sequence_length(a.lens, b, a.N);
  const int t0 = chunk * a.chunk, t1 = min(a.N, t0 + a.chunk), te = min(t1, len);
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int sl = lane % SL, cl = lane / SL, cw = warp * L::WC + cl * 2;
  const int c = r.c0 + cw;
  const int row = threadIdx.x / L::TPR, col = threadIdx.x % L::TPR * EPT;
  const int sc = r.c0 + col, valid = min(EPT, r.c1 - sc);
  const long long seq = (long long)b * a.N;
  const int subs = (a.N + K - 1) / K;
  const int cb = blockIdx.x % blocks_per_group;
  float* bcpart = a.bcpart + (((long long)cb * a.B + b) * a.N * a.G + r.g) * 2 * SP;
  float bias[EPT], skip[EPT], accD[EPT], accb[EPT];
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    bias[i] = a.dt_bias && i < valid ? a.dt_bias[sc + i] : 0.0f;
    skip[i] = a.Dskip && i < valid ? a.Dskip[sc + i] : 0.0f;
    accD[i] = accb[i] = 0.0f;
  }
  f2 A2[4], carry[4], dA[4];
  load_A<SL>(a, c, r.c1, sl * 4, A2);
  const long long bk = (long long)b * a.chunks + chunk, at = bk * a.D * SP;
  load_tile<SL>(a.back + at, c, r.c1, sl * 4, carry);
#pragma unroll
  for (int i = 0; i < 4; ++i) dA[i] = 0;
  Raw<T, EPT, VEC> nu, nd, nz, ng;
  auto fetch = [&](int t) {
    const int k = t + row, ok = k < te ? valid : 0;
    nu.load(static_cast<const T*>(a.u) + (seq + k) * a.u_row + sc, ok);
    nd.load(static_cast<const T*>(a.dt) + (seq + k) * a.dt_row + sc, ok);
    ng.load(static_cast<const T*>(a.dy) + (seq + k) * a.D + sc, ok);
    if (a.z) nz.load(static_cast<const T*>(a.z) + (seq + k) * a.z_row + sc, ok);
  };
  const int last = te > t0 ? (te - 1 - t0) / K * K + t0 : t0 - K;   // first token of the last 8
  if (last >= t0) fetch(last);
  for (int t = last; t >= t0; t -= K) {
    const Raw<T, EPT, VEC> ru = nu, rd = nd, rz = nz, rg = ng;
    const bool on = t + row < te;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const float raw = rd.get(i) + bias[i];
      sD[row * CB + col + i] = on && i < valid ? (a.softplus ? softplus(raw) : raw) : 0.0f;
      sU[row * CB + col + i] = ru.get(i);
      float g = rg.get(i);
      if (a.z) {
        const float z = rz.get(i);
        g *= z * fast_sigmoid(z);
      }
      sG[row * CB + col + i] = g;
    }
    stage_bc<T, SL, K>(sB, a.Bm, a.b_row, a, b, r.g, t, te - t);
    stage_bc<T, SL, K>(sC, a.Cm, a.c_row, a, b, r.g, t, te - t);
    __syncthreads();
    if (t - K >= t0) fetch(t - K);

    // the state in front of the 8 tokens: the mark plus the chunk's decayed start state
    f2 h0[4], h[K][4], e[K][4];
    {
      const long long mark = (long long)b * subs + t / K;
      const f2 m2 = load_pair(a.msum + mark * a.D, c, r.c1, 0, 1);
      f2 start[4];
      load_tile<SL>(a.ends + at, c, r.c1, sl * 4, start);
      load_tile<SL>(a.marks + mark * a.D * SP, c, r.c1, sl * 4, h0);
#pragma unroll
      for (int i = 0; i < 4; ++i) h0[i] = fma2(ex2_2(mul2(m2, A2[i])), start[i], h0[i]);
    }
    constexpr int YB = SL / 2;             // tokens whose C h sums leave together
    float vy[SL];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const f2 d2 = *reinterpret_cast<const f2*>(&sD[k * CB + cw]);
      const f2 du = mul2(d2, *reinterpret_cast<const f2*>(&sU[k * CB + cw]));
      f2 y = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[k][i] = ex2_2(mul2(d2, A2[i]));
        h[k][i] = fma2(e[k][i], k ? h[k - 1][i] : h0[i], mul2(du, sB[k * SP + sl * 4 + i]));
        y = fma2(h[k][i], sC[k * SP + sl * 4 + i], y);
      }
      if (a.z) {
        unpack2(y, vy[2 * (k % YB)], vy[2 * (k % YB) + 1]);
        if (k % YB == YB - 1) {
          butterfly<SL, 0, SL>(vy, lane);
          sY[(k / YB * YB + sl / 2) * CB + cw + (sl & 1)] = vy[0];
        }
      }
    }
    constexpr int RB = SL > 4 ? SL / 4 : 1;   // tokens whose p and x sums leave together
    constexpr int RV = 4 * RB;
    float vr[RV];
#pragma unroll
    for (int k = K - 1; k >= 0; --k) {
      const f2 d2 = *reinterpret_cast<const f2*>(&sD[k * CB + cw]);
      const f2 g2 = *reinterpret_cast<const f2*>(&sG[k * CB + cw]);
      const f2 du = mul2(d2, *reinterpret_cast<const f2*>(&sU[k * CB + cw]));
      f2 sp = 0, sx = 0;
      float v[8];                              // dB, dC of the lane's 4 states
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f2 dh = fma2(g2, sC[k * SP + sl * 4 + i], carry[i]);
        carry[i] = mul2(e[k][i], dh);
        const f2 p = mul2(carry[i], k ? h[k - 1][i] : h0[i]);
        sp = fma2(A2[i], p, sp);
        dA[i] = fma2(d2, p, dA[i]);
        sx = fma2(dh, sB[k * SP + sl * 4 + i], sx);
        float lo, hi;
        unpack2(mul2(dh, du), lo, hi);
        v[i] = lo + hi;
        unpack2(mul2(g2, h[k][i]), lo, hi);
        v[4 + i] = lo + hi;
      }
      // over the states: p and x of both channels
      const int j = (K - 1 - k) % RB;
      unpack2(sp, vr[4 * j], vr[4 * j + 1]);
      unpack2(sx, vr[4 * j + 2], vr[4 * j + 3]);
      if (j == RB - 1) {
        butterfly<SL, 0, RV>(vr, lane);
#pragma unroll
        for (int q = 0; q < RV / SL; ++q) {
          const int id = sl * (RV / SL) + q;    // token in the batch, then p / x, then channel
          float* dst = id & 2 ? sX : sP;
          dst[(k + RB - 1 - id / 4) * CB + cw + (id & 1)] = vr[q];
        }
      }
      // over the channels: lane cl gets the sums from index cl * 8 / CL on
      butterfly<CL, (SL == 2 ? 1 : SL == 4 ? 2 : SL == 8 ? 3 : 4), 8>(v, lane);
      constexpr int OV = CL >= 8 ? 1 : 8 / CL;
      if (CL <= 8 || cl % (CL / 8 > 0 ? CL / 8 : 1) == 0) {
#pragma unroll
        for (int q = 0; q < OV; ++q) {
          const int id = CL >= 8 ? cl / (CL / 8 > 0 ? CL / 8 : 1) : cl * OV + q;
          sW[warp][k][(id / 4) * SP + sl * 4 + id % 4] = v[q];
        }
      }
    }
    __syncthreads();
    // per (token, channel)
    if (on) {
      Raw<T, EPT, VEC> odu, odt, odz;
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const int o = row * CB + col + i;
        const float g = sG[o], u = sU[o], x = sX[o];
        odu.set(i, fmaf(skip[i], g, sD[o] * x));
        float dd = fmaf(u, x, sP[o] * kLn2);
        if (a.softplus) dd *= fast_sigmoid(rd.get(i) + bias[i]);
        odt.set(i, dd);
        accD[i] = fmaf(g, u, accD[i]);
        accb[i] += i < valid ? dd : 0.0f;
        if (a.z) {
          const float z = rz.get(i), sg = fast_sigmoid(z);
          odz.set(i, rg.get(i) * fmaf(skip[i], u, sY[o]) * sg * fmaf(z, 1.0f - sg, 1.0f));
        }
      }
      const long long o = (seq + t + row) * a.D + sc;
      odu.store(static_cast<T*>(a.du) + o, valid);
      odt.store(static_cast<T*>(a.ddt) + o, valid);
      if (a.z) odz.store(static_cast<T*>(a.dz) + o, valid);
    }
    // per (token, state): the block's channels
    for (int i = threadIdx.x; i < K * 2 * SP; i += kThreads) {
      const int k = i / (2 * SP), q = i % (2 * SP);
      if (t + k < te) {
        float v = sW[0][k][q];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) v += sW[w][k][q];
        bcpart[(long long)(t + k) * a.G * 2 * SP + q] = v;
      }
    }
  }
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
  for (int i = 0; i < 4; ++i) {
    store_pair(a.apart + bk * a.D * a.S, c, r.c1, sl * 4 + i, a.S, dA[i]);
    if (a.dstate_in && chunk == 0)
      store_pair(a.dstate_in + (long long)b * a.D * a.S, c, r.c1, sl * 4 + i, a.S, carry[i]);
  }
  // dD and ddt_bias: the 8 token rows of a channel, through shared memory in a fixed order
  __syncthreads();
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    sP[row * CB + col + i] = accD[i];
    sX[row * CB + col + i] = accb[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * CB; i += kThreads) {
    const int ch = i % CB;
    const float* src = i < CB ? sP : sX;
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) v += src[k * CB + ch];
    if (r.c0 + ch < r.c1) a.dpart[(bk * 2 + i / CB) * a.D + r.c0 + ch] = v;
  }
}

// dB and dC: the sum over the channel blocks of a group, rounded once.
template <typename T>
__global__ void __launch_bounds__(256) scan_sum_bc_kernel(ScanArgs a, int blocks_per_group, int SP) {
  const long long rows = (long long)a.B * a.N * a.G;
  TTT_GRID_LOOP(i, rows * 2 * SP) {
    const int q = (int)(i % (2 * SP)), s = q % SP;
    const long long row = i / (2 * SP);
    if (s >= a.S) continue;
    float v = 0.0f;
    for (int k = 0; k < blocks_per_group; ++k) v += a.bcpart[k * rows * 2 * SP + i];
    static_cast<T*>(q < SP ? a.dB : a.dC)[row * a.S + s] = from_f32<T>(v);
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

template <typename T, int SL, bool VEC, Kernel K>
cudaError_t launch_kernel(const ScanArgs& a, cudaStream_t s) {
  const int bpg = scan_channel_blocks(a.D, a.G, a.S);
  const dim3 grid(bpg * a.G, K == ENDS ? a.chunks - 1 : a.chunks, a.B);
  if constexpr (K == ENDS) scan_fwd_kernel<T, SL, VEC, false><<<grid, kThreads, 0, s>>>(a, bpg);
  if constexpr (K == OUTPUTS) scan_fwd_kernel<T, SL, VEC, true><<<grid, kThreads, 0, s>>>(a, bpg);
  if constexpr (K == MARKS) {
    if (a.chunks > 1) scan_marks_kernel<T, SL, VEC, true><<<grid, kThreads, 0, s>>>(a, bpg);
    else scan_marks_kernel<T, SL, VEC, false><<<grid, kThreads, 0, s>>>(a, bpg);
  }
  if constexpr (K == MAIN) scan_bwd_kernel<T, SL, VEC><<<grid, kThreads, 0, s>>>(a, bpg);
  return cudaGetLastError();
}

template <typename T, int SL, Kernel K>
cudaError_t launch_vec(const ScanArgs& a, cudaStream_t s) {
  constexpr int ept = K == MAIN ? BwdTile<SL>::EPT : Tile<SL>::EPT;
  return fits(a, ept, sizeof(T)) ? launch_kernel<T, SL, true, K>(a, s)
                                 : launch_kernel<T, SL, false, K>(a, s);
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

template <typename T, int SL>
cudaError_t launch_step(const ScanArgs& a, cudaStream_t s) {
  const long long threads = (long long)a.B * a.D * SL;
  const unsigned grid = (unsigned)((threads + kThreads - 1) / kThreads);
  const bool vec = a.S % 4 == 0 && (reinterpret_cast<uintptr_t>(a.state_out) |
                                    reinterpret_cast<uintptr_t>(a.A)) % 16 == 0;
  if (vec) scan_step_kernel<T, SL, true><<<grid, kThreads, 0, s>>>(a);
  else scan_step_kernel<T, SL, false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
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

int scan_chunks(int B, int N, int D, int G, int S, bool backward, int* chunk) {
  const long long warps = (long long)B * G * scan_channel_blocks(D, G, S) * kWarps;
  const long long want = backward ? 148 * 16 : warps < 148 * 4 ? 148 * 16 : 0;
  long long n = warps > 0 && want > warps ? (want + warps - 1) / warps : 1;
  const long long most = (N + 127) / 128;      // pieces of 128 tokens at least
  if (n > most) n = most;
  if (n > 4096) n = 4096;
  if (n < 1) n = 1;
  long long len = (N + n - 1) / n;
  len = (len + 31) / 32 * 32;                  // whole staged tiles
  if (len < 32) len = 32;
  *chunk = (int)len;
  return N > 0 ? (int)((N + len - 1) / len) : 1;
}

cudaError_t scan_fwd_ends(int dt, const ScanArgs& a, cudaStream_t s) { return launch<ENDS>(dt, a, s); }
cudaError_t scan_fwd_outputs(int dt, const ScanArgs& a, cudaStream_t s) { return launch<OUTPUTS>(dt, a, s); }
cudaError_t scan_bwd_marks(int dt, const ScanArgs& a, cudaStream_t s) { return launch<MARKS>(dt, a, s); }
cudaError_t scan_bwd_main(int dt, const ScanArgs& a, cudaStream_t s) { return launch<MAIN>(dt, a, s); }

cudaError_t scan_join(const ScanArgs& a, bool backward, cudaStream_t s) {
  const int SP = scan_padded_state(a.S);
  const unsigned grid = grid_for((long long)a.B * a.D * SP, 256);
  if (backward) scan_join_kernel<true><<<grid, 256, 0, s>>>(a, SP);
  else scan_join_kernel<false><<<grid, 256, 0, s>>>(a, SP);
  return cudaGetLastError();
}

cudaError_t scan_step(int dt, const ScanArgs& a, cudaStream_t s) {
  return dt == DT_BF16 ? launch_step_state<bf16>(a, s) : launch_step_state<float>(a, s);
}

cudaError_t scan_bwd_sum_bc(int dt, const ScanArgs& a, cudaStream_t s) {
  const int SP = scan_padded_state(a.S), bpg = scan_channel_blocks(a.D, a.G, a.S);
  const unsigned grid = grid_for((long long)a.B * a.N * a.G * 2 * SP, 256);
  if (dt == DT_BF16) scan_sum_bc_kernel<bf16><<<grid, 256, 0, s>>>(a, bpg, SP);
  else scan_sum_bc_kernel<float><<<grid, 256, 0, s>>>(a, bpg, SP);
  return cudaGetLastError();
}

}  // namespace ttt
