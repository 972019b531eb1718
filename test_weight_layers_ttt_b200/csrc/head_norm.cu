// Head norm and position rotation in one pass, from the projection's token-major rows
// [B, N, H, h] (slices of a fused projection included) to the layer's head-major [B, H, N, h]:
//     y = w * x * r,  r = (sum x^2 + eps)^(-1/2) (L2) or (mean x^2 + eps)^(-1/2) (RMS),
//     out pair p of the first `rot` elements = (a cos - b sin, b cos + a sin),
//     angle = position * inv_freq[p].
//
// HBM bound (each element is read and written once), so the layout serves the accesses: a row
// (token, head) belongs to a group of 1..32 lanes, a lane owns runs of V element pairs and
// loads both halves of each pair itself, so the rotation needs no exchange and the norm only a
// shuffle sum. The angles of a token are the same for all heads: a block takes a tile of
// tokens with all their heads and computes each cosine and sine once into shared memory, from
// a 64-bit product (fp32 loses far positions: 1e6 * 2^-24 is 0.06 of a radian) reduced to
// [-1/2, 1/2] turns.
#include "mixer.h"
#include "mixer_common.cuh"

namespace ttt {
namespace {

constexpr int kHeadThreads = 256;
constexpr int kMaxTile = 32;
constexpr double kInvTwoPi = 0.15915494309189533576888;

enum : int { PAIRS_HALVES = 0, PAIRS_INTERLEAVED = 1 };

// First and second element of pair `p`: rotated pairs first, then the elements behind `rot`
// paired the same way (the last pair of an odd h has no second element).
template <int PAIRS>
__device__ __forceinline__ void pair_at(int p, int rot, int h, int& lo, int& hi) {
  if (PAIRS == PAIRS_INTERLEAVED) {
    lo = 2 * p;
    hi = 2 * p + 1;
  } else if (p < rot / 2) {
    lo = p;
    hi = p + rot / 2;
  } else {
    lo = rot + (p - rot / 2);
    hi = lo + (h - rot + 1) / 2;
  }
}

// V pairs from p on (all of one kind; V > 1 only when every half is whole runs of V).
template <typename T, int V, int PAIRS>
__device__ __forceinline__ void load_pairs(const T* row, int p, int rot, int h, float (&a)[V],
                                           float (&b)[V]) {
  int lo, hi;
  pair_at<PAIRS>(p, rot, h, lo, hi);
  if constexpr (V == 1) {
    a[0] = to_f32(row[lo]);
    b[0] = hi < h ? to_f32(row[hi]) : 0.0f;
  } else if constexpr (PAIRS == PAIRS_INTERLEAVED) {
    float f[2][V];
    load_vec<T, V>(row + lo, f[0]);
    load_vec<T, V>(row + lo + V, f[1]);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      a[i] = f[2 * i / V][2 * i % V];
      b[i] = f[(2 * i + 1) / V][(2 * i + 1) % V];
    }
  } else {
    load_vec<T, V>(row + lo, a);
    load_vec<T, V>(row + hi, b);
  }
}

template <typename T, int V, int PAIRS>
__device__ __forceinline__ void store_pairs(T* row, int p, int rot, int h, const float (&a)[V],
                                            const float (&b)[V]) {
  int lo, hi;
  pair_at<PAIRS>(p, rot, h, lo, hi);
  if constexpr (V == 1) {
    row[lo] = from_f32<T>(a[0]);
    if (hi < h) row[hi] = from_f32<T>(b[0]);
  } else if constexpr (PAIRS == PAIRS_INTERLEAVED) {
    float f[2][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f[2 * i / V][2 * i % V] = a[i];
      f[(2 * i + 1) / V][(2 * i + 1) % V] = b[i];
    }
    store_vec<T, V>(row + lo, f[0]);
    store_vec<T, V>(row + lo + V, f[1]);
  } else {
    store_vec<T, V>(row + lo, a);
    store_vec<T, V>(row + hi, b);
  }
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int m = lanes / 2; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// One tile of `tile` tokens (all heads) per iteration; E runs of V pairs per lane, `lanes`
// lanes per row. Dynamic shared memory: float2[tile][rot / 2], and in the backward with
// weights float[2][h] behind it.
template <typename T, int V, int PAIRS, int E, bool BWD>
__global__ void __launch_bounds__(kHeadThreads) head_kernel(HeadArgs a, int tile, int lanes) {
  extern __shared__ float2 turns[];
  const long long M = (long long)a.B * a.N;
  const int half = a.rot / 2, npairs = (a.h + 1) / 2;
  const int heads = a.H[0] + a.H[1] + a.H[2];
  const int lane = threadIdx.x % lanes, group = threadIdx.x / lanes, groups = kHeadThreads / lanes;
  float dw[2][E][2][V];
  if (BWD) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int q = 0; q < V; ++q) dw[i][e][0][q] = dw[i][e][1][q] = 0.0f;
  }
  for (long long m0 = (long long)blockIdx.x * tile; m0 < M; m0 += (long long)gridDim.x * tile) {
    if (half) {
      __syncthreads();   // the tile before is done with the angles
      for (int i = threadIdx.x; i < tile * half; i += kHeadThreads) {
        const long long m = m0 + i / half;
        if (m >= M) break;
        const double pos = a.positions ? (double)a.positions[m] : (double)(a.pos0 + m % a.N);
        double turn = pos * (double)a.inv_freq[i % half] * kInvTwoPi;
        turn -= rint(turn);
        float2 cs;
        sincospif((float)(2.0 * turn), &cs.y, &cs.x);
        turns[i] = cs;
      }
      __syncthreads();
    }
    // Row i of the tile is token i % tile of head i / tile: neighbouring groups write
    // neighbouring rows of the head-major output. All lanes of a warp take every iteration.
    const int rows = tile * heads;
    for (int i0 = 0; i0 < rows; i0 += groups) {
      const int i = i0 + group;
      const long long m = m0 + i % tile;
      int head = i / tile;
      const bool live = i < rows && m < M;
      const int kind = head < a.H[0] ? 0 : head < a.H[0] + a.H[1] ? 1 : 2;
      head -= kind == 0 ? 0 : kind == 1 ? a.H[0] : a.H[0] + a.H[1];
      const long long b = m / a.N, t = m - b * a.N;
      const T* x = static_cast<const T*>(a.x[kind]) + m * a.row[kind] + (long long)head * a.h;
      const long long at = ((b * a.H[kind] + head) * a.N + t) * a.h;
      const float2* cs = turns + (i % tile) * half;
      const float* w = kind < 2 ? a.w[kind] : nullptr;
      const bool normed = kind < 2 && a.norm != TTT_NORM_NONE;
      const bool turned = kind < 2;
      float xa[E][V], xb[E][V], ga[E][V], gb[E][V], wa[E][V], wb[E][V];
      float ss = 0.0f, dot = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int p = (e * lanes + lane) * V;
        const bool on = live && p < npairs;
#pragma unroll
        for (int q = 0; q < V; ++q) {
          xa[e][q] = xb[e][q] = ga[e][q] = gb[e][q] = 0.0f;
          wa[e][q] = wb[e][q] = 1.0f;
        }
        if (!on) continue;
        if (!BWD || turned) load_pairs<T, V, PAIRS>(x, p, a.rot, a.h, xa[e], xb[e]);
        if (w) load_pairs<float, V, PAIRS>(w, p, a.rot, a.h, wa[e], wb[e]);
        if (BWD) load_pairs<T, V, PAIRS>(static_cast<const T*>(a.dout[kind]) + at, p, a.rot, a.h, ga[e], gb[e]);
#pragma unroll
        for (int q = 0; q < V; ++q) {
          ss = fmaf(xa[e][q], xa[e][q], ss);
          ss = fmaf(xb[e][q], xb[e][q], ss);
          if (BWD && turned) {
            if (p + q < half) {   // the rotation's transpose
              const float2 c = cs[p + q];
              const float u = ga[e][q], v = gb[e][q];
              ga[e][q] = u * c.x + v * c.y;
              gb[e][q] = v * c.x - u * c.y;
            }
            dot = fmaf(ga[e][q] * wa[e][q], xa[e][q], dot);
            dot = fmaf(gb[e][q] * wb[e][q], xb[e][q], dot);
          }
        }
      }
      const float inv_h = a.norm == TTT_NORM_RMS ? 1.0f / a.h : 1.0f;
      ss = group_sum(ss, lanes);
      const float r = normed ? rsqrtf(fmaf(ss, inv_h, a.eps)) : 1.0f;
      float back = 0.0f;
      if (BWD) {
        dot = group_sum(dot, lanes);
        back = normed ? r * r * r * dot * inv_h : 0.0f;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int p = (e * lanes + lane) * V;
        if (!live || p >= npairs) continue;
        float oa[V], ob[V];
#pragma unroll
        for (int q = 0; q < V; ++q) {
          if (!BWD) {
            const float u = xa[e][q] * r * wa[e][q], v = xb[e][q] * r * wb[e][q];
            if (turned && p + q < half) {
              const float2 c = cs[p + q];
              oa[q] = u * c.x - v * c.y;
              ob[q] = v * c.x + u * c.y;
            } else {
              oa[q] = u;
              ob[q] = v;
            }
          } else {
            oa[q] = fmaf(ga[e][q] * wa[e][q], r, -xa[e][q] * back);
            ob[q] = fmaf(gb[e][q] * wb[e][q], r, -xb[e][q] * back);
            if (w) {
#pragma unroll
              for (int z = 0; z < 2; ++z)
                if (kind == z) {
                  dw[z][e][0][q] = fmaf(ga[e][q] * r, xa[e][q], dw[z][e][0][q]);
                  dw[z][e][1][q] = fmaf(gb[e][q] * r, xb[e][q], dw[z][e][1][q]);
                }
            }
          }
        }
        T* out = BWD ? static_cast<T*>(a.dx[kind]) + (m * a.H[kind] + head) * a.h
                     : static_cast<T*>(a.out[kind]) + at;
        store_pairs<T, V, PAIRS>(out, p, a.rot, a.h, oa, ob);
      }
    }
  }
  if (BWD && a.partials) {
    // one row of partial weight gradients per block: groups of a warp by shuffles, warps in
    // order through shared memory
    float* acc = reinterpret_cast<float*>(turns + tile * half);
    for (int i = threadIdx.x; i < 2 * a.h; i += kHeadThreads) acc[i] = 0.0f;
    __syncthreads();
    for (int wp = 0; wp < kHeadThreads / 32; ++wp) {
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int q = 0; q < V; ++q) {
            float u = dw[z][e][0][q], v = dw[z][e][1][q];
            if (threadIdx.x / 32 != wp) continue;
            for (int m = lanes; m < 32; m *= 2) {
              u += __shfl_xor_sync(0xffffffffu, u, m);
              v += __shfl_xor_sync(0xffffffffu, v, m);
            }
            const int p = (e * lanes + lane) * V + q;
            if (threadIdx.x % 32 >= lanes || p >= npairs) continue;
            int lo, hi;
            pair_at<PAIRS>(p, a.rot, a.h, lo, hi);
            acc[z * a.h + lo] += u;
            if (hi < a.h) acc[z * a.h + hi] += v;
          }
      __syncthreads();
    }
    float* part = a.partials + (long long)blockIdx.x * 2 * a.h;
    for (int i = threadIdx.x; i < 2 * a.h; i += kHeadThreads) part[i] = acc[i];
  }
}

// Tokens of a tile: enough rows for two rounds of the block's groups, while the tiles still
// give every SM four blocks.
int head_tile(const HeadArgs& a, int groups) {
  const long long M = (long long)a.B * a.N;
  const int heads = a.H[0] + a.H[1] + a.H[2];
  int tile = 1;
  while (tile < kMaxTile && tile * heads < 2 * groups && M / (2 * tile) >= 148 * 4) tile *= 2;
  return tile;
}

template <typename T, int V, int PAIRS, int E, bool BWD>
cudaError_t launch_tiles(const HeadArgs& a, int lanes, cudaStream_t s) {
  const int tile = head_tile(a, kHeadThreads / lanes);
  const long long M = (long long)a.B * a.N, tiles = (M + tile - 1) / tile;
  // at most 32 KB of angles: a row of 256 pairs takes 32 lanes, which makes 16 tokens
  size_t smem = (size_t)tile * (a.rot / 2) * sizeof(float2);
  long long blocks = tiles;
  if (BWD) {
    blocks = head_bwd_blocks(a.B, a.N);
    if (a.partials) smem += 2 * (size_t)a.h * sizeof(float);
  }
  head_kernel<T, V, PAIRS, E, BWD><<<(unsigned)blocks, kHeadThreads, smem, s>>>(a, tile, lanes);
  return cudaGetLastError();
}

template <typename T, int V, int PAIRS, bool BWD>
cudaError_t launch_runs(const HeadArgs& a, cudaStream_t s) {
  const int runs = ((a.h + 1) / 2 + V - 1) / V;   // V pairs each
  int lanes = 1;
  while (lanes < 32 && lanes < runs) lanes *= 2;
  const int e = (runs + lanes - 1) / lanes;
  if (e <= 1) return launch_tiles<T, V, PAIRS, 1, BWD>(a, lanes, s);
  if constexpr (V <= 4)
    if (e <= 2) return launch_tiles<T, V, PAIRS, 2, BWD>(a, lanes, s);
  if constexpr (V <= 2)
    if (e <= 4) return launch_tiles<T, V, PAIRS, 4, BWD>(a, lanes, s);
  if constexpr (V <= 1)
    if (e <= 8) return launch_tiles<T, V, PAIRS, 8, BWD>(a, lanes, s);
  return cudaErrorInvalidValue;
}

// Whether every half of every row starts on V elements and holds whole runs of them.
bool fits(const HeadArgs& a, int V, int size) {
  if (a.h % (2 * V)) return false;
  if (a.pairs == PAIRS_HALVES && (a.rot / 2 % V || (a.h - a.rot) / 2 % V)) return false;
  for (int i = 0; i < 3; ++i) {
    if (!a.H[i]) continue;
    if (a.row[i] % V) return false;
    for (const void* p : {a.x[i], (const void*)a.out[i], a.dout[i], (const void*)a.dx[i]})
      if (reinterpret_cast<uintptr_t>(p) % (V * size)) return false;
  }
  for (const float* p : {a.w[0], a.w[1]})
    if (reinterpret_cast<uintptr_t>(p) % (V * 4 < 16 ? V * 4 : 16)) return false;
  return true;
}

template <typename T, int V, bool BWD>
cudaError_t launch_pairs(const HeadArgs& a, cudaStream_t s) {
  return a.pairs == PAIRS_HALVES ? launch_runs<T, V, PAIRS_HALVES, BWD>(a, s)
                                 : launch_runs<T, V, PAIRS_INTERLEAVED, BWD>(a, s);
}

template <bool BWD>
cudaError_t launch(int dt, const HeadArgs& a, cudaStream_t s) {
  if (dt == DT_BF16) {
    if (fits(a, 8, 2)) return launch_pairs<bf16, 8, BWD>(a, s);
    if (fits(a, 4, 2)) return launch_pairs<bf16, 4, BWD>(a, s);
    if (fits(a, 2, 2)) return launch_pairs<bf16, 2, BWD>(a, s);
    return launch_pairs<bf16, 1, BWD>(a, s);
  }
  if (fits(a, 4, 4)) return launch_pairs<float, 4, BWD>(a, s);
  if (fits(a, 2, 4)) return launch_pairs<float, 2, BWD>(a, s);
  return launch_pairs<float, 1, BWD>(a, s);
}

}  // namespace

long long head_bwd_blocks(int B, int N) {
  const long long M = (long long)B * N;
  return M < 148 * 4 ? M : 148 * 4;
}

cudaError_t head_fwd(int dt, const HeadArgs& a, cudaStream_t s) { return launch<false>(dt, a, s); }
cudaError_t head_bwd(int dt, const HeadArgs& a, cudaStream_t s) { return launch<true>(dt, a, s); }

}  // namespace ttt
