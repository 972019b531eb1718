// Head norm and position rotation in one pass, from the projection's token-major rows
// [B, N, H, h] (slices of a fused projection included) to the layer's head-major [B, H, N, h]:
//     y = w * x * r,  r = (sum x^2 + eps)^(-1/2) (L2) or (mean x^2 + eps)^(-1/2) (RMS),
//     out pair p of the first `rot` elements = (a cos - b sin, b cos + a sin),
//     angle = position * inv_freq[p].
//
// HBM bound (each element is read and written once), so the layout serves the accesses: a row
// (token, head) belongs to a group of 1..32 lanes, a lane owns runs of V element pairs and
// loads both halves of each pair itself, so the rotation needs no exchange and the norm only a
// shuffle sum. The angles of a token are the same for all its heads: a group keeps one token
// and its lanes the cosines and sines of their pairs in registers, each taken once, from a
// 64-bit product (fp32 loses far positions: 1e6 * 2^-24 is 0.06 of a radian) reduced to
// [-1/2, 1/2] turns. 2 x 32768 tokens of 3 x 4 heads of 256: 144 to 152 us on different cards, 5.3
// to 5.6 TB/s, 81 to 85 % of the measured copy rate; 65536 tokens of 3 x 8 heads of 128 backward:
// 219 to 226 us, 73 to 75 %.
#include <algorithm>

#include "mixer.h"
#include "mixer_common.cuh"

namespace ttt {
namespace {

constexpr int kHeadThreads = 128;
// Blocks of an SM (what the registers leave; the backward keeps two weight gradients in them)
// and rows that each thread has on their way. Two lm-sized tensors' forward of 256 elements a
// head: 162 us with one row ahead in registers, 145 us with 4 blocks of 4 rows, 137 us with 6 of
// 3; backward at 128: 320 us in registers, 224 us with 3 blocks of 3, 308 us with 4 blocks (spills).
// Forward pairs in halves of more than 256 elements that are not whole 16-byte runs spill 24 to 86
// bytes with 6.
constexpr int kFwdBlocks = 6, kBwdBlocks = 3;
// Rows of one-element accesses (V = 1) have little in flight per thread, so their backward takes
// the blocks that its registers leave room for (figures of the time): 24688 tokens of 17 bf16 heads of 81 elements
// (E = 2) 205 us with 3 blocks, 143 us with 5, 136 us with 6, 147 us with 8; 6000 tokens of 9
// heads of 255 (E = 4) 60 us with 2, 47 us with 3, 43 us with 4; of 511 (E = 8) 100 us with 2,
// 87 us with 3, 118 us with 4, and forward 52 us with 3, 43 us with 4, 49 us with 6.
constexpr int bwd_blocks(int E, int V) {
  return E * V == 1 ? 8 : E * V == 2 ? 6 : E == 4 && V == 1 ? 4 : kBwdBlocks;
}
// Forward, heads of which a part is rotated (`all` false): 69 registers where all has 64, so the 8
// blocks that those leave room for are asked for (17 heads of 81, none of it rotated: 89 us, 92 us
// without; with whole rotation 42 us at 2 x 6172 tokens of 16 heads, 43 us if it is asked for).
constexpr int fwd_blocks(int E, int V, bool all) { return !all && V == 1 && E <= 2 ? 8 : E < 8 ? kFwdBlocks : 4; }
constexpr int kFwdRows = 3, kBwdRows = 3;
constexpr double kInvTwoPi = 0.15915494309189533576888;

enum : int { PAIRS_HALVES = 0, PAIRS_INTERLEAVED = 1 };

// The backward without a norm has kernels of its own: its dx does not depend on x, which may be
// infinite, and a branch in the common kernel costs 3 % (65536 tokens of 3 x 8 heads of 128: 226
// us, 232 us with it).
enum Pass { FWD, BWD_NORMED, BWD_PLAIN };

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

// V pairs from p on as they are in memory (all of one kind; V > 1 only when every half is whole
// runs of V), or zeros; and as floats.
template <typename T, int V> struct RawPairs {
  typename Pack<T, V>::U a, b;
};
template <typename T, int V>
__device__ __forceinline__ void load_raw_pairs(RawPairs<T, V>& r, const T* row, int lo, int hi, bool on, bool on_hi) {
  load_here(row + lo, on, r.a);
  load_here(row + hi, on_hi, r.b);
}
// 2V neighbours to V first and V second elements.
template <int V>
__device__ __forceinline__ void deal(float (&a)[V], float (&b)[V]) {
  float f[2 * V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    f[i] = a[i];
    f[V + i] = b[i];
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    a[i] = f[2 * i];
    b[i] = f[2 * i + 1];
  }
}
template <typename T, int V, int PAIRS>
__device__ __forceinline__ void unpack_pairs(const RawPairs<T, V>& r, float (&a)[V], float (&b)[V]) {
  unpack<T, V>(r.a, a);
  unpack<T, V>(r.b, b);
  if constexpr (V > 1 && PAIRS == PAIRS_INTERLEAVED) deal(a, b);
}

template <typename T, int V, int PAIRS>
__device__ __forceinline__ void store_pairs(T* row, int lo, int hi, bool on_hi, const float (&a)[V],
                                            const float (&b)[V]) {
  if constexpr (V > 1 && PAIRS == PAIRS_INTERLEAVED) {
    float f[2][V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f[2 * i / V][2 * i % V] = a[i];
      f[(2 * i + 1) / V][(2 * i + 1) % V] = b[i];
    }
    store_vec<T, V>(row + lo, f[0]);
    store_vec<T, V>(row + hi, f[1]);
  } else {
    store_vec<T, V>(row + lo, a);
    if (on_hi) store_vec<T, V>(row + hi, b);
  }
}

__device__ __forceinline__ float group_sum(float v, int lanes) {
  for (int m = lanes / 2; m > 0; m /= 2) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// A walk over the rows of a group's token: the heads of q, then of k, then of v, `step` heads
// apart. All groups of a block walk alike (head - first is the same), whether or not their token
// and head exist.
template <typename T>
struct Walk {
  int kind = 0, head = 0;
  T* p[2];          // this head's row in one or two tensors
  // On to the first head of the next tensor that has any; start(kind, which) gives its row.
  template <typename F>
  __device__ __forceinline__ void enter(const HeadArgs& a, int k, int first, F&& start) {
    while (k < 3 && a.H[k] == 0) ++k;
    kind = k;
    head = first;
    if (k < 3) {
      p[0] = start(k, 0);
      p[1] = start(k, 1);
    }
  }
  template <typename F>
  __device__ __forceinline__ void next(const HeadArgs& a, int first, int step, long long s0, long long s1, F&& start) {
    head += step;
    p[0] += s0;
    p[1] += s1;
    if (head - first >= a.H[kind]) enter(a, kind + 1, first, start);
  }
};

// A thread's rows on their way: `depth` of them, `items` accesses each, at most 256 bytes of
// shared memory.
template <typename T, int V, int E, bool BWD> struct Ring {
  static constexpr bool on = V * sizeof(T) >= 4;
  static constexpr int items = E * (BWD ? 4 : 2), bytes = items * V * (int)sizeof(T);
  static constexpr int most = BWD ? kBwdRows : kFwdRows;
  static constexpr int depth = !on ? 1 : most * bytes <= 256 ? most : 256 / bytes;
};

// A tile is 2^log_tile tokens: group g takes token g % tile and every (groups / tile)-th head of
// it, so that a lane takes the angles of its pairs once for all heads, into registers, and
// neighbouring groups write neighbouring rows of the head-major output. E runs of V pairs per
// lane, `lanes` lanes per row. The first rows are on their way before the angles are taken.
// Dynamic shared memory: in the backward float[2][h], then the ring of rows.
template <typename T, int V, int PAIRS, int E, Pass P, bool ALL>
__global__ void __launch_bounds__(kHeadThreads, P != FWD ? bwd_blocks(E, V) : fwd_blocks(E, V, ALL))
    head_kernel(HeadArgs a, int log_tile, int lanes) {
  constexpr bool BWD = P != FWD, NORMED = P == BWD_NORMED;
  extern __shared__ __align__(16) float acc[];
  // The rows on their way: DEPTH of them in shared memory by asynchronous copies, each thread's
  // own, where an access has the 4 bytes that such a copy takes at least; else one in registers.
  using L = Ring<T, V, E, BWD>;
  constexpr bool RING = L::on;
  constexpr int DEPTH = L::depth, ITEMS = L::items;
  using U = typename Pack<T, V>::U;
  U* const ring = reinterpret_cast<U*>(reinterpret_cast<char*>(acc) + (BWD ? 2 * a.h * 4 + 15 & ~15 : 0)) + threadIdx.x;
  const int M = a.B * a.N, half = a.rot / 2, npairs = (a.h + 1) / 2;
  const int lane = threadIdx.x % lanes, group = threadIdx.x / lanes;
  const int first = group >> log_tile, step = (kHeadThreads / lanes) >> log_tile;
  const long long minor_step = (long long)step * a.h, major_step = minor_step * a.N;   // to the next head
  const float inv_h = a.norm == TTT_NORM_RMS ? 1.0f / a.h : 1.0f;
  int lo[E], hi[E];
  bool on[E], on_hi[E];
  float dw[2][E][2][V];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int p = (e * lanes + lane) * V;
    pair_at<PAIRS>(p, a.rot, a.h, lo[e], hi[e]);
    on[e] = p < npairs;
    on_hi[e] = on[e] && (V > 1 || hi[e] < a.h);
    if (V > 1 && PAIRS == PAIRS_INTERLEAVED) hi[e] = lo[e] + V;   // two accesses of V elements
#pragma unroll
    for (int q = 0; q < V; ++q) dw[0][e][0][q] = dw[0][e][1][q] = dw[1][e][0][q] = dw[1][e][1][q] = 0.0f;
  }

  // (x, y) -> (x cos + y s, y cos + x t). Behind the rotated pairs x and y stay as they are, for 0
  // times an infinite neighbour is NaN (ALL: there are none behind, or one, which is alone). Lanes of
  // one pair skip the rotation (2 x 6172 tokens of 16 bf16 heads of 66, 20 of it rotated: 43.4 us,
  // 44.0 us with selects), runs of pairs select (30000 tokens of 24 heads of 128, half of it rotated:
  // 68.7 us, 72.6 us with a skip).
  const auto rotate = [&](int e, float (&x)[V], float (&y)[V], const float (&c)[V], const float (&s)[V],
                          const float (&t)[V]) {
    if (!ALL && V == 1 && (e * lanes + lane) * V >= half) return;
    float u[V], v[V];
    mul_v<V>(u, x, t);
    mul_v<V>(v, y, s);
    if constexpr (!ALL && V > 1) {
#pragma unroll
      for (int q = 0; q < V; ++q)
        if ((e * lanes + lane) * V + q >= half) u[q] = v[q] = 0.0f;
    }
    fma_v<V>(x, x, c, v);
    fma_v<V>(y, y, c, u);
  };
  for (long long tile0 = (long long)blockIdx.x << log_tile; tile0 < M; tile0 += (long long)gridDim.x << log_tile) {
    const long long m = tile0 + (group & ((1 << log_tile) - 1));
    const bool live = m < M;
    const int seq = live ? (int)m / a.N : 0, t = live ? (int)m - seq * a.N : 0;
    const auto major_row = [&](int k) { return (((long long)seq * a.H[k] + first) * a.N + t) * a.h; };
    const auto source = [&](int k, int which) {   // x, and in the backward dout
      return which ? static_cast<const T*>(a.dout[k]) + major_row(k)
                   : static_cast<const T*>(a.x[k]) + m * a.row[k] + first * a.h;
    };
    const auto target = [&](int k, int) {
      return BWD ? static_cast<T*>(a.dx[k]) + (m * a.H[k] + first) * a.h : static_cast<T*>(a.out[k]) + major_row(k);
    };
    Walk<const T> in;
    Walk<T> out;
    in.enter(a, 0, first, source);
    out.enter(a, 0, first, target);
    RawPairs<T, V> rx[E], rg[E];
    int put = 0, take = 0;              // ring entries
    const auto fetch = [&]() {          // behind the last row nothing is loaded, nor waited for
      const bool row = in.kind < 3 && live && in.head < a.H[in.kind < 3 ? in.kind : 0];
      if (in.kind < 3) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const bool x = row && (!BWD || in.kind < 2);
          if constexpr (RING) {
            U* q = ring + (put * ITEMS + e * (BWD ? 4 : 2)) * kHeadThreads;
            copy_async<sizeof(U)>(q, in.p[0] + lo[e], x && on[e]);
            copy_async<sizeof(U)>(q + kHeadThreads, in.p[0] + hi[e], x && on_hi[e]);
            if (BWD) {
              copy_async<sizeof(U)>(q + 2 * kHeadThreads, in.p[1] + lo[e], row && on[e]);
              copy_async<sizeof(U)>(q + 3 * kHeadThreads, in.p[1] + hi[e], row && on_hi[e]);
            }
          } else {
            load_raw_pairs<T, V>(rx[e], in.p[0], lo[e], hi[e], x && on[e], x && on_hi[e]);
            if (BWD) load_raw_pairs<T, V>(rg[e], in.p[1], lo[e], hi[e], row && on[e], row && on_hi[e]);
          }
        }
        in.next(a, first, step, minor_step, BWD ? major_step : 0, source);
      }
      if constexpr (RING) {
        copies_commit();
        put = put + 1 == DEPTH ? 0 : put + 1;
      }
    };
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) fetch();
    float cs[E][V], sn[E][V], ns[E][V], wa[E][V], wb[E][V];   // cos, sin, -sin, weights
    const double pos = !live ? 0.0 : a.positions ? (double)a.positions[m] : (double)(a.pos0 + t);
#pragma unroll
    for (int e = 0; e < E; ++e)
#pragma unroll
      for (int q = 0; q < V; ++q) {
        const int p = (e * lanes + lane) * V + q;
        cs[e][q] = 1.0f;   // behind the rotated elements: as they are
        sn[e][q] = 0.0f;
        if (p < half) {
          double turn = pos * (double)a.inv_freq[p] * kInvTwoPi;
          turn -= rint(turn);
          sincospif((float)(2.0 * turn), &sn[e][q], &cs[e][q]);
        }
        ns[e][q] = -sn[e][q];
      }
    int kind = -1;
    bool scaled = false;
    while (out.kind < 3) {
      float xa[E][V], xb[E][V], ga[E][V], gb[E][V];
      if constexpr (RING) {
        copies_wait_but<DEPTH - 1>();
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const U* q = ring + (take * ITEMS + e * (BWD ? 4 : 2)) * kHeadThreads;
          rx[e].a = q[0];
          rx[e].b = q[kHeadThreads];
          if (BWD) {
            rg[e].a = q[2 * kHeadThreads];
            rg[e].b = q[3 * kHeadThreads];
          }
        }
        take = take + 1 == DEPTH ? 0 : take + 1;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        unpack_pairs<T, V, PAIRS>(rx[e], xa[e], xb[e]);
        if (BWD) unpack_pairs<T, V, PAIRS>(rg[e], ga[e], gb[e]);
      }
      fetch();
      const int H = a.H[out.kind];
      const auto write = [&](int e, const float (&u)[V], const float (&v)[V]) {
        if (live && out.head < H && on[e]) store_pairs<T, V, PAIRS>(out.p[0], lo[e], hi[e], on_hi[e], u, v);
      };
      if (out.kind == 2) {              // v is only laid out
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if constexpr (BWD) write(e, ga[e], gb[e]);
          else write(e, xa[e], xb[e]);
        }
        out.next(a, first, step, BWD ? minor_step : major_step, 0, target);
        continue;
      }
      if (out.kind != kind) {           // the first rows of q or k
        kind = out.kind;
        const float* w = a.w[kind];
        scaled = w != nullptr;
#pragma unroll
        for (int e = 0; e < E; ++e) {
#pragma unroll
          for (int q = 0; q < V; ++q) wa[e][q] = wb[e][q] = 1.0f;
          if (w && on[e]) load_input<float, V>(w + lo[e], wa[e]);
          if (w && on_hi[e]) load_input<float, V>(w + hi[e], wb[e]);
          if constexpr (V > 1 && PAIRS == PAIRS_INTERLEAVED) deal(wa[e], wb[e]);
        }
      }
      float r = 1.0f, back = 0.0f, ss[V] = {}, dot[V] = {}, gwa[E][V], gwb[E][V];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        fma_v<V>(ss, xa[e], xa[e], ss);
        fma_v<V>(ss, xb[e], xb[e], ss);
        if (BWD) {   // the rotation's transpose, then the weights
          rotate(e, ga[e], gb[e], cs[e], sn[e], ns[e]);
#pragma unroll
          for (int q = 0; q < V; ++q) {
            gwa[e][q] = ga[e][q];
            gwb[e][q] = gb[e][q];
          }
          if (scaled) {
            mul_v<V>(gwa[e], ga[e], wa[e]);
            mul_v<V>(gwb[e], gb[e], wb[e]);
          }
          fma_v<V>(dot, gwa[e], xa[e], dot);
          fma_v<V>(dot, gwb[e], xb[e], dot);
        }
      }
      if (BWD ? NORMED : a.norm != TTT_NORM_NONE) {
        const float s = sum_v<V>(ss), d = BWD ? sum_v<V>(dot) : 0.0f;
        r = rsqrtf(fmaf(group_sum(s, lanes), inv_h, a.eps));
        if (BWD) back = -r * group_sum(d, lanes) * inv_h;
      }
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float u[V], v[V];
        if constexpr (!BWD) {
          mul_v<V>(u, xa[e], r);
          mul_v<V>(v, xb[e], r);
          if (scaled) {
            mul_v<V>(u, u, wa[e]);
            mul_v<V>(v, v, wb[e]);
          }
          rotate(e, u, v, cs[e], ns[e], sn[e]);
          write(e, u, v);
        } else {
          // dx = r (g w - n r <g w, x> [/ h]) with n = x r, for r^3 leaves fp32's range where eps
          // and the row are small;  dw += g n
          mul_v<V>(u, xa[e], r);
          mul_v<V>(v, xb[e], r);
          if constexpr (NORMED) {
            fma_v<V>(gwa[e], u, back, gwa[e]);
            fma_v<V>(gwb[e], v, back, gwb[e]);
          }
          mul_v<V>(gwa[e], gwa[e], r);
          mul_v<V>(gwb[e], gwb[e], r);
          write(e, gwa[e], gwb[e]);
          if (a.partials) {
            if (kind == 0) {
              fma_v<V>(dw[0][e][0], ga[e], u, dw[0][e][0]);
              fma_v<V>(dw[0][e][1], gb[e], v, dw[0][e][1]);
            } else {
              fma_v<V>(dw[1][e][0], ga[e], u, dw[1][e][0]);
              fma_v<V>(dw[1][e][1], gb[e], v, dw[1][e][1]);
            }
          }
        }
      }
      out.next(a, first, step, BWD ? minor_step : major_step, 0, target);
    }
  }
  if (BWD && a.partials) {
    // one row of partial weight gradients per block: groups of a warp by shuffles, warps in
    // order through shared memory
    for (int i = threadIdx.x; i < 2 * a.h; i += kHeadThreads) acc[i] = 0.0f;
#pragma unroll
    for (int z = 0; z < 2; ++z)
#pragma unroll
      for (int e = 0; e < E; ++e)
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int q = 0; q < V; ++q)
            for (int w = lanes; w < 32; w *= 2) dw[z][e][k][q] += __shfl_xor_sync(0xffffffffu, dw[z][e][k][q], w);
    for (int wp = 0; wp < kHeadThreads / 32; ++wp) {
      __syncthreads();
      if (threadIdx.x / 32 != wp || threadIdx.x % 32 >= lanes) continue;
#pragma unroll
      for (int z = 0; z < 2; ++z)
#pragma unroll
        for (int e = 0; e < E; ++e)
#pragma unroll
          for (int q = 0; q < V; ++q) {
            const int p = (e * lanes + lane) * V + q;
            if (p >= npairs) continue;
            int lo, hi;
            pair_at<PAIRS>(p, a.rot, a.h, lo, hi);
            acc[z * a.h + lo] += dw[z][e][0][q];
            if (hi < a.h) acc[z * a.h + hi] += dw[z][e][1][q];
          }
    }
    __syncthreads();
    float* part = a.partials + (long long)blockIdx.x * 2 * a.h;
    for (int i = threadIdx.x; i < 2 * a.h; i += kHeadThreads) part[i] = acc[i];
  }
}

template <typename T, int V, int PAIRS, int E, Pass P>
cudaError_t launch_tiles(const HeadArgs& a, int lanes, long long* rows, cudaStream_t s) {
  constexpr bool BWD = P != FWD;
  // A token per group, while the tiles still give every SM four blocks.
  const long long M = (long long)a.B * a.N;
  const int groups = kHeadThreads / lanes;
  int log_tile = 0;
  while (2 << log_tile <= groups && (M >> (log_tile + 1)) >= 148 * 4) ++log_tile;
  const long long tiles = (M + (1 << log_tile) - 1) >> log_tile;
  const long long most = 148LL * bwd_blocks(E, V);   // one wave
  const long long blocks = BWD && tiles > most ? most : tiles;
  if (rows) *rows = blocks;
  size_t smem = BWD ? (2 * (size_t)a.h * sizeof(float) + 15) / 16 * 16 : 0;
  using L = Ring<T, V, E, BWD>;
  if (L::on) smem += (size_t)L::depth * L::bytes * kHeadThreads;
  if (a.rot + 1 >= a.h) head_kernel<T, V, PAIRS, E, P, true><<<(unsigned)blocks, kHeadThreads, smem, s>>>(a, log_tile, lanes);
  else head_kernel<T, V, PAIRS, E, P, false><<<(unsigned)blocks, kHeadThreads, smem, s>>>(a, log_tile, lanes);
  return cudaGetLastError();
}

template <typename T, int V, int PAIRS, Pass P>
cudaError_t launch_runs(const HeadArgs& a, long long* rows, cudaStream_t s) {
  const int runs = ((a.h + 1) / 2 + V - 1) / V;   // V pairs each
  int lanes = 1;
  while (lanes < 32 && lanes < runs) lanes *= 2;
  const int e = (runs + lanes - 1) / lanes;
  if (e <= 1) return launch_tiles<T, V, PAIRS, 1, P>(a, lanes, rows, s);
  if constexpr (V <= 4)
    if (e <= 2) return launch_tiles<T, V, PAIRS, 2, P>(a, lanes, rows, s);
  if constexpr (V <= 2)
    if (e <= 4) return launch_tiles<T, V, PAIRS, 4, P>(a, lanes, rows, s);
  if constexpr (V <= 1)
    if (e <= 8) return launch_tiles<T, V, PAIRS, 8, P>(a, lanes, rows, s);
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

template <typename T, int V, Pass P>
cudaError_t launch_pairs(const HeadArgs& a, long long* rows, cudaStream_t s) {
  return a.pairs == PAIRS_HALVES ? launch_runs<T, V, PAIRS_HALVES, P>(a, rows, s)
                                 : launch_runs<T, V, PAIRS_INTERLEAVED, P>(a, rows, s);
}

template <Pass P>
cudaError_t launch(int dt, const HeadArgs& a, long long* rows, cudaStream_t s) {
  if (dt == DT_BF16) {
    if (fits(a, 8, 2)) return launch_pairs<bf16, 8, P>(a, rows, s);
    if (fits(a, 4, 2)) return launch_pairs<bf16, 4, P>(a, rows, s);
    if (fits(a, 2, 2)) return launch_pairs<bf16, 2, P>(a, rows, s);
    return launch_pairs<bf16, 1, P>(a, rows, s);
  }
  if (fits(a, 4, 4)) return launch_pairs<float, 4, P>(a, rows, s);
  if (fits(a, 2, 4)) return launch_pairs<float, 2, P>(a, rows, s);
  return launch_pairs<float, 1, P>(a, rows, s);
}

}  // namespace

long long head_bwd_max_rows(int B, int N) {
  return std::min<long long>((long long)B * N, 148LL * bwd_blocks(1, 1));
}

cudaError_t head_fwd(int dt, const HeadArgs& a, cudaStream_t s) { return launch<FWD>(dt, a, nullptr, s); }
cudaError_t head_bwd(int dt, const HeadArgs& a, long long* rows, cudaStream_t s) {
  return a.norm == TTT_NORM_NONE ? launch<BWD_PLAIN>(dt, a, rows, s) : launch<BWD_NORMED>(dt, a, rows, s);
}

}  // namespace ttt
