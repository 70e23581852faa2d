// groupnorm.cu - GroupNorm of channels-last images with a fused activation, forward and backward.
//
// x is [N, S, C]: N images of S positions (the flattened picture or video), C channels in G groups
// of P = C / G consecutive channels. The statistics of a group run over its S * P values:
//   mu = mean(x), var = mean((x - mu)^2) (biased), s = 1 / sqrt(var + eps),
//   xhat = (x - mu) s,  z = xhat w_c + b_c,  y = act(z).
// Backward, with g = dy * act'(z) and the channel sums A_c = sum g, B_c = sum g xhat of an image:
//   dx = s (g w_c - m1 - xhat m2),  m1 = sum_{c in group} w_c A_c / (S P),  m2 = sum w_c B_c / (S P)
//   dw_c = sum over images of B_c,  db_c = sum over images of A_c.
// Unlike the row norms a group's values are not contiguous: a position's group is a run of P channels,
// P * sizeof(T) bytes (20 to 128 in practice), and positions lie C channels apart.
//
// Two passes over the image: a pass over slabs of positions that reduces every channel of the slab
// (gn_stats_kernel, gn_bwd_sums_kernel), a small kernel that joins the slabs and the channels of a
// group in a fixed order, and an elementwise pass. A thread keeps one 16-byte vector of channels and
// walks down the positions, so its per-channel sums and parameters stay in registers and every warp
// access covers whole runs of a row. The forward's sums are (mean, centred sum of squares) per
// channel, batch by batch with Chan's update: no E[x^2] - E[x]^2 cancellation.
#include "gn_common.cuh"
#include "gn_host.h"

namespace gn {
namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;  // positions a thread has in flight

struct GnShape {
  int64_t S;       // positions of an image
  int C, P, G;     // channels, channels per group, groups
  int tiles, tv;   // column tiles of a row and 16-byte vectors per tile
  int rl;          // positions a block covers at once (kThreads / tv)
  int chunks;      // slabs of an image
  int64_t rows;    // positions of a slab (the last one may be shorter)
};

// 16-byte vector `v` of a row; elements at and past C read as 0
template <typename T>
__device__ __forceinline__ void load_vec(const T* row, int v, int C, bool whole, float (&f)[Vec<T>::N]) {
  constexpr int E = Vec<T>::N;
  if (whole) {
    Vec<T>::unpack(*reinterpret_cast<const uint4*>(row + v * E), f);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = v * E + e < C ? Vec<T>::load1(row + v * E + e) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store_vec(T* row, int v, int C, bool whole, const float (&f)[Vec<T>::N]) {
  constexpr int E = Vec<T>::N;
  if (whole) {
    st_stream(row + v * E, Vec<T>::pack(f));
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (v * E + e < C) Vec<T>::store1(row + v * E + e, f[e]);
  }
}

// where a thread of the slab kernels works
struct Place {
  int n, chunk, v, lane_row;
  bool active, whole;
  int64_t r0, r1;
  template <int E>
  __device__ __forceinline__ static Place make(const GnShape& g) {
    Place p;
    const int tile = blockIdx.x % g.tiles;
    const int nc = blockIdx.x / g.tiles;
    p.chunk = nc % g.chunks;
    p.n = nc / g.chunks;
    const int i = threadIdx.x % g.tv;
    p.lane_row = threadIdx.x / g.tv;
    p.v = tile * g.tv + i;
    const int nvec = (g.C + E - 1) / E;
    p.active = p.lane_row < g.rl && p.v < nvec;
    p.whole = (p.v + 1) * E <= g.C;
    p.r0 = (int64_t)p.chunk * g.rows;
    p.r1 = p.r0 + g.rows < g.S ? p.r0 + g.rows : g.S;
    return p;
  }
};

// ---------------------------------------------------------------- forward: slab statistics
// part[n][chunk][c] = (mean, centred sum of squares) of channel c over the slab.
template <typename T>
__global__ void __launch_bounds__(kThreads) gn_stats_kernel(const T* __restrict__ x, int64_t ldx, GnShape g,
                                                            float2* __restrict__ part) {
  constexpr int E = Vec<T>::N;
  __shared__ float sm_mean[kThreads * E];
  __shared__ float sm_m2[kThreads * E];
  __shared__ float sm_cnt[kThreads];
  const Place p = Place::make<E>(g);
  float mean[E], m2[E], cnt = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) mean[e] = 0.0f, m2[e] = 0.0f;
  if (p.active) {
    const T* img = x + (int64_t)p.n * g.S * ldx;
    for (int64_t r = p.r0 + p.lane_row; r < p.r1; r += (int64_t)g.rl * kBatch) {
      float f[kBatch][E];
      int k = 0;
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int64_t rr = r + (int64_t)j * g.rl;
        if (rr < p.r1) {
          load_vec<T>(img + rr * ldx, p.v, g.C, p.whole, f[j]);
          k = j + 1;
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) f[j][e] = 0.0f;
        }
      }
      const float nk = (float)k, inv = 1.0f / nk, tot = cnt + nk;
      const float fr = nk / tot, w = cnt * fr;  // Chan: weights of the batch and of the square
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float t = 0.0f, q = 0.0f;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) t += f[j][e];
        const float bm = t * inv;
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const float d = j < k ? f[j][e] - bm : 0.0f;
          q = fmaf(d, d, q);
        }
        const float dl = bm - mean[e];
        mean[e] = fmaf(dl, fr, mean[e]);
        m2[e] += fmaf(dl * dl, w, q);
      }
      cnt = tot;
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_mean[threadIdx.x * E + e] = mean[e], sm_m2[threadIdx.x * E + e] = m2[e];
  sm_cnt[threadIdx.x] = cnt;
  __syncthreads();
  // channel j of the tile: merge the rl threads that hold it, in order
  for (int j = threadIdx.x; j < g.tv * E; j += kThreads) {
    const int c = (blockIdx.x % g.tiles) * g.tv * E + j;
    if (c >= g.C) continue;
    float mu = 0.0f, q = 0.0f, n = 0.0f;
    for (int k = 0; k < g.rl; ++k) {
      const int t = k * g.tv + j / E;
      const float nk = sm_cnt[t];
      if (nk == 0.0f) continue;
      const float tot = n + nk, dl = sm_mean[t * E + j % E] - mu;
      mu = fmaf(dl, nk / tot, mu);
      q += fmaf(dl * dl, n * (nk / tot), sm_m2[t * E + j % E]);
      n = tot;
    }
    part[((int64_t)p.n * g.chunks + p.chunk) * g.C + c] = make_float2(mu, q);
  }
}

__device__ __forceinline__ float block_sum(float v, float* red) {  // kThreads threads, fixed order
  v = group_sum<32>(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) t += red[i];
  return t;
}

// one block per (image, group): joins the slabs and the group's channels
__global__ void __launch_bounds__(kThreads) gn_stats_join_kernel(const float2* __restrict__ part, GnShape g, float eps,
                                                                 float2* __restrict__ stat, float* __restrict__ mean,
                                                                 float* __restrict__ rstd) {
  __shared__ float red[kThreads / 32];
  const int n = blockIdx.x / g.G, gr = blockIdx.x % g.G;
  const float2* base = part + (int64_t)n * g.chunks * g.C + (int64_t)gr * g.P;
  const int64_t items = (int64_t)g.chunks * g.P;
  auto count = [&](int64_t i) {
    const int64_t r0 = (i / g.P) * g.rows;
    return (float)((r0 + g.rows < g.S ? r0 + g.rows : g.S) - r0);
  };
  float t = 0.0f;
  for (int64_t i = threadIdx.x; i < items; i += kThreads) t = fmaf(count(i), base[(i / g.P) * g.C + i % g.P].x, t);
  const float total = (float)((double)g.S * g.P);
  const float mu = block_sum(t, red) / total;
  float q = 0.0f;
  for (int64_t i = threadIdx.x; i < items; i += kThreads) {
    const float2 v = base[(i / g.P) * g.C + i % g.P];
    const float d = v.x - mu;
    q += fmaf(count(i) * d, d, v.y);
  }
  const float var = block_sum(q, red) / total;
  if (threadIdx.x == 0) {
    const float s = 1.0f / sqrtf(var + eps);
    stat[blockIdx.x] = make_float2(mu, s);
    if (mean) mean[blockIdx.x] = mu;
    if (rstd) rstd[blockIdx.x] = s;
  }
}

// ---------------------------------------------------------------- forward: the elementwise pass
template <typename T, int EPI>
__global__ void __launch_bounds__(kThreads) gn_apply_kernel(const T* x, int64_t ldx, const T* __restrict__ w,
                                                            const T* __restrict__ b, const float2* __restrict__ stat,
                                                            GnShape g, T* y, int64_t ldy) {
  constexpr int E = Vec<T>::N;
  constexpr bool FAST = fast_math_for<T>();
  const Place p = Place::make<E>(g);
  if (!p.active) return;
  float mu[E], a[E], sh[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = p.v * E + e;
    if (c < g.C) {
      const float2 s = stat[(int64_t)p.n * g.G + c / g.P];
      mu[e] = s.x;
      a[e] = s.y * ld_param(w, c, 1.0f);
      sh[e] = ld_param(b, c, 0.0f);
    } else {
      mu[e] = a[e] = sh[e] = 0.0f;
    }
  }
  const int64_t img = (int64_t)p.n * g.S;
  for (int64_t r = p.r0 + p.lane_row; r < p.r1; r += g.rl) {
    float f[E];
    load_vec<T>(x + (img + r) * ldx, p.v, g.C, p.whole, f);
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = epi_fwd<EPI, FAST>(fmaf(f[e] - mu[e], a[e], sh[e]));
    store_vec<T>(y + (img + r) * ldy, p.v, g.C, p.whole, f);
  }
}

// ---------------------------------------------------------------- backward
// part[n][chunk][c] = (A_c, B_c) = (sum g, sum g xhat) of channel c over the slab
template <typename T, int EPI>
__global__ void __launch_bounds__(kThreads) gn_bwd_sums_kernel(const T* __restrict__ x, int64_t ldx,
                                                               const T* __restrict__ dy, int64_t lddy,
                                                               const T* __restrict__ w, const T* __restrict__ b,
                                                               const float* __restrict__ mean,
                                                               const float* __restrict__ rstd, GnShape g,
                                                               float2* __restrict__ part) {
  constexpr int E = Vec<T>::N;
  constexpr bool FAST = fast_math_for<T>();
  __shared__ float sm_a[kThreads * E];
  __shared__ float sm_b[kThreads * E];
  const Place p = Place::make<E>(g);
  float A[E], B[E];
#pragma unroll
  for (int e = 0; e < E; ++e) A[e] = 0.0f, B[e] = 0.0f;
  if (p.active) {
    float mu[E], s[E], wf[E], bf[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = p.v * E + e;
      const bool in = c < g.C;
      mu[e] = in ? mean[(int64_t)p.n * g.G + c / g.P] : 0.0f;
      s[e] = in ? rstd[(int64_t)p.n * g.G + c / g.P] : 0.0f;
      wf[e] = in ? ld_param(w, c, 1.0f) : 0.0f;
      bf[e] = in ? ld_param(b, c, 0.0f) : 0.0f;
    }
    const int64_t img = (int64_t)p.n * g.S;
    for (int64_t r = p.r0 + p.lane_row; r < p.r1; r += g.rl) {
      float f[E], d[E];
      load_vec<T>(x + (img + r) * ldx, p.v, g.C, p.whole, f);
      load_vec<T>(dy + (img + r) * lddy, p.v, g.C, p.whole, d);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float xh = (f[e] - mu[e]) * s[e];
        const float gg = d[e] * epi_grad<EPI, FAST>(fmaf(xh, wf[e], bf[e]));
        A[e] += gg;
        B[e] = fmaf(gg, xh, B[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) sm_a[threadIdx.x * E + e] = A[e], sm_b[threadIdx.x * E + e] = B[e];
  __syncthreads();
  for (int j = threadIdx.x; j < g.tv * E; j += kThreads) {
    const int c = (blockIdx.x % g.tiles) * g.tv * E + j;
    if (c >= g.C) continue;
    float ta = 0.0f, tb = 0.0f;
    for (int k = 0; k < g.rl; ++k) {
      ta += sm_a[k * g.tv * E + j];
      tb += sm_b[k * g.tv * E + j];
    }
    part[((int64_t)p.n * g.chunks + p.chunk) * g.C + c] = make_float2(ta, tb);
  }
}

// one block per (image, group): chan[n][0..C) = B_c, chan[n][C..2C) = A_c (the column sums over the
// images are then dw and db), stat[n][group] = (m1, m2)
template <typename T>
__global__ void __launch_bounds__(kThreads) gn_bwd_join_kernel(const float2* __restrict__ part,
                                                               const T* __restrict__ w, GnShape g,
                                                               float* __restrict__ chan, float2* __restrict__ stat) {
  __shared__ float red[kThreads / 32];
  const int n = blockIdx.x / g.G, gr = blockIdx.x % g.G;
  float m1 = 0.0f, m2 = 0.0f;
  for (int j = threadIdx.x; j < g.P; j += kThreads) {
    const int c = gr * g.P + j;
    float ta = 0.0f, tb = 0.0f;
    for (int k = 0; k < g.chunks; ++k) {
      const float2 v = part[((int64_t)n * g.chunks + k) * g.C + c];
      ta += v.x;
      tb += v.y;
    }
    chan[(int64_t)n * 2 * g.C + c] = tb;
    chan[(int64_t)n * 2 * g.C + g.C + c] = ta;
    const float wc = ld_param(w, c, 1.0f);
    m1 = fmaf(wc, ta, m1);
    m2 = fmaf(wc, tb, m2);
  }
  const float inv = 1.0f / (float)((double)g.S * g.P);
  m1 = block_sum(m1, red) * inv;
  m2 = block_sum(m2, red) * inv;
  if (threadIdx.x == 0) stat[blockIdx.x] = make_float2(m1, m2);
}

template <typename T, int EPI>
__global__ void __launch_bounds__(kThreads) gn_bwd_apply_kernel(const T* __restrict__ x, int64_t ldx, const T* dy,
                                                                int64_t lddy, const T* __restrict__ w,
                                                                const T* __restrict__ b, const float* __restrict__ mean,
                                                                const float* __restrict__ rstd,
                                                                const float2* __restrict__ stat, GnShape g, T* dx,
                                                                int64_t lddx) {
  constexpr int E = Vec<T>::N;
  constexpr bool FAST = fast_math_for<T>();
  const Place p = Place::make<E>(g);
  if (!p.active) return;
  float mu[E], s[E], wf[E], bf[E], m1[E], m2[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = p.v * E + e;
    const bool in = c < g.C;
    const int64_t gi = (int64_t)p.n * g.G + (in ? c / g.P : 0);
    mu[e] = mean[gi];
    s[e] = rstd[gi];
    m1[e] = stat[gi].x;
    m2[e] = stat[gi].y;
    wf[e] = in ? ld_param(w, c, 1.0f) : 0.0f;
    bf[e] = in ? ld_param(b, c, 0.0f) : 0.0f;
  }
  const int64_t img = (int64_t)p.n * g.S;
  for (int64_t r = p.r0 + p.lane_row; r < p.r1; r += g.rl) {
    float f[E], d[E];
    load_vec<T>(x + (img + r) * ldx, p.v, g.C, p.whole, f);
    load_vec<T>(dy + (img + r) * lddy, p.v, g.C, p.whole, d);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float xh = (f[e] - mu[e]) * s[e];
      const float gg = d[e] * epi_grad<EPI, FAST>(fmaf(xh, wf[e], bf[e]));
      f[e] = s[e] * (fmaf(gg, wf[e], -m1[e]) - xh * m2[e]);
    }
    store_vec<T>(dx + (img + r) * lddx, p.v, g.C, p.whole, f);
  }
}

// ---------------------------------------------------------------- host side

bool shape_ok(int64_t N, int64_t S, int64_t C, int64_t G) {
  return N >= 0 && S >= 0 && C > 0 && G > 0 && C % G == 0 && C <= (1 << 20) && N <= (1 << 20) && S <= INT64_MAX / 4 / C;
}

GnShape plan(int64_t N, int64_t S, int64_t C, int64_t G, int es) {
  GnShape g{};
  g.S = S;
  g.C = (int)C;
  g.G = (int)G;
  g.P = (int)(C / G);
  const int E = 16 / es;
  const int nvec = (int)((C + E - 1) / E);
  g.tiles = (nvec + 63) / 64;  // at most 64 vectors a tile: at least four positions a block
  g.tv = (nvec + g.tiles - 1) / g.tiles;
  g.rl = kThreads / g.tv;
  const int sms = sm_count() > 0 ? sm_count() : 148;
  // about eight blocks per SM over the whole tensor, a slab no shorter than one batch per thread
  int64_t chunks = (8 * (int64_t)sms + N * g.tiles - 1) / (N * g.tiles);
  const int64_t most = (S + (int64_t)g.rl * kBatch - 1) / ((int64_t)g.rl * kBatch);
  if (chunks > most) chunks = most;
  if (chunks < 1) chunks = 1;
  g.rows = (S + chunks - 1) / chunks;
  g.chunks = (int)((S + g.rows - 1) / g.rows);
  return g;
}

size_t up16(size_t v) { return (v + 15) / 16 * 16; }

template <typename T>
void* pick_apply(int epi) {
  return epi == GN_EPI_GELU_TANH ? (void*)gn_apply_kernel<T, EPI_GELU_TANH>
         : epi == GN_EPI_SILU    ? (void*)gn_apply_kernel<T, EPI_SILU>
                                 : (void*)gn_apply_kernel<T, EPI_NONE>;
}
template <typename T>
void* pick_sums(int epi) {
  return epi == GN_EPI_GELU_TANH ? (void*)gn_bwd_sums_kernel<T, EPI_GELU_TANH>
         : epi == GN_EPI_SILU    ? (void*)gn_bwd_sums_kernel<T, EPI_SILU>
                                 : (void*)gn_bwd_sums_kernel<T, EPI_NONE>;
}
template <typename T>
void* pick_bwd(int epi) {
  return epi == GN_EPI_GELU_TANH ? (void*)gn_bwd_apply_kernel<T, EPI_GELU_TANH>
         : epi == GN_EPI_SILU    ? (void*)gn_bwd_apply_kernel<T, EPI_SILU>
                                 : (void*)gn_bwd_apply_kernel<T, EPI_NONE>;
}

gn_status launch(void* kern, int64_t blocks, void** args, cudaStream_t s) {
  if (blocks > INT32_MAX) return GN_ERR_SHAPE;
  if (!kernel_attrs(kern, 0)) return GN_ERR_CUDA;
  if (cudaLaunchKernel(kern, dim3((unsigned)blocks), dim3(kThreads), args, 0, s) != cudaSuccess) return GN_ERR_CUDA;
  count_launches(1);
  return launch_status();
}

}  // namespace
}  // namespace gn

using namespace gn;

extern "C" size_t gn_groupnorm_fwd_workspace(int64_t N, int64_t S, int64_t C, int64_t G, gn_dtype dt) {
  if (!dt_ok(dt) || !shape_ok(N, S, C, G) || N == 0 || S == 0) return 0;
  const GnShape g = plan(N, S, C, G, (int)dt_size(dt));
  return up16((size_t)N * g.G * 8) + (size_t)N * g.chunks * g.C * 8;
}

extern "C" gn_status gn_groupnorm_fwd(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
                                      void* ws, size_t ws_bytes, int64_t N, int64_t S, int64_t C, int64_t G,
                                      int64_t ld_x, int64_t ld_y, float eps, gn_epilogue epi, gn_dtype dt,
                                      void* stream) {
  if (!dt_ok(dt) || !epi_ok(epi)) return GN_ERR_DTYPE;
  if (!shape_ok(N, S, C, G) || ld_x < C || ld_y < C) return GN_ERR_SHAPE;
  if (N == 0 || S == 0) return GN_OK;
  if (!x || !y) return GN_ERR_NULL;
  const size_t es = dt_size(dt);
  if (!aligned16(x) || !aligned16(y) || ld_x * es % 16 || ld_y * es % 16) return GN_ERR_ALIGN;
  if (!ws || ws_bytes < gn_groupnorm_fwd_workspace(N, S, C, G, dt)) return GN_ERR_WORKSPACE;
  if (!aligned16(ws)) return GN_ERR_ALIGN;
  cudaStream_t s = (cudaStream_t)stream;
  GnShape g = plan(N, S, C, G, (int)es);
  float2* stat = static_cast<float2*>(ws);
  float2* part = reinterpret_cast<float2*>(static_cast<char*>(ws) + up16((size_t)N * g.G * 8));
  const int64_t blocks = N * g.chunks * g.tiles;
  {
    void* args[] = {&x, &ld_x, &g, &part};
    const gn_status st =
        launch(dt == GN_BF16 ? (void*)gn_stats_kernel<__nv_bfloat16> : (void*)gn_stats_kernel<float>, blocks, args, s);
    if (st != GN_OK) return st;
  }
  {
    void* args[] = {&part, &g, &eps, &stat, &mean, &rstd};
    const gn_status st = launch((void*)gn_stats_join_kernel, N * g.G, args, s);
    if (st != GN_OK) return st;
  }
  void* args[] = {&x, &ld_x, &w, &b, &stat, &g, &y, &ld_y};
  return launch(dt == GN_BF16 ? pick_apply<__nv_bfloat16>(epi) : pick_apply<float>(epi), blocks, args, s);
}

extern "C" size_t gn_groupnorm_bwd_workspace(int64_t N, int64_t S, int64_t C, int64_t G, gn_dtype dt) {
  if (!dt_ok(dt) || !shape_ok(N, S, C, G) || N == 0 || S == 0) return 0;
  const GnShape g = plan(N, S, C, G, (int)dt_size(dt));
  return up16((size_t)N * g.G * 8) + (size_t)N * g.C * 8 + (size_t)N * g.chunks * g.C * 8;
}

extern "C" gn_status gn_groupnorm_bwd(const void* x, const void* w, const void* b, const float* mean,
                                      const float* rstd, const void* dy, void* dx, float* dw, float* db, void* ws,
                                      size_t ws_bytes, int64_t N, int64_t S, int64_t C, int64_t G, int64_t ld_x,
                                      int64_t ld_dy, int64_t ld_dx, gn_epilogue epi, gn_dtype dt, void* stream) {
  if (!dt_ok(dt) || !epi_ok(epi)) return GN_ERR_DTYPE;
  if (!shape_ok(N, S, C, G) || ld_x < C || ld_dy < C || ld_dx < C) return GN_ERR_SHAPE;
  cudaStream_t s = (cudaStream_t)stream;
  if (N == 0 || S == 0) {
    if (dw && cudaMemsetAsync(dw, 0, (size_t)C * 4, s) != cudaSuccess) return GN_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, (size_t)C * 4, s) != cudaSuccess) return GN_ERR_CUDA;
    return GN_OK;
  }
  if (!x || !mean || !rstd || !dy || !dx) return GN_ERR_NULL;
  const size_t es = dt_size(dt);
  if (!aligned16(x) || !aligned16(dy) || !aligned16(dx) || ld_x * es % 16 || ld_dy * es % 16 || ld_dx * es % 16)
    return GN_ERR_ALIGN;
  if (!ws || ws_bytes < gn_groupnorm_bwd_workspace(N, S, C, G, dt)) return GN_ERR_WORKSPACE;
  if (!aligned16(ws)) return GN_ERR_ALIGN;
  GnShape g = plan(N, S, C, G, (int)es);
  float2* stat = static_cast<float2*>(ws);
  float* chan = reinterpret_cast<float*>(static_cast<char*>(ws) + up16((size_t)N * g.G * 8));
  float2* part = reinterpret_cast<float2*>(chan + (size_t)N * g.C * 2);
  const int64_t blocks = N * g.chunks * g.tiles;
  gn_status st;
  {
    void* args[] = {&x, &ld_x, &dy, &ld_dy, &w, &b, &mean, &rstd, &g, &part};
    st = launch(dt == GN_BF16 ? pick_sums<__nv_bfloat16>(epi) : pick_sums<float>(epi), blocks, args, s);
    if (st != GN_OK) return st;
  }
  {
    void* args[] = {&part, &w, &g, &chan, &stat};
    st = launch(dt == GN_BF16 ? (void*)gn_bwd_join_kernel<__nv_bfloat16> : (void*)gn_bwd_join_kernel<float>, N * g.G,
                args, s);
    if (st != GN_OK) return st;
  }
  {
    void* args[] = {&x, &ld_x, &dy, &ld_dy, &w, &b, &mean, &rstd, &stat, &g, &dx, &ld_dx};
    st = launch(dt == GN_BF16 ? pick_bwd<__nv_bfloat16>(epi) : pick_bwd<float>(epi), blocks, args, s);
    if (st != GN_OK) return st;
  }
  return launch_colsum(chan, N, 2 * C, C, dw, db, s);
}
