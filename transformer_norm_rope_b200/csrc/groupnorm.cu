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
// Images whose groups fit on chip are read once (the resident kernels, further down). Longer ones take
// two passes: a pass over slabs of positions that reduces every channel of the slab
// (gn_stats_kernel, gn_bwd_sums_kernel), a small kernel that joins the slabs in a fixed order (and
// in the backward the channels of a group), and an elementwise pass. A thread keeps one 16-byte vector of channels and
// walks down the positions, so its per-channel sums and parameters stay in registers and every warp
// access covers whole runs of a row. The forward's sums are (mean, centred sum of squares) per
// channel, taken around a value of the slab and joined as deviations from a mean: no E[x^2] - E[x]^2 cancellation.
#include <type_traits>

#include "act_pairs.cuh"
#include "gn_common.cuh"
#include "gn_host.h"

namespace gn {
namespace {

constexpr int kThreads = 256;
// A thread's next positions are on their way, by asynchronous copies to its own places in shared memory, while
// it works on one: kRing 16-byte vectors, in the backward half of them of x and half of dy. (4 x 65536 x 512 bf16:
// 158 us forward, 224 backward; double-buffered in registers 192 and 298.)
constexpr int kRing = 8;
// blocks on an SM, by registers: a thread of fp32 images has half the channels of a bf16 one
template <typename T>
constexpr int kFwdPerSm = sizeof(T) == 4 ? 4 : 3;
template <typename T>
constexpr int kBwdPerSm = sizeof(T) == 4 ? 3 : 2;
constexpr int kBatch = 4;  // slabs are whole multiples of this many positions a thread

// `bytes` of a vector are read, the rest of its 16 is zero: the last vector of a row may not be whole (read by
// plain loads, one position after the other, such a vector made 2 x 30902 x 171 wait: forward 43 us against 26,
// backward 60 against 36)
__device__ __forceinline__ void copy16(uint4* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// f(vector) for n vectors from src on, `step` elements apart (n >= 1; the thread's places: ring[k * kThreads])
template <typename T, class F>
__device__ __forceinline__ void walk(uint4* ring, const T* src, int64_t step, int bytes, int n, F f) {
#pragma unroll
  for (int k = 0; k < kRing; ++k) {
    if (k < n) copy16(ring + k * kThreads, src + k * step, bytes);
    copy_commit();
  }
  src += kRing * step;
  int s = 0;
  for (int k = 0; k < n; ++k, src += step) {
    copy_wait<kRing - 1>();
    const uint4 u = ring[s * kThreads];
    if (k + kRing < n) copy16(ring + s * kThreads, src, bytes);
    copy_commit();
    s = s + 1 == kRing ? 0 : s + 1;
    f(u);
  }
}

// the same for two tensors
template <typename T, class F>
__device__ __forceinline__ void walk2(uint4* ring, const T* p, int64_t sp, const T* q, int64_t sq, int bytes, int n, F f) {
  constexpr int D = kRing / 2;
#pragma unroll
  for (int k = 0; k < D; ++k) {
    if (k < n) {
      copy16(ring + 2 * k * kThreads, p + k * sp, bytes);
      copy16(ring + (2 * k + 1) * kThreads, q + k * sq, bytes);
    }
    copy_commit();
  }
  p += D * sp;
  q += D * sq;
  int s = 0;
  for (int k = 0; k < n; ++k, p += sp, q += sq) {
    copy_wait<D - 1>();
    const uint4 u = ring[2 * s * kThreads], v = ring[(2 * s + 1) * kThreads];
    if (k + D < n) {
      copy16(ring + 2 * s * kThreads, p, bytes);
      copy16(ring + (2 * s + 1) * kThreads, q, bytes);
    }
    copy_commit();
    s = s + 1 == D ? 0 : s + 1;
    f(u, v);
  }
}

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
  int bytes;  // of the vector within the row
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
    p.bytes = p.whole ? 16 : (g.C - p.v * E) * (16 / E);
    p.r0 = (int64_t)p.chunk * g.rows;
    p.r1 = p.r0 + g.rows < g.S ? p.r0 + g.rows : g.S;
    return p;
  }
};

// this thread's vector of a row, or what of it lies within the row
template <typename T>
__device__ __forceinline__ void store_packed(T* row, const Place& p, int C, const uint4& u) {
  if (p.whole) {
    st_stream(row + p.v * Vec<T>::N, u);
  } else {
    float f[Vec<T>::N];
    Vec<T>::unpack(u, f);
    store_vec<T>(row, p.v, C, false, f);
  }
}

// lanes of a warp that can share one of n columns, a power of two; the sum over them (in every lane)
__device__ __forceinline__ int spare_lanes(int n) {
  int l = 1;
  while (l < 32 && l * 2 * n <= kThreads) l *= 2;
  return l;
}
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  for (int o = lanes / 2; o > 0; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// ---------------------------------------------------------------- forward: slab statistics
// part[n][chunk][slot] = (mean, centred sum of squares) over the slab of the channels that a group has in a
// column tile; slot = tile + group (neighbouring tiles share at most one group).
template <typename T>
__global__ void __launch_bounds__(kThreads, kFwdPerSm<T>) gn_stats_kernel(const T* __restrict__ x, int64_t ldx, GnShape g,
                                                            float2* __restrict__ part) {
  constexpr int E = Vec<T>::N, H = E / 2;
  __shared__ __align__(16) uint4 ring[kRing * kThreads];
  float* sm_mean = reinterpret_cast<float*>(ring);  // the copies have all been read by then
  float* sm_m2 = sm_mean + kThreads * E;
  float* sm_cnt = sm_m2 + kThreads * E;
  static_assert(sizeof(uint4) * kRing * kThreads >= 4 * (kThreads * (2 * E + 1) + 2 * 64 * E), "the sums fit the ring");
  const Place p = Place::make<E>(g);
  // sums of x - K and (x - K)^2 per channel, K the thread's first value: mean = K + s1 / n, squares
  // = s2 - s1^2 / n, which loses at most four bits while s1^2 / n <= 16 squares; where the first value is
  // further off than that, a second walk takes them around the mean
  float2 shift[H], s1[H], s2[H];
  float cnt = 0.0f;
  if (p.active && p.r0 + p.lane_row < p.r1) {
    const T* first = x + ((int64_t)p.n * g.S + p.r0 + p.lane_row) * ldx;
    const int64_t step = (int64_t)g.rl * ldx;
    const int64_t positions = (p.r1 - p.r0 - p.lane_row + g.rl - 1) / g.rl;
    cnt = (float)positions;
    float f0[E];
    load_vec<T>(first, p.v, g.C, p.whole, f0);
#pragma unroll
    for (int e = 0; e < H; ++e) shift[e] = make_float2(-f0[2 * e], -f0[2 * e + 1]);
    auto add = [&](const uint4& u) {
      float2 f[H];
      unpack2<T>(u, f);
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float2 d = add2(f[e], shift[e]);
        s1[e] = add2(s1[e], d);
        s2[e] = fma2(d, d, s2[e]);
      }
    };
    for (int round = 0; round < 2; ++round) {
#pragma unroll
      for (int e = 0; e < H; ++e) s1[e] = s2[e] = make_float2(0.0f, 0.0f);
      walk<T>(ring + threadIdx.x, first + p.v * E, step, p.bytes, (int)positions, add);
      bool again = false;
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float ax = s1[e].x * s1[e].x / cnt, ay = s1[e].y * s1[e].y / cnt;
        again |= ax > 16.0f * (s2[e].x - ax) || ay > 16.0f * (s2[e].y - ay);
      }
      if (!again || round) break;
#pragma unroll
      for (int e = 0; e < H; ++e) shift[e] = make_float2(shift[e].x - s1[e].x / cnt, shift[e].y - s1[e].y / cnt);
    }
  }
  float mean[E], m2[E];
#pragma unroll
  for (int e = 0; e < H; ++e) {
    const bool any = cnt > 0.0f;
    const float2 d = any ? make_float2(s1[e].x / cnt, s1[e].y / cnt) : make_float2(0.0f, 0.0f);
    mean[2 * e] = any ? d.x - shift[e].x : 0.0f;
    mean[2 * e + 1] = any ? d.y - shift[e].y : 0.0f;
    // (a comparison that lets NaN through)
    const float qx = any ? fmaf(-s1[e].x, d.x, s2[e].x) : 0.0f, qy = any ? fmaf(-s1[e].y, d.y, s2[e].y) : 0.0f;
    m2[2 * e] = qx < 0.0f ? 0.0f : qx;
    m2[2 * e + 1] = qy < 0.0f ? 0.0f : qy;
  }
  pdl_launch_dependents();
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e) sm_mean[threadIdx.x * E + e] = mean[e], sm_m2[threadIdx.x * E + e] = m2[e];
  sm_cnt[threadIdx.x] = cnt;
  __syncthreads();
  // channel j of the tile: as many lanes as there are to spare join the rl threads that hold it, as deviations from the first
  // one's mean (always there): mean = m0 + d, d = sum n_k (m_k - m0) / n; squares = sum of theirs + n_k (m_k - m0 - d)^2.
  // One rounding of the mean's size is left. (Merged one after the other, every step rounded the mean and the squares:
  // with 256 threads a channel the means of 15 x 1017 x 3 fp32 were off by 2.9e-7 of them, 6.6e-8 by an elementary sum.)
  const float rows = (float)(p.r1 - p.r0);
  float* ch_mean = sm_cnt + kThreads;
  float* ch_m2 = ch_mean + g.tv * E;
  const int tile = blockIdx.x % g.tiles, c_lo = tile * g.tv * E;
  const int nch = g.C - c_lo < g.tv * E ? g.C - c_lo : g.tv * E;
  const int share = spare_lanes(g.tv * E);
  for (int j0 = 0; j0 < nch; j0 += kThreads / share) {  // the same number of turns for every lane
    const int j = j0 + threadIdx.x / share, jc = j < nch ? j : nch - 1;
    const int first = (int)threadIdx.x & (share - 1);
    const float *mk = sm_mean + jc, *qk = sm_m2 + jc, *ck = sm_cnt + jc / E;  // thread k g.tv + jc / E, its value jc % E
    const float m0 = *mk;
    float d = 0.0f, q = 0.0f;
    for (int k = first; k < g.rl; k += share) {
      const float nk = ck[k * g.tv];
      if (nk > 0.0f) d = fmaf(nk, mk[k * g.tv * E] - m0, d);
    }
    d = lanes_sum(d, share) / rows;
    for (int k = first; k < g.rl; k += share) {
      const float nk = ck[k * g.tv], dl = mk[k * g.tv * E] - m0 - d;
      if (nk > 0.0f) q += fmaf(nk * dl, dl, qk[k * g.tv * E]);
    }
    q = lanes_sum(q, share);
    if (first == 0 && j < nch) ch_mean[j] = m0 + d, ch_m2[j] = q;
  }
  __syncthreads();
  // the tile's part of each group: as many neighbouring lanes as it has channels, a warp at most
  const int g_lo = c_lo / g.P, groups = (c_lo + nch - 1) / g.P - g_lo + 1;
  int team = 32;
  while (team > 1 && team / 2 >= g.P) team /= 2;
  const int lane = threadIdx.x & (team - 1), per = kThreads / team;
  auto team_sum = [&](float v) {
    for (int d = team / 2; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
    return v;
  };
  for (int i = 0; i < groups; i += per) {  // the same number of turns for every lane
    const int gi = g_lo + i + threadIdx.x / team;
    int a = gi * g.P - c_lo, b = a + g.P;
    a = a > 0 ? a : 0;
    b = b < nch ? b : nch;
    float t = 0.0f, q = 0.0f;
    for (int j = a + lane; j < b; j += team) t += ch_mean[j];
    const float mu = team_sum(t) / (float)(b - a);
    for (int j = a + lane; j < b; j += team) q += fmaf(rows * (ch_mean[j] - mu), ch_mean[j] - mu, ch_m2[j]);
    q = team_sum(q);
    if (lane == 0 && b > a)
      part[((int64_t)p.n * g.chunks + p.chunk) * (g.G + g.tiles - 1) + tile + gi] = make_float2(mu, q);
  }
}

constexpr int kJoin = 1024, kJoinFwd = 256;

template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float* red) {  // fixed order
  v = group_sum<32>(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < THREADS / 32; ++i) t += red[i];
  return t;
}

// The forward joins the channels of a group already in the slabs' blocks: one part a slab is left of a group, where
// a part a channel made the join long for wide groups and many images (3 x 36992 x 584 with one group 106 -> 93 us,
// 32 x 4096 x 512 with 32 groups 100 -> 86; images of a few groups' channels 0 to 1 us slower). The backward keeps
// its parts by channel: dw and db need them.
// one block per (image, group): joins the slabs (and the column tiles that the group crosses); a thread keeps its
// first eight parts in registers for the second round
__global__ void __launch_bounds__(kJoinFwd) gn_stats_join_kernel(const float2* __restrict__ part, GnShape g, int width,
                                                              float eps, float2* __restrict__ stat,
                                                              float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int kHeld = 8;
  __shared__ float red[kJoinFwd / 32];
  const int n = blockIdx.x / g.G, gr = blockIdx.x % g.G;
  const int c0 = gr * g.P, t0 = c0 / width, segs = (c0 + g.P - 1) / width - t0 + 1;  // width: channels of a tile
  const float2* base = part + (int64_t)n * g.chunks * (g.G + g.tiles - 1) + t0 + gr;
  const int items = g.chunks * segs;
  auto value = [&](int i) {
    const int k = segs == 1 ? i : i / segs;
    return base[(int64_t)k * (g.G + g.tiles - 1) + (segs == 1 ? 0 : i - k * segs)];
  };
  auto count = [&](int i) {  // values behind part i
    const int k = segs == 1 ? i : i / segs;
    const int64_t left = g.S - (int64_t)k * g.rows;
    const float rows = (float)(left < g.rows ? left : g.rows);
    if (segs == 1) return rows * (float)g.P;
    const int lo = (t0 + i - k * segs) * width, a = c0 > lo ? c0 : lo, b = c0 + g.P < lo + width ? c0 + g.P : lo + width;
    return rows * (float)(b - a);
  };
  pdl_launch_dependents();
  pdl_wait();
  float2 v[kHeld];
  float t = 0.0f, q = 0.0f;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    const int i = threadIdx.x + j * kJoinFwd;
    v[j] = i < items ? value(i) : make_float2(0.0f, 0.0f);
  }
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    if (threadIdx.x + j * kJoinFwd < items) t = fmaf(count(threadIdx.x + j * kJoinFwd), v[j].x, t);
  for (int i = threadIdx.x + kHeld * kJoinFwd; i < items; i += kJoinFwd) t = fmaf(count(i), value(i).x, t);
  const float total = (float)((double)g.S * g.P);
  const float mu = block_sum<kJoinFwd>(t, red) / total;
#pragma unroll
  for (int j = 0; j < kHeld; ++j)
    if (threadIdx.x + j * kJoinFwd < items) q += fmaf(count(threadIdx.x + j * kJoinFwd) * (v[j].x - mu), v[j].x - mu, v[j].y);
  for (int i = threadIdx.x + kHeld * kJoinFwd; i < items; i += kJoinFwd) {
    const float2 u = value(i);
    q += fmaf(count(i) * (u.x - mu), u.x - mu, u.y);
  }
  const float var = block_sum<kJoinFwd>(q, red) / total;
  if (threadIdx.x == 0) {
    const float s = 1.0f / sqrtf(var + eps);
    stat[blockIdx.x] = make_float2(mu, s);
    if (mean) mean[blockIdx.x] = mu;
    if (rstd) rstd[blockIdx.x] = s;
  }
}

// ---------------------------------------------------------------- forward: the elementwise pass
template <typename T, int EPI>
__global__ void __launch_bounds__(kThreads, kFwdPerSm<T>) gn_apply_kernel(const T* x, int64_t ldx, const T* __restrict__ w,
                                                            const T* __restrict__ b, const float2* __restrict__ stat,
                                                            GnShape g, T* y, int64_t ldy) {
  constexpr int E = Vec<T>::N;
  constexpr bool FAST = fast_math_for<T>();
  __shared__ __align__(16) uint4 ring[kRing * kThreads];
  const Place p = Place::make<E>(g);
  if (!p.active) return;
  pdl_wait();
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
  float2 nmu[E / 2], a2[E / 2], sh2[E / 2];
#pragma unroll
  for (int e = 0; e < E / 2; ++e) {
    nmu[e] = make_float2(-mu[2 * e], -mu[2 * e + 1]);
    a2[e] = make_float2(a[2 * e], a[2 * e + 1]);
    sh2[e] = make_float2(sh[2 * e], sh[2 * e + 1]);
  }
  // the slab from its end, which the sums read last: as much of it as L2 still holds is not read from HBM again
  const int64_t img = (int64_t)p.n * g.S;
  const int64_t left = (p.r1 - p.r0 - p.lane_row + g.rl - 1) / g.rl;  // positions of this thread
  auto one = [&](const uint4& u) {
    float2 f[E / 2];
    unpack2<T>(u, f);
#pragma unroll
    for (int e = 0; e < E / 2; ++e) f[e] = act_pair<EPI, FAST>(fma2(add2(f[e], nmu[e]), a2[e], sh2[e]));
    return pack2<T>(f);
  };
  if (left <= 0) return;
  T* dst = y + (img + p.r0 + p.lane_row + (left - 1) * g.rl) * ldy;
  const int64_t sy = (int64_t)g.rl * ldy;
  walk<T>(ring + threadIdx.x, x + (img + p.r0 + p.lane_row + (left - 1) * g.rl) * ldx + p.v * E, -(int64_t)g.rl * ldx,
          p.bytes, (int)left, [&](const uint4& u) {
            store_packed<T>(dst, p, g.C, one(u));
            dst -= sy;
          });
}

// ---------------------------------------------------------------- backward
// part[n][chunk][c] = (A_c, B_c) = (sum g, sum g xhat) of channel c over the slab
template <typename T, int EPI>
__global__ void __launch_bounds__(kThreads, kBwdPerSm<T>) gn_bwd_sums_kernel(const T* __restrict__ x, int64_t ldx,
                                                               const T* __restrict__ dy, int64_t lddy,
                                                               const T* __restrict__ w, const T* __restrict__ b,
                                                               const float* __restrict__ mean,
                                                               const float* __restrict__ rstd, GnShape g,
                                                               float2* __restrict__ part) {
  constexpr int E = Vec<T>::N;
  constexpr bool FAST = fast_math_for<T>();
  __shared__ __align__(16) uint4 ring[kRing * kThreads];
  float* sm_a = reinterpret_cast<float*>(ring);  // the copies have all been read by then
  float* sm_b = sm_a + kThreads * E;
  static_assert(sizeof(uint4) * kRing >= 4 * 2 * E, "the sums fit the ring");
  const Place p = Place::make<E>(g);
  constexpr int H = E / 2;
  float A[E], B[E];
  float2 A2[H], B2[H];
#pragma unroll
  for (int e = 0; e < H; ++e) A2[e] = B2[e] = make_float2(0.0f, 0.0f);
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
    float2 nmu[H], s2[H], w2[H], b2[H];
#pragma unroll
    for (int e = 0; e < H; ++e) {
      nmu[e] = make_float2(-mu[2 * e], -mu[2 * e + 1]);
      s2[e] = make_float2(s[2 * e], s[2 * e + 1]);
      w2[e] = make_float2(wf[2 * e], wf[2 * e + 1]);
      b2[e] = make_float2(bf[2 * e], bf[2 * e + 1]);
    }
    auto one = [&](const uint4& ux, const uint4& ud) {
      float2 f[H], d[H];
      unpack2<T>(ux, f);
      unpack2<T>(ud, d);
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float2 xh = mul2(add2(f[e], nmu[e]), s2[e]);
        const float2 gg = EPI == EPI_NONE ? d[e] : mul2(d[e], act_grad_pair<EPI, FAST>(fma2(xh, w2[e], b2[e])));
        A2[e] = add2(A2[e], gg);
        B2[e] = fma2(gg, xh, B2[e]);
      }
    };
    const int64_t row0 = (int64_t)p.n * g.S + p.r0 + p.lane_row;
    const int64_t left = (p.r1 - p.r0 - p.lane_row + g.rl - 1) / g.rl;
    if (left > 0)
      walk2<T>(ring + threadIdx.x, x + row0 * ldx + p.v * E, (int64_t)g.rl * ldx, dy + row0 * lddy + p.v * E,
               (int64_t)g.rl * lddy, p.bytes, (int)left, one);
  }
#pragma unroll
  for (int e = 0; e < H; ++e) {
    A[2 * e] = A2[e].x, A[2 * e + 1] = A2[e].y;
    B[2 * e] = B2[e].x, B[2 * e + 1] = B2[e].y;
  }
  pdl_launch_dependents();
  __syncthreads();
#pragma unroll
  for (int e = 0; e < E; ++e) sm_a[threadIdx.x * E + e] = A[e], sm_b[threadIdx.x * E + e] = B[e];
  __syncthreads();
  // as many lanes as there are to spare share the sum over the rl threads of a channel: parts of at most 16 and a tree
  // (one after the other, 256 of them, dw and db of narrow images had up to four times an elementary sum's error)
  const int share = spare_lanes(g.tv * E), lane = (int)threadIdx.x & (share - 1);
  const int c0 = (blockIdx.x % g.tiles) * g.tv * E, nch = g.C - c0 < g.tv * E ? g.C - c0 : g.tv * E;
  float2* out = part + ((int64_t)p.n * g.chunks + p.chunk) * g.C + c0;
  for (int j0 = 0; j0 < nch; j0 += kThreads / share) {  // the same number of turns for every lane
    const int j = j0 + (int)threadIdx.x / share, jc = j < nch ? j : nch - 1;
    float ta = 0.0f, tb = 0.0f;
    for (int k = lane; k < g.rl; k += share) {
      ta += sm_a[k * g.tv * E + jc];
      tb += sm_b[k * g.tv * E + jc];
    }
    if (share > 1) ta = lanes_sum(ta, share), tb = lanes_sum(tb, share);
    if (lane == 0 && j < nch) out[j] = make_float2(ta, tb);
  }
}

// folds the slabs of wide groups channel by channel, before the join: a block has 32 channels of an image, 32 threads
// each that take every 32nd slab. out[n][c] = (A_c, B_c)
__global__ void __launch_bounds__(1024) gn_bwd_fold_kernel(const float2* __restrict__ part, GnShape g, int blocks,
                                                           float2* __restrict__ out) {
  __shared__ float2 sums[32][33];
  pdl_launch_dependents();
  pdl_wait();
  const int n = blockIdx.x / blocks, c = (blockIdx.x % blocks) * 32 + (threadIdx.x & 31), k0 = threadIdx.x >> 5;
  float2 t = make_float2(0.0f, 0.0f);
  if (c < g.C) {
    const float2* src = part + (int64_t)n * g.chunks * g.C + c;
#pragma unroll 4
    for (int k = k0; k < g.chunks; k += 32) t = add2(t, src[(int64_t)k * g.C]);
  }
  sums[k0][threadIdx.x & 31] = t;
  __syncthreads();
  if (k0 == 0 && c < g.C) {
#pragma unroll
    for (int k = 1; k < 32; ++k) t = add2(t, sums[k][threadIdx.x]);
    out[(int64_t)n * g.C + c] = t;
  }
}

// one block per (image, group): chan[n][0..C) = B_c, chan[n][C..2C) = A_c (the column sums over the
// images are then dw and db), stat[n][group] = (m1, m2)
template <typename T>
__global__ void __launch_bounds__(kJoin) gn_bwd_join_kernel(const float2* __restrict__ part,
                                                               const T* __restrict__ w, GnShape g,
                                                               float* __restrict__ chan, float2* __restrict__ stat) {
  __shared__ float red[kJoin / 32];
  __shared__ float2 sums[kJoin];
  pdl_launch_dependents();
  pdl_wait();
  const int n = blockIdx.x / g.G, gr = blockIdx.x % g.G;
  float m1 = 0.0f, m2 = 0.0f;
  const int parts = g.P < kJoin ? kJoin / g.P : 1;
  int tree = 0;  // the largest power of two below the parts that hold slabs
  for (int h = 1; h < parts && h < g.chunks; h *= 2) tree = h;
  for (int b0 = 0; b0 < g.P; b0 += kJoin) {  // a thread: every `parts`-th slab of one channel
    const int j = g.P < kJoin ? (int)threadIdx.x % g.P : b0 + (int)threadIdx.x;
    const int k0 = g.P < kJoin ? (int)threadIdx.x / g.P : 0;
    float2 t = make_float2(0.0f, 0.0f);
    if (j < g.P && k0 < parts) {
      const float2* src = part + (int64_t)n * g.chunks * g.C + gr * g.P + j;
#pragma unroll 8
      for (int k = k0; k < g.chunks; k += parts) t = add2(t, src[(int64_t)k * g.C]);
    }
    sums[threadIdx.x] = t;
    __syncthreads();
    for (int h = tree; h > 0; h /= 2) {  // the parts as a tree: place k gets k + h
      if (k0 < h && k0 + h < parts) t = add2(t, sums[(k0 + h) * g.P + j]), sums[k0 * g.P + j] = t;
      __syncthreads();
    }
    if (j < g.P && k0 == 0) {
      const int c = gr * g.P + j;
      chan[(int64_t)n * 2 * g.C + c] = t.y;
      chan[(int64_t)n * 2 * g.C + g.C + c] = t.x;
      const float wc = ld_param(w, c, 1.0f);
      m1 = fmaf(wc, t.x, m1);
      m2 = fmaf(wc, t.y, m2);
    }
    __syncthreads();
  }
  const float inv = 1.0f / (float)((double)g.S * g.P);
  m1 = block_sum<kJoin>(m1, red) * inv;
  m2 = block_sum<kJoin>(m2, red) * inv;
  if (threadIdx.x == 0) stat[blockIdx.x] = make_float2(m1, m2);
}

template <typename T, int EPI>
__global__ void __launch_bounds__(kThreads, kBwdPerSm<T>) gn_bwd_apply_kernel(const T* __restrict__ x, int64_t ldx, const T* dy,
                                                                int64_t lddy, const T* __restrict__ w,
                                                                const T* __restrict__ b, const float* __restrict__ mean,
                                                                const float* __restrict__ rstd,
                                                                const float2* __restrict__ stat, GnShape g, T* dx,
                                                                int64_t lddx) {
  constexpr int E = Vec<T>::N;
  constexpr bool FAST = fast_math_for<T>();
  __shared__ __align__(16) uint4 ring[kRing * kThreads];
  const Place p = Place::make<E>(g);
  if (!p.active) return;
  pdl_wait();
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
  constexpr int H = E / 2;
  float2 nmu[H], s2[H], w2[H], b2[H], n1[H], n2[H];
#pragma unroll
  for (int e = 0; e < H; ++e) {
    nmu[e] = make_float2(-mu[2 * e], -mu[2 * e + 1]);
    s2[e] = make_float2(s[2 * e], s[2 * e + 1]);
    w2[e] = make_float2(wf[2 * e], wf[2 * e + 1]);
    b2[e] = make_float2(bf[2 * e], bf[2 * e + 1]);
    n1[e] = make_float2(-m1[2 * e], -m1[2 * e + 1]);
    n2[e] = make_float2(-m2[2 * e], -m2[2 * e + 1]);
  }
  auto one = [&](const uint4& ux, const uint4& ud) {
    float2 f[H], d[H];
    unpack2<T>(ux, f);
    unpack2<T>(ud, d);
#pragma unroll
    for (int e = 0; e < H; ++e) {
      const float2 xh = mul2(add2(f[e], nmu[e]), s2[e]);
      const float2 gg = EPI == EPI_NONE ? d[e] : mul2(d[e], act_grad_pair<EPI, FAST>(fma2(xh, w2[e], b2[e])));
      f[e] = mul2(s2[e], fma2(xh, n2[e], fma2(gg, w2[e], n1[e])));
    }
    return pack2<T>(f);
  };
  // the slab from its end, which the sums read last: as much of it as L2 still holds is not read from HBM again
  const int64_t row0 = (int64_t)p.n * g.S + p.r0 + p.lane_row;
  const int64_t left = (p.r1 - p.r0 - p.lane_row + g.rl - 1) / g.rl;
  if (left <= 0) return;
  T* out = dx + (row0 + (left - 1) * g.rl) * lddx;
  const int64_t so = (int64_t)g.rl * lddx;
  walk2<T>(ring + threadIdx.x, x + (row0 + (left - 1) * g.rl) * ldx + p.v * E, -(int64_t)g.rl * ldx,
           dy + (row0 + (left - 1) * g.rl) * lddy + p.v * E, -(int64_t)g.rl * lddy, p.bytes, (int)left,
           [&](const uint4& ux, const uint4& ud) {
             store_packed<T>(out, p, g.C, one(ux, ud));
             out -= so;
           });
}

// ---------------------------------------------------------------- resident images: one read
// When the runs of a few whole groups over an image fit the registers of a cluster of at most eight blocks,
// the cluster loads them once: block r the positions [r S / cs, (r + 1) S / cs), a thread one 16-byte
// vector of the run at every RL-th position, VPT in all, kept packed. Sums go channel by channel through
// shared memory, then across the cluster through distributed shared memory, in a fixed order. One launch,
// 2 n (forward) or 3 n (backward) values of traffic; runs are at least 64 bytes where the groups allow
// it, so that sectors are used whole.
constexpr int kResThreads = 512;

struct Bundle {
  int64_t S;
  int C, P, G;
  int groups;   // groups of a bundle
  int bv;       // its 16-byte vectors
  int bundles;  // of an image
  int cs;       // blocks of a cluster
  int rows;     // positions of a block (the last ones may have fewer)
  unsigned d_bv, d_w, d_p;  // for fdiv by bv, by the bundle's channels (whole vectors) and by P
  int lp;       // log2 of the lanes that take different channels of a group in a warp's sum
};

template <int N>
__device__ __forceinline__ void keep_packed(uint4 (&u)[N]) {  // unpack again after this; do not keep unpacked
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+r"(u[k].x), "+r"(u[k].y), "+r"(u[k].z), "+r"(u[k].w));
}

__device__ __forceinline__ uint32_t cluster_rank_() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_arrive() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ float2 peer_f2(const float2* p, int rank) {  // the same place in block `rank`
  uint32_t a;
  float2 v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
  return v;
}

// n / d for n d < 2^32 by d's magic number ceil(2^32 / d) (0 for d = 1)
__device__ __forceinline__ int fdiv(int n, unsigned m) { return m ? (int)__umulhi((unsigned)n, m) : n; }

// what a thread of the resident kernels works on
template <int E>
struct ResPlace {
  int n, c0, nch, lv, lr, rl, rank;
  bool active;
  int r0, r1;
  __device__ __forceinline__ ResPlace(const Bundle& g) {
    rank = (int)cluster_rank_();
    const int unit = blockIdx.x / g.cs;
    n = unit / g.bundles;
    c0 = (unit % g.bundles) * g.groups * g.P;
    nch = g.C - c0 < g.groups * g.P ? g.C - c0 : g.groups * g.P;
    rl = fdiv(kResThreads, g.d_bv);
    lr = fdiv(threadIdx.x, g.d_bv);
    lv = threadIdx.x - lr * g.bv;
    active = lr < rl && lv * E < nch;
    r0 = (int)(g.S < (int64_t)rank * g.rows ? g.S : rank * g.rows);
    r1 = (int)(g.S - r0 < g.rows ? g.S : r0 + g.rows);
  }
};

template <typename T, int VPT>
__device__ __forceinline__ void res_load(uint4 (&raw)[VPT], const T* x, int64_t ld, const ResPlace<Vec<T>::N>& p,
                                         int64_t S) {
  const T* base = x + ((int64_t)p.n * S + p.r0 + p.lr) * ld + p.c0 + p.lv * Vec<T>::N;
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    raw[k] = make_uint4(0, 0, 0, 0);
    if (p.active && p.r0 + p.lr + k * p.rl < p.r1) raw[k] = ld_stream(base + (int64_t)k * p.rl * ld);
  }
}

// Sums over the block's positions of NQ quantities per channel. v: this thread's E channels (0 where it is not
// active). red: NQ x kResThreads x E floats. Returns the part sums in red2[q][part][W] (W = bv E, `parts`
// parts), after a barrier; red and red2 may be the same memory (a barrier lies between).
template <int E, int NQ>
__device__ __forceinline__ int res_parts(const float (&v)[NQ][E], float* red, int W, unsigned d_w, int rl, bool in) {
  const int tid = threadIdx.x;
  if (in) {
#pragma unroll
    for (int q = 0; q < NQ; ++q)
#pragma unroll
      for (int e = 0; e < E; e += 4)
        *reinterpret_cast<float4*>(red + q * kResThreads * E + tid * E + e) =
            make_float4(v[q][e], v[q][e + 1], v[q][e + 2], v[q][e + 3]);
  }
  __syncthreads();
  const int most = W < kResThreads ? fdiv(kResThreads, d_w) : 1, parts = most < rl ? most : rl;
  const int row = W < kResThreads ? fdiv(tid, d_w) : 0, col = W < kResThreads ? tid - row * W : tid;
  // thread (part, channel) adds every parts-th position; blocks wider than kResThreads channels in rounds
  for (int c0 = 0; c0 < W; c0 += kResThreads) {
    const int c = c0 + col, part = row;
    float t[NQ];
    const bool mine = part < parts && c < W;
#pragma unroll
    for (int q = 0; q < NQ; ++q) t[q] = 0.0f;
    if (mine)
      for (int r = part; r < rl; r += parts)
#pragma unroll
        for (int q = 0; q < NQ; ++q) t[q] += red[q * kResThreads * E + r * W + c];
    __syncthreads();
    if (mine)  // the place of a position that this thread has read (rows below `parts` of its own channels)
#pragma unroll
      for (int q = 0; q < NQ; ++q) red[q * kResThreads * E + part * W + c] = t[q];
  }
  __syncthreads();
  return parts;
}

// the sum over a group's channels (from ch0, P of them) and the parts, by one warp: 2^lp lanes take different
// channels, the others different parts
__device__ __forceinline__ float warp_sum_of(const float* red, int W, int parts, int ch0, int P, int lp, int lane) {
  float t = 0.0f;
  for (int c = lane & ((1 << lp) - 1); c < P; c += 1 << lp)
    for (int k = lane >> lp; k < parts; k += 32 >> lp) t += red[k * W + ch0 + c];
  return group_sum<32>(t);
}

template <typename T, int EPI, int VPT>
__global__ void __launch_bounds__(kResThreads, VPT <= 4 ? 2 : 1)
    gn_fwd_resident_kernel(const T* x, int64_t ldx, const T* __restrict__ w, const T* __restrict__ b, Bundle g, float eps,
                           T* y, int64_t ldy, float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int E = Vec<T>::N, H = E / 2;
  constexpr bool FAST = fast_math_for<T>();
  extern __shared__ __align__(16) float smem[];
  const int W = g.bv * E;
  float* red = smem;                                        // [kResThreads][E]
  float2* own = reinterpret_cast<float2*>(red + kResThreads * E);  // [groups] (mean, centred squares) of the block
  float2* stat = own + g.groups;                            // [groups] (mean, rstd) of the image
  float* chan = reinterpret_cast<float*>(stat + g.groups);  // [3][W] mean, scale, shift of a channel
  const ResPlace<E> p(g);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ng = fdiv(p.nch, g.d_p);
  uint4 raw[VPT];
  res_load<T, VPT>(raw, x, ldx, p, g.S);
  const float cnt = (float)(p.r1 - p.r0) * (float)g.P, inv_cnt = cnt > 0.0f ? 1.0f / cnt : 0.0f;
  {
    float s[1][E];
    float2 t2[H];
#pragma unroll
    for (int e = 0; e < H; ++e) t2[e] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float2 f[H];
      unpack2<T>(raw[k], f);
#pragma unroll
      for (int e = 0; e < H; ++e) t2[e] = add2(t2[e], f[e]);
    }
#pragma unroll
    for (int e = 0; e < H; ++e) s[0][2 * e] = t2[e].x, s[0][2 * e + 1] = t2[e].y;
    const int parts = res_parts<E, 1>(s, red, W, g.d_w, p.rl, p.lr < p.rl);
    for (int i = warp; i < ng; i += kResThreads / 32) {
      const float t = warp_sum_of(red, W, parts, i * g.P, g.P, g.lp, lane);
      if (lane == 0) own[i].x = t * inv_cnt;
    }
    __syncthreads();
    keep_packed(raw);
    float2 nmu[H];
#pragma unroll
    for (int e = 0; e < H; ++e) {
      t2[e] = make_float2(0.0f, 0.0f);
      const int c = p.active ? p.lv * E + 2 * e : 0;
      nmu[e] = make_float2(-own[fdiv(c, g.d_p)].x, -own[fdiv(c + 1, g.d_p)].x);
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      if (p.active && p.r0 + p.lr + k * p.rl < p.r1) {
        float2 f[H];
        unpack2<T>(raw[k], f);
#pragma unroll
        for (int e = 0; e < H; ++e) {
          const float2 d = add2(f[e], nmu[e]);
          t2[e] = fma2(d, d, t2[e]);
        }
      }
    }
#pragma unroll
    for (int e = 0; e < H; ++e) s[0][2 * e] = t2[e].x, s[0][2 * e + 1] = t2[e].y;
    const int parts2 = res_parts<E, 1>(s, red, W, g.d_w, p.rl, p.lr < p.rl);
    for (int i = warp; i < ng; i += kResThreads / 32) {
      const float t = warp_sum_of(red, W, parts2, i * g.P, g.P, g.lp, lane);
      if (lane == 0) own[i].y = t;
    }
    keep_packed(raw);
  }
  if (g.cs > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  for (int i = threadIdx.x; i < ng; i += kResThreads) {
    const float total = (float)((double)g.S * g.P);
    float mu, q = 0.0f;
    if (g.cs > 1) {  // join the blocks' statistics in rank order
      float t = 0.0f;
      float2 v[8];
      auto count = [&](int r) {
        const int left = (int)g.S - r * g.rows;
        return left <= 0 ? 0.0f : (float)(left < g.rows ? left : g.rows) * (float)g.P;
      };
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = r < g.cs ? peer_f2(own + i, r) : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < g.cs) t = fmaf(count(r), v[r].x, t);
      mu = t / total;
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < g.cs) {
          const float d = v[r].x - mu;
          q += fmaf(count(r) * d, d, v[r].y);
        }
    } else {
      mu = own[i].x;
      q = own[i].y;
    }
    const float s = 1.0f / sqrtf(q / total + eps);
    stat[i] = make_float2(mu, s);
    if (p.rank == 0) {
      const int64_t at = (int64_t)p.n * g.G + (blockIdx.x / g.cs % g.bundles) * g.groups + i;
      if (mean) mean[at] = mu;
      if (rstd) rstd[at] = s;
    }
  }
  if (g.cs > 1) cluster_arrive();  // this block has read its peers (they may leave once all have)
  __syncthreads();
  for (int c = threadIdx.x; c < p.nch; c += kResThreads) {
    const float2 s = stat[fdiv(c, g.d_p)];
    chan[c] = s.x;
    chan[W + c] = s.y * ld_param(w, p.c0 + c, 1.0f);
    chan[2 * W + c] = ld_param(b, p.c0 + c, 0.0f);
  }
  __syncthreads();
  if (p.active) {
    float2 mu[H], a[H], sh[H];
#pragma unroll
    for (int e = 0; e < H; ++e) {
      const int c = p.lv * E + 2 * e;
      mu[e] = make_float2(-chan[c], -chan[c + 1]);
      a[e] = make_float2(chan[W + c], chan[W + c + 1]);
      sh[e] = make_float2(chan[2 * W + c], chan[2 * W + c + 1]);
    }
    T* out = y + ((int64_t)p.n * g.S + p.r0 + p.lr) * ldy + p.c0 + p.lv * E;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float2 f[H];
      unpack2<T>(raw[k], f);
#pragma unroll
      for (int e = 0; e < H; ++e) f[e] = act_pair<EPI, FAST>(fma2(add2(f[e], mu[e]), a[e], sh[e]));
      if (p.r0 + p.lr + k * p.rl < p.r1) st_stream(out + (int64_t)k * p.rl * ldy, pack2<T>(f));
    }
  }
  if (g.cs > 1) cluster_wait();
}

// chan_out[n][0..C) = B_c, [C..2C) = A_c of the image
template <typename T, int EPI, int VPT>
__global__ void __launch_bounds__(kResThreads, VPT <= 2 ? 2 : 1)
    gn_bwd_resident_kernel(const T* __restrict__ x, int64_t ldx, const T* dy, int64_t lddy, const T* __restrict__ w,
                           const T* __restrict__ b, const float* __restrict__ mean, const float* __restrict__ rstd,
                           Bundle g, T* dx, int64_t lddx, float* __restrict__ chan_out) {
  constexpr int E = Vec<T>::N, H = E / 2;
  constexpr bool FAST = fast_math_for<T>();
  extern __shared__ __align__(16) float smem[];
  const int W = g.bv * E;
  float* red = smem;                                                   // [2][kResThreads][E]
  float2* own = reinterpret_cast<float2*>(red + 2 * kResThreads * E);  // [W] (A_c, B_c) of the block
  float2* tot = own + W;                                               // [W] of the image, times w_c
  float2* stat = tot + W;                                              // [groups] (m1, m2)
  float* chan = reinterpret_cast<float*>(stat + g.groups);             // [4][W] mean, rstd, w, b of a channel
  const ResPlace<E> p(g);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int ng = fdiv(p.nch, g.d_p);
  uint4 raw[VPT], rawd[VPT];
  res_load<T, VPT>(raw, x, ldx, p, g.S);
  res_load<T, VPT>(rawd, dy, lddy, p, g.S);
  const int g0 = (blockIdx.x / g.cs % g.bundles) * g.groups;  // the bundle's first group
  for (int c = threadIdx.x; c < p.nch; c += kResThreads) {
    const int64_t at = (int64_t)p.n * g.G + g0 + fdiv(c, g.d_p);
    chan[c] = mean[at];
    chan[W + c] = rstd[at];
    chan[2 * W + c] = ld_param(w, p.c0 + c, 1.0f);
    chan[3 * W + c] = ld_param(b, p.c0 + c, 0.0f);
  }
  __syncthreads();
  float2 mu[H], s[H], wf[H], bf[H];
#pragma unroll
  for (int e = 0; e < H; ++e) {
    const int c = p.active ? p.lv * E + 2 * e : 0;
    mu[e] = make_float2(-chan[c], -chan[c + 1]);
    s[e] = make_float2(chan[W + c], chan[W + c + 1]);
    wf[e] = make_float2(chan[2 * W + c], chan[2 * W + c + 1]);
    bf[e] = make_float2(chan[3 * W + c], chan[3 * W + c + 1]);
  }
  float v[2][E];
  {
    float2 A[H], B[H];
#pragma unroll
    for (int e = 0; e < H; ++e) A[e] = B[e] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < VPT; ++k) {  // past the block's positions dy is 0 and adds nothing
      float2 f[H], d[H];
      unpack2<T>(raw[k], f);
      unpack2<T>(rawd[k], d);
#pragma unroll
      for (int e = 0; e < H; ++e) {
        const float2 xh = mul2(add2(f[e], mu[e]), s[e]);
        const float2 gg = EPI == EPI_NONE ? d[e] : mul2(d[e], act_grad_pair<EPI, FAST>(fma2(xh, wf[e], bf[e])));
        A[e] = add2(A[e], gg);
        B[e] = fma2(gg, xh, B[e]);
        if constexpr (sizeof(T) == 4) f[e] = xh, d[e] = gg;
      }
      if constexpr (sizeof(T) == 4) raw[k] = pack2<T>(f), rawd[k] = pack2<T>(d);  // as they are needed below
    }
#pragma unroll
    for (int e = 0; e < H; ++e) {
      v[0][2 * e] = p.active ? A[e].x : 0.0f, v[0][2 * e + 1] = p.active ? A[e].y : 0.0f;
      v[1][2 * e] = p.active ? B[e].x : 0.0f, v[1][2 * e + 1] = p.active ? B[e].y : 0.0f;
    }
  }
  keep_packed(raw);
  keep_packed(rawd);
  const int parts = res_parts<E, 2>(v, red, W, g.d_w, p.rl, p.lr < p.rl);
  for (int c = threadIdx.x; c < p.nch; c += kResThreads) {
    float ta = 0.0f, tb = 0.0f;
    for (int k = 0; k < parts; ++k) {
      ta += red[k * W + c];
      tb += red[kResThreads * E + k * W + c];
    }
    own[c] = make_float2(ta, tb);
  }
  if (g.cs > 1) {
    cluster_arrive();
    cluster_wait();
  } else {
    __syncthreads();
  }
  for (int c = threadIdx.x; c < p.nch; c += kResThreads) {
    float2 t = make_float2(0.0f, 0.0f);
    if (g.cs > 1) {
      float2 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r) v[r] = r < g.cs ? peer_f2(own + c, r) : make_float2(0.0f, 0.0f);
#pragma unroll
      for (int r = 0; r < 8; ++r) t = add2(t, v[r]);
    } else {
      t = own[c];
    }
    if (chan_out && p.rank == 0) {
      chan_out[(int64_t)p.n * 2 * g.C + p.c0 + c] = t.y;
      chan_out[(int64_t)p.n * 2 * g.C + g.C + p.c0 + c] = t.x;
    }
    tot[c] = mul2(t, dup2(chan[2 * W + c]));
  }
  if (g.cs > 1) cluster_arrive();  // this block has read its peers (they may leave once all have)
  __syncthreads();
  const float inv = 1.0f / (float)((double)g.S * g.P);
  for (int i = warp; i < ng; i += kResThreads / 32) {
    float m1 = 0.0f, m2 = 0.0f;
    for (int c = lane; c < g.P; c += 32) {
      const float2 t = tot[i * g.P + c];
      m1 += t.x;
      m2 += t.y;
    }
    m1 = group_sum<32>(m1) * inv;
    m2 = group_sum<32>(m2) * inv;
    if (lane == 0) stat[i] = make_float2(m1, m2);
  }
  __syncthreads();
  if (p.active) {
    float2 m1[H], m2[H];
#pragma unroll
    for (int e = 0; e < H; ++e) {
      const float2 u = stat[fdiv(p.lv * E + 2 * e, g.d_p)], t = stat[fdiv(p.lv * E + 2 * e + 1, g.d_p)];
      m1[e] = make_float2(-u.x, -t.x);
      m2[e] = make_float2(-u.y, -t.y);
    }
    T* out = dx + ((int64_t)p.n * g.S + p.r0 + p.lr) * lddx + p.c0 + p.lv * E;
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      float2 f[H], d[H];
      unpack2<T>(raw[k], f);
      unpack2<T>(rawd[k], d);
#pragma unroll
      for (int e = 0; e < H; ++e) {
        float2 xh = f[e], gg = d[e];
        if constexpr (sizeof(T) == 2) {
          xh = mul2(add2(f[e], mu[e]), s[e]);
          if constexpr (EPI != EPI_NONE) gg = mul2(d[e], act_grad_pair<EPI, FAST>(fma2(xh, wf[e], bf[e])));
        }
        f[e] = mul2(s[e], fma2(xh, m2[e], fma2(gg, wf[e], m1[e])));
      }
      if (p.r0 + p.lr + k * p.rl < p.r1) st_stream(out + (int64_t)k * p.rl * lddx, pack2<T>(f));
    }
  }
  if (g.cs > 1) cluster_wait();
}

// ---------------------------------------------------------------- host side

bool shape_ok(int64_t N, int64_t S, int64_t C, int64_t G) {
  return N >= 0 && S >= 0 && C > 0 && G > 0 && C % G == 0 && C <= (1 << 20) && N <= (1 << 20) && S <= INT64_MAX / 4 / C;
}

GnShape plan(int64_t N, int64_t S, int64_t C, int64_t G, int es, bool fwd) {
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
  // the blocks that are resident at once, a slab no shorter than one batch per thread
  const int per_sm = es == 4 ? (fwd ? kFwdPerSm<float> : kBwdPerSm<float>)
                             : (fwd ? kFwdPerSm<__nv_bfloat16> : kBwdPerSm<__nv_bfloat16>);
  int64_t chunks = per_sm * (int64_t)sms / (N * g.tiles);
  if (chunks < 1) chunks = 1;
  const int64_t most = (S + (int64_t)g.rl * kBatch - 1) / ((int64_t)g.rl * kBatch);
  if (chunks > most) chunks = most;
  if (chunks < 1) chunks = 1;
  // in whole batches: what is left of one is read position by position, a memory latency each
  const int64_t batch = (int64_t)g.rl * kBatch;
  g.rows = (S + chunks - 1) / chunks;
  if (g.rows > batch) g.rows = (g.rows + batch - 1) / batch * batch;
  g.chunks = (int)((S + g.rows - 1) / g.rows);
  return g;
}

// From about twelve parts a thread of the join on, folding the slabs by channels first, on all SMs, is faster than its
// own launch costs: 1 x 4846 x 1020 bf16 with one group 37 us without, 25 with; 2 x 8192 x 512 with 4 groups (18
// parts) 28 both; 2 x 4096 x 640 with 8 (6 parts) 23.9 and 24.6.
bool folds(const GnShape& g) { return (int64_t)g.chunks * g.P > 12 * kJoin; }

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

gn_status launch(void* kern, int64_t blocks, void** args, cudaStream_t s, bool waits, int threads = kThreads) {
  if (blocks > INT32_MAX) return GN_ERR_SHAPE;
  if (!kernel_attrs(kern, 0)) return GN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = s;
  // a kernel that waits for the one before it on the device (pdl_wait) may be launched while that one ends
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = GN_PDL;
  cfg.attrs = attr;
  cfg.numAttrs = waits ? 1 : 0;
  if (cudaLaunchKernelExC(&cfg, kern, args) != cudaSuccess) return GN_ERR_CUDA;
  count_launches(1);
  return launch_status();
}

// How the resident kernels would take the shape; cs == 0: it does not fit. most: the vectors a thread
// may hold (of each tensor). A bundle is the fewest groups whose run is whole vectors, widened to 64 bytes
// while that still fits; the cluster has as many blocks as it takes to fill the SMs or to hold the run.
Bundle plan_resident(int64_t N, int64_t S, int64_t C, int64_t G, int es, int most, int* vpt) {
  Bundle g{};
  g.S = S;
  g.C = (int)C;
  g.G = (int)G;
  g.P = (int)(C / G);
  g.cs = 0;
  const int64_t run = (int64_t)g.P * es;  // bytes of one group at one position
  if (C * es % 16 || S > (1 << 20)) return g;
  int per = 1;
  while (per * run % 16) per *= 2;  // run * per is whole vectors for some power of two up to 16
  if (per > G) return g;
  int64_t bv = per * run / 16;
  auto fits = [&](int64_t v, int64_t cs) { return v <= kResThreads && (S + cs - 1) / cs <= (kResThreads / v) * (int64_t)most; };
  // beyond 4 MiB in all, only images of which a block holds a bundle by itself, a few vectors a thread: else
  // the two passes, whose many short-lived loads keep memory busier, are faster (2 x 4096 x 640 bf16 forward: 27
  // us on chip, 19 in two passes; 2 x 1024 x 640: 8 and 13). The backward goes by the same bytes of x, though it holds
  // dy as well: 2 x 1024 x 640 13.3 on chip and 16.3, 1 x 4096 x 512 18.5 and 17.6, 4 x 1024 x 640 25.7 and 19.5; where
  // one block holds a bundle it errs, by 3 us in 23 at 8 x 256 x 1280
  if (!fits(bv, 8) || (N * S * C * es > (4 << 20) && S > (kResThreads / bv) * 4)) return g;
  while (bv < 4 && per * 2 <= G && fits(bv * 2, 8)) per *= 2, bv *= 2;
  // many small images: wider bundles while there are blocks enough, so that a block's threads have work
  const int sms = sm_count() > 0 ? sm_count() : 148;
  while (per * 2 <= G && N * ((G + 2 * per - 1) / (2 * per)) >= 2 * sms && bv * 2 <= kResThreads &&
         S <= (kResThreads / (bv * 2)) * 4)
    per *= 2, bv *= 2;
  g.groups = per;
  g.bv = (int)bv;
  g.bundles = (int)((G + per - 1) / per);
  const int64_t units = N * g.bundles;
  int cs = 1;
  while (cs < 8 && (!fits(bv, cs) || (units * cs < 2 * sms && (S + cs - 1) / cs > 2 * (kResThreads / bv)))) cs *= 2;
  const int64_t need = ((S + cs - 1) / cs + kResThreads / bv - 1) / (kResThreads / bv);
  *vpt = need <= 2 ? (int)need : need <= 8 ? (int)(need + 1) / 2 * 2 : (int)(need + 3) / 4 * 4;
  g.cs = cs;
  g.rows = (int)((S + cs - 1) / cs);
  auto magic = [](int64_t d) { return d > 1 ? (unsigned)(((1ull << 32) + d - 1) / d) : 0u; };
  g.d_bv = magic(bv);
  g.d_w = magic(bv * 16 / es);
  g.d_p = magic(g.P);
  while (g.lp < 5 && (1 << g.lp) < g.P) ++g.lp;
  return g;
}

template <typename T, int EPI>
void* pick_fwd_res(int vpt) {
  return vpt <= 1   ? (void*)gn_fwd_resident_kernel<T, EPI, 1>
         : vpt <= 2 ? (void*)gn_fwd_resident_kernel<T, EPI, 2>
         : vpt <= 4 ? (void*)gn_fwd_resident_kernel<T, EPI, 4>
         : vpt <= 6 ? (void*)gn_fwd_resident_kernel<T, EPI, 6>
         : vpt <= 8 ? (void*)gn_fwd_resident_kernel<T, EPI, 8>
         : vpt <= 12 ? (void*)gn_fwd_resident_kernel<T, EPI, 12>
                    : (void*)gn_fwd_resident_kernel<T, EPI, 16>;
}
template <typename T, int EPI>
void* pick_bwd_res(int vpt) {
  return vpt <= 1   ? (void*)gn_bwd_resident_kernel<T, EPI, 1>
         : vpt <= 2 ? (void*)gn_bwd_resident_kernel<T, EPI, 2>
         : vpt <= 4 ? (void*)gn_bwd_resident_kernel<T, EPI, 4>
         : vpt <= 6 ? (void*)gn_bwd_resident_kernel<T, EPI, 6>
                    : (void*)gn_bwd_resident_kernel<T, EPI, 8>;
}
template <typename T>
void* pick_res(bool fwd, int epi, int vpt) {
  if (fwd)
    return epi == GN_EPI_GELU_TANH ? pick_fwd_res<T, EPI_GELU_TANH>(vpt)
           : epi == GN_EPI_SILU    ? pick_fwd_res<T, EPI_SILU>(vpt)
                                   : pick_fwd_res<T, EPI_NONE>(vpt);
  return epi == GN_EPI_GELU_TANH ? pick_bwd_res<T, EPI_GELU_TANH>(vpt)
         : epi == GN_EPI_SILU    ? pick_bwd_res<T, EPI_SILU>(vpt)
                                 : pick_bwd_res<T, EPI_NONE>(vpt);
}
constexpr int kFwdMost = 16, kBwdMost = 8;  // vectors a thread may hold of each tensor: 64 registers in all

size_t res_smem(const Bundle& g, int es, bool fwd) {
  const size_t E = 16 / es, W = (size_t)g.bv * E;
  return fwd ? (kResThreads * E + 4 * g.groups + 3 * W) * 4 : (2 * kResThreads * E + 4 * W + 2 * g.groups + 4 * W) * 4;
}

gn_status launch_resident(void* kern, const Bundle& g, int64_t N, size_t smem, void** args, cudaStream_t s) {
  const int64_t blocks = N * g.bundles * g.cs;
  if (blocks > INT32_MAX) return GN_ERR_SHAPE;
  if (!kernel_attrs(kern, smem)) return GN_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kResThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)g.cs;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelExC(&cfg, kern, args) != cudaSuccess) return GN_ERR_CUDA;
  count_launches(1);
  return launch_status();
}

}  // namespace
}  // namespace gn

using namespace gn;

extern "C" size_t gn_groupnorm_fwd_workspace(int64_t N, int64_t S, int64_t C, int64_t G, gn_dtype dt) {
  if (!dt_ok(dt) || !shape_ok(N, S, C, G) || N == 0 || S == 0) return 0;
  int vpt = 0;
  if (plan_resident(N, S, C, G, (int)dt_size(dt), kFwdMost, &vpt).cs) return 0;
  const GnShape g = plan(N, S, C, G, (int)dt_size(dt), true);
  return up16((size_t)N * g.G * 8) + (size_t)N * g.chunks * (g.G + g.tiles - 1) * 8;
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
  cudaStream_t s = (cudaStream_t)stream;
  int vpt = 0;
  Bundle r = plan_resident(N, S, C, G, (int)es, kFwdMost, &vpt);
  if (r.cs) {
    void* args[] = {&x, &ld_x, &w, &b, &r, &eps, &y, &ld_y, &mean, &rstd};
    return launch_resident(dt == GN_BF16 ? pick_res<__nv_bfloat16>(true, epi, vpt) : pick_res<float>(true, epi, vpt), r, N,
                           res_smem(r, (int)es, true), args, s);
  }
  if (!ws || ws_bytes < gn_groupnorm_fwd_workspace(N, S, C, G, dt)) return GN_ERR_WORKSPACE;
  if (!aligned16(ws)) return GN_ERR_ALIGN;
  GnShape g = plan(N, S, C, G, (int)es, true);
  float2* stat = static_cast<float2*>(ws);
  float2* part = reinterpret_cast<float2*>(static_cast<char*>(ws) + up16((size_t)N * g.G * 8));
  const int64_t blocks = N * g.chunks * g.tiles;
  void* args0[] = {&x, &ld_x, &g, &part};
  gn_status st = launch(dt == GN_BF16 ? (void*)gn_stats_kernel<__nv_bfloat16> : (void*)gn_stats_kernel<float>, blocks, args0,
                        s, false);
  if (st != GN_OK) return st;
  int width = g.tv * (int)(16 / es);
  void* args1[] = {&part, &g, &width, &eps, &stat, &mean, &rstd};
  st = launch((void*)gn_stats_join_kernel, N * G, args1, s, true, kJoinFwd);
  if (st != GN_OK) return st;
  void* args2[] = {&x, &ld_x, &w, &b, &stat, &g, &y, &ld_y};
  return launch(dt == GN_BF16 ? pick_apply<__nv_bfloat16>(epi) : pick_apply<float>(epi), blocks, args2, s, true);
}

extern "C" size_t gn_groupnorm_bwd_workspace(int64_t N, int64_t S, int64_t C, int64_t G, gn_dtype dt) {
  if (!dt_ok(dt) || !shape_ok(N, S, C, G) || N == 0 || S == 0) return 0;
  int vpt = 0;
  if (plan_resident(N, S, C, G, (int)dt_size(dt), kBwdMost, &vpt).cs) return (size_t)N * C * 8;
  const GnShape g = plan(N, S, C, G, (int)dt_size(dt), false);
  return up16((size_t)N * g.G * 8) + (size_t)N * g.C * 8 + (size_t)N * (g.chunks + (folds(g) ? 1 : 0)) * g.C * 8;
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
  int vpt = 0;
  Bundle r = plan_resident(N, S, C, G, (int)es, kBwdMost, &vpt);
  if (r.cs) {
    float* chan = dw || db ? static_cast<float*>(ws) : nullptr;
    void* args[] = {&x, &ld_x, &dy, &ld_dy, &w, &b, &mean, &rstd, &r, &dx, &ld_dx, &chan};
    const gn_status st = launch_resident(dt == GN_BF16 ? pick_res<__nv_bfloat16>(false, epi, vpt) : pick_res<float>(false, epi, vpt),
                                         r, N, res_smem(r, (int)es, false), args, s);
    if (st != GN_OK || !chan) return st;
    return launch_colsum(chan, N, 2 * C, C, dw, db, s);
  }
  GnShape g = plan(N, S, C, G, (int)es, false);
  float2* stat = static_cast<float2*>(ws);
  float* chan = reinterpret_cast<float*>(static_cast<char*>(ws) + up16((size_t)N * g.G * 8));
  float2* part = reinterpret_cast<float2*>(chan + (size_t)N * g.C * 2);
  const int64_t blocks = N * g.chunks * g.tiles;
  void* args0[] = {&x, &ld_x, &dy, &ld_dy, &w, &b, &mean, &rstd, &g, &part};
  gn_status st = launch(dt == GN_BF16 ? pick_sums<__nv_bfloat16>(epi) : pick_sums<float>(epi), blocks, args0, s, false);
  if (st != GN_OK) return st;
  GnShape joined = g;
  if (folds(g)) {
    int blocks_n = (int)((C + 31) / 32);
    float2* sums = part + (size_t)N * g.chunks * g.C;
    void* fold[] = {&part, &g, &blocks_n, &sums};
    st = launch((void*)gn_bwd_fold_kernel, N * blocks_n, fold, s, true, 1024);
    if (st != GN_OK) return st;
    part = sums;
    joined.chunks = 1;
  }
  void* args1[] = {&part, &w, &joined, &chan, &stat};
  st = launch(dt == GN_BF16 ? (void*)gn_bwd_join_kernel<__nv_bfloat16> : (void*)gn_bwd_join_kernel<float>, N * G, args1, s,
              true, kJoin);
  if (st != GN_OK) return st;
  void* args2[] = {&x, &ld_x, &dy, &ld_dy, &w, &b, &mean, &rstd, &stat, &g, &dx, &ld_dx};
  st = launch(dt == GN_BF16 ? pick_bwd<__nv_bfloat16>(epi) : pick_bwd<float>(epi), blocks, args2, s, true);
  if (st != GN_OK) return st;
  return launch_colsum(chan, N, 2 * C, C, dw, db, s);
}
