// quant_fp8.cu - 8-bit operands (e4m3) with one fp32 scale for each block of 128 values.
//
// A block of values v is held as codes q and a scale s with v ~ q s:
//   s = max(amax, 2^-110) / 448,  amax = max |v| over the block  (448: the largest e4m3 value),
//   q = e4m3(v / s), the fp32 quotient rounded to nearest even.
// A block that holds a NaN or an infinity gets the scale NaN and NaN codes: whatever reads it sees NaN.
// The floor keeps s a normal number whose reciprocal is finite; an all-zero block has zero codes.
//
// The quotient is the correctly rounded one without a division per value: with i = 1 / s correctly
// rounded once per block, r = v i, then r + (v - r s) i with both steps fused is v / s rounded to
// nearest (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990, theorem on the last step of a division). Ties of bf16 values over a scale
// derived from one of them are common, so a quotient one ulp off would flip codes.
#include "gn_common.cuh"
#include "gn_host.h"

namespace gn {
namespace {

constexpr int kBlk = 128;
constexpr float kE4m3Max = 448.0f;
constexpr float kAmaxFloor = 7.70371978e-34f;  // 2^-110

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float quotient(float v, float s, float i) {
  const float r = v * i;
  return fmaf(fmaf(-r, s, v), i, r);
}

// scale of a block from its largest magnitude (NaN or infinity: NaN); 1 / 448 rounded is 0x3b124925
__device__ __forceinline__ float block_scale(float amax) {
  return amax <= 3.402823466e38f ? quotient(fmaxf(amax, kAmaxFloor), kE4m3Max, 1.0f / kE4m3Max) : __int_as_float(0x7fffffff);
}

// 1 / s: correctly rounded where the quotient has to be, else the hardware's approximation (1 ulp)
template <bool EXACT>
__device__ __forceinline__ float inverse(float s) {
  return EXACT ? __frcp_rn(s) : __fdividef(1.0f, s);
}

// v / s for a value that is itself an fp32 evaluation (EXACT false): one rounding of 1 / s more is no
// more than what v already carries
template <bool EXACT>
__device__ __forceinline__ float scaled(float v, float s, float i) {
  return EXACT ? quotient(v, s, i) : v * i;
}

// two codes, lo in the low byte
__device__ __forceinline__ uint32_t code2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool EXACT>
__device__ __forceinline__ uint32_t code4(const float* v, float s, float i) {
  if constexpr (!EXACT) {
    const float2 lo = mul2(make_float2(v[0], v[1]), dup2(i)), hi = mul2(make_float2(v[2], v[3]), dup2(i));
    return code2(lo.x, lo.y) | code2(hi.x, hi.y) << 16;
  }
  return code2(scaled<EXACT>(v[0], s, i), scaled<EXACT>(v[1], s, i)) |
         code2(scaled<EXACT>(v[2], s, i), scaled<EXACT>(v[3], s, i)) << 16;
}

// The activation and its derivative for values on their way to codes. The hardware tanh (error 2^-11) of
// the bf16 epilogues would move one code in a hundred; on bf16 inputs the exponential and the divide are the
// approximate ones (together about 1e-6), on fp32 inputs the accurate ones.
template <int EPI, bool FAST>
__device__ __forceinline__ float q_act(float z) {
  if constexpr (!FAST || EPI == EPI_NONE) {
    return epi_fwd<EPI, false>(z);
  } else if constexpr (EPI == EPI_SILU) {
    return __fdividef(z, 1.0f + __expf(-z));
  } else {  // z (1 + tanh u) / 2 = z sigmoid(2 u)
    const float u2 = z * fmaf(2.0f * kGeluK * kGeluC, z * z, 2.0f * kGeluK);
    return __fdividef(z, 1.0f + __expf(-u2));
  }
}
template <int EPI, bool FAST>
__device__ __forceinline__ float q_grad(float z) {
  if constexpr (!FAST || EPI == EPI_NONE) {
    return epi_grad<EPI, false>(z);
  } else if constexpr (EPI == EPI_SILU) {
    const float s = __fdividef(1.0f, 1.0f + __expf(-z));
    return s * fmaf(z, 1.0f - s, 1.0f);
  } else {  // with p = sigmoid(2 u): p + z p (1 - p) (2 u)'; 1 - p = a / (1 + a) without cancellation
    const float z2 = z * z;
    const float u2 = z * fmaf(2.0f * kGeluK * kGeluC, z2, 2.0f * kGeluK);
    const float a = __expf(-fabsf(u2));
    const float r = __fdividef(1.0f, 1.0f + a), ra = r * a;
    const float p = u2 >= 0.0f ? r : ra, n = u2 >= 0.0f ? ra : r;
    return p * fmaf(z * n, fmaf(6.0f * kGeluK * kGeluC, z2, 2.0f * kGeluK), 1.0f);
  }
}

// The largest of each of K values over L lanes (K a power of two <= L): every step exchanges the half of the
// values that the partner keeps, so K values take about K + log2(L / K) shuffles, not K log2(L), and leave each
// lane with one value's result, that of index value_of_lane<K, L>(lane). lane_of_value gives a lane of
// this lane's group that holds value k.
template <int K, int L>
__device__ __forceinline__ float group_max(float (&v)[K], int lane) {
  int h = L / 2;
#pragma unroll
  for (int n = K; n > 1; n /= 2, h /= 2) {
    const bool up = lane & h;
#pragma unroll
    for (int j = 0; j < n / 2; ++j) {
      const float keep = up ? v[j + n / 2] : v[j], send = up ? v[j] : v[j + n / 2];
      v[j] = max_nan(keep, __shfl_xor_sync(0xffffffffu, send, h));
    }
  }
  float m = v[0];
#pragma unroll
  for (; h > 0; h /= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, h));
  return m;
}
template <int K, int L>
__device__ __forceinline__ int value_of_lane(int lane) { return (lane & (L - 1)) / (L / K); }
template <int K, int L>
__device__ __forceinline__ int lane_of_value(int lane, int k) { return (lane & ~(L - 1)) | k * (L / K); }

// vector v of a row of n elements (E to a vector), 0 past the end: a predicated load, and the elements of a
// last vector that is not whole
template <typename T>
__device__ __forceinline__ uint4 load_raw(const T* row, int v, int n) {
  constexpr int E = Vec<T>::N;
  uint4 u = make_uint4(0, 0, 0, 0);
  if (v < n / E) {
    u = ld_stream(row + v * E);
  } else if (v * E < n) {
    float f[E];
#pragma unroll
    for (int e = 0; e < E; ++e) f[e] = v * E + e < n ? Vec<T>::load1(row + v * E + e) : 0.0f;
    u = Vec<T>::pack(f);
  }
  return u;
}

// E codes of vector v of a row of n codes
template <int E, bool EXACT>
__device__ __forceinline__ void store_codes(uint8_t* row, int v, int n, const float* f, float s, float i) {
  uint32_t w[E / 4];
#pragma unroll
  for (int k = 0; k < E / 4; ++k) w[k] = code4<EXACT>(f + 4 * k, s, i);
  uint8_t* out = row + v * E;
  if ((v + 1) * E <= n) {
    if constexpr (E == 8) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint32_t*>(out) = w[0];
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (v * E + e < n) out[e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
  }
}

// ---------------------------------------------------------------- norm + quantise, blocks along the row
// The row is read once and stays in registers, VPT vectors a thread: statistics (mean, then centred
// squares), normalise, activate, then each run of 128 / E threads holds a block of 128 values, finds its
// amax with shuffles and writes the codes. A row belongs to the warps of one block (TEAM of blockDim.x
// threads) or, up to 128 vectors, to one warp of eight (TEAM 32, no barrier). Bound by HBM: 3 bytes a
// value in and out for bf16.
template <typename T, int NORM, int EPI, int VPT, bool WARP>
__global__ void __launch_bounds__(WARP ? 256 : VPT == 4 ? 512 : 1024) norm_quant_kernel(const T* __restrict__ x, const T* __restrict__ g,
                                                                       const T* __restrict__ beta,
                                                                       uint8_t* __restrict__ q, float* __restrict__ scale,
                                                                       float* __restrict__ mean, float* __restrict__ rstd,
                                                                       int64_t rows, int hidden, int64_t ldx, int64_t ldq,
                                                                       int64_t lds, float eps, int gemma, int pvec) {
  constexpr int E = Vec<T>::N;
  constexpr int L = kBlk / E;  // threads of a block of values
  constexpr bool FAST = fast_math_for<T>();
  constexpr bool EXACT = NORM == GN_NORM_NONE && EPI == EPI_NONE;
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t m = WARP ? (int64_t)blockIdx.x * 8 + warp : (int64_t)blockIdx.x;
  if (WARP && m >= rows) return;
  const int t = WARP ? lane : threadIdx.x;
  const int team = WARP ? 32 : (int)blockDim.x;
  const T* row = x + m * ldx;
  const bool ragged = (team * VPT) * E != hidden;  // some of the threads' values lie past the row
  uint4 raw[VPT];
  if (hidden % E == 0) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      raw[k] = make_uint4(0, 0, 0, 0);
      if ((t + k * team) * E < hidden) raw[k] = ld_stream(row + (t + k * team) * E);
    }
  } else {
#pragma unroll
    for (int k = 0; k < VPT; ++k) raw[k] = load_raw<T>(row, t + k * team, hidden);
  }
  float f[VPT][E];
#pragma unroll
  for (int k = 0; k < VPT; ++k) Vec<T>::unpack(raw[k], f[k]);
  auto total = [&](float v, int slot) {  // over the row's threads, in a fixed order
    v = group_sum<32>(v);
    if constexpr (!WARP) {
      if (lane == 0) red[slot][warp] = v;
      __syncthreads();
      v = lane < (int)(blockDim.x >> 5) ? red[slot][lane] : 0.0f;
      v = group_sum<32>(v);
    }
    return v;
  };
  float mu = 0.0f, r = 1.0f;
  if constexpr (NORM != GN_NORM_NONE) {
    const float n = (float)hidden;
    float2 acc = make_float2(0.0f, 0.0f);
    if constexpr (NORM == GN_NORM_LN) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int e = 0; e < E; e += 2) acc = add2(acc, make_float2(f[k][e], f[k][e + 1]));
      mu = __fdiv_rn(total(acc.x + acc.y, 0), n);
      acc = make_float2(0.0f, 0.0f);
    }
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
      const int left = hidden - (t + k * team) * E;  // elements of the row from this vector on
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        float2 d = make_float2(f[k][e], f[k][e + 1]);
        if constexpr (NORM == GN_NORM_LN) {
          d = add2(d, dup2(-mu));
          if (ragged) d = make_float2(e < left ? d.x : 0.0f, e + 1 < left ? d.y : 0.0f);
          f[k][e] = d.x, f[k][e + 1] = d.y;
        }
        acc = fma2(d, d, acc);
      }
    }
    r = __frcp_rn(__fsqrt_rn(__fdiv_rn(total(acc.x + acc.y, 1), n) + eps));
    if (t == 0) {
      if (mean && NORM == GN_NORM_LN) mean[m] = mu;
      if (rstd) rstd[m] = r;
    }
  }
  if constexpr (NORM != GN_NORM_NONE) {
    if (pvec && g && (NORM == GN_NORM_RMS || beta)) {  // both parameters, 16 bytes at a time
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        const int v = t + k * team;
        uint4 uw = make_uint4(0, 0, 0, 0), ub = uw;
        if ((v + 1) * E <= hidden) {
          uw = __ldg(reinterpret_cast<const uint4*>(g + v * E));
          if (NORM == GN_NORM_LN) ub = __ldg(reinterpret_cast<const uint4*>(beta + v * E));
        } else if (v * E < hidden) {
          uw = load_raw<T>(g, v, hidden);
          if (NORM == GN_NORM_LN) ub = load_raw<T>(beta, v, hidden);
        }
        float2 w[E / 2], b[E / 2];
        unpack2<T>(uw, w);
        unpack2<T>(ub, b);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) {
          const float2 z = mul2(make_float2(f[k][2 * e], f[k][2 * e + 1]), dup2(r));
          const float2 o = NORM == GN_NORM_LN ? fma2(z, w[e], b[e]) : mul2(z, gemma ? add2(w[e], dup2(1.0f)) : w[e]);
          f[k][2 * e] = o.x, f[k][2 * e + 1] = o.y;
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int c = (t + k * team) * E + e;
          if (c < hidden) {
            const float w = ld_param(g, c, 1.0f) + (NORM == GN_NORM_RMS && gemma ? 1.0f : 0.0f);
            f[k][e] = fmaf(f[k][e] * r, w, NORM == GN_NORM_LN ? ld_param(beta, c, 0.0f) : 0.0f);
          }
        }
    }
  }
  float am[VPT];
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    am[k] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      if constexpr (EPI != EPI_NONE) f[k][e] = q_act<EPI, FAST>(f[k][e]);
      am[k] = max_nan(am[k], fabsf(f[k][e]));
    }
  }
  // each lane makes the scale of one of its group's VPT blocks
  const float s = block_scale(group_max<VPT, L>(am, lane)), i = inverse<EXACT>(s);
  {
    const int v = t + value_of_lane<VPT, L>(lane) * team;
    if (lane % (L / VPT) == 0 && v / L * kBlk < hidden) scale[m * lds + v / L] = s;
  }
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = t + k * team, src = lane_of_value<VPT, L>(lane, k);
    const float ik = __shfl_sync(0xffffffffu, i, src), sk = EXACT ? __shfl_sync(0xffffffffu, s, src) : 0.0f;
    if (v * E < hidden) store_codes<E, EXACT>(q + m * ldq, v, hidden, f[k], sk, ik);
  }
}

// ---------------------------------------------------------------- tiles of 128 x 128
// One block per tile: v = x, or dy * act'(x) (GRAD), read once, 64 values a thread in registers. Warp w
// has the rows 16 w..: for bf16 a thread has 8 consecutive rows (lanes 0-15 the first eight of the warp's
// 16, lanes 16-31 the others) x 8 columns, for fp32 all 16 rows x 4 columns. So a row's block is a run of
// lanes (amax by shuffles, codes stored from registers, 128 bytes a row), and a column's is the warp's
// rows and then the eight warps (shared memory). The transposed codes of a thread are R consecutive bytes
// of each of its columns: they meet in a 16 KiB byte tile (16-byte chunk j of column c at j ^ key(c), so
// that neither side conflicts) and leave as 128-byte runs. Both ways and the bias gradient in one read:
// 6 bytes a value for a bf16 gradient. Bound by HBM.
constexpr int kTileThreads = 256;

struct QuantArgs {
  const void* x;
  const void* dy;
  uint8_t* q;
  float* scale;
  uint8_t* qt;
  float* scale_t;
  float* colsum;
  int64_t rows, cols, ldx, lddy, ldq, lds, ldqt, ldst;
};

template <typename T, int EPI, bool GRAD, bool TILE>
__global__ void __launch_bounds__(kTileThreads, 2) quant_tile_kernel(const QuantArgs a) {
  constexpr int E = Vec<T>::N;
  constexpr int L = kBlk / E;         // lanes of a row: 16 or 32
  constexpr int R = 64 / E;           // rows of a thread: 8 or 16
  constexpr bool FAST = fast_math_for<T>();
  constexpr bool EXACT = !GRAD || EPI == EPI_NONE;
  __shared__ __align__(16) uint8_t bytes[kBlk * kBlk];
  __shared__ float red_max[8][kBlk], red_sum[GRAD ? 8 : 1][kBlk];
  __shared__ __align__(16) float col_scale[kBlk], col_inv[kBlk];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t r0 = (int64_t)blockIdx.y * kBlk, c0 = (int64_t)blockIdx.x * kBlk;
  const int nr = a.rows - r0 < kBlk ? (int)(a.rows - r0) : kBlk;
  const int nc = a.cols - c0 < kBlk ? (int)(a.cols - c0) : kBlk;
  const int lv = lane % L;                          // vector of the row
  const int row0 = 16 * warp + (lane / L) * R;      // first row of the thread
  const T* x = static_cast<const T*>(a.x) + r0 * a.ldx + c0;
  const T* dy = GRAD ? static_cast<const T*>(a.dy) + r0 * a.lddy + c0 : nullptr;
  // whole tiles: every load of the thread is issued before the first value is used
  const bool whole = nr == kBlk && nc == kBlk;
  uint4 raw[R], rawd[GRAD ? R : 1];
  if (whole) {
#pragma unroll
    for (int i = 0; i < R; ++i) raw[i] = ld_stream(x + (row0 + i) * a.ldx + lv * E);
    if constexpr (GRAD) {
#pragma unroll
      for (int i = 0; i < R; ++i) rawd[i] = ld_stream(dy + (row0 + i) * a.lddy + lv * E);
    }
  } else {
#pragma unroll
    for (int i = 0; i < R; ++i) {
      raw[i] = load_raw<T>(x + (row0 + i) * a.ldx, lv, row0 + i < nr ? nc : 0);
      if constexpr (GRAD) rawd[i] = load_raw<T>(dy + (row0 + i) * a.lddy, lv, row0 + i < nr ? nc : 0);
    }
  }
  float f[R][E];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    Vec<T>::unpack(raw[i], f[i]);
    if constexpr (GRAD) {  // past the last row and column z and dy are 0: 0 * act'(0) = 0
      float d[E];
      Vec<T>::unpack(rawd[i], d);
#pragma unroll
      for (int e = 0; e < E; ++e) f[i][e] = d[e] * q_grad<EPI, FAST>(f[i][e]);
    }
  }
  float cmax[E], csum[E];
#pragma unroll
  for (int e = 0; e < E; ++e) cmax[e] = csum[e] = 0.0f;
  float rmax[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    rmax[i] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float m = fabsf(f[i][e]);
      rmax[i] = max_nan(rmax[i], m);
      cmax[e] = max_nan(cmax[e], m);
      if constexpr (GRAD) csum[e] += f[i][e];
    }
  }
  float all = 0.0f;
  if (a.qt || TILE || (GRAD && a.colsum)) {
    if constexpr (L == 16) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        cmax[e] = max_nan(cmax[e], __shfl_xor_sync(0xffffffffu, cmax[e], 16));
        if constexpr (GRAD) csum[e] += __shfl_xor_sync(0xffffffffu, csum[e], 16);
      }
    }
    if (lane < L) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        red_max[warp][lv * E + e] = cmax[e];
        if constexpr (GRAD) red_sum[warp][lv * E + e] = csum[e];
      }
    }
    __syncthreads();
    if constexpr (TILE) {
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max_nan(m, red_max[w][lane + 32 * k]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      all = m;
    } else if (a.qt) {  // a thread per column makes its scale
      if (threadIdx.x < kBlk) {
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = max_nan(m, red_max[w][threadIdx.x]);
        const float s = block_scale(m);
        col_scale[threadIdx.x] = s;
        col_inv[threadIdx.x] = inverse<EXACT>(s);
        if (threadIdx.x < nc) a.scale_t[(c0 + threadIdx.x) * a.ldst + blockIdx.y] = s;
      }
    }
    if constexpr (GRAD) {
      if (a.colsum && threadIdx.x < nc) {
        float t = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) t += red_sum[w][threadIdx.x];
        a.colsum[(int64_t)blockIdx.y * a.cols + c0 + threadIdx.x] = t;
      }
    }
  }
  const float s_all = TILE ? block_scale(all) : 0.0f, i_all = TILE ? inverse<EXACT>(s_all) : 0.0f;
  if (TILE && threadIdx.x == 0) {
    if (a.q) a.scale[(int64_t)blockIdx.y * a.lds + blockIdx.x] = s_all;
    if (a.qt) a.scale_t[(int64_t)blockIdx.x * a.ldst + blockIdx.y] = s_all;
  }
  if (a.q) {
    float s = s_all, inv = i_all;
    if constexpr (!TILE) {  // each lane makes the scale of one of its group's rows
      s = block_scale(group_max<R, L>(rmax, lane));
      inv = inverse<EXACT>(s);
      const int i = row0 + value_of_lane<R, L>(lane);
      if (lane % (L / R) == 0 && i < nr) a.scale[(r0 + i) * a.lds + blockIdx.x] = s;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int src = lane_of_value<R, L>(lane, i);
      const float ii = TILE ? inv : __shfl_sync(0xffffffffu, inv, src);
      const float si = TILE ? s : EXACT ? __shfl_sync(0xffffffffu, s, src) : 0.0f;
      if (row0 + i < nr && lv * E < nc) store_codes<E, EXACT>(a.q + (r0 + row0 + i) * a.ldq + c0, lv, nc, f[i], si, ii);
    }
  }
  if (!a.qt) return;
  if constexpr (!TILE) __syncthreads();  // the columns' scales
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int c = lv * E + e;
    const float s = TILE ? s_all : EXACT ? col_scale[c] : 0.0f, inv = TILE ? i_all : col_inv[c];
    uint32_t w[R / 4];
#pragma unroll
    for (int k = 0; k < R / 4; ++k) {
      const float v[4] = {f[4 * k][e], f[4 * k + 1][e], f[4 * k + 2][e], f[4 * k + 3][e]};
      w[k] = code4<EXACT>(v, s, inv);
    }
    uint8_t* at = bytes + c * kBlk + ((warp ^ (lv & 7)) << 4);
    if constexpr (R == 8) *reinterpret_cast<uint2*>(at + 8 * (lane / L)) = make_uint2(w[0], w[1]);
    else *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __syncthreads();
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int idx = it * kTileThreads + threadIdx.x, c = idx >> 3, j = idx & 7;
    if (c >= nc || 16 * j >= nr) continue;
    const uint4 v = *reinterpret_cast<const uint4*>(bytes + c * kBlk + ((j ^ ((c / E) & 7)) << 4));
    uint8_t* out = a.qt + (c0 + c) * a.ldqt + r0 + 16 * j;
    if (16 * j + 16 <= nr) {
      *reinterpret_cast<uint4*>(out) = v;
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if (16 * j + k < nr) out[k] = (uint8_t)(w[k / 4] >> (8 * (k % 4)));
    }
  }
}

// ---------------------------------------------------------------- host side

// variants of the row kernel: 0-2: one warp per row, 1, 2 or 4 vectors a lane; 3, 4: one block per row, 1
// or 4 vectors a thread
template <typename T, int NORM, int EPI>
void* pick_norm_shape(int shape) {
  return shape == 0   ? (void*)norm_quant_kernel<T, NORM, EPI, 1, true>
         : shape == 1 ? (void*)norm_quant_kernel<T, NORM, EPI, 2, true>
         : shape == 2 ? (void*)norm_quant_kernel<T, NORM, EPI, 4, true>
         : shape == 3 ? (void*)norm_quant_kernel<T, NORM, EPI, 1, false>
                      : (void*)norm_quant_kernel<T, NORM, EPI, 4, false>;
}
template <typename T, int NORM>
void* pick_norm_epi(int epi, int shape) {
  return epi == GN_EPI_GELU_TANH ? pick_norm_shape<T, NORM, EPI_GELU_TANH>(shape)
         : epi == GN_EPI_SILU    ? pick_norm_shape<T, NORM, EPI_SILU>(shape)
                                 : pick_norm_shape<T, NORM, EPI_NONE>(shape);
}
template <typename T>
void* pick_norm(int norm, int epi, int shape) {
  return norm == GN_NORM_LN    ? pick_norm_epi<T, GN_NORM_LN>(epi, shape)
         : norm == GN_NORM_RMS ? pick_norm_epi<T, GN_NORM_RMS>(epi, shape)
                               : pick_norm_epi<T, GN_NORM_NONE>(epi, shape);
}
template <typename T>
void* pick_tile(int epi, bool grad, bool tile) {
  if (!grad) return tile ? (void*)quant_tile_kernel<T, EPI_NONE, false, true> : (void*)quant_tile_kernel<T, EPI_NONE, false, false>;
  return epi == GN_EPI_GELU_TANH ? (void*)quant_tile_kernel<T, EPI_GELU_TANH, true, false>
         : epi == GN_EPI_SILU    ? (void*)quant_tile_kernel<T, EPI_SILU, true, false>
                                 : (void*)quant_tile_kernel<T, EPI_NONE, true, false>;
}

int64_t blocks_of(int64_t n) { return (n + kBlk - 1) / kBlk; }

}  // namespace
}  // namespace gn

using namespace gn;

extern "C" gn_status gn_norm_quant_fp8(const void* x, const void* g, const void* beta, void* q, float* scale,
                                       float* mean, float* rstd, int64_t rows, int64_t hidden, int64_t ld_x,
                                       int64_t ld_q, int64_t ld_s, float eps, gn_norm norm, int gemma,
                                       gn_epilogue epi, gn_dtype dt, void* stream) {
  if (!dt_ok(dt) || !epi_ok(epi)) return GN_ERR_DTYPE;
  if (norm != GN_NORM_RMS && norm != GN_NORM_LN && norm != GN_NORM_NONE) return GN_ERR_SHAPE;
  if (rows < 0 || hidden <= 0 || rows > INT32_MAX || ld_x < hidden || ld_q < hidden || ld_s < blocks_of(hidden))
    return GN_ERR_SHAPE;
  if (hidden > (dt == GN_BF16 ? 16384 : 8192)) return GN_ERR_UNSUPPORTED;
  if (rows == 0) return GN_OK;
  if (!x || !q || !scale) return GN_ERR_NULL;
  if (!aligned16(x) || !aligned16(q) || ld_x * dt_size(dt) % 16 || ld_q % 16) return GN_ERR_ALIGN;
  int pvec = (!g || aligned16(g)) && (!beta || aligned16(beta));  // parameters read 16 bytes at a time
  const int e = (int)(16 / dt_size(dt));
  const int nvec = (int)((hidden + e - 1) / e);
  // up to 128 vectors: a warp per row; above, a block per row with four vectors a thread, or one while
  // the rows do not fill the SMs anyway and the latency of a row counts
  int shape, threads = 256;
  int64_t blocks = (rows + 7) / 8;
  if (nvec <= 128 && (rows > sm_count() || nvec <= 32)) {
    shape = nvec <= 32 ? 0 : nvec <= 64 ? 1 : 2;
  } else {
    shape = nvec <= 1024 && rows <= sm_count() ? 3 : 4;
    const int per = shape == 3 ? 1 : 4;
    threads = ((nvec + per - 1) / per + 31) / 32 * 32;
    blocks = rows;
  }
  void* kern = dt == GN_BF16 ? pick_norm<__nv_bfloat16>(norm, epi, shape) : pick_norm<float>(norm, epi, shape);
  int h = (int)hidden;
  void* args[] = {&x, &g, &beta, &q, &scale, &mean, &rstd, &rows, &h, &ld_x, &ld_q, &ld_s, &eps, &gemma, &pvec};
  if (!kernel_attrs(kern, 0)) return GN_ERR_CUDA;
  if (cudaLaunchKernel(kern, dim3((unsigned)blocks), dim3((unsigned)threads), args, 0, (cudaStream_t)stream) != cudaSuccess)
    return GN_ERR_CUDA;
  count_launches(1);
  return launch_status();
}

extern "C" size_t gn_quant_fp8_workspace(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0) return 0;
  return (size_t)blocks_of(rows) * cols * 4;
}

extern "C" gn_status gn_quant_fp8(const void* x, const void* dy, void* q, float* scale, void* qt, float* scale_t,
                                  float* db, void* ws, size_t ws_bytes, int64_t rows, int64_t cols, int64_t ld_x,
                                  int64_t ld_dy, int64_t ld_q, int64_t ld_s, int64_t ld_qt, int64_t ld_st,
                                  gn_fp8_block block, gn_epilogue epi, gn_dtype dt, void* stream) {
  if (!dt_ok(dt) || !epi_ok(epi)) return GN_ERR_DTYPE;
  const bool tile = block == GN_FP8_TILE;
  if (block != GN_FP8_VEC && block != GN_FP8_TILE) return GN_ERR_SHAPE;
  if (rows < 0 || cols <= 0 || rows > 65535ll * kBlk || cols > INT32_MAX || ld_x < cols || (dy && ld_dy < cols)) return GN_ERR_SHAPE;
  if (q && (ld_q < cols || ld_s < blocks_of(cols))) return GN_ERR_SHAPE;
  if (qt && (ld_qt < rows || ld_st < blocks_of(rows))) return GN_ERR_SHAPE;
  if ((tile && dy) || (!dy && epi != GN_EPI_NONE)) return GN_ERR_UNSUPPORTED;
  cudaStream_t s = (cudaStream_t)stream;
  if (rows == 0) {
    if (db && cudaMemsetAsync(db, 0, (size_t)cols * 4, s) != cudaSuccess) return GN_ERR_CUDA;
    return GN_OK;
  }
  if (!x || (!q && !qt) || (q && !scale) || (qt && !scale_t)) return GN_ERR_NULL;
  if (!aligned16(x) || ld_x * dt_size(dt) % 16 || (dy && (!aligned16(dy) || ld_dy * dt_size(dt) % 16))) return GN_ERR_ALIGN;
  if ((q && (!aligned16(q) || ld_q % 16)) || (qt && (!aligned16(qt) || ld_qt % 16))) return GN_ERR_ALIGN;
  if (db && (!ws || ws_bytes < gn_quant_fp8_workspace(rows, cols))) return GN_ERR_WORKSPACE;
  if (db && !aligned16(ws)) return GN_ERR_ALIGN;
  QuantArgs a{x, dy, static_cast<uint8_t*>(q), scale, static_cast<uint8_t*>(qt), scale_t,
              db ? static_cast<float*>(ws) : nullptr, rows, cols, ld_x, ld_dy, ld_q, ld_s, ld_qt, ld_st};
  void* kern = dt == GN_BF16 ? pick_tile<__nv_bfloat16>(epi, dy != nullptr, tile) : pick_tile<float>(epi, dy != nullptr, tile);
  if (!kernel_attrs(kern, 0)) return GN_ERR_CUDA;
  void* args[] = {&a};
  if (cudaLaunchKernel(kern, dim3((unsigned)blocks_of(cols), (unsigned)blocks_of(rows)), dim3(kTileThreads), args, 0,
                       s) != cudaSuccess)
    return GN_ERR_CUDA;
  count_launches(1);
  const gn_status st = launch_status();
  if (st != GN_OK || !db) return st;
  return launch_colsum(a.colsum, blocks_of(rows), cols, cols, db, nullptr, s);
}
