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

// scale of a block from its largest magnitude (NaN or infinity: NaN)
__device__ __forceinline__ float block_scale(float amax) {
  return amax <= 3.402823466e38f ? __fdiv_rn(fmaxf(amax, kAmaxFloor), kE4m3Max) : __int_as_float(0x7fffffff);
}

__device__ __forceinline__ float quotient(float v, float s, float i) {
  const float r = v * i;
  return fmaf(fmaf(-r, s, v), i, r);
}

// two codes, lo in the low byte
__device__ __forceinline__ uint32_t code2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- norm + quantise, row blocks
// One block per row: statistics (mean, then centred squares), then each run of 128 / E threads takes
// a 128-value block of the row.
constexpr int kRowThreads = 256;

__device__ __forceinline__ float row_sum(float v, float* red) {
  v = group_sum<32>(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < kRowThreads / 32; ++i) t += red[i];
  return t;
}

template <typename T, int NORM, int EPI>
__global__ void __launch_bounds__(kRowThreads) norm_quant_kernel(const T* __restrict__ x, const T* __restrict__ g,
                                                                 const T* __restrict__ beta, uint8_t* __restrict__ q,
                                                                 float* __restrict__ scale, float* __restrict__ mean,
                                                                 float* __restrict__ rstd, int hidden, int64_t ldx,
                                                                 int64_t ldq, int64_t lds, float eps, int gemma) {
  constexpr int E = Vec<T>::N;
  constexpr int L = kBlk / E;  // threads of a block of values
  __shared__ float red[kRowThreads / 32];
  const int64_t m = blockIdx.x;
  const T* row = x + m * ldx;
  const int nvec = (hidden + E - 1) / E;
  auto load = [&](int v, float (&f)[E]) {
    if ((v + 1) * E <= hidden) {
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(row + v * E), f);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) f[e] = v * E + e < hidden ? Vec<T>::load1(row + v * E + e) : 0.0f;
    }
  };
  float mu = 0.0f, r = 1.0f;
  if (NORM != GN_NORM_NONE) {
    const float inv = 1.0f / (float)hidden;
    if (NORM == GN_NORM_LN) {
      float t = 0.0f;
      for (int v = threadIdx.x; v < nvec; v += kRowThreads) {
        float f[E];
        load(v, f);
#pragma unroll
        for (int e = 0; e < E; ++e) t += f[e];
      }
      mu = row_sum(t, red) * inv;
    }
    float t = 0.0f;
    for (int v = threadIdx.x; v < nvec; v += kRowThreads) {
      float f[E];
      load(v, f);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = v * E + e < hidden ? f[e] - mu : 0.0f;
        t = fmaf(d, d, t);
      }
    }
    r = 1.0f / sqrtf(fmaf(row_sum(t, red), inv, eps));
    if (threadIdx.x == 0) {
      if (mean && NORM == GN_NORM_LN) mean[m] = mu;
      if (rstd) rstd[m] = r;
    }
  }
  for (int v0 = 0; v0 < nvec; v0 += kRowThreads) {
    const int v = v0 + threadIdx.x;
    float f[E];
    float amax = 0.0f;
    if (v < nvec) {
      load(v, f);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = v * E + e;
        float z = f[e];
        if (c >= hidden) {
          z = 0.0f;
        } else {
          if (NORM == GN_NORM_LN) z = fmaf((z - mu) * r, ld_param(g, c, 1.0f), ld_param(beta, c, 0.0f));
          if (NORM == GN_NORM_RMS) z = z * r * (ld_param(g, c, 1.0f) + (gemma ? 1.0f : 0.0f));
          z = epi_fwd<EPI, false>(z);
        }
        f[e] = z;
        amax = max_nan(amax, fabsf(z));
      }
    }
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (v >= nvec) continue;
    const float s = block_scale(amax), i = __frcp_rn(s);
    if (v % L == 0) scale[m * lds + v / L] = s;
    uint8_t* out = q + m * ldq + (int64_t)v * E;
    uint32_t w[E / 4];
#pragma unroll
    for (int k = 0; k < E / 4; ++k)
      w[k] = code2(quotient(f[4 * k], s, i), quotient(f[4 * k + 1], s, i)) |
             code2(quotient(f[4 * k + 2], s, i), quotient(f[4 * k + 3], s, i)) << 16;
    if ((v + 1) * E <= hidden) {
      if constexpr (E == 8) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t*>(out) = w[0];
    } else {
      for (int e = 0; v * E + e < hidden; ++e) out[e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
    }
  }
}

// ---------------------------------------------------------------- tiles of 128 x 128
// One block per tile: v = x, or dy * act'(x) (GRAD). q / scale get the tile by rows, qt / scale_t its
// transpose; blocks of 128 values along a row (VEC) or of the whole tile (GN_FP8_TILE). colsum, when
// given, gets the tile's column sums (row tile blockIdx.y of a [row tiles, cols] matrix).
constexpr int kTileThreads = 256;
constexpr int kTileLd = kBlk + 1;

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
__global__ void __launch_bounds__(kTileThreads) quant_tile_kernel(const QuantArgs a) {
  extern __shared__ float tile[];  // [128][kTileLd]
  __shared__ float amax_r[kBlk], amax_c[kBlk];
  const int64_t r0 = (int64_t)blockIdx.y * kBlk, c0 = (int64_t)blockIdx.x * kBlk;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dy);
  for (int i = threadIdx.x; i < kBlk * kBlk; i += kTileThreads) {
    const int r = i / kBlk, c = i % kBlk;
    float v = 0.0f;
    if (r0 + r < a.rows && c0 + c < a.cols) {
      v = Vec<T>::load1(x + (r0 + r) * a.ldx + c0 + c);
      if constexpr (GRAD) v = Vec<T>::load1(dy + (r0 + r) * a.lddy + c0 + c) * epi_grad<EPI, false>(v);
    }
    tile[r * kTileLd + c] = v;
  }
  __syncthreads();
  {
    const int k = threadIdx.x % kBlk;
    float m = 0.0f;
    if (threadIdx.x < kBlk) {
      for (int c = 0; c < kBlk; ++c) m = max_nan(m, fabsf(tile[k * kTileLd + c]));
      amax_r[k] = m;
    } else {
      float t = 0.0f;
      for (int r = 0; r < kBlk; ++r) {
        m = max_nan(m, fabsf(tile[r * kTileLd + k]));
        t += tile[r * kTileLd + k];
      }
      amax_c[k] = m;
      if (a.colsum && c0 + k < a.cols) a.colsum[(int64_t)blockIdx.y * a.cols + c0 + k] = t;
    }
  }
  __syncthreads();
  float all = 0.0f;
  if constexpr (TILE)
    for (int k = 0; k < kBlk; ++k) all = max_nan(all, amax_r[k]);
  for (int i = threadIdx.x; i < kBlk * kBlk; i += kTileThreads) {
    const int u = i / kBlk, k = i % kBlk;
    if (a.q && r0 + u < a.rows && c0 + k < a.cols) {
      const float s = block_scale(TILE ? all : amax_r[u]);
      a.q[(r0 + u) * a.ldq + c0 + k] = (uint8_t)code2(quotient(tile[u * kTileLd + k], s, __frcp_rn(s)), 0.0f);
      if (!TILE && k == 0) a.scale[(r0 + u) * a.lds + blockIdx.x] = s;
    }
    if (a.qt && c0 + u < a.cols && r0 + k < a.rows) {
      const float s = block_scale(TILE ? all : amax_c[u]);
      a.qt[(c0 + u) * a.ldqt + r0 + k] = (uint8_t)code2(quotient(tile[k * kTileLd + u], s, __frcp_rn(s)), 0.0f);
      if (!TILE && k == 0) a.scale_t[(c0 + u) * a.ldst + blockIdx.y] = s;
    }
  }
  if (TILE && threadIdx.x == 0) {
    const float s = block_scale(all);
    if (a.q) a.scale[(int64_t)blockIdx.y * a.lds + blockIdx.x] = s;
    if (a.qt) a.scale_t[(int64_t)blockIdx.x * a.ldst + blockIdx.y] = s;
  }
}

// ---------------------------------------------------------------- host side

template <typename T, int NORM>
void* pick_norm(int epi) {
  return epi == GN_EPI_GELU_TANH ? (void*)norm_quant_kernel<T, NORM, EPI_GELU_TANH>
         : epi == GN_EPI_SILU    ? (void*)norm_quant_kernel<T, NORM, EPI_SILU>
                                 : (void*)norm_quant_kernel<T, NORM, EPI_NONE>;
}
template <typename T>
void* pick_norm(int norm, int epi) {
  return norm == GN_NORM_LN    ? pick_norm<T, GN_NORM_LN>(epi)
         : norm == GN_NORM_RMS ? pick_norm<T, GN_NORM_RMS>(epi)
                               : pick_norm<T, GN_NORM_NONE>(epi);
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
  void* kern = dt == GN_BF16 ? pick_norm<__nv_bfloat16>(norm, epi) : pick_norm<float>(norm, epi);
  int h = (int)hidden;
  void* args[] = {&x, &g, &beta, &q, &scale, &mean, &rstd, &h, &ld_x, &ld_q, &ld_s, &eps, &gemma};
  if (!kernel_attrs(kern, 0)) return GN_ERR_CUDA;
  if (cudaLaunchKernel(kern, dim3((unsigned)rows), dim3(kRowThreads), args, 0, (cudaStream_t)stream) != cudaSuccess)
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
  const size_t smem = (size_t)kBlk * kTileLd * 4;
  if (!kernel_attrs(kern, smem)) return GN_ERR_CUDA;
  void* args[] = {&a};
  if (cudaLaunchKernel(kern, dim3((unsigned)blocks_of(cols), (unsigned)blocks_of(rows)), dim3(kTileThreads), args, smem,
                       s) != cudaSuccess)
    return GN_ERR_CUDA;
  count_launches(1);
  const gn_status st = launch_status();
  if (st != GN_OK || !db) return st;
  return launch_colsum(a.colsum, blocks_of(rows), cols, cols, db, nullptr, s);
}
