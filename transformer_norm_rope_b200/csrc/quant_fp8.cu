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
#include <type_traits>

#include "act_pairs.cuh"
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

// 1 / sqrt(v), rounded twice. One per row or block: next to a value's own roundings the hardware's
// approximations (2 ulp for all of a row) would move two to three times as many codes.
__device__ __forceinline__ float inverse_root(float v) { return __frcp_rn(__fsqrt_rn(v)); }

// two codes, lo in the low byte
__device__ __forceinline__ uint32_t code2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// four codes of v / s, i = 1 / s: the quotient on pairs. (v i alone saves an instruction a value and moves
// two to three times as many codes: 112 us against 121 at 32760 x 5120.)
__device__ __forceinline__ uint32_t code4(const float* v, float s, float i) {
  const float2 a = make_float2(v[0], v[1]), b = make_float2(v[2], v[3]), ii = dup2(i);
  float2 lo = mul2(a, ii), hi = mul2(b, ii);
  const float2 ns = dup2(-s);
  lo = fma2(fma2(lo, ns, a), ii, lo);
  hi = fma2(fma2(hi, ns, b), ii, hi);
  return code2(lo.x, lo.y) | code2(hi.x, hi.y) << 16;
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
template <int E>
__device__ __forceinline__ void store_codes(uint8_t* row, int v, int n, const float* f, float s, float i) {
  uint32_t w[E / 4];
#pragma unroll
  for (int k = 0; k < E / 4; ++k) w[k] = code4(f + 4 * k, s, i);
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
// The row is read once from HBM: statistics, then normalise, activate, and each run of 128 / E lanes holds a
// block of 128 values, finds its amax with shuffles and writes the codes. Bound by HBM (3 bytes a value in
// and out for bf16) only if the instructions stay near ten a value, so what a row costs once should be
// paid by few threads:
//   * norm_quant_warp_kernel, rows of up to 128 vectors: one warp per row, 1, 2 or 4 vectors a lane in
//     registers;
//   * norm_quant_stage_kernel, rows of up to 1024 vectors: one warp per row, which a bulk copy brings to the
//     warp's own stage in shared memory; the warp reads it there once for the statistics and once for the
//     codes, so that few registers and twenty warps suffice. At 32760 x 5120 bf16 LayerNorm: a row in the
//     registers of 160 threads 169 us, in those of one warp (12 warps an SM) 154 us, so: 110 us (RMSNorm 94, no norm 89);
//   * norm_quant_row_kernel: one block per row, for longer rows and while there are too few rows to fill
//     the SMs, where a row's latency counts.
constexpr int kWarpRows = 16;

// the packed vectors are unpacked again after this, not kept unpacked in twice the registers
template <int N>
__device__ __forceinline__ void keep_packed(uint4 (&u)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+r"(u[k].x), "+r"(u[k].y), "+r"(u[k].z), "+r"(u[k].w));
}

template <typename T, int NORM, int EPI, int VPT>
__global__ void __launch_bounds__(32 * kWarpRows, 2)
    norm_quant_warp_kernel(const T* __restrict__ x, const T* __restrict__ g, const T* __restrict__ beta,
                           uint8_t* __restrict__ q, float* __restrict__ scale, float* __restrict__ mean,
                           float* __restrict__ rstd, int64_t rows, int hidden, int64_t ldx, int64_t ldq, int64_t lds,
                           float eps, int gemma) {
  constexpr int E = Vec<T>::N, H = E / 2;
  constexpr int L = kBlk / E;  // lanes of a block of values
  constexpr bool FAST = fast_math_for<T>();
  constexpr int kGroup = VPT;  // vectors whose scales are made together
  static_assert(VPT == 1 || VPT == 2 || VPT == 4, "a power of two");
  extern __shared__ __align__(16) uint4 params[];  // [1 or 2][32 VPT] vectors: weight, bias
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if constexpr (NORM != GN_NORM_NONE) {
    for (int v = threadIdx.x; v < 32 * VPT; v += 32 * kWarpRows) {
      float w[E], b[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        w[e] = v * E + e < hidden ? ld_param(g, v * E + e, 1.0f) : 0.0f;
        b[e] = NORM == GN_NORM_LN && v * E + e < hidden ? ld_param(beta, v * E + e, 0.0f) : 0.0f;
      }
      params[v] = Vec<T>::pack(w);
      if (NORM == GN_NORM_LN) params[32 * VPT + v] = Vec<T>::pack(b);
    }
    __syncthreads();
  }
  const float inv_n = 1.0f / (float)hidden;
  const float2 gem = dup2(NORM == GN_NORM_RMS && gemma ? 1.0f : 0.0f);
  const bool aligned = hidden % E == 0, full = hidden == 32 * VPT * E;
  for (int64_t m = (int64_t)blockIdx.x * kWarpRows + warp; m < rows; m += (int64_t)gridDim.x * kWarpRows) {
    const T* row = x + m * ldx;
    uint4 raw[VPT];
    if (aligned) {
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        raw[k] = make_uint4(0, 0, 0, 0);
        if ((lane + 32 * k) * E < hidden) raw[k] = ld_stream(row + (lane + 32 * k) * E);
      }
    } else {
#pragma unroll
      for (int k = 0; k < VPT; ++k) raw[k] = load_raw<T>(row, lane + 32 * k, hidden);
    }
    float mu = 0.0f, r = 1.0f;
    if constexpr (NORM == GN_NORM_RMS) {
      float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float2 f[H];
        unpack2<T>(raw[k], f);
#pragma unroll
        for (int e = 0; e < H; ++e) acc = fma2(f[e], f[e], acc);
      }
      r = inverse_root(fmaf(group_sum<32>(acc.x + acc.y), inv_n, eps));
    } else if constexpr (NORM == GN_NORM_LN) {
      float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < VPT; ++k) {
        float2 f[H];
        unpack2<T>(raw[k], f);
#pragma unroll
        for (int e = 0; e < H; ++e) acc = add2(acc, f[e]);
      }
      mu = group_sum<32>(acc.x + acc.y) * inv_n;
      acc = make_float2(0.0f, 0.0f);
      keep_packed(raw);
      if (full) {
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          float2 f[H];
          unpack2<T>(raw[k], f);
#pragma unroll
          for (int e = 0; e < H; ++e) {
            const float2 d = add2(f[e], dup2(-mu));
            acc = fma2(d, d, acc);
          }
        }
      } else {  // some of the lanes' values lie past the row
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
          float2 f[H];
          unpack2<T>(raw[k], f);
          const int left = hidden - (lane + 32 * k) * E;  // elements of the row from this vector on
#pragma unroll
          for (int e = 0; e < H; ++e) {
            const float2 d = add2(f[e], dup2(-mu));
            acc = fma2(d, make_float2(2 * e < left ? d.x : 0.0f, 2 * e + 1 < left ? d.y : 0.0f), acc);
          }
        }
      }
      r = inverse_root(fmaf(group_sum<32>(acc.x + acc.y), inv_n, eps));
    }
    if constexpr (NORM != GN_NORM_NONE) {
      keep_packed(raw);
      if (lane == 0) {
        if (mean && NORM == GN_NORM_LN) mean[m] = mu;
        if (rstd) rstd[m] = r;
      }
    }
#pragma unroll
    for (int k0 = 0; k0 < VPT; k0 += kGroup) {
      if (32 * k0 * E >= hidden) break;
      float f[kGroup][E];
      float am[kGroup];
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        const int v = lane + 32 * (k0 + j);
        float2 z[H];
        unpack2<T>(raw[k0 + j], z);
        if constexpr (NORM != GN_NORM_NONE) {
          float2 w[H], b[H];
          unpack2<T>(params[v], w);
          if constexpr (NORM == GN_NORM_LN) unpack2<T>(params[32 * VPT + v], b);
#pragma unroll
          for (int e = 0; e < H; ++e) {
            if constexpr (NORM == GN_NORM_LN) z[e] = fma2(mul2(add2(z[e], dup2(-mu)), dup2(r)), w[e], b[e]);
            else z[e] = mul2(mul2(z[e], dup2(r)), add2(w[e], gem));
          }
        }
        am[j] = 0.0f;
#pragma unroll
        for (int e = 0; e < H; ++e) {
          if constexpr (EPI != EPI_NONE) z[e] = act_pair<EPI, FAST>(z[e]);
          f[j][2 * e] = z[e].x, f[j][2 * e + 1] = z[e].y;
          am[j] = max_nan(am[j], max_nan(fabsf(f[j][2 * e]), fabsf(f[j][2 * e + 1])));
        }
      }
      // each lane makes the scale of one of its group's blocks
      const float s = block_scale(group_max<kGroup, L>(am, lane)), i = __frcp_rn(s);
      const int vs = lane + 32 * (k0 + value_of_lane<kGroup, L>(lane));
      if (lane % (L / kGroup) == 0 && vs / L * kBlk < hidden) scale[m * lds + vs / L] = s;
#pragma unroll
      for (int j = 0; j < kGroup; ++j) {
        const int v = lane + 32 * (k0 + j), src = lane_of_value<kGroup, L>(lane, j);
        const float ij = __shfl_sync(0xffffffffu, i, src), sj = __shfl_sync(0xffffffffu, s, src);
        if (v * E < hidden) store_codes<E>(q + m * ldq, v, hidden, f[j], sj, ij);
      }
    }
  }
}

constexpr int kStageWarps = 20;

template <typename T, int NORM, int EPI>
__global__ void __launch_bounds__(32 * kStageWarps, 1)
    norm_quant_stage_kernel(const T* __restrict__ x, const T* __restrict__ g, const T* __restrict__ beta,
                            uint8_t* __restrict__ q, float* __restrict__ scale, float* __restrict__ mean,
                            float* __restrict__ rstd, int64_t rows, int hidden, int64_t ldx, int64_t ldq, int64_t lds,
                            float eps, int gemma, int slot, unsigned* err) {
  constexpr int E = Vec<T>::N, H = E / 2;
  constexpr int L = kBlk / E;  // lanes of a block of values
  constexpr bool FAST = fast_math_for<T>();
  constexpr int kParams = NORM == GN_NORM_LN ? 2 : NORM == GN_NORM_RMS ? 1 : 0;
  // the parameters, `slot` vectors each, then a row per warp
  extern __shared__ __align__(16) uint4 smem_rows[];
  __shared__ uint64_t bars[kStageWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = (int)(blockDim.x >> 5);
  uint4* params = smem_rows;
  uint4* stage = smem_rows + slot * (kParams + warp);
  uint64_t* bar = &bars[warp];
  const int nfull = hidden / E, nvec = (hidden + E - 1) / E;
  const int kfull = nfull / 32;  // rounds of 32 vectors in which every lane has a whole one
  const uint32_t bulk = (uint32_t)nfull * 16u;
  const int64_t step = (int64_t)gridDim.x * warps;
  const int64_t first = (int64_t)blockIdx.x * warps + warp;
  if (lane == 0) {
    mbar_init(bar, 1);
    mbar_fence_init();
    if (first < rows) {
      mbar_expect_tx(bar, bulk);
      bulk_g2s(stage, x + first * ldx, bulk, bar);
    }
  }
  if constexpr (kParams > 0) {
    for (int v = threadIdx.x; v < slot; v += (int)blockDim.x) {
      float w[E], b[E];
#pragma unroll
      for (int e = 0; e < E; ++e) {
        w[e] = v * E + e < hidden ? ld_param(g, v * E + e, 1.0f) : 0.0f;
        b[e] = NORM == GN_NORM_LN && v * E + e < hidden ? ld_param(beta, v * E + e, 0.0f) : 0.0f;
      }
      params[v] = Vec<T>::pack(w);
      if (NORM == GN_NORM_LN) params[slot + v] = Vec<T>::pack(b);
    }
  }
  __syncthreads();
  const float inv_n = 1.0f / (float)hidden;
  const float2 gem = dup2(NORM == GN_NORM_RMS && gemma ? 1.0f : 0.0f);
  uint32_t ph = 0;
  for (int64_t m = first; m < rows; m += step) {
    if (!__all_sync(0xffffffffu, mbar_wait(bar, ph, err))) {
      (void)mbar_wait(bar, ph, err);  // the copy gets a second limit to land before the warp leaves
      return;
    }
    ph ^= 1u;
    if (nvec > nfull) {  // the last vector is not whole: copied by value, zeros behind the row
      if (lane == (nfull & 31)) stage[nfull] = load_raw<T>(x + m * ldx, nfull, hidden);
      __syncwarp();
    }
    float mu = 0.0f, r = 1.0f;
    if constexpr (NORM == GN_NORM_RMS) {
      float2 acc = make_float2(0.0f, 0.0f);
#pragma unroll 4
      for (int v = lane; v < nvec; v += 32) {
        float2 f[H];
        unpack2<T>(stage[v], f);
#pragma unroll
        for (int e = 0; e < H; ++e) acc = fma2(f[e], f[e], acc);
      }
      r = inverse_root(fmaf(group_sum<32>(acc.x + acc.y), inv_n, eps));
    }
    if constexpr (NORM == GN_NORM_LN) {
      // sums of x - K and (x - K)^2 for a K near the mean (that of the row's first 32 vectors): mean
      // = K + d, var = mean((x - K)^2) - d^2, which loses at most three bits while d^2 <= 4 var; a row whose
      // beginning is further off than that gets a second pass around its mean
      auto sums = [&](float k, float2& s1, float2& s2) {
        s1 = s2 = make_float2(0.0f, 0.0f);
        const float2 nk = dup2(-k);
#pragma unroll 4
        for (int j = 0; j < kfull; ++j) {
          float2 f[H];
          unpack2<T>(stage[lane + 32 * j], f);
#pragma unroll
          for (int e = 0; e < H; ++e) {
            const float2 d = add2(f[e], nk);
            s1 = add2(s1, d);
            s2 = fma2(d, d, s2);
          }
        }
        const int v = lane + 32 * kfull;
        if (v < nvec) {
          float2 f[H];
          unpack2<T>(stage[v], f);
          const int left = hidden - v * E;
#pragma unroll
          for (int e = 0; e < H; ++e) {
            const float2 t = add2(f[e], nk);
            const float2 d = make_float2(2 * e < left ? t.x : 0.0f, 2 * e + 1 < left ? t.y : 0.0f);
            s1 = add2(s1, d);
            s2 = fma2(d, d, s2);
          }
        }
      };
      float2 f[H], t = make_float2(0.0f, 0.0f);  // (nvec > 128: the first 32 vectors are whole)
      unpack2<T>(stage[lane], f);
#pragma unroll
      for (int e = 0; e < H; ++e) t = add2(t, f[e]);
      // K of a bf16 row has a bf16's bits: then x - K is exact. Its discarded bits would be K's own, the same for all
      // values of one binade, and add up in the mean (off by 1.05e-7 of it over 32760 rows so, 5e-8 rounded)
      auto near = [](float v) { return sizeof(T) == 2 ? __bfloat162float(__float2bfloat16_rn(v)) : v; };
      float k = near(group_sum<32>(t.x + t.y) * (1.0f / (32 * E)));
      float2 s1, s2;
      sums(k, s1, s2);
      float d = group_sum<32>(s1.x + s1.y) * inv_n;
      float var = fmaf(-d, d, group_sum<32>(s2.x + s2.y) * inv_n);
      if (!(d * d <= 4.0f * var)) {  // uniform over the warp
        k = near(k + d);
        sums(k, s1, s2);
        d = group_sum<32>(s1.x + s1.y) * inv_n;
        var = fmaf(-d, d, group_sum<32>(s2.x + s2.y) * inv_n);
      }
      mu = k + d;
      r = inverse_root((var < 0.0f ? 0.0f : var) + eps);
    }
    if constexpr (NORM != GN_NORM_NONE) {
      if (lane == 0) {
        if (mean && NORM == GN_NORM_LN) mean[m] = mu;
        if (rstd) rstd[m] = r;
      }
    }
    uint8_t* qrow = q + m * ldq;
    auto four = [&](int k0, auto checked) {  // vectors lane + 32 (k0 .. k0 + 3)
      constexpr bool CHECK = decltype(checked)::value;
      float f[4][E], am[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = lane + 32 * (k0 + j);
        am[j] = 0.0f;
        if (CHECK && v >= nvec) {
#pragma unroll
          for (int e = 0; e < E; ++e) f[j][e] = 0.0f;
          continue;
        }
        float2 z[H];
        unpack2<T>(stage[v], z);
        if constexpr (NORM != GN_NORM_NONE) {
          float2 w[H];
          unpack2<T>(params[v], w);
          if constexpr (NORM == GN_NORM_LN) {
            float2 b[H];
            unpack2<T>(params[slot + v], b);
#pragma unroll
            for (int e = 0; e < H; ++e) z[e] = fma2(mul2(add2(z[e], dup2(-mu)), dup2(r)), w[e], b[e]);
          } else {
#pragma unroll
            for (int e = 0; e < H; ++e) z[e] = mul2(mul2(z[e], dup2(r)), add2(w[e], gem));
          }
        }
#pragma unroll
        for (int e = 0; e < H; ++e) {
          if constexpr (EPI != EPI_NONE) z[e] = act_pair<EPI, FAST>(z[e]);
          f[j][2 * e] = z[e].x, f[j][2 * e + 1] = z[e].y;
          am[j] = max_nan(am[j], max_nan(fabsf(z[e].x), fabsf(z[e].y)));
        }
      }
      // each lane makes the scale of one of its group's four blocks
      const float s = block_scale(group_max<4, L>(am, lane)), i = __frcp_rn(s);
      const int vs = lane + 32 * (k0 + value_of_lane<4, L>(lane));
      if (lane % (L / 4) == 0 && (!CHECK || vs / L * kBlk < hidden)) scale[m * lds + vs / L] = s;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int v = lane + 32 * (k0 + j), src = lane_of_value<4, L>(lane, j);
        const float ij = __shfl_sync(0xffffffffu, i, src), sj = __shfl_sync(0xffffffffu, s, src);
        if (!CHECK || v < nvec) store_codes<E>(qrow, v, CHECK ? hidden : INT32_MAX, f[j], sj, ij);
      }
    };
    int k0 = 0;
    for (; k0 + 4 <= kfull; k0 += 4) four(k0, std::false_type{});
    if (32 * k0 < nvec) four(k0, std::true_type{});
    __syncwarp();  // every lane has read the row: the next one may take its place
    if (lane == 0 && m + step < rows) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      mbar_expect_tx(bar, bulk);
      bulk_g2s(stage, x + (m + step) * ldx, bulk, bar);
    }
  }
}

template <typename T, int NORM, int EPI, int VPT>
__global__ void __launch_bounds__(VPT == 4 ? 512 : 1024) norm_quant_row_kernel(const T* __restrict__ x, const T* __restrict__ g,
                                                                       const T* __restrict__ beta,
                                                                       uint8_t* __restrict__ q, float* __restrict__ scale,
                                                                       float* __restrict__ mean, float* __restrict__ rstd,
                                                                       int hidden, int64_t ldx, int64_t ldq,
                                                                       int64_t lds, float eps, int gemma, int pvec) {
  constexpr int E = Vec<T>::N;
  constexpr int L = kBlk / E;  // threads of a block of values
  constexpr bool FAST = fast_math_for<T>();
  __shared__ float red[2][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t m = blockIdx.x;
  const int t = threadIdx.x;
  const int team = (int)blockDim.x;
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
    if (lane == 0) red[slot][warp] = v;
    __syncthreads();
    return group_sum<32>(lane < (int)(blockDim.x >> 5) ? red[slot][lane] : 0.0f);
  };
  float mu = 0.0f, r = 1.0f;
  if constexpr (NORM != GN_NORM_NONE) {
    const float inv_n = 1.0f / (float)hidden;
    float2 acc = make_float2(0.0f, 0.0f);
    if constexpr (NORM == GN_NORM_LN) {
#pragma unroll
      for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int e = 0; e < E; e += 2) acc = add2(acc, make_float2(f[k][e], f[k][e + 1]));
      mu = total(acc.x + acc.y, 0) * inv_n;
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
    r = inverse_root(fmaf(total(acc.x + acc.y, 1), inv_n, eps));
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
    for (int e = 0; e < E; e += 2) {
      if constexpr (EPI != EPI_NONE) {
        const float2 z = act_pair<EPI, FAST>(make_float2(f[k][e], f[k][e + 1]));
        f[k][e] = z.x, f[k][e + 1] = z.y;
      }
      am[k] = max_nan(am[k], max_nan(fabsf(f[k][e]), fabsf(f[k][e + 1])));
    }
  }
  // each lane makes the scale of one of its group's VPT blocks
  const float s = block_scale(group_max<VPT, L>(am, lane)), i = __frcp_rn(s);
  {
    const int v = t + value_of_lane<VPT, L>(lane) * team;
    if (lane % (L / VPT) == 0 && v / L * kBlk < hidden) scale[m * lds + v / L] = s;
  }
#pragma unroll
  for (int k = 0; k < VPT; ++k) {
    const int v = t + k * team, src = lane_of_value<VPT, L>(lane, k);
    const float ik = __shfl_sync(0xffffffffu, i, src), sk = __shfl_sync(0xffffffffu, s, src);
    if (v * E < hidden) store_codes<E>(q + m * ldq, v, hidden, f[k], sk, ik);
  }
}

// ---------------------------------------------------------------- tiles of 128 x 128
// One block per tile: v = x, or dy * act'(x) (GRAD), read once, 32 values a thread in registers. Warp w
// has the rows 8 w..: for bf16 a thread has 4 consecutive rows (lanes 0-15 the first four of the warp's
// eight, lanes 16-31 the others) x 8 columns, for fp32 all 8 rows x 4 columns. So a row's block is a run of
// lanes (amax by shuffles, codes stored from registers, 128 bytes a row), and a column's is the warp's
// rows and then the sixteen warps (shared memory). The transposed codes of a thread are R consecutive
// bytes of each of its columns: they meet in a 16 KiB byte tile (16-byte chunk j of column c at j ^ key(c),
// so that neither side conflicts) and leave as 128-byte runs. A block walks over tiles and has the next
// one's vectors copied to each thread's own place in shared memory while it works on this one (a gradient of
// 16384 x 5120: 156 us without, 123 with). Both ways and the bias gradient in one read: 6 bytes a value for a
// bf16 gradient. Bound by the instructions of a value (4.1 TB/s of those bytes, two thirds of a copy's rate).
constexpr int kTileThreads = 512, kTileWarps = 16;

struct QuantArgs {
  const void* x;
  const void* dy;
  uint8_t* q;
  float* scale;
  uint8_t* qt;
  float* scale_t;
  float* colsum;
  int64_t rows, cols, ldx, lddy, ldq, lds, ldqt, ldst;
  unsigned row_tiles, col_tiles;
};

// 16 bytes of a row into this thread's place in shared memory, `bytes` of them read and the rest zero
__device__ __forceinline__ void copy16(uint4* dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(bytes) : "memory");
}

template <typename T, int EPI, bool GRAD, bool TILE>
__global__ void __launch_bounds__(kTileThreads, 2) quant_tile_kernel(const QuantArgs a) {
  constexpr int E = Vec<T>::N;
  constexpr int L = kBlk / E;         // lanes of a row: 16 or 32
  constexpr int R = 32 / E;           // rows of a thread: 4 or 8
  constexpr bool FAST = fast_math_for<T>();
  // the next tile, each thread's own vectors: [x and dy][R][threads]; then what the block shares
  extern __shared__ __align__(16) uint4 ahead[];
  uint8_t* bytes = reinterpret_cast<uint8_t*>(ahead + (GRAD ? 2 : 1) * R * kTileThreads);
  float(*red_max)[kBlk] = reinterpret_cast<float(*)[kBlk]>(bytes + kBlk * kBlk);
  float* col_scale = red_max[kTileWarps];
  float* col_inv = col_scale + kBlk;
  float(*red_sum)[kBlk] = reinterpret_cast<float(*)[kBlk]>(col_inv + kBlk);  // GRAD
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lv = lane % L;                          // vector of the row
  const int row0 = 8 * warp + (lane / L) * R;       // first row of the thread
  const unsigned tiles = (unsigned)a.col_tiles * (unsigned)a.row_tiles;
  auto fetch = [&](unsigned tile) {
    const unsigned ty = tile / a.col_tiles;
    const int64_t r0 = (int64_t)ty * kBlk, c = (int64_t)(tile - ty * a.col_tiles) * kBlk + lv * E;
    const int64_t left = (a.cols - c) * (int64_t)sizeof(T);
    const int most = left <= 0 ? 0 : left < 16 ? (int)left : 16;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int64_t r = r0 + row0 + i;
      const bool in = r < a.rows && most > 0;
      copy16(ahead + i * kTileThreads + threadIdx.x, static_cast<const T*>(a.x) + (in ? r * a.ldx + c : 0), in ? most : 0);
      if constexpr (GRAD)
        copy16(ahead + (R + i) * kTileThreads + threadIdx.x, static_cast<const T*>(a.dy) + (in ? r * a.lddy + c : 0),
               in ? most : 0);
    }
  };
  fetch(blockIdx.x);
  for (unsigned tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const unsigned tile_y = tile / a.col_tiles, tile_x = tile - tile_y * a.col_tiles;
    const int64_t r0 = (int64_t)tile_y * kBlk, c0 = (int64_t)tile_x * kBlk;
    const int nr = a.rows - r0 < kBlk ? (int)(a.rows - r0) : kBlk;
    const int nc = a.cols - c0 < kBlk ? (int)(a.cols - c0) : kBlk;
    uint4 raw[R], rawd[GRAD ? R : 1];
    asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll
    for (int i = 0; i < R; ++i) {
      raw[i] = ahead[i * kTileThreads + threadIdx.x];
      if constexpr (GRAD) rawd[i] = ahead[(R + i) * kTileThreads + threadIdx.x];
    }
    if (tile + gridDim.x < tiles) fetch(tile + gridDim.x);
    float f[R][E];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      Vec<T>::unpack(raw[i], f[i]);
      if constexpr (GRAD) {  // past the last row and column z and dy are 0: 0 * act'(0) = 0
        float d[E];
        Vec<T>::unpack(rawd[i], d);
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float2 v = mul2(make_float2(d[e], d[e + 1]), act_grad_pair<EPI, FAST>(make_float2(f[i][e], f[i][e + 1])));
          f[i][e] = v.x, f[i][e + 1] = v.y;
        }
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
      if constexpr (TILE) {
        float m = cmax[0];
#pragma unroll
        for (int e = 1; e < E; ++e) m = max_nan(m, cmax[e]);
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (lane == 0) red_max[0][warp] = m;
      }
      if ((GRAD || !TILE) && lane < L) {
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          if constexpr (!TILE)
            *reinterpret_cast<float4*>(&red_max[warp][lv * E + e]) = make_float4(cmax[e], cmax[e + 1], cmax[e + 2], cmax[e + 3]);
          if constexpr (GRAD)
            *reinterpret_cast<float4*>(&red_sum[warp][lv * E + e]) = make_float4(csum[e], csum[e + 1], csum[e + 2], csum[e + 3]);
        }
      }
      __syncthreads();
      if constexpr (TILE) {
#pragma unroll
        for (int w = 0; w < kTileWarps; w += 4) {
          const float4 v = *reinterpret_cast<const float4*>(&red_max[0][w]);
          all = max_nan(all, max_nan(max_nan(v.x, v.y), max_nan(v.z, v.w)));
        }
      } else if (a.qt) {  // a thread per column makes its scale
        if (threadIdx.x < kBlk) {
          float m = 0.0f;
#pragma unroll
          for (int w = 0; w < kTileWarps; ++w) m = max_nan(m, red_max[w][threadIdx.x]);
          const float s = block_scale(m);
          col_scale[threadIdx.x] = s;
          col_inv[threadIdx.x] = __frcp_rn(s);
          if (threadIdx.x < nc) a.scale_t[(c0 + threadIdx.x) * a.ldst + tile_y] = s;
        }
      }
      if constexpr (GRAD) {
        if (a.colsum && threadIdx.x < nc) {
          float t = 0.0f;
#pragma unroll
          for (int w = 0; w < kTileWarps; ++w) t += red_sum[w][threadIdx.x];
          a.colsum[(int64_t)tile_y * a.cols + c0 + threadIdx.x] = t;
        }
      }
    }
    const float s_all = TILE ? block_scale(all) : 0.0f, i_all = TILE ? __frcp_rn(s_all) : 0.0f;
    if (TILE && threadIdx.x == 0) {
      if (a.q) a.scale[(int64_t)tile_y * a.lds + tile_x] = s_all;
      if (a.qt) a.scale_t[(int64_t)tile_x * a.ldst + tile_y] = s_all;
    }
    // where R codes of column c (vector lv of the row) go: chunk row / 16 of the column; its 8-byte halves change
    // places on every other eight vectors
    auto put = [&](int c, const uint32_t* w) {
      uint8_t* at = bytes + c * kBlk + (((warp >> 1) ^ (lv & 7)) << 4) + 8 * ((warp & 1) ^ ((lv >> 3) & 1));
      if constexpr (R == 4) *reinterpret_cast<uint32_t*>(at + 4 * (lane / L)) = w[0];
      else *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[1]);
    };
    if constexpr (TILE) {  // one scale: the codes are made once and their bytes transposed four by four
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        uint32_t w[R], t[4][R / 4];
#pragma unroll
        for (int i = 0; i < R; ++i) w[i] = code4(f[i] + e, s_all, i_all);
        if (a.q) {
#pragma unroll
          for (int i = 0; i < R; ++i) {
            const int c = lv * E + e;
            if (row0 + i >= nr || c >= nc) continue;
            uint8_t* out = a.q + (r0 + row0 + i) * a.ldq + c0 + c;
            if (c + 4 <= nc) {
              *reinterpret_cast<uint32_t*>(out) = w[i];
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                if (c + k < nc) out[k] = (uint8_t)(w[i] >> (8 * k));
            }
          }
        }
        if (a.qt) {
#pragma unroll
          for (int k = 0; k < R / 4; ++k) {
            const uint32_t *u = w + 4 * k;
            const uint32_t p = __byte_perm(u[0], u[1], 0x5140), q = __byte_perm(u[2], u[3], 0x5140);
            const uint32_t x = __byte_perm(u[0], u[1], 0x7362), y = __byte_perm(u[2], u[3], 0x7362);
            t[0][k] = __byte_perm(p, q, 0x5410);
            t[1][k] = __byte_perm(p, q, 0x7632);
            t[2][k] = __byte_perm(x, y, 0x5410);
            t[3][k] = __byte_perm(x, y, 0x7632);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) put(lv * E + e + k, t[k]);
        }
      }
    } else {
      if (a.q) {  // each lane makes the scale of one of its group's rows
        const float s = block_scale(group_max<R, L>(rmax, lane)), inv = __frcp_rn(s);
        const int ir = row0 + value_of_lane<R, L>(lane);
        if (lane % (L / R) == 0 && ir < nr) a.scale[(r0 + ir) * a.lds + tile_x] = s;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const int src = lane_of_value<R, L>(lane, i);
          const float ii = __shfl_sync(0xffffffffu, inv, src), si = __shfl_sync(0xffffffffu, s, src);
          if (row0 + i < nr && lv * E < nc) store_codes<E>(a.q + (r0 + row0 + i) * a.ldq + c0, lv, nc, f[i], si, ii);
        }
      }
      if (a.qt) {
        __syncthreads();  // the columns' scales
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int c = lv * E + e;
          const float s = col_scale[c], inv = col_inv[c];
          uint32_t w[R / 4];
#pragma unroll
          for (int k = 0; k < R / 4; ++k) {
            const float v[4] = {f[4 * k][e], f[4 * k + 1][e], f[4 * k + 2][e], f[4 * k + 3][e]};
            w[k] = code4(v, s, inv);
          }
          put(c, w);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < kBlk * 8 / kTileThreads; ++it) {
      const int idx = it * kTileThreads + threadIdx.x, c = idx >> 3, j = idx & 7;
      if (!a.qt || c >= nc || 16 * j >= nr) continue;
      uint4 v = *reinterpret_cast<const uint4*>(bytes + c * kBlk + ((j ^ ((c / E) & 7)) << 4));
      if ((c / E) & 8) v = make_uint4(v.z, v.w, v.x, v.y);
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
    __syncthreads();  // the next tile's sums and bytes take these places
  }
}

// ---------------------------------------------------------------- host side

// shape 1, 2, 4: one warp per row with that many vectors a lane; 0: staged rows; -1, -4: one block per row with
// 1 or 4 vectors a thread
template <typename T, int NORM, int EPI>
void* pick_norm_shape(int shape) {
  switch (shape) {
    case 1: return (void*)norm_quant_warp_kernel<T, NORM, EPI, 1>;
    case 2: return (void*)norm_quant_warp_kernel<T, NORM, EPI, 2>;
    case 4: return (void*)norm_quant_warp_kernel<T, NORM, EPI, 4>;
    case 0: return (void*)norm_quant_stage_kernel<T, NORM, EPI>;
    case -1: return (void*)norm_quant_row_kernel<T, NORM, EPI, 1>;
    default: return (void*)norm_quant_row_kernel<T, NORM, EPI, 4>;
  }
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
  if (tile) return (void*)quant_tile_kernel<T, EPI_NONE, true, true>;
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
  const int lanes = (nvec + 31) / 32;  // vectors a lane of a warp would hold
  const int sms = sm_count() > 0 ? sm_count() : 148;
  int h = (int)hidden;
  const int vectors = norm == GN_NORM_LN ? 2 : norm == GN_NORM_RMS ? 1 : 0;  // parameters
  if (lanes <= 4 && (lanes == 1 || rows > 4 * sms)) {
    const int shape = lanes <= 2 ? lanes : 4;
    void* kern = dt == GN_BF16 ? pick_norm<__nv_bfloat16>(norm, epi, shape) : pick_norm<float>(norm, epi, shape);
    const size_t smem = (size_t)vectors * 32 * shape * 16;
    const int most = persistent_grid(kern, 32 * kWarpRows, smem, 0);
    if (most <= 0) return GN_ERR_CUDA;
    const int64_t blocks = (rows + kWarpRows - 1) / kWarpRows;
    void* args[] = {&x, &g, &beta, &q, &scale, &mean, &rstd, &rows, &h, &ld_x, &ld_q, &ld_s, &eps, &gemma};
    if (cudaLaunchKernel(kern, dim3((unsigned)(blocks < most ? blocks : most)), dim3(32 * kWarpRows), args, smem,
                         (cudaStream_t)stream) != cudaSuccess)
      return GN_ERR_CUDA;
  } else if (nvec > 128 && nvec <= 1024 && rows > 4 * sms) {
    void* kern = dt == GN_BF16 ? pick_norm<__nv_bfloat16>(norm, epi, 0) : pick_norm<float>(norm, epi, 0);
    int slot = (nvec + 7) / 8 * 8;
    const size_t room = smem_optin() > 1024 ? smem_optin() - 1024 : 0;  // the barriers are static
    int warps = (int)(room / ((size_t)slot * 16)) - vectors;
    if (warps > kStageWarps) warps = kStageWarps;
    if (warps < 1) return GN_ERR_UNSUPPORTED;
    const size_t smem = (size_t)(vectors + warps) * slot * 16;
    if (!kernel_attrs(kern, smem)) return GN_ERR_CUDA;
    unsigned* err = device_err_word();
    if (!err) return GN_ERR_CUDA;
    const int64_t blocks = (rows + warps - 1) / warps;
    void* args[] = {&x, &g, &beta, &q, &scale, &mean, &rstd, &rows, &h, &ld_x, &ld_q, &ld_s, &eps, &gemma, &slot, &err};
    if (cudaLaunchKernel(kern, dim3((unsigned)(blocks < sms ? blocks : sms)), dim3((unsigned)(32 * warps)), args, smem,
                         (cudaStream_t)stream) != cudaSuccess)
      return GN_ERR_CUDA;
  } else {
    const int per = nvec <= 1024 && rows <= sms ? 1 : 4;
    void* kern = dt == GN_BF16 ? pick_norm<__nv_bfloat16>(norm, epi, -per) : pick_norm<float>(norm, epi, -per);
    const int threads = ((nvec + per - 1) / per + 31) / 32 * 32;
    void* args[] = {&x, &g, &beta, &q, &scale, &mean, &rstd, &h, &ld_x, &ld_q, &ld_s, &eps, &gemma, &pvec};
    if (!kernel_attrs(kern, 0)) return GN_ERR_CUDA;
    if (cudaLaunchKernel(kern, dim3((unsigned)rows), dim3((unsigned)threads), args, 0, (cudaStream_t)stream) != cudaSuccess)
      return GN_ERR_CUDA;
  }
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
  // (a dy of no rows may well be a null pointer)
  if ((tile && dy) || (!dy && rows > 0 && epi != GN_EPI_NONE)) return GN_ERR_UNSUPPORTED;
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
  // only the gradient's kernels form column sums: those of a matrix as it is go through them as dy * 1
  if (db && !dy) dy = x, ld_dy = ld_x;
  QuantArgs a{x, dy, static_cast<uint8_t*>(q), scale, static_cast<uint8_t*>(qt), scale_t,
              db ? static_cast<float*>(ws) : nullptr, rows, cols, ld_x, ld_dy, ld_q, ld_s, ld_qt, ld_st,
              (unsigned)blocks_of(rows), (unsigned)blocks_of(cols)};
  void* kern = dt == GN_BF16 ? pick_tile<__nv_bfloat16>(epi, dy != nullptr, tile) : pick_tile<float>(epi, dy != nullptr, tile);
  const size_t smem = (size_t)kTileThreads * (dt == GN_BF16 ? 4 : 8) * 16 * (dy ? 2 : 1) + kBlk * kBlk +
                      (kTileWarps * (dy ? 2 : 1) + 2) * kBlk * 4;
  const int most = persistent_grid(kern, kTileThreads, smem, 0);
  if (most <= 0) return GN_ERR_CUDA;
  const int64_t tiles = blocks_of(rows) * blocks_of(cols);
  if (tiles > INT32_MAX) return GN_ERR_SHAPE;  // far above any device's memory
  void* args[] = {&a};
  if (cudaLaunchKernel(kern, dim3((unsigned)(tiles < most ? tiles : most)), dim3(kTileThreads), args, smem, s) != cudaSuccess)
    return GN_ERR_CUDA;
  count_launches(1);
  const gn_status st = launch_status();
  if (st != GN_OK || !db) return st;
  return launch_colsum(a.colsum, blocks_of(rows), cols, cols, db, nullptr, s);
}
