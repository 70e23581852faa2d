// linear_fp8.cu - matrix product of two 8-bit (e4m3) operands with block scales:
//   y[m, n] = act( sum_b sa[m, b] sb[n', b] sum_{k in block b} A[m, k] B[n, k]  + d[n] ),
// b over the blocks of 128 of the contraction, n' = n / 128 (a weight's 128 x 128 blocks) or n.
// A product of two e4m3 values is exact in fp32; the block sums and the scaled total are fp32.
#include "gn_common.cuh"
#include "gn_host.h"

namespace gn {
namespace {

constexpr int64_t kMaxRows = 65535ll * 128;
constexpr int kT = 64, kKC = 32, kBlk = 128;

struct Fp8Args {
  const uint8_t* A;
  const float* sa;
  const uint8_t* B;
  const float* sb;
  const float* d;
  void* y;
  int64_t M, N, K, lda, ldsa, ldb, ldsb, ldy;
  int b_rows, accumulate;
};

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  float f;
  asm("cvt.f32.f16 %0, %1;" : "=f"(f) : "h"((uint16_t)(h & 0xffff)));
  return f;
}

template <int EPI, bool F32>
__global__ void __launch_bounds__(256) linear_fp8_simple_kernel(const Fp8Args a) {
  __shared__ float As[kKC][kT + 1], Bs[kKC][kT + 1];
  const int64_t m0 = (int64_t)blockIdx.y * kT, n0 = (int64_t)blockIdx.x * kT;
  const int tr = threadIdx.x / 16, tc = threadIdx.x % 16;
  float acc[4][4] = {}, part[4][4] = {};
  for (int64_t k0 = 0; k0 < a.K; k0 += kKC) {
    for (int i = threadIdx.x; i < kT * kKC; i += 256) {
      const int r = i / kKC, k = i % kKC;
      const bool kin = k0 + k < a.K;
      As[k][r] = kin && m0 + r < a.M ? e4m3_to_f32(a.A[(m0 + r) * a.lda + k0 + k]) : 0.0f;
      Bs[k][r] = kin && n0 + r < a.N ? e4m3_to_f32(a.B[(n0 + r) * a.ldb + k0 + k]) : 0.0f;
    }
    __syncthreads();
    for (int k = 0; k < kKC; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[i][j] = fmaf(As[k][tr * 4 + i], Bs[k][tc * 4 + j], part[i][j]);
    __syncthreads();
    if ((k0 + kKC) % kBlk == 0 || k0 + kKC >= a.K) {
      const int64_t b = k0 / kBlk;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t m = m0 + tr * 4 + i, n = n0 + tc * 4 + j;
          if (m < a.M && n < a.N) acc[i][j] = fmaf(a.sa[m * a.ldsa + b] * a.sb[n / a.b_rows * a.ldsb + b], part[i][j], acc[i][j]);
          part[i][j] = 0.0f;
        }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + tr * 4 + i, n = n0 + tc * 4 + j;
      if (m >= a.M || n >= a.N) continue;
      const float z = epi_fwd<EPI, !F32>(acc[i][j] + (a.d ? a.d[n] : 0.0f));
      if constexpr (F32) {
        float* p = static_cast<float*>(a.y) + m * a.ldy + n;
        *p = a.accumulate ? *p + z : z;
      } else {
        static_cast<__nv_bfloat16*>(a.y)[m * a.ldy + n] = __float2bfloat16_rn(z);
      }
    }
}

}  // namespace
}  // namespace gn

using namespace gn;

extern "C" gn_status gn_linear_fp8(const void* A, const float* sa, const void* B, const float* sb, const float* d,
                                   void* y, int64_t M, int64_t N, int64_t K, int64_t ld_a, int64_t ld_sa, int64_t ld_b,
                                   int64_t ld_sb, int64_t ld_y, int64_t b_rows, int accumulate, gn_epilogue epi,
                                   gn_dtype out, void* stream) {
  if (!dt_ok(out) || !epi_ok(epi)) return GN_ERR_DTYPE;
  const int64_t kb = (K + kBlk - 1) / kBlk;
  if (M < 0 || N < 0 || K <= 0 || M > kMaxRows || N > INT32_MAX || K > INT32_MAX || (b_rows != 1 && b_rows != kBlk))
    return GN_ERR_SHAPE;
  if (ld_a < K || ld_b < K || ld_sa < kb || ld_sb < kb || ld_y < N) return GN_ERR_SHAPE;
  if (out == GN_F32 ? epi != GN_EPI_NONE : accumulate != 0) return GN_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return GN_OK;
  if (!A || !sa || !B || !sb || !y) return GN_ERR_NULL;
  if (!aligned16(A) || !aligned16(B) || !aligned16(y) || ld_a % 16 || ld_b % 16 || ld_y * dt_size(out) % 16 ||
      (d && !aligned16(d)) || (reinterpret_cast<uintptr_t>(sa) & 3) ||
      (reinterpret_cast<uintptr_t>(sb) & 3))
    return GN_ERR_ALIGN;
  Fp8Args a{static_cast<const uint8_t*>(A), sa, static_cast<const uint8_t*>(B), sb, d, y, M, N, K, ld_a, ld_sa, ld_b, ld_sb,
            ld_y, (int)b_rows, accumulate != 0};
  void* kern = out == GN_F32             ? (void*)linear_fp8_simple_kernel<EPI_NONE, true>
               : epi == GN_EPI_GELU_TANH ? (void*)linear_fp8_simple_kernel<EPI_GELU_TANH, false>
               : epi == GN_EPI_SILU      ? (void*)linear_fp8_simple_kernel<EPI_SILU, false>
                                         : (void*)linear_fp8_simple_kernel<EPI_NONE, false>;
  const dim3 grid((unsigned)((N + kT - 1) / kT), (unsigned)((M + kT - 1) / kT));
  if (grid.y > 65535) return GN_ERR_UNSUPPORTED;
  void* args[] = {&a};
  if (cudaLaunchKernel(kern, grid, dim3(256), args, 0, (cudaStream_t)stream) != cudaSuccess) return GN_ERR_CUDA;
  count_launches(1);
  return launch_status();
}
