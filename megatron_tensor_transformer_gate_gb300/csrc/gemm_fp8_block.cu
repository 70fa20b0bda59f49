// gemm_fp8_block.cu — C[M, N] = Σ_b sa[b]·sb[b]·Σ_{k in block b} qa·qb over
// K blocks of 128, E4M3 codes with fp32 scales, C in bf16 or fp32.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "fp8_block.h"
#include "gemm.h"
#include "profile.h"

namespace tp {
namespace {

// CUDA-core form: 64×64 tiles, 4×4 outputs a thread, 32-deep K slices staged
// in shared memory as fp32; a K block's sum is kept apart and scaled once.
constexpr int ST = 64, SK = 32;

__device__ __forceinline__ float e4m3_to_float(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

__global__ void __launch_bounds__(256)
    gemm_fp8_block_simt(const GemmFp8Block p, int64_t n_tiles) {
  __shared__ float as[SK][ST + 1], bs[SK][ST + 1];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int64_t m0 = blockIdx.x / n_tiles * ST, n0 = blockIdx.x % n_tiles * ST;
  float acc[4][4] = {};
  for (int64_t kb = 0; kb * kFp8Group < p.K; ++kb) {
    float part[4][4] = {};
    for (int ks = 0; ks < kFp8Group; ks += SK) {
      const int64_t k0 = kb * kFp8Group + ks;
      if (k0 >= p.K) break;
      __syncthreads();
      for (int i = tid; i < ST * SK; i += 256) {
        const int r = i / SK, k = i % SK;
        const bool in = k0 + k < p.K;
        as[k][r] = in && m0 + r < p.M
                       ? e4m3_to_float(p.qa[(m0 + r) * p.lda + k0 + k]) : 0.0f;
        bs[k][r] = in && n0 + r < p.N
                       ? e4m3_to_float(p.qb[(n0 + r) * p.ldb + k0 + k]) : 0.0f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < SK; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            part[i][j] += as[k][ty * 4 + i] * bs[k][tx * 4 + j];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
        if (m < p.M && n < p.N) {
          const float sa = p.sa[kb * p.ldsa +
                                (p.a_group == kFp8Row ? m : m / kFp8Group)];
          const float sb = p.sb[kb * p.ldsb +
                                (p.b_group == kFp8Row ? n : n / kFp8Group)];
          acc[i][j] += part[i][j] * (sa * sb);
        }
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t m = m0 + ty * 4 + i, n = n0 + tx * 4 + j;
      if (m < p.M && n < p.N) {
        if (p.out_f32)
          static_cast<float*>(p.c)[m * p.ldc + n] = acc[i][j];
        else
          static_cast<__nv_bfloat16*>(p.c)[m * p.ldc + n] =
              __float2bfloat16_rn(acc[i][j]);
      }
    }
}

}  // namespace

int gemm_fp8_block(const GemmFp8Block& p, void* stream, unsigned* status) {
  (void)status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t mt = (p.M + ST - 1) / ST, nt = (p.N + ST - 1) / ST;
  if (mt * nt > INT32_MAX) return cudaErrorInvalidValue;
  {
    ProfScope ps(s, KF_GEMM_TC_FP8, 2.0 * p.M * p.N * p.K,
                 (double)(p.M + p.N) * p.K + (p.out_f32 ? 4.0 : 2.0) * p.M * p.N);
    gemm_fp8_block_simt<<<(unsigned)(mt * nt), 256, 0, s>>>(p, nt);
  }
  count_launch();
  return cudaGetLastError();
}

}  // namespace tp
