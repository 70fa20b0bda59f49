// fp8_block.h — host launchers of the block-scaled E4M3 operators.
//
// A quantized matrix [rows, cols] is E4M3 codes (row pitch a multiple of 16
// bytes) and fp32 scales with one row for each block of 128 columns:
// s[c / 128][r] (TP_FP8_ROW: 1×128 groups) or s[c / 128][r / 128]
// (TP_FP8_BLOCK: 128×128 blocks).  The element's value is q·s.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace tp {

constexpr int kFp8Group = 128;
constexpr int kFp8Row = 0;     // tp_fp8_group
constexpr int kFp8Block = 1;

// Where the codes of a matrix and of its transpose go; q or qt may be null.
struct Fp8BlockOut {
  uint8_t* q = nullptr;
  int64_t ldq = 0;
  float* s = nullptr;
  int64_t lds = 0;
  uint8_t* qt = nullptr;
  int64_t ldqt = 0;
  float* st = nullptr;
  int64_t ldst = 0;
};

// fp8_block.cu; all return a cudaError_t value.
// dtype: tp_dtype of x (TP_F32 or TP_BF16).
int quantize_fp8_block(int dtype, int group, int64_t rows, int64_t cols,
                       const void* x, int64_t ldx, const Fp8BlockOut& o,
                       void* stream);
// The codes of A = SiLU(G) ⊙ U, gu = [G | U] (bf16, [T, 2f]).
int swiglu_fp8_fwd(int64_t T, int64_t f, const void* gu, int64_t ldgu,
                   const Fp8BlockOut& o, void* stream);
// The codes of [dG | dU] ([T, 2f]) from dA [T, f] and gu.
int swiglu_fp8_bwd(int64_t T, int64_t f, const void* da, int64_t ldda,
                   const void* gu, int64_t ldgu, const Fp8BlockOut& o,
                   void* stream);
// x1 = x + r (r and x1 may be null), the codes of RMSNorm(x1)·γ, rstd, and
// the norm's output in bf16 (y, may be null).
int add_rmsnorm_fp8_fwd(int64_t T, int64_t h, float eps, const void* x,
                        const void* r, const void* gamma, void* x1, void* y,
                        float* rstd, uint8_t* q, int64_t ldq, float* s,
                        int64_t lds, unsigned* status, void* stream);

// gemm_fp8_block.cu: C[M, N] = Σ over K blocks sa·sb·Σ_k qa·qb.
struct GemmFp8Block {
  int64_t M = 0, N = 0, K = 0;
  const uint8_t *qa = nullptr, *qb = nullptr;
  int64_t lda = 0, ldb = 0;
  const float *sa = nullptr, *sb = nullptr;
  int64_t ldsa = 0, ldsb = 0;
  int a_group = kFp8Row, b_group = kFp8Block;
  int out_f32 = 0;
  void* c = nullptr;
  int64_t ldc = 0;
};
int gemm_fp8_block(const GemmFp8Block& p, void* stream, unsigned* status);
// What it takes for sizes M, N, K on `sms` SMs.
enum Fp8BlockForm { kFp8Thin = 0, kFp8Narrow = 1, kFp8Wide = 2 };   // tp.h
struct Fp8BlockPlan {
  int form = kFp8Wide;
  int rows = 256;      // of A a tile
  int split = 1;       // parts of K
};
Fp8BlockPlan plan_fp8_block(int64_t M, int64_t N, int64_t K, int b_group,
                            int sms);
// gemm_fp8_block_thin.cu: its form for M ≤ 8.
int gemm_fp8_block_thin(const GemmFp8Block& p, cudaStream_t s);

}  // namespace tp
