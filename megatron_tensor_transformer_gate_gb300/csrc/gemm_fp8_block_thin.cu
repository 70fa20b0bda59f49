// gemm_fp8_block_thin.cu — the block-scaled E4M3 product for at most eight
// rows of A (single tokens, and a few of them).
//
// Its cost is one read of B and the latency around it, so nothing stands
// between B and the arithmetic: each lane loads B's codes from global memory
// straight into the registers that mma.sync m16n8k32 takes them from (B's rows
// on the 16 side, A's on the 8 side).  The order of k inside a K block is free
// as long as A and B agree on it: lane (g, t) of a warp (g = lane / 4,
// t = lane mod 4) reads 16 neighbouring codes at 16t and at 64 + 16t of rows
// g and g + 8 of B and g of A, and each 64 codes make the operands of two
// instructions.  A K block's sum is scaled and added in fp32.
//
// Measured beside the tcgen05 form for few rows, whose barriers, ring, TMEM
// and cluster sum are what a small product waits for (µs, weight from DRAM):
// 1×512×2000 3.3 against 4.4, 1×4096×4096 5.5 against 7.6 (2.5 is the read of
// B at copy speed, 2.0 the smallest launch), 1×8192×8192 15.8 / 16.3,
// 1×28672×8192 41.0 / 42.2, 1×8192×28672 43.2 / 42.1, 8×28672×8192 42.8 / 42.4;
// with a second group of eight rows it falls behind (16×8192×28672 65 / 42),
// so nine rows are where that form starts.  Bound by DRAM: 5.7 TB/s at
// 1×28672×8192.  Eight warps of three K blocks in flight, two CTAs an SM, were
// the best of 4 to 8 warps and 2 to 5 blocks at 1×4096×4096.
#include <cuda_bf16.h>

#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "fp8_block.h"
#include "gemm.h"

namespace tp {
namespace {

constexpr int BK = 128;
constexpr int TOKENS = 8;    // at most, rows of A
constexpr int ROWS = 16;     // of B a CTA
constexpr int WARPS = 8;     // K blocks are dealt to them in turn
constexpr int U = 3;         // K blocks of a warp in flight
constexpr int CTAS = 2;      // on an SM

struct ThinParams {
  const uint8_t *r, *t;      // B's codes (16 rows a CTA), A's
  int64_t ldr, ldt;
  const float *sr, *st;
  int64_t ldsr, ldst;
  int r_row, t_row;          // a scale for each row (1) or for 128 rows (0)
  int R, T, K;
  void* c;
  int64_t ldc;
};

// 16 codes of which `valid` exist (no others are read: a row may end where
// its codes do), zeros after them.
__device__ __forceinline__ uint4 codes16(const uint8_t* p, int valid) {
  if (valid >= 16) {
    uint4 u;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
                 : "l"(p));
    return u;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (j < valid) w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void mma_e4m3(float (&c)[4], uint32_t a0,
                                         uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <int OUT_F32>
__global__ void __launch_bounds__(32 * WARPS, CTAS)
    gemm_fp8_block_thin_kernel(const ThinParams p) {
  __shared__ float part_sum[WARPS][TOKENS][ROWS + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int r0 = blockIdx.x * ROWS;
  // rows that do not exist stand for row 0 and are not stored
  const int gl = r0 + g < p.R ? r0 + g : 0, gh = r0 + g + 8 < p.R ? r0 + g + 8 : 0;
  const uint8_t* rl = p.r + gl * p.ldr + 16 * t;
  const uint8_t* rh = p.r + gh * p.ldr + 16 * t;
  const float* srl = p.sr + (p.r_row ? gl : gl / BK);
  const float* srh = p.sr + (p.r_row ? gh : gh / BK);
  const uint8_t* tr = p.t + (g < p.T ? g : 0) * p.ldt + 16 * t;
  const float* st0 = p.st + (p.t_row && 2 * t < p.T ? 2 * t : 0);
  const float* st1 = p.st + (p.t_row && 2 * t + 1 < p.T ? 2 * t + 1 : 0);
  float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};

  struct Block {
    uint4 lo[2], hi[2], tok[2];   // 64 codes each of rows g, g + 8 and A's
    float wl, wh, w0, w1;
  };
  auto load = [&](Block& x, int64_t kb, auto tail) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int64_t at = kb * BK + 64 * j;
      const int valid = decltype(tail)::value ? (int)(p.K - at) - 16 * t : 16;
      x.lo[j] = codes16(rl + at, valid);
      x.hi[j] = codes16(rh + at, valid);
      x.tok[j] = codes16(tr + at, valid);
    }
    x.wl = __ldg(srl + kb * p.ldsr);
    x.wh = __ldg(srh + kb * p.ldsr);
    x.w0 = __ldg(st0 + kb * p.ldst);
    x.w1 = __ldg(st1 + kb * p.ldst);
  };
  auto add = [&](const Block& x) {
    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 &l = x.lo[j], &h = x.hi[j], &z = x.tok[j];
      mma_e4m3(c, l.x, h.x, l.y, h.y, z.x, z.y);
      mma_e4m3(c, l.z, h.z, l.w, h.w, z.z, z.w);
    }
    acc[0] = fmaf(c[0], x.wl * x.w0, acc[0]);
    acc[1] = fmaf(c[1], x.wl * x.w1, acc[1]);
    acc[2] = fmaf(c[2], x.wh * x.w0, acc[2]);
    acc[3] = fmaf(c[3], x.wh * x.w1, acc[3]);
  };
  // a block's registers are loaded anew as soon as it is added
  const int full = p.K / BK;
  Block x[U];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (warp + u * WARPS < full)
      load(x[u], warp + u * WARPS, std::false_type{});
  for (int kb = warp; kb < full; kb += WARPS * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (kb + u * WARPS >= full) break;
      add(x[u]);
      if (kb + (u + U) * WARPS < full)
        load(x[u], kb + (u + U) * WARPS, std::false_type{});
    }
  }
  if (p.K % BK && full % WARPS == warp) {   // the block that K ends in
    load(x[0], full, std::true_type{});
    add(x[0]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    part_sum[warp][2 * t + (i & 1)][g + 8 * (i >> 1)] = acc[i];
  __syncthreads();

  // the warps' sums in warp order
  const int tok = tid >> 4, row = tid & 15;
  if (tok < p.T && tok < TOKENS && r0 + row < p.R) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) v += part_sum[k][tok][row];
    const int64_t at = tok * p.ldc + r0 + row;
    if (OUT_F32)
      static_cast<float*>(p.c)[at] = v;
    else
      static_cast<__nv_bfloat16*>(p.c)[at] = __float2bfloat16(v);
  }
}

}  // namespace

int gemm_fp8_block_thin(const GemmFp8Block& g, cudaStream_t s) {
  ThinParams p;
  memset(&p, 0, sizeof(p));
  p.r = g.qb;
  p.t = g.qa;
  p.ldr = g.ldb;
  p.ldt = g.lda;
  p.sr = g.sb;
  p.st = g.sa;
  p.ldsr = g.ldsb;
  p.ldst = g.ldsa;
  p.r_row = g.b_group == kFp8Row;
  p.t_row = g.a_group == kFp8Row;
  p.R = (int)g.N;
  p.T = (int)g.M;
  p.K = (int)g.K;
  p.c = g.c;
  p.ldc = g.ldc;
  const unsigned grid = (unsigned)((g.N + ROWS - 1) / ROWS);
  if (g.out_f32)
    gemm_fp8_block_thin_kernel<1><<<grid, 32 * WARPS, 0, s>>>(p);
  else
    gemm_fp8_block_thin_kernel<0><<<grid, 32 * WARPS, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace tp
