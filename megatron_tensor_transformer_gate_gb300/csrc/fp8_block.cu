// fp8_block.cu — the operators that write block-scaled E4M3 codes:
// quantization, SwiGLU (forward and backward) and residual + RMSNorm.
//
// With amax the largest magnitude of a block of 128 (1×128 or 128×128),
//   r = 448 / amax,  s = amax / 448  (fp32),  q = e4m3(x·r),
// values are taken in fp32 straight from the producing formula (SwiGLU, norm:
// no rounding to bf16 in between) and rounded once, to E4M3.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "fp8.cuh"
#include "fp8_block.h"
#include "gemm.h"
#include "profile.h"

namespace tp {
namespace {

// ------------------------------------------------------------ tile kernel --
// One CTA per 128×128 tile of the output matrix.  A source gives eight
// consecutive columns of one row as fp32 (columns beyond the end as 0).
constexpr int TILE = 128;
constexpr int TILE_THREADS = 256;

template <typename T>
__device__ __forceinline__ void load8(const T* p, int valid, bool vec,
                                      float* v);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p,
                                                     int valid, bool vec,
                                                     float* v) {
  if (vec && valid >= 8) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y),
                 c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
    v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = j < valid ? __bfloat162float(p[j]) : 0.0f;
  }
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, int valid,
                                             bool vec, float* v) {
  if (vec && valid >= 8) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)),
                 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = j < valid ? p[j] : 0.0f;
  }
}

template <typename T>
struct CopySource {
  const T* x;
  int64_t ld;
  bool vec;
  __device__ void load(int64_t r, int64_t c, int64_t cols, float* v) const {
    load8(x + r * ld + c, (int)(cols - c < 8 ? cols - c : 8), vec, v);
  }
  __device__ int64_t col_tile(int64_t j, int64_t) const { return j; }
};

// A = SiLU(G)·U.
struct SwigluSource {
  const __nv_bfloat16* gu;
  int64_t ld, f;
  bool vec;
  __device__ void load(int64_t r, int64_t c, int64_t cols, float* v) const {
    const int valid = (int)(cols - c < 8 ? cols - c : 8);
    const __nv_bfloat16* p = gu + r * ld + c;
    float g[8], u[8];
    load8(p, valid, vec, g);
    load8(p + f, valid, vec, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = g[j] * sigmoid_f(g[j]) * u[j];
  }
  __device__ int64_t col_tile(int64_t j, int64_t) const { return j; }
};

// [dG | dU]: dG = dA·U·s·(1 + G·(1 − s)), dU = dA·G·s with s = σ(G).
struct SwigluBwdSource {
  const __nv_bfloat16 *da, *gu;
  int64_t ldda, ld, f;
  bool vec;
  __device__ static float dgate(float a, float g, float u) {
    const float s = sigmoid_f(g);
    return a * u * s * (1.0f + g * (1.0f - s));
  }
  __device__ static float dup(float a, float g) { return a * g * sigmoid_f(g); }
  __device__ void load(int64_t r, int64_t c, int64_t cols, float* v) const {
    const __nv_bfloat16* pa = da + r * ldda;
    const __nv_bfloat16* pg = gu + r * ld;
    if (vec && (c >= f || c + 8 <= f)) {   // all eight on one side
      const bool up = c >= f;
      const int64_t k = up ? c - f : c;
      const int valid = (int)(f - k < 8 ? f - k : 8);
      float a[8], g[8], u[8];
      load8(pa + k, valid, true, a);
      load8(pg + k, valid, true, g);
      if (up) {
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = dup(a[j], g[j]);
      } else {
        load8(pg + f + k, valid, true, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = dgate(a[j], g[j], u[j]);
      }
      return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t cj = c + j;
      v[j] = 0.0f;
      if (cj < f)
        v[j] = dgate(__bfloat162float(pa[cj]), __bfloat162float(pg[cj]),
                     __bfloat162float(pg[f + cj]));
      else if (cj < cols)
        v[j] = dup(__bfloat162float(pa[cj - f]), __bfloat162float(pg[cj - f]));
    }
  }
  // the dG tile and the dU tile of the same hidden units run side by side, so
  // that the second reads dA and G from L2
  __device__ int64_t col_tile(int64_t j, int64_t n) const {
    return (j & 1) ? (n + 1) / 2 + (j >> 1) : (j >> 1);
  }
};

__device__ __forceinline__ void store8(uint8_t* p, uint2 c, int valid) {
  if (valid >= 8) {
    *reinterpret_cast<uint2*>(p) = c;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid) p[j] = (uint8_t)((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
  }
}

// Thread (warp w, half-warp g, lane l of 16) holds rows 16w + 8g + i and
// columns 8l + j, i, j < 8: a row's codes leave as 16 lanes × 8 bytes, a
// column's largest magnitude takes one shuffle and one pass through shared
// memory, and eight rows of a column pack into one 8-byte shared-memory store
// of the transposed tile.
template <typename SRC, int GROUP>
__global__ void __launch_bounds__(TILE_THREADS, 2)
    quantize_tile_kernel(const SRC src, int64_t rows, int64_t cols,
                         int64_t col_tiles, const Fp8BlockOut o) {
  __shared__ float cmax[8][TILE];
  __shared__ __align__(16) uint8_t tile_t[TILE * TILE];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = lane >> 4, l = lane & 15;
  const int64_t rt = blockIdx.x / col_tiles;
  const int64_t ct = src.col_tile(blockIdx.x - rt * col_tiles, col_tiles);
  const int64_t r0 = rt * TILE + warp * 16 + half * 8;
  const int64_t c0 = ct * TILE + l * 8;

  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + i < rows && c0 < cols) {
      src.load(r0 + i, c0, cols, v[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
    }
  }

  float colr[8];   // the factor of each of this thread's columns
  float rowr[8];   // and of each of its rows
  if (GROUP == kFp8Row) {
    if (o.q != nullptr) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[i][j]));
#pragma unroll
        for (int d = 8; d > 0; d >>= 1)
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        rowr[i] = block_factor(m);
        if (l == 0 && r0 + i < rows) o.s[ct * o.lds + r0 + i] = block_scale(m);
      }
    }
    if (o.qt != nullptr) {
      float cm[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float m = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i][j]));
        cm[j] = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
      }
      if (half == 0) {
#pragma unroll
        for (int j = 0; j < 8; ++j) cmax[warp][l * 8 + j] = cm[j];
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float m = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = fmaxf(m, cmax[w][l * 8 + j]);
        colr[j] = block_factor(m);
        if (warp == 0 && half == 0 && c0 + j < cols)
          o.st[rt * o.ldst + c0 + j] = block_scale(m);
      }
    }
  } else {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[i][j]));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) cmax[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = fmaxf(m, cmax[0][w]);
    const float f = block_factor(m);
#pragma unroll
    for (int j = 0; j < 8; ++j) colr[j] = rowr[j] = f;
    if (tid == 0) {
      if (o.q != nullptr) o.s[ct * o.lds + rt] = block_scale(m);
      if (o.qt != nullptr) o.st[rt * o.ldst + ct] = block_scale(m);
    }
  }

  if (o.q != nullptr && c0 < cols) {
    const int valid = (int)(cols - c0 < 8 ? cols - c0 : 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (r0 + i < rows) {
        const float f = rowr[i];
        uint2 c;
        c.x = e4m3x4(__fmul_rn(v[i][0], f), __fmul_rn(v[i][1], f),
                     __fmul_rn(v[i][2], f), __fmul_rn(v[i][3], f));
        c.y = e4m3x4(__fmul_rn(v[i][4], f), __fmul_rn(v[i][5], f),
                     __fmul_rn(v[i][6], f), __fmul_rn(v[i][7], f));
        store8(o.q + (r0 + i) * o.ldq + c0, c, valid);
      }
    }
  }
  if (o.qt != nullptr) {
    // transposed tile: column c's 128 bytes in 16 chunks of 8, chunk k stored
    // at k ^ (c / 8) so that the 16 lanes' stores (columns 8 apart) and the
    // reads below each touch every bank once
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float f = colr[j];
      uint2 c;
      c.x = e4m3x4(__fmul_rn(v[0][j], f), __fmul_rn(v[1][j], f),
                   __fmul_rn(v[2][j], f), __fmul_rn(v[3][j], f));
      c.y = e4m3x4(__fmul_rn(v[4][j], f), __fmul_rn(v[5][j], f),
                   __fmul_rn(v[6][j], f), __fmul_rn(v[7][j], f));
      const int chunk = (warp * 2 + half) ^ l;
      *reinterpret_cast<uint2*>(tile_t + (l * 8 + j) * TILE + chunk * 8) = c;
    }
    __syncthreads();
    const int64_t rr = rt * TILE + l * 8;   // eight rows of the source
    const int valid = (int)(rows - rr < 8 ? rows - rr : 8);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = warp * 16 + i * 2 + half;
      const int64_t cc = ct * TILE + c;
      const int chunk = l ^ (c >> 3);
      const uint2 u =
          *reinterpret_cast<const uint2*>(tile_t + c * TILE + chunk * 8);
      if (cc < cols && valid > 0) store8(o.qt + cc * o.ldqt + rr, u, valid);
    }
  }
}

template <typename SRC>
int launch_tiles(const SRC& src, int group, int64_t rows, int64_t cols,
                 const Fp8BlockOut& o, double bytes, cudaStream_t s) {
  const int64_t ct = (cols + TILE - 1) / TILE, rt = (rows + TILE - 1) / TILE;
  if (ct * rt > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(ct * rt);
  {
    ProfScope ps(s, KF_QUANT, 0.0, bytes);
    if (group == kFp8Row)
      quantize_tile_kernel<SRC, kFp8Row>
          <<<grid, TILE_THREADS, 0, s>>>(src, rows, cols, ct, o);
    else
      quantize_tile_kernel<SRC, kFp8Block>
          <<<grid, TILE_THREADS, 0, s>>>(src, rows, cols, ct, o);
  }
  count_launch();
  return cudaGetLastError();
}

bool vec_rows(const void* p, int64_t ld, int elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (ld * elem) % 16 == 0;
}

double out_bytes(const Fp8BlockOut& o, int64_t rows, int64_t cols) {
  return (double)rows * cols * ((o.q != nullptr) + (o.qt != nullptr));
}

// ----------------------------------------------------- residual + RMSNorm --
// One CTA per row; the row stays in registers (V vectors of eight columns a
// thread), 16 neighbouring threads hold one group of 128.
template <int V>
__global__ void __launch_bounds__(256)
    add_rmsnorm_fp8_kernel(const __nv_bfloat16* x, const __nv_bfloat16* r,
                           const __nv_bfloat16* __restrict__ gamma,
                           __nv_bfloat16* x1, __nv_bfloat16* y,
                           float* __restrict__ rstd, uint8_t* q, int64_t ldq,
                           float* s, int64_t lds, int64_t h, float eps,
                           bool vec) {
  __shared__ float red[8];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  float v[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int64_t c = (int64_t)(k * 256 + tid) * 8;
    const int valid = (int)(h - c < 8 ? h - c : 8);
    if (valid > 0) {
      // x1 may be x or r: plain loads, each element read before it is written
      float a[8];
      if (vec) {
        const uint4 u = *reinterpret_cast<const uint4*>(x + row * h + c);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 t = unpack_bf16x2(w[j]);
          a[2 * j] = t.x;
          a[2 * j + 1] = t.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          a[j] = j < valid ? __bfloat162float(x[row * h + c + j]) : 0.0f;
      }
      if (r != nullptr) {
        float b[8];
        if (vec) {
          const uint4 u = *reinterpret_cast<const uint4*>(r + row * h + c);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 t = unpack_bf16x2(w[j]);
            b[2 * j] = t.x;
            b[2 * j + 1] = t.y;
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            b[j] = j < valid ? __bfloat162float(r[row * h + c + j]) : 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j)   // the stored stream is what is normed
          a[j] = __bfloat162float(__float2bfloat16_rn(a[j] + b[j]));
      }
      if (x1 != nullptr) {
        if (vec) {
          uint4 u;
          u.x = pack_bf16x2(a[0], a[1]);
          u.y = pack_bf16x2(a[2], a[3]);
          u.z = pack_bf16x2(a[4], a[5]);
          u.w = pack_bf16x2(a[6], a[7]);
          *reinterpret_cast<uint4*>(x1 + row * h + c) = u;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < valid) x1[row * h + c + j] = __float2bfloat16_rn(a[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        v[k][j] = a[j];
        ss += a[j] * a[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[k][j] = 0.0f;
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if ((tid & 31) == 0) red[tid >> 5] = ss;
  __syncthreads();
  float tot = 0.0f;
#pragma unroll
  for (int w = 0; w < 8; ++w) tot += red[w];
  const float rs = rsqrtf(tot / (float)h + eps);
  if (tid == 0) rstd[row] = rs;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int64_t c = (int64_t)(k * 256 + tid) * 8;
    const int valid = (int)(h - c < 8 ? h - c : 8);
    float g[8];
    load8(gamma + c, valid, vec, g);
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[k][j] = v[k][j] * rs * g[j];
      m = fmaxf(m, fabsf(v[k][j]));
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (valid > 0) {
      const float f = block_factor(m);
      uint2 u;
      u.x = e4m3x4(__fmul_rn(v[k][0], f), __fmul_rn(v[k][1], f),
                   __fmul_rn(v[k][2], f), __fmul_rn(v[k][3], f));
      u.y = e4m3x4(__fmul_rn(v[k][4], f), __fmul_rn(v[k][5], f),
                   __fmul_rn(v[k][6], f), __fmul_rn(v[k][7], f));
      store8(q + row * ldq + c, u, valid);
      if ((tid & 15) == 0) s[(c >> 7) * lds + row] = block_scale(m);
      if (y != nullptr) {
        if (vec) {
          uint4 w;
          w.x = pack_bf16x2(v[k][0], v[k][1]);
          w.y = pack_bf16x2(v[k][2], v[k][3]);
          w.z = pack_bf16x2(v[k][4], v[k][5]);
          w.w = pack_bf16x2(v[k][6], v[k][7]);
          *reinterpret_cast<uint4*>(y + row * h + c) = w;
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < valid) y[row * h + c + j] = __float2bfloat16_rn(v[k][j]);
        }
      }
    }
  }
}

}  // namespace

int quantize_fp8_block(int dtype, int group, int64_t rows, int64_t cols,
                       const void* x, int64_t ldx, const Fp8BlockOut& o,
                       void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == 0) {
    const CopySource<float> src{static_cast<const float*>(x), ldx,
                                vec_rows(x, ldx, 4)};
    return launch_tiles(src, group, rows, cols, o,
                        4.0 * rows * cols + out_bytes(o, rows, cols), s);
  }
  const CopySource<__nv_bfloat16> src{static_cast<const __nv_bfloat16*>(x),
                                      ldx, vec_rows(x, ldx, 2)};
  return launch_tiles(src, group, rows, cols, o,
                      2.0 * rows * cols + out_bytes(o, rows, cols), s);
}

int swiglu_fp8_fwd(int64_t T, int64_t f, const void* gu, int64_t ldgu,
                   const Fp8BlockOut& o, void* stream) {
  const SwigluSource src{static_cast<const __nv_bfloat16*>(gu), ldgu, f,
                         vec_rows(gu, ldgu, 2) && f % 8 == 0};
  return launch_tiles(src, kFp8Row, T, f, o, 4.0 * T * f + out_bytes(o, T, f),
                      static_cast<cudaStream_t>(stream));
}

int swiglu_fp8_bwd(int64_t T, int64_t f, const void* da, int64_t ldda,
                   const void* gu, int64_t ldgu, const Fp8BlockOut& o,
                   void* stream) {
  const SwigluBwdSource src{
      static_cast<const __nv_bfloat16*>(da),
      static_cast<const __nv_bfloat16*>(gu), ldda, ldgu, f,
      vec_rows(gu, ldgu, 2) && vec_rows(da, ldda, 2) && f % 8 == 0};
  return launch_tiles(src, kFp8Row, T, 2 * f, o,
                      6.0 * T * f + out_bytes(o, T, 2 * f),
                      static_cast<cudaStream_t>(stream));
}

int add_rmsnorm_fp8_fwd(int64_t T, int64_t h, float eps, const void* x,
                        const void* r, const void* gamma, void* x1, void* y,
                        float* rstd, uint8_t* q, int64_t ldq, float* s,
                        int64_t lds, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto bf = [](const void* p) { return static_cast<const __nv_bfloat16*>(p); };
  auto al = [](const void* p) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;   // null counts
  };
  const bool vec =
      h % 8 == 0 && al(x) && al(r) && al(gamma) && al(x1) && al(y);
  auto* o1 = static_cast<__nv_bfloat16*>(x1);
  auto* oy = static_cast<__nv_bfloat16*>(y);
  {
    ProfScope ps(st, KF_NORM, 4.0 * T * h,
                 (2.0 + 2.0 * (r != nullptr) + 2.0 * (x1 != nullptr) +
                  2.0 * (y != nullptr) + 1.0) * T * h);
    const unsigned grid = (unsigned)T;
    if (h <= 2048)
      add_rmsnorm_fp8_kernel<1><<<grid, 256, 0, st>>>(
          bf(x), bf(r), bf(gamma), o1, oy, rstd, q, ldq, s, lds, h, eps, vec);
    else if (h <= 4096)
      add_rmsnorm_fp8_kernel<2><<<grid, 256, 0, st>>>(
          bf(x), bf(r), bf(gamma), o1, oy, rstd, q, ldq, s, lds, h, eps, vec);
    else if (h <= 8192)
      add_rmsnorm_fp8_kernel<4><<<grid, 256, 0, st>>>(
          bf(x), bf(r), bf(gamma), o1, oy, rstd, q, ldq, s, lds, h, eps, vec);
    else
      add_rmsnorm_fp8_kernel<8><<<grid, 256, 0, st>>>(
          bf(x), bf(r), bf(gamma), o1, oy, rstd, q, ldq, s, lds, h, eps, vec);
  }
  count_launch();
  return cudaGetLastError();
}

}  // namespace tp
