// fp8_block.cu — the operators that write block-scaled E4M3 codes:
// quantization, SwiGLU (forward and backward) and residual + RMSNorm.
//
// With amax the largest magnitude of a block of 128 (1×128 or 128×128),
//   r = 448 / amax,  s = amax / 448  (fp32),  q = e4m3(x·r),
// values are taken in fp32 straight from the producing formula (SwiGLU, norm:
// no rounding to bf16 in between) and rounded once, to E4M3.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "common.cuh"
#include "fp8.cuh"
#include "fp8_block.h"
#include "gemm.h"
#include "profile.h"

namespace tp {
namespace {

// ------------------------------------------------------------ tile kernel --
// One CTA per 128×128 tile of the output matrix.  Thread (warp w, half-warp g,
// lane l of 16) holds R rows (2w + g)·R + i and columns 8l + j.  A thread's
// loads are issued BATCH rows at a time before any is used (a source's
// raw()): the registers of the CTAs on an SM are the buffer of what is in
// flight.  A source's R, BATCH and CTAS (on an SM) are what its values leave
// room for: bf16 values are kept as loaded (8 rows, four CTAs of 256
// threads), computed ones as fp32 (4 rows, two CTAs of 512).
constexpr int TILE = 128;

__device__ __forceinline__ void unpack8(const uint4& u, float* v) {
  const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y),
               c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
}
// Eight elements; those at and beyond `valid` are 0 and not read.
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p, int valid,
                                       bool vec) {
  if (vec && valid >= 8) return __ldg(reinterpret_cast<const uint4*>(p));
  uint32_t w[4] = {0, 0, 0, 0};
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < valid) w[j >> 1] |= (uint32_t)h[j] << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A source: raw() loads eight columns of a row (columns at and beyond `cols`
// give 0), value() makes them fp32.
struct CopyBf16 {
  static constexpr int RAW = 1, R = 8, BATCH = 8, CTAS = 4;
  const __nv_bfloat16* x;
  int64_t ld;
  bool vec;
  __device__ __forceinline__ void raw(int64_t r, int64_t c, int64_t cols,
                                      uint4* u) const {
    u[0] = load8(x + r * ld + c, (int)(cols - c < 8 ? cols - c : 8), vec);
  }
  __device__ __forceinline__ void value(const uint4* u, int64_t, float* v) const {
    unpack8(u[0], v);
  }
  __device__ int64_t col_tile(int64_t j, int64_t) const { return j; }
};

struct CopyF32 {
  static constexpr int RAW = 2, R = 4, BATCH = 4, CTAS = 2;
  const float* x;
  int64_t ld;
  bool vec;
  __device__ __forceinline__ void raw(int64_t r, int64_t c, int64_t cols,
                                      uint4* u) const {
    const float* p = x + r * ld + c;
    if (vec && cols - c >= 8) {
      u[0] = __ldg(reinterpret_cast<const uint4*>(p));
      u[1] = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    } else {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = c + j < cols ? __float_as_uint(p[j]) : 0u;
      u[0] = make_uint4(w[0], w[1], w[2], w[3]);
      u[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  __device__ __forceinline__ void value(const uint4* u, int64_t, float* v) const {
    v[0] = __uint_as_float(u[0].x); v[1] = __uint_as_float(u[0].y);
    v[2] = __uint_as_float(u[0].z); v[3] = __uint_as_float(u[0].w);
    v[4] = __uint_as_float(u[1].x); v[5] = __uint_as_float(u[1].y);
    v[6] = __uint_as_float(u[1].z); v[7] = __uint_as_float(u[1].w);
  }
  __device__ int64_t col_tile(int64_t j, int64_t) const { return j; }
};

// σ(x), the quotient by the approximate division (2 ulp): the values only go
// to E4M3, and an IEEE division is a third of the kernel's instructions.
__device__ __forceinline__ float sigmoid_approx(float x) {
  return __fdividef(1.0f, 1.0f + __expf(-x));
}

// A = SiLU(G)·U.
template <bool VEC>   // 16-byte loads: f a multiple of 8, rows aligned
struct SwigluSource {
  static constexpr int RAW = 2, R = 4, BATCH = 4, CTAS = 2;
  const __nv_bfloat16* gu;
  int64_t ld, f;
  __device__ __forceinline__ void raw(int64_t r, int64_t c, int64_t cols,
                                      uint4* u) const {
    const int valid = (int)(cols - c < 8 ? cols - c : 8);
    const __nv_bfloat16* p = gu + r * ld + c;
    u[0] = load8(p, VEC ? 8 : valid, VEC);
    u[1] = load8(p + f, VEC ? 8 : valid, VEC);
  }
  __device__ __forceinline__ void value(const uint4* x, int64_t, float* v) const {
    float g[8], u[8];
    unpack8(x[0], g);
    unpack8(x[1], u);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = g[j] * sigmoid_approx(g[j]) * u[j];
  }
  __device__ int64_t col_tile(int64_t j, int64_t) const { return j; }
};

// [dG | dU]: dG = dA·U·s·(1 + G·(1 − s)), dU = dA·G·s with s = σ(G).  The
// multiplier of the up side is read for dG alone; which side a column is on
// may change inside eight columns when f is not a multiple of 8.
template <bool VEC>
struct SwigluBwdSource {
  static constexpr int RAW = 3, R = 4, BATCH = 2, CTAS = 2;
  const __nv_bfloat16 *da, *gu;
  int64_t ldda, ld, f;
  __device__ __forceinline__ void raw(int64_t r, int64_t c, int64_t cols,
                                      uint4* u) const {
    const __nv_bfloat16* pa = da + r * ldda;
    const __nv_bfloat16* pg = gu + r * ld;
    if (VEC) {   // all eight columns on one side
      const bool up = c >= f;
      const int64_t k = up ? c - f : c;
      u[0] = __ldg(reinterpret_cast<const uint4*>(pa + k));
      u[1] = __ldg(reinterpret_cast<const uint4*>(pg + k));
      u[2] = up ? make_uint4(0, 0, 0, 0)
                : __ldg(reinterpret_cast<const uint4*>(pg + f + k));
      return;
    }
    const uint16_t* ha = reinterpret_cast<const uint16_t*>(pa);
    const uint16_t* hg = reinterpret_cast<const uint16_t*>(pg);
    uint32_t w[3][4] = {};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int64_t cj = c + j;
      const int sh = 16 * (j & 1);
      if (cj < f) {
        w[0][j >> 1] |= (uint32_t)ha[cj] << sh;
        w[1][j >> 1] |= (uint32_t)hg[cj] << sh;
        w[2][j >> 1] |= (uint32_t)hg[f + cj] << sh;
      } else if (cj < cols) {
        w[0][j >> 1] |= (uint32_t)ha[cj - f] << sh;
        w[1][j >> 1] |= (uint32_t)hg[cj - f] << sh;
      }
    }
#pragma unroll
    for (int k = 0; k < 3; ++k)
      u[k] = make_uint4(w[k][0], w[k][1], w[k][2], w[k][3]);
  }
  __device__ __forceinline__ void value(const uint4* x, int64_t c,
                                        float* v) const {
    float a[8], g[8], u[8];
    unpack8(x[0], a);
    unpack8(x[1], g);
    unpack8(x[2], u);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = sigmoid_approx(g[j]);
      v[j] = c + (VEC ? 0 : j) < f ? a[j] * u[j] * s * (1.0f + g[j] * (1.0f - s))
                       : a[j] * g[j] * s;
    }
  }
  // the dG tile and the dU tile of the same hidden units run side by side, so
  // that the second reads dA and G from L2
  __device__ int64_t col_tile(int64_t j, int64_t n) const {
    return (j & 1) ? (n + 1) / 2 + (j >> 1) : (j >> 1);
  }
};

// What a thread keeps of its R×8 elements: bf16 as loaded, else fp32.
template <typename SRC>
struct Held {
  static constexpr int R = SRC::R;
  float v[R][8];
  __device__ __forceinline__ void take(const SRC& src, int i, const uint4* u,
                                       int64_t c) {
    src.value(u, c, v[i]);
  }
  __device__ __forceinline__ void row(int i, float* o) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = v[i][j];
  }
  __device__ __forceinline__ float at(int i, int j) const { return v[i][j]; }
  __device__ __forceinline__ float row_max(int i) const {
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[i][j]));
    return m;
  }
  __device__ __forceinline__ void col_max(float* m) const {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[j] = 0.0f;
#pragma unroll
      for (int i = 0; i < R; ++i) m[j] = fmaxf(m[j], fabsf(v[i][j]));
    }
  }
};
// Largest magnitudes two at a time on the packed values (a bf16 maximum is
// exact; like fmaxf it takes the other operand where one is NaN).
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  __nv_bfloat162 x, y;
  a &= 0x7FFF7FFFu;
  b &= 0x7FFF7FFFu;
  memcpy(&x, &a, 4);
  memcpy(&y, &b, 4);
  x = __hmax2(x, y);
  memcpy(&a, &x, 4);
  return a;
}
template <>
struct Held<CopyBf16> {
  uint4 u[8];
  __device__ __forceinline__ void take(const CopyBf16&, int i, const uint4* x,
                                       int64_t) {
    u[i] = x[0];
  }
  __device__ __forceinline__ void row(int i, float* o) const { unpack8(u[i], o); }
  __device__ __forceinline__ uint32_t word(int i, int w) const {
    return w == 0 ? u[i].x : w == 1 ? u[i].y : w == 2 ? u[i].z : u[i].w;
  }
  __device__ __forceinline__ float at(int i, int j) const {
    const float2 t = unpack_bf16x2(word(i, j >> 1));
    return j & 1 ? t.y : t.x;
  }
  __device__ __forceinline__ float row_max(int i) const {
    const uint32_t m = max_abs2(max_abs2(u[i].x, u[i].y),
                                max_abs2(u[i].z, u[i].w));
    const float2 t = unpack_bf16x2(max_abs2(m, 0));
    return fmaxf(t.x, t.y);
  }
  __device__ __forceinline__ void col_max(float* m) const {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t x = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) x = max_abs2(x, word(i, w));
      const float2 t = unpack_bf16x2(x);
      m[2 * w] = t.x;
      m[2 * w + 1] = t.y;
    }
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

__device__ __forceinline__ uint2 codes8(const float* v, float f) {
  uint2 c;
  c.x = e4m3x4(__fmul_rn(v[0], f), __fmul_rn(v[1], f), __fmul_rn(v[2], f),
               __fmul_rn(v[3], f));
  c.y = e4m3x4(__fmul_rn(v[4], f), __fmul_rn(v[5], f), __fmul_rn(v[6], f),
               __fmul_rn(v[7], f));
  return c;
}

// A row's codes leave as 16 lanes × 8 bytes; a column's largest magnitude
// takes one shuffle and one pass through shared memory; R rows of a column
// pack into one R-byte shared-memory store of the transposed tile, whose rows
// then leave the same way.
template <typename SRC, int GROUP>
__global__ void __launch_bounds__(2048 / SRC::R, SRC::CTAS)
    quantize_tile_kernel(const SRC src, int64_t rows, int64_t cols,
                         int64_t col_tiles, const Fp8BlockOut o) {
  constexpr int R = SRC::R, WARPS = 64 / R;
  __shared__ __align__(16) float cmax[WARPS][TILE];
  __shared__ __align__(16) uint8_t tile_t[TILE * TILE];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = lane >> 4, l = lane & 15;
  const int64_t rt = blockIdx.x / col_tiles;
  const int64_t ct = src.col_tile(blockIdx.x - rt * col_tiles, col_tiles);
  const int64_t r0 = rt * TILE + (warp * 2 + half) * R;
  const int64_t c0 = ct * TILE + l * 8;

  Held<SRC> h;
#pragma unroll
  for (int b = 0; b < R; b += SRC::BATCH) {
    uint4 u[SRC::BATCH][SRC::RAW];
#pragma unroll
    for (int i = 0; i < SRC::BATCH; ++i) {
#pragma unroll
      for (int k = 0; k < SRC::RAW; ++k) u[i][k] = make_uint4(0, 0, 0, 0);
      if (r0 + b + i < rows && c0 < cols) src.raw(r0 + b + i, c0, cols, u[i]);
    }
#pragma unroll
    for (int i = 0; i < SRC::BATCH; ++i) h.take(src, b + i, u[i], c0);
  }

  float colr[8];   // the factor of each of this thread's columns
  float rowr[R];   // and of each of its rows
  if (GROUP == kFp8Row) {
    if (o.q != nullptr) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float m = h.row_max(i);
#pragma unroll
        for (int d = 8; d > 0; d >>= 1)
          m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        rowr[i] = block_factor(m);
        if (l == 0 && r0 + i < rows) o.s[ct * o.lds + r0 + i] = block_scale(m);
      }
    }
    if (o.qt != nullptr) {
      float cm[8];
      h.col_max(cm);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        cm[j] = fmaxf(cm[j], __shfl_xor_sync(0xffffffffu, cm[j], 16));
      if (half == 0) {
        float4* d = reinterpret_cast<float4*>(&cmax[warp][l * 8]);
        d[0] = make_float4(cm[0], cm[1], cm[2], cm[3]);
        d[1] = make_float4(cm[4], cm[5], cm[6], cm[7]);
      }
      __syncthreads();
      if (tid < TILE) {   // a column each: its factor, and its scale
        float m = cmax[0][tid];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) m = fmaxf(m, cmax[w][tid]);
        const int64_t c = ct * TILE + tid;
        if (c < cols) o.st[rt * o.ldst + c] = block_scale(m);
        cmax[0][tid] = block_factor(m);   // read by this thread alone so far
      }
      __syncthreads();
      const float4* d = reinterpret_cast<const float4*>(&cmax[0][l * 8]);
      const float4 x = d[0], y = d[1];
      colr[0] = x.x; colr[1] = x.y; colr[2] = x.z; colr[3] = x.w;
      colr[4] = y.x; colr[5] = y.y; colr[6] = y.z; colr[7] = y.w;
    }
  } else {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < R; ++i) m = fmaxf(m, h.row_max(i));
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (lane == 0) cmax[0][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) m = fmaxf(m, cmax[0][w]);
    const float f = block_factor(m);
#pragma unroll
    for (int j = 0; j < 8; ++j) colr[j] = f;
#pragma unroll
    for (int i = 0; i < R; ++i) rowr[i] = f;
    if (tid == 0) {
      if (o.q != nullptr) o.s[ct * o.lds + rt] = block_scale(m);
      if (o.qt != nullptr) o.st[rt * o.ldst + ct] = block_scale(m);
    }
  }

  if (o.q != nullptr && c0 < cols) {
    const int valid = (int)(cols - c0 < 8 ? cols - c0 : 8);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (r0 + i < rows) {
        float v[8];
        h.row(i, v);
        store8(o.q + (r0 + i) * o.ldq + c0, codes8(v, rowr[i]), valid);
      }
    }
  }
  if (o.qt != nullptr) {
    // transposed tile: column c's 128 bytes in 16 chunks of 8, chunk k stored
    // at k ^ (c / 8) so that the lanes' stores (columns 8 apart) and the reads
    // below each touch every bank once
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      uint8_t* d = tile_t + (l * 8 + j) * TILE;
      const float f = colr[j];
      const uint32_t lo =
          e4m3x4(__fmul_rn(h.at(0, j), f), __fmul_rn(h.at(1, j), f),
                 __fmul_rn(h.at(2, j), f), __fmul_rn(h.at(3, j), f));
      if constexpr (R == 8) {
        const uint32_t hi =
            e4m3x4(__fmul_rn(h.at(4, j), f), __fmul_rn(h.at(5, j), f),
                   __fmul_rn(h.at(6, j), f), __fmul_rn(h.at(7, j), f));
        *reinterpret_cast<uint2*>(d + ((warp * 2 + half) ^ l) * 8) =
            make_uint2(lo, hi);
      } else {
        *reinterpret_cast<uint32_t*>(d + (warp ^ l) * 8 + half * 4) = lo;
      }
    }
    __syncthreads();
    const int64_t rr = rt * TILE + l * 8;   // eight rows of the source
    const int valid = (int)(rows - rr < 8 ? rows - rr : 8);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = (warp * R + i) * 2 + half;
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
          <<<grid, 2048 / SRC::R, 0, s>>>(src, rows, cols, ct, o);
    else
      quantize_tile_kernel<SRC, kFp8Block>
          <<<grid, 2048 / SRC::R, 0, s>>>(src, rows, cols, ct, o);
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
// One CTA per row, which stays in registers: V vectors of eight columns a
// thread, 16 neighbouring threads hold one group of 128.  γ is read before the
// row's sum is known, so that its latency is not paid after the barrier.
template <int THREADS, int V, int CTAS, bool VEC>
__global__ void __launch_bounds__(THREADS, CTAS)
    add_rmsnorm_fp8_kernel(const __nv_bfloat16* x, const __nv_bfloat16* r,
                           const __nv_bfloat16* __restrict__ gamma,
                           __nv_bfloat16* x1, __nv_bfloat16* y,
                           float* __restrict__ rstd, uint8_t* q, int64_t ldq,
                           float* s, int64_t lds, int h, float eps) {
  __shared__ float red[THREADS / 32];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  // x1 may be x or r: no read-only loads, and each element is read before it
  // is written, by the same thread
  auto load = [&](const __nv_bfloat16* p, int c) -> uint4 {
    if (VEC) return *reinterpret_cast<const uint4*>(p + c);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j < h)
        w[j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[c + j]
                     << (16 * (j & 1));
    return make_uint4(w[0], w[1], w[2], w[3]);
  };
  auto save = [&](__nv_bfloat16* p, int c, const uint4& u) {
    if (VEC) {
      *reinterpret_cast<uint4*>(p + c) = u;
    } else {
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < h)
          reinterpret_cast<uint16_t*>(p)[c + j] =
              (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
    }
  };
  uint4 u[V], ur[V], g[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * THREADS + tid) * 8;
    u[k] = ur[k] = make_uint4(0, 0, 0, 0);
    if (c < h) {
      u[k] = load(x + row * h, c);
      if (r != nullptr) ur[k] = load(r + row * h, c);
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * THREADS + tid) * 8;
    g[k] = make_uint4(0, 0, 0, 0);
    if (c < h) g[k] = load8(gamma + c, h - c < 8 ? h - c : 8, VEC);
  }
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * THREADS + tid) * 8;
    if (r != nullptr) {   // the stored stream is what is normed
      float a[8], b[8];
      unpack8(u[k], a);
      unpack8(ur[k], b);
      u[k].x = pack_bf16x2(a[0] + b[0], a[1] + b[1]);
      u[k].y = pack_bf16x2(a[2] + b[2], a[3] + b[3]);
      u[k].z = pack_bf16x2(a[4] + b[4], a[5] + b[5]);
      u[k].w = pack_bf16x2(a[6] + b[6], a[7] + b[7]);
    }
    if (x1 != nullptr && c < h) save(x1 + row * h, c, u[k]);
    float a[8];
    unpack8(u[k], a);
#pragma unroll
    for (int j = 0; j < 8; ++j) ss += a[j] * a[j];
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if ((tid & 31) == 0) red[tid >> 5] = ss;
  __syncthreads();
  float tot = 0.0f;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) tot += red[w];
  const float rs = rsqrtf(tot / (float)h + eps);
  if (tid == 0) rstd[row] = rs;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * THREADS + tid) * 8;
    float v[8], gm[8];
    unpack8(u[k], v);
    unpack8(g[k], gm);
    float m = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[j] = v[j] * rs * gm[j];
      m = fmaxf(m, fabsf(v[j]));
    }
#pragma unroll
    for (int d = 8; d > 0; d >>= 1)
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    if (c < h) {
      store8(q + row * ldq + c, codes8(v, block_factor(m)), VEC ? 8 : h - c);
      if ((tid & 15) == 0) s[(c >> 7) * lds + row] = block_scale(m);
      if (y != nullptr)
        save(y + row * h, c,
             make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                        pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])));
    }
  }
}

}  // namespace

int quantize_fp8_block(int dtype, int group, int64_t rows, int64_t cols,
                       const void* x, int64_t ldx, const Fp8BlockOut& o,
                       void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == 0) {
    const CopyF32 src{static_cast<const float*>(x), ldx, vec_rows(x, ldx, 4)};
    return launch_tiles(src, group, rows, cols, o,
                        4.0 * rows * cols + out_bytes(o, rows, cols), s);
  }
  const CopyBf16 src{static_cast<const __nv_bfloat16*>(x), ldx,
                     vec_rows(x, ldx, 2)};
  return launch_tiles(src, group, rows, cols, o,
                      2.0 * rows * cols + out_bytes(o, rows, cols), s);
}

int swiglu_fp8_fwd(int64_t T, int64_t f, const void* gu, int64_t ldgu,
                   const Fp8BlockOut& o, void* stream) {
  const auto* x = static_cast<const __nv_bfloat16*>(gu);
  const double bytes = 4.0 * T * f + out_bytes(o, T, f);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (vec_rows(gu, ldgu, 2) && f % 8 == 0)
    return launch_tiles(SwigluSource<true>{x, ldgu, f}, kFp8Row, T, f, o, bytes,
                        s);
  return launch_tiles(SwigluSource<false>{x, ldgu, f}, kFp8Row, T, f, o, bytes,
                      s);
}

int swiglu_fp8_bwd(int64_t T, int64_t f, const void* da, int64_t ldda,
                   const void* gu, int64_t ldgu, const Fp8BlockOut& o,
                   void* stream) {
  const auto* a = static_cast<const __nv_bfloat16*>(da);
  const auto* x = static_cast<const __nv_bfloat16*>(gu);
  const double bytes = 6.0 * T * f + out_bytes(o, T, 2 * f);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (vec_rows(gu, ldgu, 2) && vec_rows(da, ldda, 2) && f % 8 == 0)
    return launch_tiles(SwigluBwdSource<true>{a, x, ldda, ldgu, f}, kFp8Row, T,
                        2 * f, o, bytes, s);
  return launch_tiles(SwigluBwdSource<false>{a, x, ldda, ldgu, f}, kFp8Row, T,
                      2 * f, o, bytes, s);
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
    auto go = [&](auto vec_kernel, auto any_kernel, int threads) {
      auto k = vec ? vec_kernel : any_kernel;
      k<<<(unsigned)T, threads, 0, st>>>(bf(x), bf(r), bf(gamma), o1, oy, rstd,
                                         q, ldq, s, lds, (int)h, eps);
    };
    if (h <= 1024)
      go(add_rmsnorm_fp8_kernel<128, 1, 12, true>,
         add_rmsnorm_fp8_kernel<128, 1, 8, false>, 128);
    else if (h <= 2048)
      go(add_rmsnorm_fp8_kernel<256, 1, 6, true>,
         add_rmsnorm_fp8_kernel<256, 1, 4, false>, 256);
    else if (h <= 4096)
      go(add_rmsnorm_fp8_kernel<512, 1, 3, true>,
         add_rmsnorm_fp8_kernel<512, 1, 2, false>, 512);
    else if (h <= 8192)
      go(add_rmsnorm_fp8_kernel<512, 2, 3, true>,
         add_rmsnorm_fp8_kernel<512, 2, 2, false>, 512);
    else
      go(add_rmsnorm_fp8_kernel<1024, 2, 1, true>,
         add_rmsnorm_fp8_kernel<1024, 2, 1, false>, 1024);
  }
  count_launch();
  return cudaGetLastError();
}

}  // namespace tp
