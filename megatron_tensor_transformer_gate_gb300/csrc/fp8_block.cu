// fp8_block.cu — the operators that write block-scaled E4M3 codes:
// quantization, SwiGLU (forward and backward) and residual + RMSNorm.
//
// All of them read and write every byte once, so DRAM is their floor (figures
// here are against a copy's 6.67 TB/s, device time of a launch, inputs not in
// L2).
//
// With amax the largest magnitude of a block of 128 (1×128 or 128×128),
//   r = 448 / amax,  s = amax / 448  (fp32),  q = e4m3(x·r),
// values are taken in fp32 straight from the producing formula (SwiGLU, norm:
// no rounding to bf16 in between) and rounded once, to E4M3.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
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
// flight.  A source's shapes (rows a thread, BATCH, CTAs on an SM) are what its
// values leave room for: bf16 values are kept as loaded (8 rows, four CTAs of
// 256 threads), computed ones as fp32.  For these three CTAs of 256 threads
// (8 rows) overlap loads and arithmetic better than two of 512 (4 rows), whose
// phases fall into step: SwiGLU both ways 97 against 109 µs at 8192×11008,
// fp32 8192×8192 62 against 68.
//
// Measured: 128×128 blocks and their transpose of a bf16 8192×28672 142 µs
// (6.6 TB/s, 99 %); row scales both ways of 8192×8192 45.5 µs (5.9 TB/s, 89 %),
// of 8192×8191 (rows on two bytes) 68; of fp32 8192×8192 62 (97 %); SwiGLU both
// ways 8192×11008 97 µs (84 %).  With row scales both ways a value is scaled
// and rounded twice, by different factors: instructions, and the two barriers
// around the columns' maxima, count beside DRAM there.  Loading the next tile
// asynchronously while one is worked on measured slower.
constexpr int TILE = 128;

__device__ __forceinline__ void unpack8(const uint4& u, float* v) {
  const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y),
               c = unpack_bf16x2(u.z), d = unpack_bf16x2(u.w);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
}
// 16 bytes in pieces of W that are W-aligned.
template <int W>
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 u;
  if constexpr (W == 16) {
    u = __ldg(static_cast<const uint4*>(p));
  } else if constexpr (W == 8) {
    const uint2 a = __ldg(static_cast<const uint2*>(p)),
                b = __ldg(static_cast<const uint2*>(p) + 1);
    u = make_uint4(a.x, a.y, b.x, b.y);
  } else if constexpr (W == 4) {
    const uint32_t* w = static_cast<const uint32_t*>(p);
    u = make_uint4(__ldg(w), __ldg(w + 1), __ldg(w + 2), __ldg(w + 3));
  } else {
    const uint16_t* h = static_cast<const uint16_t*>(p);
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = (uint32_t)__ldg(h + 2 * j) | ((uint32_t)__ldg(h + 2 * j + 1) << 16);
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return u;
}
// Eight bf16; those at and beyond `valid` are 0 and not read.
template <int W>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* p, int valid) {
  if (valid >= 8) return load16<W>(p);
  uint32_t w[4] = {0, 0, 0, 0};
  const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < valid) w[j >> 1] |= (uint32_t)h[j] << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <int W>
__device__ __forceinline__ void save8(__nv_bfloat16* p, const uint4& u,
                                      int valid) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  if (W == 16) {   // rows of a multiple of eight
    *reinterpret_cast<uint4*>(p) = u;
  } else if (W == 8 && valid >= 8) {
    reinterpret_cast<uint2*>(p)[0] = make_uint2(u.x, u.y);
    reinterpret_cast<uint2*>(p)[1] = make_uint2(u.z, u.w);
  } else if (W == 4 && valid >= 8) {
#pragma unroll
    for (int j = 0; j < 4; ++j) reinterpret_cast<uint32_t*>(p)[j] = w[j];
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < valid)
        reinterpret_cast<uint16_t*>(p)[j] =
            (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
  }
}

// How many of a thread's eight columns exist, of `left`; WHOLE: all of them.
template <bool WHOLE>
__device__ __forceinline__ int columns(int64_t left) {
  return WHOLE || left >= 8 ? 8 : (int)left;
}

// Rows a thread, rows whose loads are issued together, CTAs on an SM.  A source
// has one for rows alone, one for tiles and one for few tiles.
template <int R_, int BATCH_, int CTAS_>
struct Shape {
  static constexpr int R = R_, BATCH = BATCH_, CTAS = CTAS_;
};

// A source: raw() loads eight columns of a row (W: the bytes that its rows'
// starts and pitch are multiples of, at most 16) (columns at and beyond `cols`
// give 0), value() makes them fp32.
template <int W>
struct CopyBf16 {
  static constexpr int RAW = 1;
  using Rows = Shape<8, 8, 4>;
  using Tile = Shape<8, 8, 4>;
  using Few = Tile;
  const __nv_bfloat16* x;
  int64_t ld;
  template <bool WHOLE>
  __device__ __forceinline__ void raw(int64_t r, int64_t c, int64_t cols,
                                      uint4* u) const {
    u[0] = load8<W>(x + r * ld + c, columns<WHOLE>(cols - c));
  }
  __device__ int64_t col_tile(int64_t j, int64_t) const { return j; }
};

template <int W>
struct CopyF32 {
  static constexpr int RAW = 2;
  using Rows = Shape<4, 4, 4>;
  using Tile = Shape<8, 1, 3>;
  using Few = Shape<4, 4, 2>;
  const float* x;
  int64_t ld;
  template <bool WHOLE>
  __device__ __forceinline__ void raw(int64_t r, int64_t c, int64_t cols,
                                      uint4* u) const {
    const float* p = x + r * ld + c;
    if (WHOLE || cols - c >= 8) {
      u[0] = load16<W>(p);
      u[1] = load16<W>(p + 4);
    } else {
      uint32_t w[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = c + j < cols ? __float_as_uint(p[j]) : 0u;
      u[0] = make_uint4(w[0], w[1], w[2], w[3]);
      u[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
  __device__ __forceinline__ void value(const uint4* u, int64_t,
                                        float* v) const {
    v[0] = __uint_as_float(u[0].x); v[1] = __uint_as_float(u[0].y);
    v[2] = __uint_as_float(u[0].z); v[3] = __uint_as_float(u[0].w);
    v[4] = __uint_as_float(u[1].x); v[5] = __uint_as_float(u[1].y);
    v[6] = __uint_as_float(u[1].z); v[7] = __uint_as_float(u[1].w);
  }
  __device__ int64_t col_tile(int64_t j, int64_t) const { return j; }
};

// σ(x) = 1 / (1 + 2^(−x·log2 e)) by the special-function unit's exponential
// and reciprocal (1 and 2 ulp; 1 + inf gives 0): the values only go to E4M3,
// and an IEEE division or a denormal-preserving exponential would be a third
// of these kernels' instructions, which are what bounds them.
__device__ __forceinline__ float sigmoid_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;"
      : "=f"(r)
      : "f"(1.0f + ex2_approx(x * -1.4426950408889634f)));
  return r;
}

// A = SiLU(G)·U.
template <int W>
struct SwigluSource {
  static constexpr int RAW = 2;
  using Rows = Shape<4, 4, 4>;
  using Tile = Shape<8, 1, 3>;
  using Few = Shape<4, 4, 2>;
  const __nv_bfloat16* gu;
  int64_t ld, f;
  template <bool WHOLE>
  __device__ __forceinline__ void raw(int64_t r, int64_t c, int64_t cols,
                                      uint4* u) const {
    const int valid = columns<WHOLE || W == 16>(cols - c);   // 16: f % 8 == 0
    const __nv_bfloat16* p = gu + r * ld + c;
    u[0] = load8<W>(p, valid);
    u[1] = load8<W>(p + f, valid);
  }
  __device__ __forceinline__ void value(const uint4* x, int64_t,
                                        float* v) const {
    float g[8], u[8];
    unpack8(x[0], g);
    unpack8(x[1], u);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      v[j] = g[j] * sigmoid_approx(g[j]) * u[j];
  }
  __device__ int64_t col_tile(int64_t j, int64_t) const { return j; }
};

// [dG | dU]: dG = dA·U·s·(1 + G·(1 − s)), dU = dA·G·s with s = σ(G).  The
// multiplier of the up side is read for dG alone; which side a column is on
// may change inside eight columns when f is not a multiple of 8.
template <int W>   // 16: f a multiple of 8
struct SwigluBwdSource {
  static constexpr int RAW = 3;
  using Rows = Shape<4, 2, 4>;
  using Tile = Shape<4, 2, 2>;
  using Few = Tile;
  const __nv_bfloat16 *da, *gu;
  int64_t ldda, ld, f;
  template <bool WHOLE>
  __device__ __forceinline__ void raw(int64_t r, int64_t c, int64_t cols,
                                      uint4* u) const {
    const __nv_bfloat16* pa = da + r * ldda;
    const __nv_bfloat16* pg = gu + r * ld;
    const bool up = c >= f;
    if (W == 16 || up || c + 8 <= f) {   // all eight columns on one side
      const int64_t k = up ? c - f : c;
      const int valid = columns<WHOLE || W == 16>(cols - c);
      u[0] = load8<W>(pa + k, valid);
      u[1] = load8<W>(pg + k, valid);
      u[2] = up ? make_uint4(0, 0, 0, 0) : load8<W>(pg + f + k, valid);
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
      v[j] = c + (W == 16 ? 0 : j) < f
                 ? a[j] * u[j] * s * (1.0f + g[j] * (1.0f - s))
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
template <typename SRC, int ROWS>
struct Held {
  static constexpr int R = ROWS;
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
// max(m, |a|) on two packed values (a bf16 maximum is exact; like fmaxf it
// takes the other operand where one is NaN).
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t a) {
  __nv_bfloat162 x, y;
  memcpy(&x, &m, 4);
  memcpy(&y, &a, 4);
  x = __hmax2(x, __habs2(y));
  memcpy(&m, &x, 4);
  return m;
}
template <int W>
struct Held<CopyBf16<W>, 8> {
  static constexpr int R = 8;
  uint4 u[8];
  __device__ __forceinline__ void take(const CopyBf16<W>&, int i,
                                       const uint4* x, int64_t) {
    u[i] = x[0];
  }
  __device__ __forceinline__ void row(int i, float* o) const {
    unpack8(u[i], o);
  }
  __device__ __forceinline__ uint32_t word(int i, int w) const {
    return w == 0 ? u[i].x : w == 1 ? u[i].y : w == 2 ? u[i].z : u[i].w;
  }
  __device__ __forceinline__ float at(int i, int j) const {
    const float2 t = unpack_bf16x2(word(i, j >> 1));
    return j & 1 ? t.y : t.x;
  }
  __device__ __forceinline__ float row_max(int i) const {
    const float2 t = unpack_bf16x2(
        max_abs2(max_abs2(max_abs2(max_abs2(0u, u[i].x), u[i].y), u[i].z),
                 u[i].w));
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

// A thread's elements of rows r0 and on, columns c0 to c0 + 7.
template <bool WHOLE, int BATCH, typename SRC, int R>
__device__ __forceinline__ void load_held(Held<SRC, R>& h, const SRC& src,
                                          int64_t r0, int64_t c0, int64_t rows,
                                          int64_t cols) {
#pragma unroll
  for (int b = 0; b < R; b += BATCH) {
    uint4 u[BATCH][SRC::RAW];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      if (!WHOLE) {
#pragma unroll
        for (int k = 0; k < SRC::RAW; ++k) u[i][k] = make_uint4(0, 0, 0, 0);
      }
      if (WHOLE || (r0 + b + i < rows && c0 < cols))
        src.template raw<WHOLE>(r0 + b + i, c0, cols, u[i]);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) h.take(src, b + i, u[i], c0);
  }
}

template <bool WHOLE>
__device__ __forceinline__ void store8(uint8_t* p, uint2 c, int valid) {
  if (WHOLE || valid >= 8) {
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

// An IEEE division is a dozen instructions, so lanes share them: of the lanes
// that know a block's amax some get its factor (want_scale false), the others
// its scale, from the same division.
__device__ __forceinline__ float factor_or_scale(float amax, bool want_scale) {
  const float a = fmaxf(amax, kBlockAmaxFloor);
  const float x = __fdiv_rn(want_scale ? a : kE4M3Max,
                            want_scale ? kE4M3Max : a);
  return want_scale && amax == 0.0f ? 1.0f : x;
}

// Maxima of R rows over the 16 lanes of a half-warp, row l mod R in lane l:
// halving exchanges (R − 1 shuffles) instead of one reduction a row.
template <int R>
__device__ __forceinline__ float rows_max(float (&m)[R], int l) {
  const bool b0 = l & 1, b1 = l & 2, b2 = l & 4;
  float x[R / 2];
#pragma unroll
  for (int j = 0; j < R / 2; ++j)
    x[j] = fmaxf(b0 ? m[2 * j + 1] : m[2 * j],
                 __shfl_xor_sync(0xffffffffu, b0 ? m[2 * j] : m[2 * j + 1], 1));
  float y[R / 4];
#pragma unroll
  for (int j = 0; j < R / 4; ++j)
    y[j] = fmaxf(b1 ? x[2 * j + 1] : x[2 * j],
                 __shfl_xor_sync(0xffffffffu, b1 ? x[2 * j] : x[2 * j + 1], 2));
  float z;
  if constexpr (R == 8)
    z = fmaxf(b2 ? y[1] : y[0],
              __shfl_xor_sync(0xffffffffu, b2 ? y[0] : y[1], 4));
  else
    z = fmaxf(y[0], __shfl_xor_sync(0xffffffffu, y[0], 4));
  return fmaxf(z, __shfl_xor_sync(0xffffffffu, z, 8));
}

// Scratch of a CTA: the warps' column maxima, the transposed codes.
template <int R>
struct TileScratch {
  __align__(16) float cmax[64 / R][TILE];
  __align__(16) float colf[TILE];
  __align__(16) uint8_t t[TILE * TILE];
};

// The codes and scales of tile (rt, ct).  A row's codes leave as 16 lanes × 8
// bytes; a column's largest magnitude takes one shuffle and one pass through
// shared memory; R rows of a column pack into one R-byte shared-memory store
// of the transposed tile, whose rows then leave the same way.
template <int GROUP, bool WHOLE, typename H>
__device__ __forceinline__ void emit_tile(const H& h, const Fp8BlockOut& o,
                                          int64_t rows, int64_t cols,
                                          int64_t rt, int64_t ct,
                                          TileScratch<H::R>& sm) {
  constexpr int R = H::R, WARPS = 64 / R;
  float(&cmax)[WARPS][TILE] = sm.cmax;
  uint8_t* tile_t = sm.t;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int half = lane >> 4, l = lane & 15;
  const int64_t r0 = rt * TILE + (warp * 2 + half) * R;
  const int64_t c0 = ct * TILE + l * 8;
  // this thread's rows and columns that exist
  const int nr = WHOLE || rows - r0 >= R ? R : (int)(rows - r0);
  const int nc = columns<WHOLE>(cols - c0);
  float colr[8];   // the factor of each of this thread's columns
  float rowr[R];   // and of each of its rows
  if (GROUP == kFp8Row) {
    // The columns' maxima first: their pass through shared memory, and the
    // divisions of 256 threads, run while the rows' codes are made.
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
      if (tid < 2 * TILE) {   // a column each: its factor, its scale
        const int c = tid & (TILE - 1);
        float m = cmax[0][c];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) m = fmaxf(m, cmax[w][c]);
        const float x = factor_or_scale(m, tid >= TILE);
        if (tid < TILE)
          sm.colf[c] = x;
        else if (ct * TILE + c < cols)
          o.st[rt * o.ldst + ct * TILE + c] = x;
      }
    }
    if (o.q != nullptr) {
      float m[R];
#pragma unroll
      for (int i = 0; i < R; ++i) m[i] = h.row_max(i);
      // lanes 0 to 7 get the factors, 8 to 15 the scales, of row l mod R
      const float x = factor_or_scale(rows_max<R>(m, l), l & 8);
      if (l >= 8 && l < 8 + R && l - 8 < nr)
        o.s[ct * o.lds + r0 + l - 8] = x;
#pragma unroll
      for (int i = 0; i < R; ++i)
        rowr[i] = __shfl_sync(0xffffffffu, x, (lane & 16) | i);
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

  if (o.q != nullptr && nc > 0) {
    uint8_t* q = o.q + r0 * o.ldq + c0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i < nr) {
        float v[8];
        h.row(i, v);
        store8<WHOLE>(q, codes8(v, rowr[i]), nc);
      }
      q += o.ldq;
    }
  }
  if (GROUP == kFp8Row && o.qt != nullptr) {
    __syncthreads();   // the columns' factors
    const float4* d = reinterpret_cast<const float4*>(&sm.colf[l * 8]);
    const float4 x = d[0], y = d[1];
    colr[0] = x.x; colr[1] = x.y; colr[2] = x.z; colr[3] = x.w;
    colr[4] = y.x; colr[5] = y.y; colr[6] = y.z; colr[7] = y.w;
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
    const int valid = columns<WHOLE>(rows - rr);
    // columns 2R·warp + half + 2i of the tile
    const int first = warp * 2 * R + half;
    const int64_t left = cols - ct * TILE - first;
    const int nt = WHOLE || left >= TILE ? TILE : (int)left;
    uint8_t* q = o.qt + (ct * TILE + first) * o.ldqt + rr;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int c = first + 2 * i;
      const int chunk = l ^ (c >> 3);
      const uint2 u =
          *reinterpret_cast<const uint2*>(tile_t + c * TILE + chunk * 8);
      if (2 * i < nt && valid > 0) store8<WHOLE>(q, u, valid);
      q += 2 * o.ldqt;
    }
  }
}

// Row scales alone (no transpose): a half-warp takes R rows of one group of 128
// columns, nothing passes through shared memory, and a single row spreads over
// as many half-warps as it has groups.  8192×8192 bf16 33 µs (6.1 TB/s, 91 %),
// SwiGLU 8192×11008 80 µs (84 %), 1×28672 2.4 µs (1×128 2.3).
template <bool WHOLE, typename SRC>
__device__ __forceinline__ void emit_rows(const SRC& src, int64_t r0,
                                          int64_t c0, int64_t ct, int64_t rows,
                                          int64_t cols, const Fp8BlockOut& o) {
  constexpr int R = SRC::Rows::R;
  const int lane = threadIdx.x & 31, l = lane & 15;
  Held<SRC, R> h;
  load_held<WHOLE, SRC::Rows::BATCH>(h, src, r0, c0, rows, cols);
  float m[R];
#pragma unroll
  for (int i = 0; i < R; ++i) m[i] = h.row_max(i);
  // lanes 0 to 7 get the factors, 8 to 15 the scales, of row l mod R
  const float x = factor_or_scale(rows_max<R>(m, l), l & 8);
  if (l >= 8 && l < 8 + R && r0 + l - 8 < rows)
    o.s[ct * o.lds + r0 + l - 8] = x;
  const int nc = columns<WHOLE>(cols - c0);
  uint8_t* q = o.q + r0 * o.ldq + c0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float f = __shfl_sync(0xffffffffu, x, (lane & 16) | i);
    if (WHOLE || (r0 + i < rows && nc > 0)) {
      float v[8];
      h.row(i, v);
      store8<WHOLE>(q, codes8(v, f), nc);
    }
    q += o.ldq;
  }
}
template <typename SRC>
__global__ void __launch_bounds__(256, SRC::Rows::CTAS)
    quantize_rows_kernel(const SRC src, int64_t rows, int64_t cols,
                         int64_t col_tiles, const Fp8BlockOut o) {
  constexpr int R = SRC::Rows::R;
  const int l = threadIdx.x & 15;
  const int64_t hw = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  const int64_t rt = hw / col_tiles;
  const int64_t ct = src.col_tile(hw - rt * col_tiles, col_tiles);
  const int64_t r0 = rt * R, c0 = ct * TILE + l * 8;   // r0 ≥ rows: no work
  if (__all_sync(0xffffffffu, r0 + R <= rows && c0 + 8 <= cols))
    emit_rows<true>(src, r0, c0, ct, rows, cols, o);
  else
    emit_rows<false>(src, r0, c0, ct, rows, cols, o);
}

template <typename SRC, int GROUP, typename SHAPE>
__global__ void __launch_bounds__(2048 / SHAPE::R, SHAPE::CTAS)
    quantize_tile_kernel(const SRC src, int64_t rows, int64_t cols,
                         int64_t col_tiles, const Fp8BlockOut o) {
  constexpr int R = SHAPE::R, BATCH = SHAPE::BATCH;
  __shared__ TileScratch<R> sm;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t rt = blockIdx.x / col_tiles;
  const int64_t ct = src.col_tile(blockIdx.x - rt * col_tiles, col_tiles);
  const int64_t r0 = rt * TILE + (warp * 2 + (lane >> 4)) * R;
  const int64_t c0 = ct * TILE + (lane & 15) * 8;

  // tiles that are whole (all but the last of an axis) are spared every bound
  Held<SRC, R> h;
  if (rows - rt * TILE >= TILE && cols - ct * TILE >= TILE) {
    load_held<true, BATCH>(h, src, r0, c0, rows, cols);
    emit_tile<GROUP, true>(h, o, rows, cols, rt, ct, sm);
  } else {
    load_held<false, BATCH>(h, src, r0, c0, rows, cols);
    emit_tile<GROUP, false>(h, o, rows, cols, rt, ct, sm);
  }
}

// The SwiGLU backward where dG's and dU's tiles line up (f a multiple of 128):
// one CTA makes both from one read of dA, G and U and one σ; dU waits in
// shared memory, each thread's in its own slots, while dG leaves.  8192×11008
// both ways 189 µs (4.8 TB/s, 72 %; 223 with a CTA for each of the two), rows
// alone 138 (78 %, against 154).  Bound by issue, like the tiles above, and by
// what two CTAs of 512 threads can have in flight (all four rows' loads at once
// spill; 256 threads of eight rows 195 to 229).
struct Fp32Rows {};
constexpr int PAIR_SMEM = 128 * 128 * 4;
using PairShape = Shape<4, 2, 2>;
constexpr int PAIR_THREADS = 2048 / PairShape::R;
__global__ void __launch_bounds__(PAIR_THREADS, PairShape::CTAS)
    swiglu_bwd_pair_kernel(const SwigluBwdSource<16> src, int64_t rows,
                           int64_t pairs, const Fp8BlockOut o) {
  extern __shared__ float4 kept[];   // [row][half of eight][thread]
  constexpr int R = PairShape::R, BATCH = PairShape::BATCH;
  __shared__ TileScratch<R> sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t rt = blockIdx.x / pairs, ct = blockIdx.x - rt * pairs;
  const int64_t r0 = rt * TILE + (warp * 2 + (lane >> 4)) * R;
  const int64_t c0 = ct * TILE + (lane & 15) * 8;
  Held<Fp32Rows, R> h;
#pragma unroll
  for (int b = 0; b < R; b += BATCH) {
    uint4 x[BATCH][3];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
#pragma unroll
      for (int k = 0; k < 3; ++k) x[i][k] = make_uint4(0, 0, 0, 0);
      if (r0 + b + i < rows)
        src.raw<true>(r0 + b + i, c0, 2 * src.f, x[i]);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      float a[8], g[8], u[8];
      unpack8(x[i][0], a);
      unpack8(x[i][1], g);
      unpack8(x[i][2], u);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = sigmoid_approx(g[j]);
        h.v[b + i][j] = a[j] * u[j] * s * (1.0f + g[j] * (1.0f - s));
        u[j] = a[j] * g[j] * s;
      }
      float4* k = kept + (b + i) * 2 * PAIR_THREADS + tid;
      k[0] = make_float4(u[0], u[1], u[2], u[3]);
      k[PAIR_THREADS] = make_float4(u[4], u[5], u[6], u[7]);
    }
  }
  const bool whole = rows - rt * TILE >= TILE;
  if (whole)
    emit_tile<kFp8Row, true>(h, o, rows, 2 * src.f, rt, ct, sm);
  else
    emit_tile<kFp8Row, false>(h, o, rows, 2 * src.f, rt, ct, sm);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const float4* k = kept + i * 2 * PAIR_THREADS + tid;
    const float4 a = k[0], b = k[PAIR_THREADS];
    h.v[i][0] = a.x; h.v[i][1] = a.y; h.v[i][2] = a.z; h.v[i][3] = a.w;
    h.v[i][4] = b.x; h.v[i][5] = b.y; h.v[i][6] = b.z; h.v[i][7] = b.w;
  }
  __syncthreads();   // the scratch is read
  if (whole)
    emit_tile<kFp8Row, true>(h, o, rows, 2 * src.f, rt, pairs + ct, sm);
  else
    emit_tile<kFp8Row, false>(h, o, rows, 2 * src.f, rt, pairs + ct, sm);
}

// BLOCKS: whether the source is also quantized in 128×128 blocks.
template <bool BLOCKS, typename SRC>
int launch_tiles(const SRC& src, int group, int64_t rows, int64_t cols,
                 const Fp8BlockOut& o, double bytes, cudaStream_t s) {
  const int64_t ct = (cols + TILE - 1) / TILE, rt = (rows + TILE - 1) / TILE;
  if (ct * rt > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(ct * rt);
  {
    ProfScope ps(s, KF_QUANT, 0.0, bytes);
    if (o.qt == nullptr && group == kFp8Row) {
      const int64_t half_warps = ct * ((rows + SRC::Rows::R - 1) / SRC::Rows::R);
      quantize_rows_kernel<SRC><<<(unsigned)((half_warps + 15) / 16), 256, 0,
                                  s>>>(src, rows, cols, ct, o);
    } else {
      auto go = [&](auto shape) {
        using SHAPE = decltype(shape);
        if constexpr (BLOCKS) {
          if (group != kFp8Row) {
            quantize_tile_kernel<SRC, kFp8Block, SHAPE>
                <<<grid, 2048 / SHAPE::R, 0, s>>>(src, rows, cols, ct, o);
            return;
          }
        }
        quantize_tile_kernel<SRC, kFp8Row, SHAPE>
            <<<grid, 2048 / SHAPE::R, 0, s>>>(src, rows, cols, ct, o);
      };
      // Few tiles wait for their loads, not for each other: all of a thread's
      // loads at once and half the rows (SwiGLU 777×1536 4.8 against 6.2 µs,
      // 2048×4096 13.8 / 14.3, 4096×4096 24.2 / 23.1; fp32 777×1000 6.0 / 9.1).
      if (grid <= 4u * (unsigned)device_sm_count())
        go(typename SRC::Few{});
      else
        go(typename SRC::Tile{});
    }
  }
  count_launch();
  return cudaGetLastError();
}

// The largest power of two, at most 16, that the address and the byte pitch
// are multiples of (a null address is a multiple of any).
int width(const void* p, int64_t pitch) {
  const uint64_t m = reinterpret_cast<uintptr_t>(p) | (uint64_t)pitch | 16u;
  return (int)(m & -m);
}

double out_bytes(const Fp8BlockOut& o, int64_t rows, int64_t cols) {
  return (double)rows * cols * ((o.q != nullptr) + (o.qt != nullptr));
}

// ----------------------------------------------------- residual + RMSNorm --
// Sets a kernel's dynamic shared memory limit once per device.
template <typename K>
int allow_smem(K kernel, int bytes, std::atomic<bool> (&done)[64]) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev].load()) return cudaSuccess;
  err = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (err == cudaSuccess) done[dev].store(true);
  return err;
}

struct NormArgs {
  // x1 may be x or r: no read-only loads, and each element is read before it
  // is written, by the same thread
  const __nv_bfloat16 *x, *r, *gamma;
  __nv_bfloat16 *x1, *y;
  float* rstd;
  uint8_t* q;
  int64_t ldq;
  float* s;
  int64_t lds;
  int64_t rows;
  int h;
  float eps;
  unsigned* status;
};

// u + ur rounded to bf16 (the stored stream is what is normed), and its sum
// of squares.
__device__ __forceinline__ float add_squares(uint4& u, const uint4& ur,
                                             bool add) {
  float a[8];
  if (add) {
    float b[8];
    unpack8(u, a);
    unpack8(ur, b);
    u.x = pack_bf16x2(a[0] + b[0], a[1] + b[1]);
    u.y = pack_bf16x2(a[2] + b[2], a[3] + b[3]);
    u.z = pack_bf16x2(a[4] + b[4], a[5] + b[5]);
    u.w = pack_bf16x2(a[6] + b[6], a[7] + b[7]);
  }
  unpack8(u, a);
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) ss += a[j] * a[j];
  return ss;
}

// Eight columns of a normed row: codes, the scale of the 16 lanes' 128
// columns, y.  All lanes of a half-warp call it; valid ≤ 0 writes nothing.
template <int W>
__device__ __forceinline__ void emit_norm(const NormArgs& p, int64_t row,
                                          int c, int valid, const uint4& u,
                                          const uint4& g, float rs) {
  float v[8], gm[8];
  unpack8(u, v);
  unpack8(g, gm);
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = v[j] * rs * gm[j];
    m = fmaxf(m, fabsf(v[j]));
  }
#pragma unroll
  for (int d = 8; d > 0; d >>= 1)
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  // the half-warp's lane 8 gets the scale, lane 0 the factor of all
  const int lane = threadIdx.x & 31;
  const float x = factor_or_scale(m, lane & 8);
  const float f = __shfl_sync(0xffffffffu, x, lane & 16);
  if ((lane & 15) == 8 && c - 64 < p.h) p.s[(c >> 7) * p.lds + row] = x;
  if (valid <= 0) return;
  store8<W == 16>(p.q + row * p.ldq + c, codes8(v, f), valid);
  if (p.y != nullptr)
    save8<W>(p.y + row * p.h + c,
             make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                        pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7])),
             valid);
}

template <int W>
__device__ __forceinline__ uint4 load8_plain(const __nv_bfloat16* p,
                                             int valid) {
  if (W == 16) return *reinterpret_cast<const uint4*>(p);
  if (W == 8 && valid >= 8) {
    const uint2 a = reinterpret_cast<const uint2*>(p)[0],
                b = reinterpret_cast<const uint2*>(p)[1];
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  if (W == 4 && valid >= 8) {
    const uint32_t* a = reinterpret_cast<const uint32_t*>(p);
    return make_uint4(a[0], a[1], a[2], a[3]);
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < valid)
      w[j >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[j]
                   << (16 * (j & 1));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Threads of a row of h columns with V vectors of eight columns each: whole
// warps, no more than the row has work for.
int norm_threads(int h, int V) {
  const int vectors = (h + 7) / 8;
  return ((vectors + V - 1) / V + 31) / 32 * 32;
}

// At most THREADS threads a row, which stays in their registers (V vectors of
// eight columns each, 16 neighbouring threads hold one group of 128); a warp
// per row (eight rows a CTA) up to 512 columns, else a CTA per row.  γ is read
// before the row's sum is known, so that its latency is not paid after it.
// Few rows are bound by latency (1×8192 2.9 µs, 600×8192 10: load, sum, output
// in turn), 1001×4100 (rows on eight bytes, 3.3 waves of CTAs) by it 11 µs.
template <int THREADS, int V, int CTAS, int W>
__global__ void __launch_bounds__(THREADS == 32 ? 256 : THREADS, CTAS)
    add_rmsnorm_fp8_kernel(const NormArgs p) {
  constexpr bool WARP = THREADS == 32;
  __shared__ float red[THREADS / 32];
  const int threads = WARP ? 32 : blockDim.x;
  const int tid = WARP ? threadIdx.x & 31 : threadIdx.x;
  const int64_t row =
      WARP ? (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5) : blockIdx.x;
  if (WARP && row >= p.rows) return;
  const int h = p.h;
  const __nv_bfloat16* x = p.x + row * h;
  const __nv_bfloat16* r = p.r + row * h;
  uint4 u[V], ur[V], g[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * threads + tid) * 8;
    u[k] = ur[k] = make_uint4(0, 0, 0, 0);
    if (c < h) {
      u[k] = load8_plain<W>(x + c, h - c);
      if (p.r != nullptr) ur[k] = load8_plain<W>(r + c, h - c);
    }
  }
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * threads + tid) * 8;
    g[k] = make_uint4(0, 0, 0, 0);
    if (c < h) g[k] = load8<W>(p.gamma + c, h - c);
  }
  float ss = 0.0f;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * threads + tid) * 8;
    ss += add_squares(u[k], ur[k], p.r != nullptr);
    if (p.x1 != nullptr && c < h) save8<W>(p.x1 + row * h + c, u[k], h - c);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if (!WARP) {
    if ((tid & 31) == 0) red[tid >> 5] = ss;
    __syncthreads();
    ss = 0.0f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w)
      if (w * 32 < threads) ss += red[w];
  }
  const float rs = rsqrtf(ss / (float)h + p.eps);
  if (tid == 0) p.rstd[row] = rs;
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * threads + tid) * 8;
    emit_norm<W>(p, row, c, h - c, u[k], g[k], rs);
  }
}

// Many rows of 16-byte aligned vectors: a CTA works through every gridDim-th
// row, thread 0 copying x and r of the rows to come into a ring of one or two
// stages (bulk copies), so that loads are in flight all the time and γ is
// read once.  Waits are bounded; the block agrees on every outcome.
// Bound by DRAM: 8192×8192 with the bf16 output 97 µs (6.2 TB/s, 93 %),
// without 77 (92 %), 8192×4096 40 (88 %), 8192×2048 21 (83 %).
constexpr int MAX_STAGES = 2;
template <int THREADS, int V, int CTAS>
__global__ void __launch_bounds__(THREADS, CTAS)
    add_rmsnorm_fp8_staged_kernel(const NormArgs p, int stages) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ uint64_t full[MAX_STAGES];
  __shared__ float red[2][THREADS / 32];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, threads = blockDim.x, h = p.h;
  const int nin = p.r != nullptr ? 2 : 1;
  const uint32_t row_bytes = (uint32_t)h * 2;
  if (tid == 0) {
    for (int i = 0; i < stages; ++i) mbar_init(&full[i], 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  auto issue = [&](int64_t row, int sg) {
    uint8_t* d = ring + (size_t)sg * nin * row_bytes;
    mbar_arrive_expect_tx(&full[sg], nin * row_bytes);
    bulk_g2s(d, p.x + row * h, row_bytes, &full[sg]);
    if (nin == 2) bulk_g2s(d + row_bytes, p.r + row * h, row_bytes, &full[sg]);
  };
  const int64_t step = gridDim.x;
  if (tid == 0)
    for (int i = 0; i < stages; ++i)
      if (blockIdx.x + i * step < p.rows) issue(blockIdx.x + i * step, i);
  uint4 g[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    const int c = (k * threads + tid) * 8;
    g[k] = c < h ? load16<16>(p.gamma + c) : make_uint4(0, 0, 0, 0);
  }
  int sg = 0;
  uint32_t par = 0;
  int64_t row = blockIdx.x;
  bool odd = false;
  for (; row < p.rows; row += step) {
    const bool got = mbar_wait(&full[sg], par,
                               reinterpret_cast<volatile int*>(&abort_flag),
                               p.status, 61);
    if (!__syncthreads_and(got)) break;
    const uint8_t* in = ring + (size_t)sg * nin * row_bytes;
    uint4 u[V];
    float ss = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = (k * threads + tid) * 8;
      u[k] = make_uint4(0, 0, 0, 0);
      uint4 ur = u[k];
      if (c < h) {
        u[k] = *reinterpret_cast<const uint4*>(in + c * 2);
        if (nin == 2)
          ur = *reinterpret_cast<const uint4*>(in + row_bytes + c * 2);
      }
      ss += add_squares(u[k], ur, nin == 2);
      if (p.x1 != nullptr && c < h)
        *reinterpret_cast<uint4*>(p.x1 + row * h + c) = u[k];
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    if ((tid & 31) == 0) red[odd][tid >> 5] = ss;
    __syncthreads();   // the sums are there, the stage is read
    if (tid == 0 && row + stages * step < p.rows) issue(row + stages * step, sg);
    ss = 0.0f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w)
      if (w * 32 < threads) ss += red[odd][w];
    odd = !odd;
    const float rs = rsqrtf(ss / (float)h + p.eps);
    if (tid == 0) p.rstd[row] = rs;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int c = (k * threads + tid) * 8;
      emit_norm<16>(p, row, c, h - c, u[k], g[k], rs);
    }
    if (++sg == stages) {
      sg = 0;
      par ^= 1;
    }
  }
  if (row < p.rows && tid == 0) {
    // gave up: let the copies in flight land before the block exits
    volatile int no_abort = 0;
    for (int i = 0; i < stages && row + i * step < p.rows; ++i) {
      mbar_wait(&full[sg], par, &no_abort, nullptr, 0);
      if (++sg == stages) {
        sg = 0;
        par ^= 1;
      }
    }
  }
}

template <int THREADS, int V, int CTAS>
int launch_norm_staged(const NormArgs& p, int stages, cudaStream_t s) {
  static std::atomic<bool> done[64];
  auto kernel = add_rmsnorm_fp8_staged_kernel<THREADS, V, CTAS>;
  // V vectors of 16 bytes a thread, x and r
  const int err = allow_smem(kernel, MAX_STAGES * 2 * V * THREADS * 16, done);
  if (err) return err;
  const size_t smem = (size_t)stages * (p.r != nullptr ? 2 : 1) * p.h * 2;
  // CTAS on an SM with all THREADS; of smaller ones more fit
  const int threads = norm_threads(p.h, V);
  const int64_t grid = std::min<int64_t>(
      p.rows, (int64_t)device_sm_count() * (CTAS * THREADS / threads));
  kernel<<<(unsigned)grid, threads, smem, s>>>(p, stages);
  return cudaGetLastError();
}

template <int W>
int launch_norm(const NormArgs& p, cudaStream_t s) {
  const unsigned T = (unsigned)p.rows;
  if (p.h <= 256)
    add_rmsnorm_fp8_kernel<32, 1, 4, W><<<(T + 7) / 8, 256, 0, s>>>(p);
  else if (p.h <= 512)
    add_rmsnorm_fp8_kernel<32, 2, 4, W><<<(T + 7) / 8, 256, 0, s>>>(p);
  else if (p.h <= 1024)
    add_rmsnorm_fp8_kernel<128, 1, 8, W>
        <<<T, norm_threads(p.h, 1), 0, s>>>(p);
  else if (p.h <= 2048)
    add_rmsnorm_fp8_kernel<256, 1, 4, W>
        <<<T, norm_threads(p.h, 1), 0, s>>>(p);
  else if (p.h <= 4096)
    add_rmsnorm_fp8_kernel<512, 1, 2, W>
        <<<T, norm_threads(p.h, 1), 0, s>>>(p);
  else if (p.h <= 8192)
    add_rmsnorm_fp8_kernel<512, 2, 2, W>
        <<<T, norm_threads(p.h, 2), 0, s>>>(p);
  else
    add_rmsnorm_fp8_kernel<1024, 2, 1, W>
        <<<T, norm_threads(p.h, 2), 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

int quantize_fp8_block(int dtype, int group, int64_t rows, int64_t cols,
                       const void* x, int64_t ldx, const Fp8BlockOut& o,
                       void* stream) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int es = dtype == 0 ? 4 : 2;
  const double bytes = (double)es * rows * cols + out_bytes(o, rows, cols);
  auto go = [&](const auto& src) {
    return launch_tiles<true>(src, group, rows, cols, o, bytes, s);
  };
  const int w = width(x, ldx * es);
  if (dtype == 0) {
    const auto* p = static_cast<const float*>(x);
    if (w == 16) return go(CopyF32<16>{p, ldx});
    return go(CopyF32<4>{p, ldx});
  }
  const auto* p = static_cast<const __nv_bfloat16*>(x);
  switch (w) {
    case 16: return go(CopyBf16<16>{p, ldx});
    case 8: return go(CopyBf16<8>{p, ldx});
    case 4: return go(CopyBf16<4>{p, ldx});
    default: return go(CopyBf16<2>{p, ldx});
  }
}

int swiglu_fp8_fwd(int64_t T, int64_t f, const void* gu, int64_t ldgu,
                   const Fp8BlockOut& o, void* stream) {
  const auto* x = static_cast<const __nv_bfloat16*>(gu);
  const double bytes = 4.0 * T * f + out_bytes(o, T, f);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](const auto& src) {
    return launch_tiles<false>(src, kFp8Row, T, f, o, bytes, s);
  };
  switch (std::min(width(gu, ldgu * 2), width(nullptr, f * 2))) {
    case 16: return go(SwigluSource<16>{x, ldgu, f});
    case 8: return go(SwigluSource<8>{x, ldgu, f});
    case 4: return go(SwigluSource<4>{x, ldgu, f});
    default: return go(SwigluSource<2>{x, ldgu, f});
  }
}

int swiglu_fp8_bwd(int64_t T, int64_t f, const void* da, int64_t ldda,
                   const void* gu, int64_t ldgu, const Fp8BlockOut& o,
                   void* stream) {
  const auto* a = static_cast<const __nv_bfloat16*>(da);
  const auto* x = static_cast<const __nv_bfloat16*>(gu);
  const double bytes = 6.0 * T * f + out_bytes(o, T, 2 * f);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  auto go = [&](const auto& src) {
    return launch_tiles<false>(src, kFp8Row, T, 2 * f, o, bytes, s);
  };
  switch (std::min({width(gu, ldgu * 2), width(da, ldda * 2),
                    width(nullptr, f * 2)})) {
    case 16: break;
    case 8: return go(SwigluBwdSource<8>{a, x, ldda, ldgu, f});
    case 4: return go(SwigluBwdSource<4>{a, x, ldda, ldgu, f});
    default: return go(SwigluBwdSource<2>{a, x, ldda, ldgu, f});
  }
  const SwigluBwdSource<16> src{a, x, ldda, ldgu, f};
  // Where tiles are too few to fill the SMs, two CTAs finish them sooner than
  // one (separate / pair in µs, rows alone: 1×28672 2.8 / 6.0, 64×28672 5.6 /
  // 8.0, 128×28672 9.4 / 9.0, 512×28672 27.9 / 25.6, 512×4096 6.5 / 7.1; both
  // ways: 128×28672 11.9 / 12.1, 256×4096 6.0 / 8.4, 512×4096 8.1 / 9.1,
  // 8192×11008 223 / 189).
  if (f % TILE || T * f < device_sm_count() * 3 / 2 * (TILE * TILE))
    return go(src);
  static std::atomic<bool> done[64];
  const int err = allow_smem(swiglu_bwd_pair_kernel, PAIR_SMEM, done);
  if (err) return err;
  const int64_t pairs = f / TILE, rt = (T + TILE - 1) / TILE;
  {
    ProfScope ps(s, KF_QUANT, 0.0, bytes);
    swiglu_bwd_pair_kernel<<<(unsigned)(pairs * rt), PAIR_THREADS, PAIR_SMEM,
                             s>>>(
        src, T, pairs, o);
  }
  count_launch();
  return cudaGetLastError();
}

int add_rmsnorm_fp8_fwd(int64_t T, int64_t h, float eps, const void* x,
                        const void* r, const void* gamma, void* x1, void* y,
                        float* rstd, uint8_t* q, int64_t ldq, float* s,
                        int64_t lds, unsigned* status, void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto bf = [](const void* p) { return static_cast<const __nv_bfloat16*>(p); };
  const NormArgs p{bf(x), bf(r), bf(gamma), static_cast<__nv_bfloat16*>(x1),
                   static_cast<__nv_bfloat16*>(y), rstd, q, ldq, s, lds, T,
                   (int)h, eps, status};
  int w = width(gamma, h * 2);
  for (const void* a : {x, r, (const void*)x1, (const void*)y})
    w = std::min(w, width(a, 0));
  int err;
  {
    ProfScope ps(st, KF_NORM, 4.0 * T * h,
                 (2.0 + 2.0 * (r != nullptr) + 2.0 * (x1 != nullptr) +
                  2.0 * (y != nullptr) + 1.0) * T * h);
    // The ring pays where a CTA has rows to run ahead on (one CTA a row /
    // ring in µs: 600×8192 10.0 / 10.2, 1000×8192 15.6 / 14.1, 600×16384 with y
    // 21.8 / 18.5, 600×2048 4.1 / 4.7, 2000×2048 8.6 / 8.0, 1000×1024 3.8 /
    // 4.4, 2000×1024 5.9 / 5.9).  Its second stage helps long rows without y
    // (8192×8192 78 against 79 to 81 µs) and costs the others (with y 96
    // against 112: more reads in flight between the writes).
    const int ctas = h <= 1024 ? 12 : h <= 2048 ? 8 : h <= 4096 ? 4 : 2;
    const bool many = T >= (int64_t)device_sm_count() * std::max(3, ctas);
    const int stages = y == nullptr && h > 4096 ? 2 : 1;
    if (w == 16 && h > 512 && many) {
      if (h <= 1024)
        err = launch_norm_staged<128, 1, 12>(p, stages, st);
      else if (h <= 2048)
        err = launch_norm_staged<128, 2, 8>(p, stages, st);
      else if (h <= 4096)
        err = launch_norm_staged<256, 2, 4>(p, stages, st);
      else if (h <= 8192)
        err = launch_norm_staged<512, 2, 2>(p, stages, st);
      else
        err = launch_norm_staged<512, 4, 1>(p, stages, st);
    } else if (w == 16) {
      err = launch_norm<16>(p, st);
    } else if (w == 8) {
      err = launch_norm<8>(p, st);
    } else if (w == 4) {
      err = launch_norm<4>(p, st);
    } else {
      err = launch_norm<2>(p, st);
    }
  }
  count_launch();
  return err;
}

}  // namespace tp
