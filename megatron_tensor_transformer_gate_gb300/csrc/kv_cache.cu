// kv_cache.cu — rows of K and V into the pages of a key-value cache, and back.
//
// A vector (one head of one token, d elements) is the unit of both calls: d/8
// lanes move 16 bytes of its row each.  Quantized, its largest magnitude is
// found by exchanges among these lanes, so that every value is read once.
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8.cuh"
#include "gemm.h"
#include "kv_cache.cuh"
#include "kv_cache.h"
#include "profile.h"

namespace tp {
namespace {

constexpr int THREADS = 256;

struct Args {
  tp_kv_cache c;
  KvRows r;
  int per_seq;   // rows of a sequence (start == nullptr)
  unsigned* status;
};

// Eight elements of a 16-bit row as fp32.
template <int DT>
__device__ __forceinline__ void unpack8(uint4 u, float (&x)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = pair_to_f32<DT>(w[j]);
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
  }
}
template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = DT == TP_BF16 ? pack_bf16x2(x[2 * j], x[2 * j + 1])
                         : pack_f16x2(x[2 * j], x[2 * j + 1]);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A finite value that fp16 does not hold (it has infinities and NaN).
__device__ __forceinline__ bool beyond_f16(const float (&x)[8]) {
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    bad |= fabsf(x[j]) > kF16Max && !isinf(x[j]);
  return bad;
}

// Vector `vec` of the call: row, K or V, head; the lane's eight elements of
// it in the rows' tensor and in the pool, and its scale.
template <int D>
struct Place {
  bool there = false;
  int64_t row_at, pool_at, scale_at;
  int which;
};
template <int D>
__device__ __forceinline__ Place<D> place(const Args& a) {
  constexpr int LANES = D / 8;
  Place<D> r;
  const int64_t vec =
      ((int64_t)blockIdx.x * THREADS + threadIdx.x) / LANES;
  const int lane = threadIdx.x % LANES;
  const int per_row = 2 * a.c.n_kv;
  const int64_t row = vec / per_row;
  const int in_row = (int)(vec - row * per_row);
  r.which = in_row >= a.c.n_kv;
  const int head = in_row - r.which * a.c.n_kv;
  int seq, pos, offset;
  if (row >= a.r.rows ||
      !kv_token_of(a.c, a.r.start, a.per_seq, row, &seq, &pos))
    return r;
  const int64_t page = page_of(a.c, seq, pos, &offset, a.status);
  if (page < 0) return r;
  r.there = true;
  r.row_at = row * (r.which ? a.r.v_row : a.r.k_row) +
             head * (r.which ? a.r.v_head : a.r.k_head) + 8 * lane;
  r.pool_at = page * a.c.page_stride + offset * a.c.token_stride +
              head * a.c.head_stride + 8 * lane;
  r.scale_at = page * a.c.s_page_stride + offset * a.c.s_token_stride +
               head * a.c.s_head_stride;
  return r;
}

template <int SRC, int CACHE, int D>
__global__ void __launch_bounds__(THREADS) write_kernel(const Args a) {
  const Place<D> p = place<D>(a);
  uint4 u = make_uint4(0, 0, 0, 0);
  if (p.there)
    u = *reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(p.which ? a.r.v : a.r.k) + p.row_at);
  void* pool = p.which ? a.c.v : a.c.k;
  if constexpr (SRC == CACHE) {
    if (p.there)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pool) + p.pool_at) = u;
  } else {
    float x[8];
    unpack8<SRC>(u, x);
    if constexpr (CACHE != TP_FP8) {
      if (CACHE == TP_F16 && beyond_f16(x))
        record_error(a.status, kDevRange, 41);
      if (p.there)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(pool) + p.pool_at) =
            pack8<CACHE>(x);
    } else {
      float amax = 0.0f;   // fmaxf leaves NaN out
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
#pragma unroll
      for (int o = D / 16; o > 0; o >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const float r = block_factor(amax);
      if (p.there) {
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(pool) + p.pool_at) =
            make_uint2(e4m3x4(x[0] * r, x[1] * r, x[2] * r, x[3] * r),
                       e4m3x4(x[4] * r, x[5] * r, x[6] * r, x[7] * r));
        if (threadIdx.x % (D / 8) == 0)
          (p.which ? a.c.vs : a.c.ks)[p.scale_at] = block_scale(amax);
      }
    }
  }
}

template <int CACHE, int DST, int D>
__global__ void __launch_bounds__(THREADS) read_kernel(const Args a) {
  const Place<D> p = place<D>(a);
  if (!p.there) return;
  const void* pool = p.which ? a.c.v : a.c.k;
  uint4* dst = reinterpret_cast<uint4*>(
      static_cast<uint16_t*>(p.which ? a.r.v : a.r.k) + p.row_at);
  float x[8];
  if constexpr (CACHE == TP_FP8) {
    const uint2 u = *reinterpret_cast<const uint2*>(
        static_cast<const uint8_t*>(pool) + p.pool_at);
    const float s = (p.which ? a.c.vs : a.c.ks)[p.scale_at];
    const uint32_t w[2] = {u.x, u.y};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f =
          pair_to_f32<TP_FP8>((w[j >> 1] >> (16 * (j & 1))) & 0xffffu);
      x[2 * j] = f.x * s;
      x[2 * j + 1] = f.y * s;
    }
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(
        static_cast<const uint16_t*>(pool) + p.pool_at);
    if constexpr (CACHE == DST) {
      *dst = u;
      return;
    }
    unpack8<CACHE>(u, x);
  }
  if (DST == TP_F16 && beyond_f16(x)) record_error(a.status, kDevRange, 42);
  *dst = pack8<DST>(x);
}

using Kernel = void (*)(const Args);

template <int SRC, int D>
Kernel write_for(int cache) {
  return cache == TP_BF16  ? write_kernel<SRC, TP_BF16, D>
         : cache == TP_F16 ? write_kernel<SRC, TP_F16, D>
                           : write_kernel<SRC, TP_FP8, D>;
}
template <int DST, int D>
Kernel read_for(int cache) {
  return cache == TP_BF16  ? read_kernel<TP_BF16, DST, D>
         : cache == TP_F16 ? read_kernel<TP_F16, DST, D>
                           : read_kernel<TP_FP8, DST, D>;
}

int launch(Kernel k, const tp_kv_cache& c, const KvRows& r, unsigned* status,
           void* stream) {
  Args a;
  a.c = c;
  a.r = r;
  a.per_seq = (int)(r.rows / c.b);
  a.status = status;
  const int64_t threads = r.rows * 2 * c.n_kv * (c.d / 8);
  const int64_t grid = (threads + THREADS - 1) / THREADS;
  const double size = c.dtype == TP_FP8 ? c.d + 4 : 2 * c.d;
  ProfScope prof(stream, KF_KV_CACHE, 0.0,
                 2.0 * r.rows * c.n_kv * (size + 2 * c.d));
  count_launch(1);
  k<<<(unsigned)grid, THREADS, 0, static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError();
}

}  // namespace

int kv_cache_write(const tp_kv_cache& c, int dtype, const KvRows& r,
                   unsigned* status, void* stream) {
  const Kernel k =
      dtype == TP_BF16
          ? (c.d == 128 ? write_for<TP_BF16, 128>(c.dtype)
                        : write_for<TP_BF16, 64>(c.dtype))
          : (c.d == 128 ? write_for<TP_F16, 128>(c.dtype)
                        : write_for<TP_F16, 64>(c.dtype));
  return launch(k, c, r, status, stream);
}

int kv_cache_read(const tp_kv_cache& c, int dtype, const KvRows& r,
                  unsigned* status, void* stream) {
  const Kernel k = dtype == TP_BF16
                       ? (c.d == 128 ? read_for<TP_BF16, 128>(c.dtype)
                                     : read_for<TP_BF16, 64>(c.dtype))
                       : (c.d == 128 ? read_for<TP_F16, 128>(c.dtype)
                                     : read_for<TP_F16, 64>(c.dtype));
  return launch(k, c, r, status, stream);
}

}  // namespace tp
