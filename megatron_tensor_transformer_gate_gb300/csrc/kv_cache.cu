// kv_cache.cu — rows of K and V into the pages of a key-value cache, and back.
//
// A vector (one head of one token, d elements) is the unit of both calls: a
// team of d/16 lanes moves two pieces of eight elements each of it, its halves'
// l-th.  The cost is one read and one write of the vectors.  With few vectors a
// thread has one of them, and what stands in front of it (the row's sequence,
// its length, its page: a chain of loads) it looks up for itself.  With many it
// has four, whose loads are all in flight before the first is used, and a CTA's
// look-ups are made once a row.  New rows are read while their places are looked
// up.  Quantized, four vectors' largest magnitudes are found together by halving
// exchanges that leave one vector's in each lane (or two), which then divides
// for it alone.
//
// Measured (GB300, copy 6.8 TB/s): 79970 tokens of fp16 to E4M3 84 µs (0.87 of a
// copy, bound by DRAM and the look-ups in front of a CTA's loads), back to fp16
// 71767 in 75 (0.87); 256 tokens 2.6 µs, one 2.2: a chain of three loads and a
// launch.
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

// Whether a finite value of x is none of its fp16 form u (which has infinities
// and NaN): looked for where u has an infinity, or its largest value.
__device__ __forceinline__ bool beyond_f16(const float (&x)[8], uint4 u) {
  auto h = [](uint32_t v) { return __habs2(*reinterpret_cast<__half2*>(&v)); };
  const __half2 m = __hmax2(__hmax2(h(u.x), h(u.y)), __hmax2(h(u.z), h(u.w)));
  const float2 f = __half22float2(m);
  if (fmaxf(f.x, f.y) < kF16Max) return false;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    bad |= fabsf(x[j]) > kF16Max && !isinf(x[j]);
  return bad;
}

__device__ __forceinline__ int64_t mul(int a, int b) { return (int64_t)a * b; }

// Where the pool has a row's vectors: offsets of its heads' first one (−1: the
// row is no token, or its page is none of the pool's) and of its scale.
struct RowPlace {
  int64_t pool, scale;
};
__device__ __forceinline__ RowPlace place_of(const Args& a, int64_t row) {
  RowPlace p = {-1, 0};
  int seq, pos, offset;
  if (row < a.r.rows &&
      kv_token_of(a.c, a.r.start, a.per_seq, row, &seq, &pos)) {
    const int64_t page = page_of(a.c, seq, pos, &offset, a.status);
    if (page >= 0) {
      p.pool = page * a.c.page_stride + mul(offset, (int)a.c.token_stride);
      p.scale = page * a.c.s_page_stride + mul(offset, (int)a.c.s_token_stride);
    }
  }
  return p;
}

// A CTA has U·VECS neighbouring vectors, (row, head) in this order, of K
// (blockIdx.y = 0) or of V, of which a team takes every VECS-th.
template <int D, int U>
struct Team {
  static constexpr int LANES = D / 16, VECS = THREADS / LANES, HALF = D / 2;
  static constexpr int ROWS = U == 1 ? 1 : U * VECS + 1;   // of a CTA, at most
  RowPlace own;            // U == 1: of the vector's row
  int row, head;           // vector 0: its row in the CTA's, its head
  int skip, skip_h, n_kv;  // to the next one
  int row_s, head_s, pool_head_s, scale_head_s;   // strides
  int in_row, left;        // vector 0 of the CTA in its row; rows from row0 on
  int64_t row0;
  uint16_t* rows;          // the lane's elements of the CTA's first row
  unsigned char* pool;
  float* scales;
  const RowPlace* places;

  __device__ __forceinline__ explicit Team(const Args& a) {
    const int tid = threadIdx.x;
    const bool v = blockIdx.y;
    n_kv = a.c.n_kv;
    row_s = (int)(v ? a.r.v_row : a.r.k_row);
    head_s = (int)(v ? a.r.v_head : a.r.k_head);
    pool_head_s = (int)a.c.head_stride;
    scale_head_s = (int)a.c.s_head_stride;
    const int64_t vec0 = (int64_t)blockIdx.x * (U * VECS);
    row0 = vec0 >> 31 ? vec0 / n_kv : (int)vec0 / n_kv;
    in_row = (int)(vec0 - row0 * n_kv);
    left = (int)min(a.r.rows - row0, (int64_t)INT32_MAX);
    const int at = in_row + tid / LANES;
    row = at / n_kv;
    head = at - row * n_kv;
    rows = static_cast<uint16_t*>(v ? a.r.v : a.r.k) + row0 * row_s +
           8 * (tid % LANES);
    pool = static_cast<unsigned char*>(v ? a.c.v : a.c.k);
    scales = v ? a.c.vs : a.c.ks;
    skip = VECS / n_kv;
    skip_h = VECS - skip * n_kv;
  }
  // Looks the vectors' places up (all threads of the CTA).
  __device__ __forceinline__ void look_up(const Args& a,
                                          RowPlace (&room)[ROWS]) {
    if constexpr (U == 1) {
      own = place_of(a, row0 + row);
    } else {
      const int n = (in_row + U * VECS - 1) / n_kv + 1;
      for (int i = threadIdx.x; i < n; i += THREADS)
        room[i] = place_of(a, row0 + i);
      places = room;
      __syncthreads();
    }
  }
  __device__ __forceinline__ void next() {
    row += skip;
    head += skip_h;
    if (head >= n_kv) {
      head -= n_kv;
      ++row;
    }
  }
  __device__ __forceinline__ RowPlace place() const {
    if constexpr (U == 1)
      return own;
    else
      return places[row];
  }
  // The lane's pieces in the rows' tensor and in the pool, whose elements have
  // SIZE bytes.
  __device__ __forceinline__ uint16_t* in_rows() const {
    return rows + mul(row, row_s) + mul(head, head_s);
  }
  template <int SIZE>
  __device__ __forceinline__ unsigned char* in_pool(const RowPlace& p) const {
    return pool + (p.pool + mul(head, pool_head_s) +
                   8 * (int)(threadIdx.x % LANES)) *
                      SIZE;
  }
  __device__ __forceinline__ float* scale(const RowPlace& p) const {
    return scales + p.scale + mul(head, scale_head_s);
  }
};
__device__ __forceinline__ uint4& at16(void* p) {
  return *static_cast<uint4*>(p);
}
__device__ __forceinline__ uint2& at8(void* p) {
  return *static_cast<uint2*>(p);
}

// The largest magnitude of a lane's eight elements, NaN left out (NaN where
// there is nothing else).
template <int DT>
__device__ __forceinline__ float amax8(uint4 u) {
  if constexpr (DT == TP_BF16) {
    auto h = [](uint32_t x) {
      return __habs2(*reinterpret_cast<__nv_bfloat162*>(&x));
    };
    const __nv_bfloat162 m =
        __hmax2(__hmax2(h(u.x), h(u.y)), __hmax2(h(u.z), h(u.w)));
    const float2 f = __bfloat1622float2(m);
    return fmaxf(f.x, f.y);
  } else {
    auto h = [](uint32_t x) { return __habs2(*reinterpret_cast<__half2*>(&x)); };
    const __half2 m =
        __hmax2(__hmax2(h(u.x), h(u.y)), __hmax2(h(u.z), h(u.w)));
    const float2 f = __half22float2(m);
    return fmaxf(f.x, f.y);
  }
}
// One step of the exchange: 2·N vectors' values in x, of which a lane keeps the
// half that its bit O names.
template <int N, int O, int U>
__device__ __forceinline__ void keep_half(float (&x)[U]) {
  const bool upper = threadIdx.x & O;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float send = upper ? x[i] : x[i + N];
    const float mine = upper ? x[i + N] : x[i];
    x[i] = fmaxf(mine, __shfl_xor_sync(0xffffffffu, send, O));
  }
}
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float r) {
  return make_uint2(e4m3x4(x[0] * r, x[1] * r, x[2] * r, x[3] * r),
                    e4m3x4(x[4] * r, x[5] * r, x[6] * r, x[7] * r));
}

template <int SRC, int CACHE, int D, int U>
__global__ void __launch_bounds__(THREADS, 4)
    write_kernel(const Args a) {
  using T = Team<D, U>;
  static_assert(U == 1 || U == 4, "the exchange of maxima");
  __shared__ RowPlace room[T::ROWS];
  T t(a);
  T of = t;
  uint4 in[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    in[u][0] = in[u][1] = make_uint4(0, 0, 0, 0);
    if (of.row < t.left) {
      uint16_t* const src = of.in_rows();
      in[u][0] = at16(src);
      in[u][1] = at16(src + T::HALF);
    }
    if (u + 1 < U) of.next();
  }
  t.look_up(a, room);
  if constexpr (CACHE == TP_FP8) {
    float amax[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      amax[u] = fmaxf(amax8<SRC>(in[u][0]), amax8<SRC>(in[u][1]));
    constexpr int LOW = U == 1 ? T::LANES : T::LANES / 4;   // lanes a vector
    if constexpr (U == 4) {
      keep_half<2, T::LANES / 2>(amax);
      keep_half<1, T::LANES / 4>(amax);
    }
#pragma unroll
    for (int o = LOW / 2; o > 0; o >>= 1)
      amax[0] = fmaxf(amax[0], __shfl_xor_sync(0xffffffffu, amax[0], o));
    amax[0] = fmaxf(amax[0], 0.0f);
    const float r = block_factor(amax[0]), s = block_scale(amax[0]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const RowPlace p = t.place();
      float f = r, su = s;
      if constexpr (U == 4) {   // from the lane that has vector u's
        const int from = (threadIdx.x & 31 & ~(T::LANES - 1)) + u * LOW;
        f = __shfl_sync(0xffffffffu, r, from);
        su = __shfl_sync(0xffffffffu, s, from);
      }
      if (p.pool >= 0) {
        unsigned char* const dst = t.template in_pool<1>(p);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float x[8];
          unpack8<SRC>(in[u][h], x);
          at8(dst + h * T::HALF) = codes8(x, f);
        }
        if (threadIdx.x % T::LANES == 0) *t.scale(p) = su;
      }
      if (u + 1 < U) t.next();
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const RowPlace p = t.place();
      if (p.pool >= 0) {
        unsigned char* const dst = t.template in_pool<2>(p);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint4 y = in[u][h];
          if constexpr (SRC != CACHE) {
            float x[8];
            unpack8<SRC>(y, x);
            y = pack8<CACHE>(x);
            if (CACHE == TP_F16 && beyond_f16(x, y))
              record_error(a.status, kDevRange, 41);
          }
          at16(dst + 2 * h * T::HALF) = y;
        }
      }
      if (u + 1 < U) t.next();
    }
  }
}

template <int DST, int CACHE, int D, int U>
__global__ void __launch_bounds__(THREADS, 4)
    read_kernel(const Args a) {
  using T = Team<D, U>;
  __shared__ RowPlace room[T::ROWS];
  T t(a);
  t.look_up(a, room);
  T of = t;
  uint4 in[U][2];
  float scale[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const RowPlace p = of.place();
    in[u][0] = in[u][1] = make_uint4(0, 0, 0, 0);
    scale[u] = 0.0f;
    if (p.pool >= 0) {
      if constexpr (CACHE == TP_FP8) {
        unsigned char* const src = of.template in_pool<1>(p);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint2 x = at8(src + h * T::HALF);
          in[u][h].x = x.x;
          in[u][h].y = x.y;
        }
        scale[u] = *of.scale(p);
      } else {
        unsigned char* const src = of.template in_pool<2>(p);
#pragma unroll
        for (int h = 0; h < 2; ++h) in[u][h] = at16(src + 2 * h * T::HALF);
      }
    }
    if (u + 1 < U) of.next();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (t.place().pool >= 0) {
      uint16_t* const dst = t.in_rows();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint4 y = in[u][h];
        if constexpr (CACHE != DST) {
          float x[8];
          if constexpr (CACHE == TP_FP8) {
            const uint32_t w[2] = {y.x, y.y};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f =
                  pair_to_f32<TP_FP8>((w[j >> 1] >> (16 * (j & 1))) & 0xffffu);
              x[2 * j] = f.x * scale[u];
              x[2 * j + 1] = f.y * scale[u];
            }
          } else {
            unpack8<CACHE>(y, x);
          }
          y = pack8<DST>(x);
          if (DST == TP_F16 && beyond_f16(x, y))
            record_error(a.status, kDevRange, 42);
        }
        at16(dst + h * T::HALF) = y;
      }
    }
    if (u + 1 < U) t.next();
  }
}

using Kernel = void (*)(const Args);

template <bool WRITE, int ROWS_DT, int CACHE, int D, int U>
Kernel kernel() {
  if constexpr (WRITE)
    return write_kernel<ROWS_DT, CACHE, D, U>;
  else
    return read_kernel<ROWS_DT, CACHE, D, U>;
}
template <bool WRITE, int ROWS_DT, int D, int U>
Kernel kernel_of(int cache) {
  return cache == TP_BF16  ? kernel<WRITE, ROWS_DT, TP_BF16, D, U>()
         : cache == TP_F16 ? kernel<WRITE, ROWS_DT, TP_F16, D, U>()
                           : kernel<WRITE, ROWS_DT, TP_FP8, D, U>();
}
template <bool WRITE, int U>
Kernel kernel_of(int dtype, int d, int cache) {
  return dtype == TP_BF16 ? (d == 128 ? kernel_of<WRITE, TP_BF16, 128, U>(cache)
                                      : kernel_of<WRITE, TP_BF16, 64, U>(cache))
                          : (d == 128 ? kernel_of<WRITE, TP_F16, 128, U>(cache)
                                      : kernel_of<WRITE, TP_F16, 64, U>(cache));
}

// Vectors of a thread: as many as keep its loads in flight where there are
// enough vectors to give every SM four CTAs of them, else one.
constexpr int MANY = 4;

template <bool WRITE>
int launch(const tp_kv_cache& c, int dtype, const KvRows& r, unsigned* status,
           void* stream) {
  Args a;
  a.c = c;
  a.r = r;
  a.per_seq = (int)(r.rows / c.b);
  a.status = status;
  const int64_t vecs = r.rows * c.n_kv;   // of K, and as many of V
  const int64_t of_cta = THREADS / (c.d / 16);
  const bool many = vecs >= 2 * MANY * of_cta * device_sm_count();
  const Kernel k = many ? kernel_of<WRITE, MANY>(dtype, c.d, c.dtype)
                        : kernel_of<WRITE, 1>(dtype, c.d, c.dtype);
  const int64_t per = of_cta * (many ? MANY : 1);
  const double size = c.dtype == TP_FP8 ? c.d + 4 : 2 * c.d;
  ProfScope prof(stream, KF_KV_CACHE, 0.0, 2.0 * vecs * (size + 2 * c.d));
  count_launch(1);
  k<<<dim3((unsigned)((vecs + per - 1) / per), 2), THREADS, 0,
      static_cast<cudaStream_t>(stream)>>>(a);
  return cudaGetLastError();
}

}  // namespace

int kv_cache_write(const tp_kv_cache& c, int dtype, const KvRows& r,
                   unsigned* status, void* stream) {
  return launch<true>(c, dtype, r, status, stream);
}

int kv_cache_read(const tp_kv_cache& c, int dtype, const KvRows& r,
                  unsigned* status, void* stream) {
  return launch<false>(c, dtype, r, status, stream);
}

}  // namespace tp
