// kv_cache.cu — rows of K and V into the pages of a key-value cache, and back.
//
// A vector (one head of one token, d elements) is the unit of both calls: a
// team of d/8 lanes moves 16 bytes of its row each.  The cost is one read and
// one write of the vectors.  With few vectors a thread has one of them, and what
// stands in front of it (the row's sequence, its length, its page: a chain of
// loads) it looks up for itself.  With many it has eight, whose loads are all in
// flight before the first is used, and a CTA's look-ups are made once a row.
// Quantized, eight vectors' largest magnitudes are found together by halving
// exchanges that leave one vector's in each lane (or two), which then divides
// for it alone.
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

// A CTA has U·VECS neighbouring vectors, (row, K or V, head) in this order, of
// which a team takes every VECS-th.
template <int D, int U>
struct Team {
  static constexpr int LANES = D / 8, VECS = THREADS / LANES;
  // rows of a CTA's vectors: two vectors a row at least, and both ends cut
  static constexpr int ROWS = U == 1 ? 1 : U * VECS / 2 + 1;
  static_assert(ROWS <= THREADS, "a thread for each row");
  RowPlace own;     // U == 1: of the vector's row
  int row, head;    // vector 0: its row in the CTA's; head, or n_kv + head of V
  int skip, skip_h; // to the next one
  int64_t row0;
  Args const* args;
  const RowPlace* places;

  __device__ __forceinline__ Team(const Args& a, RowPlace (&room)[ROWS])
      : args(&a), places(room) {
    const int per_row = 2 * a.c.n_kv, tid = threadIdx.x;
    const int64_t vec0 = (int64_t)blockIdx.x * (U * VECS);
    row0 = vec0 >> 31 ? vec0 / per_row : (int)vec0 / per_row;
    const int in_row = (int)(vec0 - row0 * per_row);
    const int v = in_row + tid / LANES;
    row = v / per_row;
    head = v - row * per_row;
    if constexpr (U == 1) {
      own = place_of(a, row0 + row);
    } else {
      const int rows = (in_row + U * VECS - 1) / per_row + 1;
      if (tid < rows) room[tid] = place_of(a, row0 + tid);
      skip = VECS / per_row;
      skip_h = VECS - skip * per_row;
      __syncthreads();
    }
  }
  __device__ __forceinline__ void next() {
    row += skip;
    head += skip_h;
    if (head >= 2 * args->c.n_kv) {
      head -= 2 * args->c.n_kv;
      ++row;
    }
  }
  __device__ __forceinline__ RowPlace place() const {
    if constexpr (U == 1)
      return own;
    else
      return places[row];
  }
  __device__ __forceinline__ bool is_v() const { return head >= args->c.n_kv; }
  __device__ __forceinline__ int kv_head() const {
    return head - (is_v() ? args->c.n_kv : 0);
  }
  // The lane's eight elements in the rows' tensor, and their offset in the pool.
  __device__ __forceinline__ uint4* in_rows() const {
    const bool v = is_v();
    return reinterpret_cast<uint4*>(
        static_cast<uint16_t*>(v ? args->r.v : args->r.k) +
        row0 * (v ? args->r.v_row : args->r.k_row) +
        mul(row, (int)(v ? args->r.v_row : args->r.k_row)) +
        mul(kv_head(), (int)(v ? args->r.v_head : args->r.k_head)) +
        8 * (threadIdx.x % LANES));
  }
  __device__ __forceinline__ int64_t in_pool(const RowPlace& p) const {
    return p.pool + mul(kv_head(), (int)args->c.head_stride) +
           8 * (threadIdx.x % LANES);
  }
  __device__ __forceinline__ void* pool() const {
    return is_v() ? args->c.v : args->c.k;
  }
  __device__ __forceinline__ float* scale(const RowPlace& p) const {
    return (is_v() ? args->c.vs : args->c.ks) + p.scale +
           mul(kv_head(), (int)args->c.s_head_stride);
  }
};

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
__global__ void __launch_bounds__(THREADS) write_kernel(const Args a) {
  using T = Team<D, U>;
  static_assert(U == 1 || U == 8, "the exchange of maxima");
  __shared__ RowPlace room[T::ROWS];
  T t(a, room);
  const T first = t;
  uint4 in[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    in[u] = make_uint4(0, 0, 0, 0);
    if (t.place().pool >= 0) in[u] = *t.in_rows();
    if (u + 1 < U) t.next();
  }
  t = first;
  if constexpr (CACHE == TP_FP8) {
    float amax[U];
#pragma unroll
    for (int u = 0; u < U; ++u) amax[u] = amax8<SRC>(in[u]);
    float r = 0.0f;
    constexpr int LOW = U == 1 ? T::LANES : T::LANES / 8;   // lanes a vector
    if constexpr (U == 8) {
      keep_half<4, T::LANES / 2>(amax);
      keep_half<2, T::LANES / 4>(amax);
      keep_half<1, T::LANES / 8>(amax);
    }
#pragma unroll
    for (int o = LOW / 2; o > 0; o >>= 1)
      amax[0] = fmaxf(amax[0], __shfl_xor_sync(0xffffffffu, amax[0], o));
    amax[0] = fmaxf(amax[0], 0.0f);
    r = block_factor(amax[0]);
    const float s = block_scale(amax[0]);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const RowPlace p = t.place();
      float f = r, su = s;
      if constexpr (U == 8) {   // from the lane that has vector u's
        const int from = (threadIdx.x & 31 & ~(T::LANES - 1)) + u * LOW;
        f = __shfl_sync(0xffffffffu, r, from);
        su = __shfl_sync(0xffffffffu, s, from);
      }
      if (p.pool >= 0) {
        float x[8];
        unpack8<SRC>(in[u], x);
        *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.pool()) +
                                  t.in_pool(p)) = codes8(x, f);
        if (threadIdx.x % T::LANES == 0) *t.scale(p) = su;
      }
      if (u + 1 < U) t.next();
    }
  } else {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const RowPlace p = t.place();
      if (p.pool >= 0) {
        if constexpr (SRC != CACHE) {
          float x[8];
          unpack8<SRC>(in[u], x);
          if (CACHE == TP_F16 && beyond_f16(x))
            record_error(a.status, kDevRange, 41);
          in[u] = pack8<CACHE>(x);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(t.pool()) +
                                  t.in_pool(p)) = in[u];
      }
      if (u + 1 < U) t.next();
    }
  }
}

template <int DST, int CACHE, int D, int U>
__global__ void __launch_bounds__(THREADS) read_kernel(const Args a) {
  using T = Team<D, U>;
  __shared__ RowPlace room[T::ROWS];
  T t(a, room);
  const T first = t;
  uint4 in[U];
  float scale[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const RowPlace p = t.place();
    in[u] = make_uint4(0, 0, 0, 0);
    scale[u] = 0.0f;
    if (p.pool >= 0) {
      if constexpr (CACHE == TP_FP8) {
        const uint2 x = *reinterpret_cast<const uint2*>(
            static_cast<const uint8_t*>(t.pool()) + t.in_pool(p));
        in[u].x = x.x;
        in[u].y = x.y;
        scale[u] = *t.scale(p);
      } else {
        in[u] = *reinterpret_cast<const uint4*>(
            static_cast<const uint16_t*>(t.pool()) + t.in_pool(p));
      }
    }
    if (u + 1 < U) t.next();
  }
  t = first;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (t.place().pool >= 0) {
      if constexpr (CACHE != DST) {
        float x[8];
        if constexpr (CACHE == TP_FP8) {
          const uint32_t w[2] = {in[u].x, in[u].y};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 f =
                pair_to_f32<TP_FP8>((w[j >> 1] >> (16 * (j & 1))) & 0xffffu);
            x[2 * j] = f.x * scale[u];
            x[2 * j + 1] = f.y * scale[u];
          }
        } else {
          unpack8<CACHE>(in[u], x);
        }
        if (DST == TP_F16 && beyond_f16(x))
          record_error(a.status, kDevRange, 42);
        in[u] = pack8<DST>(x);
      }
      *t.in_rows() = in[u];
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
constexpr int MANY = 8;

template <bool WRITE>
int launch(const tp_kv_cache& c, int dtype, const KvRows& r, unsigned* status,
           void* stream) {
  Args a;
  a.c = c;
  a.r = r;
  a.per_seq = (int)(r.rows / c.b);
  a.status = status;
  const int64_t vecs = r.rows * 2 * c.n_kv, of_cta = THREADS / (c.d / 8);
  const bool many = vecs >= 4 * MANY * of_cta * device_sm_count();
  const Kernel k = many ? kernel_of<WRITE, MANY>(dtype, c.d, c.dtype)
                        : kernel_of<WRITE, 1>(dtype, c.d, c.dtype);
  const int64_t per = of_cta * (many ? MANY : 1);
  const double size = c.dtype == TP_FP8 ? c.d + 4 : 2 * c.d;
  ProfScope prof(stream, KF_KV_CACHE, 0.0, vecs * (size + 2.0 * c.d));
  count_launch(1);
  k<<<(unsigned)((vecs + per - 1) / per), THREADS, 0,
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
