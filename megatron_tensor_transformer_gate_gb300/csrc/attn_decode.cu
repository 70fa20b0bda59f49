// attn_decode.cu — attention of the newest tokens over a paged key-value cache.
//
// One CTA per row and query head, its four warps taking every fourth token
// with a running maximum and sum each (x_t = scale·q·k_t, o = Σ e^(x_t − m)·v_t,
// l = Σ e^(x_t − m); a new maximum rescales o and l), joined at the end.
#include <cuda_runtime.h>

#include <cmath>

#include "gemm.h"
#include "kv_cache.cuh"
#include "kv_cache.h"
#include "profile.h"

namespace tp {
namespace {

constexpr int WARPS = 4;

struct Params {
  tp_kv_cache c;
  DecodeArgs a;
  int per_seq;
  unsigned* status;
};

// The lane's D/32 elements of a vector.
template <int DT, int D>
__device__ __forceinline__ void load(const void* base, int64_t at, int lane,
                                     float (&x)[D / 32]) {
  constexpr int N = D / 32;
  const int64_t e = at + lane * N;
#pragma unroll
  for (int j = 0; j < N; j += 2) {
    const uint32_t u =
        DT == TP_FP8
            ? *reinterpret_cast<const uint16_t*>(
                  static_cast<const uint8_t*>(base) + e + j)
            : *reinterpret_cast<const uint32_t*>(
                  static_cast<const uint16_t*>(base) + e + j);
    const float2 f = pair_to_f32<DT>(u);
    x[j] = f.x;
    x[j + 1] = f.y;
  }
}

template <int DT, int CACHE, int D>
__global__ void __launch_bounds__(32 * WARPS) decode_kernel(const Params p) {
  constexpr int N = D / 32;
  const tp_kv_cache& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x / p.a.n_q;
  const int head = (int)(blockIdx.x - row * p.a.n_q);
  const int kvh = head / (p.a.n_q / c.n_kv);
  const int seq = (int)(row / p.per_seq);
  // tokens 0 … n − 1 are seen, of those that the table can list
  int64_t n = c.lens[seq] - (int64_t)(seq + 1) * p.per_seq + row + 1;
  if (n > (int64_t)c.table_cols * c.page) {
    n = (int64_t)c.table_cols * c.page;
    record_error(p.status, kDevPage, 43);
  }
  float q[N], o[N] = {}, m = -INFINITY, l = 0.0f;
  load<DT, D>(p.a.q, row * p.a.q_row + head * p.a.q_head, lane, q);
  const float scale = p.a.scale * 1.4426950408889634f;
  for (int64_t t = warp; t < n; t += WARPS) {
    int offset;
    const int64_t page = page_of(c, seq, (int)t, &offset, p.status);
    if (page < 0) continue;
    const int64_t at = page * c.page_stride + offset * c.token_stride +
                       kvh * c.head_stride;
    float k[N], v[N];
    load<CACHE, D>(c.k, at, lane, k);
    load<CACHE, D>(c.v, at, lane, v);
    float x = 0.0f, sk = 1.0f, sv = 1.0f;
    if (CACHE == TP_FP8) {
      const int64_t sat = page * c.s_page_stride + offset * c.s_token_stride +
                          kvh * c.s_head_stride;
      sk = c.ks[sat];
      sv = c.vs[sat];
    }
#pragma unroll
    for (int j = 0; j < N; ++j) x = fmaf(q[j], k[j], x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    x *= sk * scale;
    const float top = fmaxf(m, x), f = exp2f(m - top), w = exp2f(x - top);
    l = fmaf(l, f, w);
#pragma unroll
    for (int j = 0; j < N; ++j) o[j] = fmaf(o[j], f, w * sv * v[j]);
    m = top;
  }
  __shared__ float sm[WARPS], sl[WARPS], so[WARPS][D];
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < N; ++j) so[warp][lane * N + j] = o[j];
  __syncthreads();
  const int e = threadIdx.x;
  float top = -INFINITY, sum = 0.0f, acc = 0.0f;
  for (int w = 0; w < WARPS; ++w) top = fmaxf(top, sm[w]);
  for (int w = 0; w < WARPS; ++w) {
    if (sm[w] == -INFINITY) continue;
    const float f = exp2f(sm[w] - top);
    sum += f * sl[w];
    if (e < D) acc += f * so[w][e];
  }
  const float v = sum == 0.0f ? 0.0f : acc / sum;
  if (e < D) {
    const int64_t at = row * p.a.o_row + head * p.a.o_head + e;
    if (DT == TP_BF16)
      static_cast<__nv_bfloat16*>(p.a.out)[at] = __float2bfloat16(v);
    else
      static_cast<__half*>(p.a.out)[at] = __float2half(v);
  }
  if (e == 0 && p.a.lse != nullptr)
    p.a.lse[row * p.a.n_q + head] =
        sum == 0.0f ? -INFINITY
                    : (top + log2f(sum)) * 0.69314718055994531f;
}

using Kernel = void (*)(const Params);

template <int DT, int D>
Kernel kernel_for(int cache) {
  return cache == TP_BF16  ? decode_kernel<DT, TP_BF16, D>
         : cache == TP_F16 ? decode_kernel<DT, TP_F16, D>
                           : decode_kernel<DT, TP_FP8, D>;
}

}  // namespace

size_t attn_decode_ws_bytes(const tp_kv_cache&, int64_t, int) { return 0; }

int attn_decode(const tp_kv_cache& c, int dtype, const DecodeArgs& a,
                unsigned* status, void* stream) {
  Params p;
  p.c = c;
  p.a = a;
  p.per_seq = (int)(a.rows / c.b);
  p.status = status;
  const Kernel k = dtype == TP_BF16
                       ? (c.d == 128 ? kernel_for<TP_BF16, 128>(c.dtype)
                                     : kernel_for<TP_BF16, 64>(c.dtype))
                       : (c.d == 128 ? kernel_for<TP_F16, 128>(c.dtype)
                                     : kernel_for<TP_F16, 64>(c.dtype));
  // the lengths, and with them the work, are known on the device alone
  ProfScope prof(stream, KF_ATTN_DECODE, 0.0, 0.0);
  count_launch(1);
  k<<<(unsigned)(a.rows * a.n_q), 32 * WARPS, 0,
      static_cast<cudaStream_t>(stream)>>>(p);
  return cudaGetLastError();
}

}  // namespace tp
