// attn_decode.cu — attention of the newest tokens over a paged key-value cache.
//
//   x_t = scale·q·k_t,  o = Σ_t e^(x_t)·v_t / Σ_t e^(x_t)
//
// The cost is one read of the cached K and V, so every byte of them is read
// once for all query rows of a kv head (a unit: up to 32 rows, 8·NT), and what
// the SMs read is shared out evenly whatever the sequences' lengths: all units'
// blocks of 64 tokens, laid end to end, are cut into as many equal pieces as
// there are CTAs.  A CTA walks its piece segment by segment (a segment: the
// part of one unit in it).  A unit that lies in one CTA is finished there;
// one that is cut leaves partial results (o normalised, log₂ of its sum) in the
// workspace, at most two a CTA, which a second kernel joins in CTA order:
//   L = max lse_c, o = Σ 2^(lse_c − L)·o_c / Σ 2^(lse_c − L).
//
// In a CTA each of four warps takes every fourth step of 16 tokens and runs an
// online softmax of its own, so that nothing waits on another warp before the
// segment's end.  Its K and V rows come by asynchronous 16-byte copies into a
// ring of the warp's own.  Both products are mma.sync m16n8k16 with the cache
// on the 16 side: Sᵀ = K·Qᵀ (16 tokens × 8 rows) and Oᵀ += Vᵀ·Pᵀ (16 elements
// × 8 rows), K by ldmatrix, Vᵀ by its transposing form; between them P is
// transposed in registers (movmatrix).  With few rows a group the
// tensor cores' 128-row instructions would idle on padding and cost a pass of
// the codes through shared memory; here E4M3 codes become fp16 operands in
// registers.
//
// Precision: scores, maxima, sums and o are fp32.  Over fp16 values and E4M3
// codes the operands are fp16, q divided by a power of two that brings its
// largest element to [1, 2) (exact but for elements below 2^-14 of it).  P is
// rounded to fp16 (2^-11); over bf16 values, where bf16 (2^-8) would show in
// the output, it is the sum of two bf16 parts, 2^-16, at the price of a second
// product.  A code's scale is multiplied into its score, and into its weight in
// front of the product with V: w = 2^(x + log₂ s_v − M) with a running maximum
// M of its own, so that scales of any size keep the weights in fp16's range.
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "gemm.h"
#include "kv_cache.cuh"
#include "kv_cache.h"
#include "profile.h"

namespace tp {
namespace {

constexpr int WARPS = 4;
constexpr int THREADS = 32 * WARPS;
constexpr int CTAS = 2;               // on an SM
constexpr int STEP = 16;              // tokens of a warp at a time
constexpr int BLOCK = STEP * WARPS;   // tokens of a CTA at a time
constexpr int MIN_BLOCKS = 2;         // of a CTA, where there is little to do
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.69314718055994531f;

// Where the first part of a unit that is cut lies, for the join.
struct Cut {
  int seq, head, tile;   // tile < 0: this CTA begins no such unit
  int first_slot;        // its slot, 2·CTA or 2·CTA + 1
  int parts;             // CTAs that hold a part; the others' slots are 2·CTA
};

struct Params {
  tp_kv_cache c;
  DecodeArgs a;
  int per_seq;           // new tokens of a sequence
  int group;             // query heads of a kv head
  int tiles;             // row tiles of a kv head
  float* part_o;         // [2·CTAs][8·NT][D]
  float* part_lse;       // [2·CTAs][8·NT], log₂
  Cut* cuts;             // [CTAs]
  unsigned* status;
};

template <int CACHE, int D, int NT>
struct Conf {
  static constexpr int SIZE = CACHE == TP_FP8 ? 1 : 2;
  static constexpr int ROW = D * SIZE;             // bytes
  static constexpr int ROWS = 8 * NT;
  static constexpr int TILE = STEP * ROW;
  // K, V, the scales and the valid tokens of a step
  static constexpr int STAGE = 2 * TILE + (CACHE == TP_FP8 ? 128 : 0);
  static constexpr int STAGES = ROW == 256 ? 3 : ROW == 128 ? 6 : 8;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int JOIN = ROWS * (D + 4) * 4;  // of a warp, over its ring
  static constexpr int SMEM = WARPS * (RING > JOIN ? RING : JOIN);
  static constexpr bool QREG = NT < 4;             // Q in registers
  static constexpr int QSMEM = QREG ? 0 : ROWS * D * 2;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src,
                                           bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void ldmatrix(uint32_t a, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(a)
      : "memory");
}
__device__ __forceinline__ void ldmatrix_trans(uint32_t a, uint32_t (&r)[4]) {
  asm volatile(
      "ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(a)
      : "memory");
}
// Lane (g, t) of an 8×8 matrix (row g, columns 2t and 2t + 1) gets its
// transpose's.
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;"
               : "=r"(y)
               : "r"(x));
  return y;
}
template <bool BF>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4],
                                    uint32_t b0, uint32_t b1) {
  if constexpr (BF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Two E4M3 codes (the lower 16 bits) as fp16.
__device__ __forceinline__ uint32_t codes_f16(uint32_t u) {
  uint32_t y;
  asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t}"
      : "=r"(y)
      : "r"(u));
  return y;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte offset of 16-byte chunk ch of row r in a tile, spread so that eight
// rows' same chunk lie in different banks.
template <int ROW>
__device__ __forceinline__ uint32_t spread(int r, int ch) {
  return ROW >= 128 ? r * ROW + ((ch ^ (r & 7)) << 4)
                    : r * ROW + ((ch ^ ((r >> 1) & 3)) << 4);
}

// A sequence's tokens that are followed, and the blocks they take (at least
// one, so that a sequence without any has its rows written too).
__device__ __forceinline__ int tokens_of(const tp_kv_cache& c, int seq) {
  const int64_t cap = (int64_t)c.table_cols * c.page;
  const int n = c.lens[seq];
  return n < 0 ? 0 : n > cap ? (int)cap : n;
}
__device__ __forceinline__ int blocks_of(int n) {
  return n <= BLOCK ? 1 : (n - 1) / BLOCK + 1;
}

// The pages of a warp's next tokens: lane l holds table entries base + l and
// base + 32 + l of a sequence, the second ones read ahead.
struct Pages {
  const int32_t* row;
  int base, end, cur, next;   // entries from `end` on are not read
  __device__ __forceinline__ int get(int col) const {
    return col < end ? row[col] : -1;
  }
  __device__ __forceinline__ void start(const int32_t* r, int first, int last,
                                        int lane) {
    row = r;
    base = first;
    end = last;
    cur = get(base + lane);
    next = get(base + 32 + lane);
  }
  __device__ __forceinline__ void move_to(int col, int lane) {
    while (col >= base + 32) {
      base += 32;
      cur = next;
      next = get(base + 32 + lane);
    }
  }
  __device__ __forceinline__ int at(int col) const {   // base ≤ col < base + 64
    const int a = __shfl_sync(0xffffffffu, cur, col - base);
    const int b = __shfl_sync(0xffffffffu, next, col - base);
    return col - base < 32 ? a : b;
  }
};

template <int CACHE, int D, int NT>
__global__ void __launch_bounds__(THREADS, CTAS)
    decode_kernel(const Params p) {
  using C = Conf<CACHE, D, NT>;
  constexpr bool FP8 = CACHE == TP_FP8, BF = CACHE == TP_BF16;
  constexpr int KS = D / 16;          // steps of 16 elements
  constexpr int ROW = C::ROW, CHUNKS = ROW / 16;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ int64_t sum_of[WARPS];
  __shared__ int64_t s_before;
  __shared__ int s_seq;
  __shared__ uint32_t valid_of[WARPS][C::STAGES];
  __shared__ float s_m[WARPS][C::ROWS], s_top[WARPS][C::ROWS],
      s_l[WARPS][C::ROWS];
  const tp_kv_cache& c = p.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  const int per_block = c.n_kv * p.tiles;   // units of a sequence

  // ---- this CTA's piece: blocks [at, stop) of all, and where `at` lies
  int64_t at, stop;
  int64_t total;
  {
    const int span = (c.b + THREADS - 1) / THREADS;
    const int i0 = min(tid * span, c.b), i1 = min(i0 + span, c.b);
    int64_t sum = 0;
    for (int i = i0; i < i1; ++i) sum += blocks_of(tokens_of(c, i));
    int64_t inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    if (lane == 31) sum_of[warp] = inc;
    __syncthreads();
    int64_t before = inc - sum;
    total = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
      if (w < warp) before += sum_of[w];
      total += sum_of[w];
    }
    total *= per_block;
    const int64_t most = (total + MIN_BLOCKS - 1) / MIN_BLOCKS;
    const int64_t ctas = most < gridDim.x ? most : gridDim.x;
    if (blockIdx.x >= ctas) {
      if (tid == 0) p.cuts[blockIdx.x].tile = -1;
      return;
    }
    at = total * blockIdx.x / ctas;
    stop = total * (blockIdx.x + 1) / ctas;
    before *= per_block;
    sum *= per_block;
    if (before <= at && at < before + sum) {   // one thread
      int i = i0;
      for (;; ++i) {
        const int64_t w = (int64_t)blocks_of(tokens_of(c, i)) * per_block;
        if (at < before + w) break;
        before += w;
      }
      s_seq = i;
      s_before = before;
    }
    __syncthreads();
    if (tid == 0) p.cuts[blockIdx.x].tile = -1;
  }
  const int64_t begin = at;
  int seq = s_seq;
  int64_t before = s_before;   // blocks in front of the sequence

  const uint32_t ring = smem_u32(smem) + warp * C::RING;
  unsigned char* const q_smem =
      smem + WARPS * (C::RING > C::JOIN ? C::RING : C::JOIN);
  const float scale = p.a.scale * LOG2E;
  const char* const kpool = static_cast<const char*>(c.k);
  const int64_t to_v = static_cast<const char*>(c.v) - kpool;
  const bool whole_pages = c.page % STEP == 0;

  while (at < stop) {
    // ---- the segment: blocks [blk0, blk1) of a unit
    const int len = max(c.lens[seq], 0);
    const int n = tokens_of(c, seq);
    const int nb = blocks_of(n);
    const int unit = (int)((at - before) / nb);
    const int blk0 = (int)((at - before) - (int64_t)unit * nb);
    const int blk1 = (int)min((int64_t)nb, blk0 + (stop - at));
    const int kvh = unit / p.tiles, tile = unit - kvh * p.tiles;
    const int row0 = tile * C::ROWS, rows = p.per_seq * p.group;
    const int64_t qrow = (int64_t)seq * p.per_seq;
    if (len > n && tid == 0) record_error(p.status, kDevPage, 43);

    // ---- Q: lane (g, t) holds elements of row 8·nt + g as the products take
    // them (over codes, four neighbours of a step instead of two and two)
    uint32_t q[C::QREG ? NT : 1][KS][2];
    float qf[NT][2];      // scale of the lane's rows 8·nt + 2·t4 (+ 1)
    int lim[NT][2];       // tokens that they see
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = row0 + 8 * nt + g;
      const bool there = r < rows;
      const int j = there ? r / p.group : 0;
      const uint16_t* src =
          static_cast<const uint16_t*>(p.a.q) + (qrow + j) * p.a.q_row +
          (there ? (int64_t)(kvh * p.group + r - j * p.group) * p.a.q_head : 0);
      uint32_t u[KS][2];
      float amax = 0.0f;
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int e0 = 16 * s + (FP8 ? 4 : 2) * t4, e1 = e0 + (FP8 ? 2 : 8);
        u[s][0] = there ? *reinterpret_cast<const uint32_t*>(src + e0) : 0u;
        u[s][1] = there ? *reinterpret_cast<const uint32_t*>(src + e1) : 0u;
      }
      float f = 1.0f;
      if (!BF) {
        float2 x[KS][2];
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            x[s][h] = p.a.bf16 ? unpack_bf16x2(u[s][h]) : unpack_f16x2(u[s][h]);
            amax = fmaxf(amax, fmaxf(fabsf(x[s][h].x), fabsf(x[s][h].y)));
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // 2^e ≤ amax < 2^(e + 1), and q·2^-e
        const int e =
            amax == 0.0f
                ? 0
                : min((int)(__float_as_uint(amax) >> 23) - 127, 126);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
        f = e >= -126 ? __uint_as_float((uint32_t)(127 + e) << 23)
                      : 5.8774717541114375e-39f;   // 2^-127
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            u[s][h] = pack_f16x2(x[s][h].x * down, x[s][h].y * down);
      }
      f *= scale;
      qf[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t4);
      qf[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int rr = row0 + 8 * nt + 2 * t4 + h;
        lim[nt][h] = rr < rows
                         ? min(n, len - p.per_seq + 1 + rr / p.group)
                         : n;
      }
      if constexpr (C::QREG) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          q[nt][s][0] = u[s][0];
          q[nt][s][1] = u[s][1];
        }
      } else if (warp == 0) {   // [nt][s][lane] pairs of registers
#pragma unroll
        for (int s = 0; s < KS; ++s)
          reinterpret_cast<uint2*>(q_smem)[(nt * KS + s) * 32 + lane] =
              make_uint2(u[s][0], u[s][1]);
      }
    }
    if constexpr (!C::QREG) __syncthreads();

    // ---- the warp's steps: 16 tokens from 64·blk + 16·warp on
    const int first = blk0 * BLOCK + warp * STEP;
    const int steps =
        first < n ? min(blk1 - blk0, (n - 1 - first) / BLOCK + 1) : 0;
    const int64_t head_at = (int64_t)kvh * c.head_stride * C::SIZE;
    Pages pg;
    pg.start(c.table + (int64_t)seq * c.table_stride,
             steps > 0 ? first / c.page : 0, n > 0 ? (n - 1) / c.page + 1 : 0,
             lane);
    auto issue = [&](int i, int stage) {
      const int t0 = first + i * BLOCK;
      const uint32_t dst = ring + stage * C::STAGE;
      // lane r < 16: the place of token t0 + r
      const int tok = t0 + (lane & 15);
      bool in = tok < n;
      int64_t page;
      int off;
      if (whole_pages) {
        const int col = t0 / c.page;
        pg.move_to(col, lane);
        page = pg.at(col);
        off = tok - col * c.page;
      } else {
        const int col0 = t0 / c.page;
        pg.move_to(col0, lane);
        const int col = (in ? tok : t0) / c.page;
        page = pg.at(col);
        off = tok - col * c.page;
      }
      if (in && (page < 0 || page >= c.pages)) {
        in = false;
        record_error(p.status, kDevPage, 44);
      }
      const uint32_t valid = __ballot_sync(0xffffffffu, in) & 0xffffu;
      if (lane == 0) valid_of[warp][stage] = valid;
      if (FP8) {   // scales of K in lanes 0 to 15, of V in the others
        const int64_t sat = in ? page * c.s_page_stride +
                                     off * c.s_token_stride +
                                     kvh * c.s_head_stride
                               : 0;
        cp_async4(reinterpret_cast<float*>(smem + warp * C::RING +
                                           stage * C::STAGE + 2 * C::TILE) +
                      lane,
                  (lane < 16 ? c.ks : c.vs) + sat, in);
      }
      int64_t place = in ? (page * c.page_stride + off * c.token_stride) *
                                   C::SIZE +
                               head_at
                         : 0;
      constexpr int LANES = CHUNKS;            // of a row
      constexpr int PER = 32 / LANES;          // rows of an instruction
      const int ch = lane % LANES, sub = lane / LANES;
#pragma unroll
      for (int k = 0; k < STEP / PER; ++k) {
        const int r = k * PER + sub;
        const int64_t pl = __shfl_sync(0xffffffffu, place, r);
        const char* src = kpool + pl + 16 * ch;
        const bool ok = (valid >> r) & 1;
        const uint32_t d = dst + spread<ROW>(r, ch);
        cp_async16(d, src, ok);
        cp_async16(d + C::TILE, src + to_v, ok);
      }
    };

    float o[KS][NT][4];
    float m[NT][2], top[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int s = 0; s < KS; ++s)
#pragma unroll
        for (int j = 0; j < 4; ++j) o[s][nt][j] = 0.0f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[nt][h] = top[nt][h] = -INFINITY;
        l[nt][h] = 0.0f;
      }
    }
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) {
      if (s < steps) issue(s, s);
      cp_async_commit();
    }
    int stage = 0;
    for (int i = 0; i < steps; ++i) {
      cp_async_wait<C::STAGES - 2>();
      __syncwarp();
      {
        const int ahead = i + C::STAGES - 1;
        int to = stage + C::STAGES - 1;
        if (to >= C::STAGES) to -= C::STAGES;
        if (ahead < steps) issue(ahead, to);
        cp_async_commit();
      }
      const uint32_t kt = ring + stage * C::STAGE, vt = kt + C::TILE;
      const uint32_t valid = valid_of[warp][stage];
      const int t0 = first + i * BLOCK;

      // ---- Sᵀ = K·Qᵀ
      float sc[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j) sc[nt][j] = 0.0f;
      auto add_scores = [&](const uint32_t(&a)[4], int s) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if constexpr (C::QREG) {
            mma<BF>(sc[nt], a, q[nt][s][0], q[nt][s][1]);
          } else {
            const uint2 u =
                reinterpret_cast<const uint2*>(q_smem)[(nt * KS + s) * 32 +
                                                       lane];
            mma<BF>(sc[nt], a, u.x, u.y);
          }
        }
      };
      if constexpr (FP8) {
#pragma unroll
        for (int s = 0; s < KS; s += 2) {
          // rows 0–7 and 8–15 of chunk s, then of chunk s + 1
          uint32_t u[4];
          ldmatrix(kt + spread<ROW>((lane & 7) + (lane & 8), s + (lane >> 4)),
                   u);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a[4] = {
                codes_f16(u[2 * h]), codes_f16(u[2 * h + 1]),
                codes_f16(u[2 * h] >> 16), codes_f16(u[2 * h + 1] >> 16)};
            add_scores(a, s + h);
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint32_t a[4];
          ldmatrix(kt + spread<ROW>(lane & 15, 2 * s + (lane >> 4)), a);
          add_scores(a, s);
        }
      }

      // ---- softmax of the lane's rows 2·t4, 2·t4 + 1 at tokens g and g + 8
      float sk[2] = {1.0f, 1.0f}, lv[2] = {0.0f, 0.0f};
      if (FP8) {
        const float* ss = reinterpret_cast<const float*>(
            smem + (kt - smem_u32(smem)) + 2 * C::TILE);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          sk[h] = ss[g + 8 * h];
          lv[h] = lg2_approx(ss[16 + g + 8 * h]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sc[nt][j] *= FP8 ? qf[nt][j & 1] * sk[j >> 1] : qf[nt][j & 1];
      const bool mixed = p.per_seq > 1 && t0 > len - p.per_seq + 1 - STEP;
      if (valid != 0xffffu || mixed) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = g + 8 * (j >> 1);
            if (!((valid >> k) & 1) || t0 + k >= lim[nt][j & 1])
              sc[nt][j] = -INFINITY;
          }
      }
      bool more = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          more |= fmaxf(sc[nt][h], sc[nt][2 + h]) > m[nt][h];
          if (FP8)
            more |= fmaxf(sc[nt][h] + lv[0], sc[nt][2 + h] + lv[1]) >
                    top[nt][h];
        }
      if (__any_sync(0xffffffffu, more)) {   // new maxima
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = fmaxf(m[nt][h], fmaxf(sc[nt][h], sc[nt][2 + h]));
            float y = x;
            if (FP8)
              y = fmaxf(top[nt][h],
                        fmaxf(sc[nt][h] + lv[0], sc[nt][2 + h] + lv[1]));
#pragma unroll
            for (int z = 4; z < 32; z <<= 1) {
              x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, z));
              if (FP8) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, z));
            }
            if (!FP8) y = x;
            // 0 where there was nothing yet
            l[nt][h] *= m[nt][h] == -INFINITY ? 0.0f : ex2_approx(m[nt][h] - x);
            const float f = top[nt][h] == -INFINITY
                                ? 0.0f
                                : ex2_approx(top[nt][h] - y);
            m[nt][h] = x;
            top[nt][h] = y;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              o[s][nt][h] *= f;
              o[s][nt][2 + h] *= f;
            }
          }
      }
      // weights: 0 where a row has seen nothing yet
      uint32_t b[NT][2], b2[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float ref = m[nt][j & 1] == -INFINITY ? 0.0f : m[nt][j & 1];
          w[j] = ex2_approx(sc[nt][j] - ref);
          l[nt][j & 1] += w[j];
          if (FP8) {
            const float far =
                top[nt][j & 1] == -INFINITY ? 0.0f : top[nt][j & 1];
            w[j] = sc[nt][j] == -INFINITY
                       ? 0.0f
                       : ex2_approx(sc[nt][j] + lv[j >> 1] - far);
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (BF) {
            const uint32_t hi = pack_bf16x2(w[2 * h], w[2 * h + 1]);
            const float2 f = unpack_bf16x2(hi);
            b[nt][h] = movmatrix(hi);
            b2[nt][h] =
                movmatrix(pack_bf16x2(w[2 * h] - f.x, w[2 * h + 1] - f.y));
          } else {
            b[nt][h] = movmatrix(pack_f16x2(w[2 * h], w[2 * h + 1]));
          }
        }
      }

      // ---- Oᵀ += Vᵀ·Pᵀ
      auto add_values = [&](const uint32_t(&a)[4], int s) {
        if (!mixed) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma<BF>(o[s][nt], a, b[nt][0], b[nt][1]);
            if (BF) mma<BF>(o[s][nt], a, b2[nt][0], b2[nt][1]);
          }
          return;
        }
        // Rows of several new tokens see different ends of this step.  What
        // a later token's v holds (NaN, say) must not reach a row that does
        // not see it through a weight of 0: one product for each of them.
        const int j1 = min(p.per_seq - 1, (row0 + C::ROWS - 1) / p.group);
        for (int j = row0 / p.group; j <= j1; ++j) {
          const int end = len - p.per_seq + 1 + j - t0;   // tokens seen
          uint32_t cut[4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int k = 2 * t4 + 8 * h;
            const uint32_t keep = (k < end ? 0xffffu : 0u) |
                                  (k + 1 < end ? 0xffff0000u : 0u);
            cut[2 * h] = a[2 * h] & keep;
            cut[2 * h + 1] = a[2 * h + 1] & keep;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float x[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            mma<BF>(x, cut, b[nt][0], b[nt][1]);
            if (BF) mma<BF>(x, cut, b2[nt][0], b2[nt][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((row0 + 8 * nt + 2 * t4 + (e & 1)) / p.group == j)
                o[s][nt][e] += x[e];
          }
        }
      };
      if constexpr (FP8) {
#pragma unroll
        for (int s = 0; s < KS; s += 2) {
          uint32_t u[4];
          ldmatrix_trans(
              vt + spread<ROW>((lane & 7) + (lane & 8), s + (lane >> 4)), u);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // elements 2g and 2g + 1 of tokens 2t, 2t + 1 to pairs of tokens
            const uint32_t x = __byte_perm(u[2 * h], 0, 0x3120),
                           y = __byte_perm(u[2 * h + 1], 0, 0x3120);
            const uint32_t a[4] = {codes_f16(x), codes_f16(x >> 16),
                                   codes_f16(y), codes_f16(y >> 16)};
            add_values(a, s + h);
          }
        }
      } else {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          uint32_t a[4];
          ldmatrix_trans(vt + spread<ROW>((lane & 7) + ((lane >> 1) & 8),
                                          2 * s + ((lane >> 3) & 1)),
                         a);
          add_values(a, s);
        }
      }
      if (++stage == C::STAGES) stage = 0;
    }
    cp_async_wait<0>();

    // ---- the warps' results together
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int z = 4; z < 32; z <<= 1)
          l[nt][h] += __shfl_xor_sync(0xffffffffu, l[nt][h], z);
        if (g == 0) {
          const int r = 8 * nt + 2 * t4 + h;
          s_m[warp][r] = m[nt][h];
          s_top[warp][r] = top[nt][h];
          s_l[warp][r] = l[nt][h];
        }
      }
    __syncthreads();   // every warp's ring is read
    float* const join = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * nt + 2 * t4 + h;
        float all = s_top[0][r];
#pragma unroll
        for (int w = 1; w < WARPS; ++w) all = fmaxf(all, s_top[w][r]);
        const float f = top[nt][h] == -INFINITY
                            ? 0.0f
                            : ex2_approx(top[nt][h] - all);
        float* dst = join + (warp * C::ROWS + r) * (D + 4);
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const int e0 = 16 * s + (FP8 ? 2 * g : g);
          dst[e0] = o[s][nt][h] * f;
          dst[e0 + (FP8 ? 1 : 8)] = o[s][nt][2 + h] * f;
        }
      }
    __syncthreads();
    const bool part = blk0 > 0 || blk1 < nb;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (at != begin);
    constexpr int QUADS = D / 4;
    for (int i = tid; i < C::ROWS * QUADS; i += THREADS) {
      const int r = i / QUADS, e = 4 * (i - r * QUADS);
      const int rr = row0 + r;
      if (rr >= rows) break;
      float mm = s_m[0][r], tt = s_top[0][r];
#pragma unroll
      for (int w = 1; w < WARPS; ++w) {
        mm = fmaxf(mm, s_m[w][r]);
        tt = fmaxf(tt, s_top[w][r]);
      }
      float sum = 0.0f;
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float4 x = *reinterpret_cast<const float4*>(
            join + (w * C::ROWS + r) * (D + 4) + e);
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
        // a warp without a maximum has l = 0, or NaN of NaN scores
        sum = s_m[w][r] == -INFINITY
                  ? sum + s_l[w][r]
                  : fmaf(s_l[w][r], ex2_approx(s_m[w][r] - mm), sum);
      }
      const bool none = sum == 0.0f;
      const float f = none ? 0.0f : (FP8 ? ex2_approx(tt - mm) : 1.0f) / sum;
      v.x *= f;
      v.y *= f;
      v.z *= f;
      v.w *= f;
      const float lse2 = none ? -INFINITY : mm + log2f(sum);
      if (part) {
        *reinterpret_cast<float4*>(p.part_o + (slot * C::ROWS + r) * D + e) =
            v;
        if (e == 0) p.part_lse[slot * C::ROWS + r] = lse2;
      } else {
        const int j = rr / p.group;
        const int head = kvh * p.group + rr - j * p.group;
        const int64_t row = qrow + j;
        uint16_t* dst = static_cast<uint16_t*>(p.a.out) + row * p.a.o_row +
                        head * p.a.o_head + e;
        *reinterpret_cast<uint2*>(dst) =
            p.a.bf16 ? make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w))
                     : make_uint2(pack_f16x2(v.x, v.y), pack_f16x2(v.z, v.w));
        if (e == 0 && p.a.lse != nullptr)
          p.a.lse[row * p.a.n_q + head] = lse2 * LN2;
      }
    }
    if (blk0 == 0 && blk1 < nb && tid == 0) {
      // the CTA of the unit's last block: total·c / ctas ≤ it
      const int64_t most = (total + MIN_BLOCKS - 1) / MIN_BLOCKS;
      const int64_t ctas = most < gridDim.x ? most : gridDim.x;
      const int64_t last = at + nb - 1;
      const int end = (int)(((last + 1) * ctas - 1) / total);
      Cut cut;
      cut.seq = seq;
      cut.head = kvh;
      cut.tile = tile;
      cut.first_slot = (int)slot;
      cut.parts = end - (int)blockIdx.x + 1;
      p.cuts[blockIdx.x] = cut;
    }
    at += blk1 - blk0;
    if (at < stop && at - before >= (int64_t)nb * per_block) {
      before += (int64_t)nb * per_block;
      ++seq;
    }
    __syncthreads();   // the joined results are read
  }
}

// Joins the parts of the units that were cut: CTA (i, r) row r of the one that
// CTA i of the first kernel begins, if there is one.
constexpr int JOIN_THREADS = 256;
template <int D>
__global__ void __launch_bounds__(JOIN_THREADS)
    join_kernel(const Params p, int tile_rows) {
  constexpr int TEAM = D / 4, TEAMS = JOIN_THREADS / TEAM;
  __shared__ float s_max[JOIN_THREADS / 32];
  __shared__ float s_sum[TEAMS];
  __shared__ float4 s_o[TEAMS][TEAM];
  const Cut cut = p.cuts[blockIdx.x];
  const int r = blockIdx.y, rr = cut.tile * tile_rows + r;
  if (cut.tile < 0 || rr >= p.per_seq * p.group) return;
  const int tid = threadIdx.x;
  auto slot_of = [&](int i) -> int64_t {
    return i == 0 ? cut.first_slot : 2 * ((int64_t)blockIdx.x + i);
  };
  float top = -INFINITY;
  for (int i = tid; i < cut.parts; i += JOIN_THREADS)
    top = fmaxf(top, p.part_lse[slot_of(i) * tile_rows + r]);
#pragma unroll
  for (int z = 16; z > 0; z >>= 1)
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, z));
  if ((tid & 31) == 0) s_max[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < JOIN_THREADS / 32; ++w) top = fmaxf(top, s_max[w]);
  // parts i, i + TEAMS, …: each team its own, then the teams in order
  const int team = tid / TEAM, e = tid % TEAM;
  float sum = 0.0f;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i = team; i < cut.parts; i += TEAMS) {
    const int64_t at = slot_of(i) * tile_rows + r;
    const float x = p.part_lse[at];
    const float w = x == -INFINITY ? 0.0f : ex2_approx(x - top);
    const float4 u = *reinterpret_cast<const float4*>(p.part_o + at * D + 4 * e);
    sum += w;
    v.x = fmaf(w, u.x, v.x);
    v.y = fmaf(w, u.y, v.y);
    v.z = fmaf(w, u.z, v.z);
    v.w = fmaf(w, u.w, v.w);
  }
  s_o[team][e] = v;
  if (e == 0) s_sum[team] = sum;
  __syncthreads();
  if (team != 0) return;
  for (int k = 1; k < TEAMS; ++k) {
    const float4 u = s_o[k][e];
    sum += s_sum[k];
    v.x += u.x;
    v.y += u.y;
    v.z += u.z;
    v.w += u.w;
  }
  const bool none = sum == 0.0f;
  const float f = none ? 0.0f : 1.0f / sum;
  const int j = rr / p.group;
  const int head = cut.head * p.group + rr - j * p.group;
  const int64_t row = (int64_t)cut.seq * p.per_seq + j;
  uint16_t* dst = static_cast<uint16_t*>(p.a.out) + row * p.a.o_row +
                  head * p.a.o_head + 4 * e;
  v.x *= f;
  v.y *= f;
  v.z *= f;
  v.w *= f;
  *reinterpret_cast<uint2*>(dst) =
      p.a.bf16 ? make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w))
               : make_uint2(pack_f16x2(v.x, v.y), pack_f16x2(v.z, v.w));
  if (e == 0 && p.a.lse != nullptr)
    p.a.lse[row * p.a.n_q + head] =
        none ? -INFINITY : (top + log2f(sum)) * LN2;
}

// Rows of a unit's tile: as few as hold them, 32 at most.
int tile_rows_of(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

struct Layout {
  size_t o, lse, cuts, bytes;
};
Layout layout_of(int ctas, int tile_rows, int d) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  Layout l;
  l.o = 0;
  l.lse = up((size_t)2 * ctas * tile_rows * d * 4);
  l.cuts = l.lse + up((size_t)2 * ctas * tile_rows * 4);
  l.bytes = l.cuts + up((size_t)ctas * sizeof(Cut));
  return l;
}

template <int CACHE, int D, int NT>
int launch(const Params& p, int ctas, cudaStream_t s) {
  using C = Conf<CACHE, D, NT>;
  constexpr int bytes = C::SMEM + C::QSMEM;
  static std::atomic<uint64_t> ready{0};   // devices whose attribute is set
  int dev = 0;
  int err = cudaGetDevice(&dev);
  if (err) return err;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    err = cudaFuncSetAttribute(decode_kernel<CACHE, D, NT>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               bytes);
    if (err) return err;
    ready.fetch_or(bit);
  }
  decode_kernel<CACHE, D, NT><<<ctas, THREADS, bytes, s>>>(p);
  return cudaGetLastError();
}
template <int CACHE, int D>
int launch_rows(const Params& p, int tile_rows, int ctas, cudaStream_t s) {
  return tile_rows == 8    ? launch<CACHE, D, 1>(p, ctas, s)
         : tile_rows == 16 ? launch<CACHE, D, 2>(p, ctas, s)
                           : launch<CACHE, D, 4>(p, ctas, s);
}
template <int CACHE>
int launch_d(const Params& p, int tile_rows, int ctas, cudaStream_t s) {
  return p.c.d == 128 ? launch_rows<CACHE, 128>(p, tile_rows, ctas, s)
                      : launch_rows<CACHE, 64>(p, tile_rows, ctas, s);
}

}  // namespace

size_t attn_decode_ws_bytes(const tp_kv_cache& c, int64_t rows, int n_q) {
  const int64_t unit = rows / c.b * (n_q / c.n_kv);
  return layout_of(CTAS * device_sm_count(), tile_rows_of(unit), c.d).bytes;
}

int attn_decode(const tp_kv_cache& c, int dtype, const DecodeArgs& a,
                unsigned* status, void* stream) {
  Params p;
  p.c = c;
  p.a = a;
  p.a.bf16 = dtype == TP_BF16;
  p.per_seq = (int)(a.rows / c.b);
  p.group = a.n_q / c.n_kv;
  const int64_t unit = (int64_t)p.per_seq * p.group;
  const int tile_rows = tile_rows_of(unit);
  p.tiles = (int)((unit + tile_rows - 1) / tile_rows);
  p.status = status;
  const int ctas = CTAS * device_sm_count();
  const Layout l = layout_of(ctas, tile_rows, c.d);
  char* ws = static_cast<char*>(a.ws);
  p.part_o = reinterpret_cast<float*>(ws + l.o);
  p.part_lse = reinterpret_cast<float*>(ws + l.lse);
  p.cuts = reinterpret_cast<Cut*>(ws + l.cuts);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the lengths, and with them the work, are known on the device alone
  ProfScope prof(stream, KF_ATTN_DECODE, 0.0, 0.0);
  count_launch(2);
  const int err = c.dtype == TP_BF16  ? launch_d<TP_BF16>(p, tile_rows, ctas, s)
                  : c.dtype == TP_F16 ? launch_d<TP_F16>(p, tile_rows, ctas, s)
                                      : launch_d<TP_FP8>(p, tile_rows, ctas, s);
  if (err) return err;
  const dim3 grid(ctas, (unsigned)(unit < tile_rows ? unit : tile_rows));
  if (c.d == 128)
    join_kernel<128><<<grid, JOIN_THREADS, 0, s>>>(p, tile_rows);
  else
    join_kernel<64><<<grid, JOIN_THREADS, 0, s>>>(p, tile_rows);
  return cudaGetLastError();
}

}  // namespace tp
