// attn_decode.cu — attention of the newest tokens over a paged key-value cache.
//
//   x_t = scale·q·k_t,  o = Σ_t e^(x_t)·v_t / Σ_t e^(x_t)
//
// The cost is one read of the cached K and V, so every byte of them is read
// once for all query rows of a kv head (a unit: up to 32 rows, 8·NT), and what
// the SMs read is shared out evenly whatever the sequences' lengths: all units'
// blocks of 64 or 128 tokens, laid end to end with a fixed extra for each unit,
// are cut into as many equal pieces as there are CTAs, two an SM.  A CTA walks
// its piece segment by segment (a segment: the part of one unit in it).  A unit
// that lies in one CTA is finished there; one that is cut leaves partial
// results (o normalised, M and the sum l relative to it) in the workspace, at
// most two a CTA, which a second kernel joins in CTA order:
//   L = max M_c, o = Σ l_c·2^(M_c − L)·o_c / Σ l_c·2^(M_c − L).
//
// In a CTA each of four warps takes every fourth step of 16 tokens (32 where
// their rows are 128 bytes or less) and runs an online softmax of its own, so
// that nothing waits on another warp before the segment's end.  Its K and V
// rows come by asynchronous 16-byte copies into a ring of the warp's own, the
// next segment's behind this one's.  Both products are mma.sync m16n8k16 with
// the cache on the 16 side: Sᵀ = K·Qᵀ (16 tokens × 8 rows) and Oᵀ += Vᵀ·Pᵀ (16
// elements × 8 rows), K by ldmatrix, Vᵀ by its transposing form; between them P
// is transposed in registers (movmatrix).  At eight rows that takes 14 to 16 %
// of the tensor pipe; the tensor cores' 128-row instructions cost the same for
// one row as for 128 and read shared memory, where codes would have to be
// written again as fp16.  E4M3 codes become fp16 operands in registers here.
//
// Measured (GB300, copy 6.8 TB/s): 32 sequences of 32768 in bf16 630 µs = 1.0
// of a copy, in E4M3 335 to 348 = 0.97 to 0.93; one of 131072 in bf16 89 µs
// (0.88: 4 µs until the first copies are in flight, 4 for the join and its
// launch); 64 of 61 to 8192 in E4M3 44.5 µs (0.68: the start, 512 segments' ends,
// latencies between a step's dependent instructions); with 32 rows over codes
// 364 µs for 1.6 GB (0.65: those latencies alone, eight warps an SM at 250
// registers a thread), over bf16 475 for 3.1 GB (0.96).
//
// Precision: scores, maxima, sums and o are fp32.  Over fp16 values and E4M3
// codes the operands are fp16, q divided by a power of two that brings its
// largest element to [1, 2) (exact but for elements below 2^-14 of it).  P is
// rounded to fp16 in front of the product with V: by 2^-11 of a weight, of those
// below 2^-25 of the largest by 2^-36 of that one (weights lie between 2^11 and
// 2^15 at a row's maximum); the denominator adds up the weights in fp32, in front
// of that rounding.  Over bf16 values, where bf16 (2^-8) would show in the
// output, P is the sum of two bf16 parts, 2^-16, at the price of a second
// product.  A code's scale is multiplied into its score, and into its weight in
// front of the product with V: t = x + log₂ s_v, w = 2^(t − M) with M near the
// running maximum of t (BELOW), so that scales of any size keep the weights of
// the sum in fp16's range; the denominator is Σ w / s_v, relative to the same M
// (fp32's range leaves s_v a factor of 2^100 from token to token; for vectors
// without a value see SMALLEST).  Like x itself t is rounded to 2^-24 of its
// size, so that scales count while |x| is below 2^20.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "gemm.h"
#include "kv_cache.cuh"
#include "kv_cache.h"
#include "profile.h"

namespace tp {
namespace {

constexpr int CTAS = 2;   // on an SM
// M of a row that has seen nothing: below every t and finite, so that nothing
// needs a case of its own (2^(−∞ − M) = 0, 2^(M − t) = 0).
constexpr float NOTHING = -3e38f;
// Over codes a vector without a value counts in the denominator alone: one whose
// scale is below SMALLEST (the cache's writer makes none as small), or of zeros,
// to which the writer gives the scale 1.  What stands for its scale is far below
// others', so that M is not its and small values keep their weights' bits.
constexpr float SMALLEST = 1.5407439555097887e-33f;   // 2^-109
constexpr float NO_VALUE = 8.271806125530277e-25f;    // 2^-80
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
  float2* part_l;        // [2·CTAs][8·NT]: M and l
  Cut* cuts;             // [CTAs]
  unsigned* status;
  // the cache's strides (elements; a product of two is formed in 64 bits)
  int page, pages, page_s, token_s, head_s, s_page_s, s_token_s, s_head_s;
  int units;                 // of a sequence
  int cap;                   // tokens that a row of the table can list (≤ 2^30)
  int skip_cols, skip_off;   // a block's tokens in pages and the rest
  int whole;                 // no unit is cut: each is one slot
  // ⌊n / page⌋ = n·page_mul >> page_shift for n ≤ 2^30: page_mul =
  // ⌈2^page_shift / page⌉ is off by less than page·2^-page_shift of itself,
  // and page_shift = 30 + ⌈log₂ page⌉
  uint32_t page_mul;
  int page_shift;
  __device__ __forceinline__ int col_of(int n) const {
    return (int)((uint64_t)(uint32_t)n * page_mul >> page_shift);
  }
};
__device__ __forceinline__ int64_t mul(int a, int b) { return (int64_t)a * b; }

template <int CACHE, int D, int NT>
struct Conf {
  static constexpr int SIZE = CACHE == TP_FP8 ? 1 : 2;
  static constexpr int ROW = D * SIZE;             // bytes
  static constexpr int ROWS = 8 * NT;
  // The reference M is set to 2^BELOW below a row's largest t, and the sums are
  // rescaled when a t comes to lie more than 2^SLACK further above it: some row
  // of 32 has a new maximum in nearly every step of a short segment, one beyond
  // 2^4 seldom (16x65536 with 32 rows: over codes 401 µs without slack, 368 with
  // 2^4; over bf16 513, 477 and with 2^8 475).  fp16 weights are
  // as large as they may be, 2^15 where fp16 ends at 2^16, so that small ones
  // keep their bits; bf16 has as many exponents as fp32.
  static constexpr float BELOW = CACHE == TP_BF16 ? 0.0f : 11.0f;
  static constexpr float SLACK = CACHE == TP_BF16 ? 8.0f : 4.0f;
  // Sums over codes are kept 2^-RAISE of their size, Σ w·2^-RAISE / s_v: w is up
  // to 2^15 and s_v from 2^-109 to 2^119, between which 2^20 tokens' sum stays
  // in fp32's range at the one end, and 2^-18 of a w / s_v at the other.
  static constexpr float RAISE = CACHE == TP_FP8 ? 12.0f : 0.0f;
  static constexpr float LOWER = CACHE == TP_FP8 ? 0x1p-12f : 1.0f;   // 2^-RAISE
  static constexpr int WARPS = 4;
  static constexpr int THREADS = 32 * WARPS;
  // tokens of a warp: that are loaded, and that are worked on at a time
  static constexpr int STEP = ROW == 256 ? 16 : 32;
  static constexpr int PART = ROW == 256 || NT == 4 ? 16 : 32;
  static constexpr int BLOCK = STEP * WARPS;       // of a CTA
  // A segment's fixed cost in blocks of work (64x8192 in E4M3: 55, 49, 45 and
  // 51 µs with 128, 256, 512 and 1024 tokens, in fp16 with heads of 64 48.8,
  // 44.2, 39.8 and 42.2, 31x2047 28.2, 27.5, 26.3 and 28.2; 256x1000 in fp16 with
  // heads of 128 21.0, 22.3, 24.9 and 28.3).
  static constexpr int EXTRA = (ROW == 256 ? 128 : 512) / BLOCK;
  static constexpr int TILE = STEP * ROW;
  // K, V and the scales of a step
  static constexpr int STAGE = 2 * TILE + (CACHE == TP_FP8 ? 8 * STEP : 0);
  static constexpr int STAGES = STEP * ROW >= 4096 ? 3 : 5;
  static constexpr int RING = STAGES * STAGE;
  static constexpr bool QREG = NT < 4;             // Q in registers
  static constexpr int JOIN = (WARPS / 2) * 8 * (D + 4) * 4;
  static constexpr int QSMEM = QREG ? 0 : ROWS * D * 2;
  static constexpr int ALIGN = 256;
  static constexpr int SMEM =
      WARPS * RING + (JOIN > QSMEM ? JOIN : QSMEM) + ALIGN;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src)
               : "memory");
}
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
// Four E4M3 codes as two pairs of fp16.
__device__ __forceinline__ void codes_f16(uint32_t u, uint32_t& lo,
                                          uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(u));
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte offset of 16-byte chunk ch of row r in a tile, spread so that eight
// rows' same chunk lie in different banks.  Rows lie on multiples of their
// size, so chunk ch ^ x lies at that of ch with 16·x flipped in.
template <int ROW>
__device__ __forceinline__ uint32_t spread(int r, int ch) {
  return ROW >= 128 ? r * ROW + ((ch ^ (r & 7)) << 4)
                    : r * ROW + ((ch ^ ((r >> 1) & 3)) << 4);
}

// A sequence's tokens that are followed.
__device__ __forceinline__ int tokens_of(const Params& p, int seq) {
  return min(max(p.c.lens[seq], 0), p.cap);
}
// The blocks they take (at least one, so that a sequence without any has its
// rows written too).
template <int BLOCK>
__device__ __forceinline__ int blocks_of(int n) {
  return n <= BLOCK ? 1 : (n - 1) / BLOCK + 1;
}
// `total` slots cut into `ctas` pieces of which the first `more` have one slot
// more than the others (`share`).
struct Pieces {
  int total, ctas, share, more;
  __device__ __forceinline__ int begin(int cta) const {
    return cta * share + min(cta, more);
  }
  __device__ __forceinline__ int cta_of(int slot) const {
    const int edge = more * (share + 1);
    return slot < edge ? slot / (share + 1) : more + (slot - edge) / share;
  }
};

// A finite output that fp16 does not hold: recorded, unless it is beyond fp16's
// end by what the weights' rounding to fp16 adds to a mean of such values (2^-11)
// and the sums' to that.
__device__ __noinline__ float4 to_f16_range(float4 v, unsigned* status) {
  auto held = [&](float x) {
    if (!(fabsf(x) > kF16Max) || isinf(x)) return x;
    if (fabsf(x) < kF16Max * (1.0f + 0x1p-10f)) return copysignf(kF16Max, x);
    record_error(status, kDevRange, 45);
    return x;
  };
  return make_float4(held(v.x), held(v.y), held(v.z), held(v.w));
}
// Elements e … e + 3 of a row's head.  F16: the output may be fp16 (over bf16
// values it is not; the question alone takes 2 % with 32 rows).
template <bool F16>
__device__ __forceinline__ void store4(const Params& p, int64_t row, int head,
                                       int e, float4 v) {
  const DecodeArgs& a = p.a;
  uint16_t* dst = static_cast<uint16_t*>(a.out) + row * a.o_row +
                  head * a.o_head + e;
  if (F16 && !a.bf16 &&
      fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))) >
          kF16Max)
    v = to_f16_range(v, p.status);
  *reinterpret_cast<uint2*>(dst) =
      F16 && !a.bf16
          ? make_uint2(pack_f16x2(v.x, v.y), pack_f16x2(v.z, v.w))
          : make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

// The pages of a warp's next tokens: lane l holds entries base + l and
// base + 32 + l of a table row, the second ones read ahead.
struct Pages {
  int base, end, cur, next;   // entries from `end` on are not read
  __device__ __forceinline__ int get(const int32_t* row, int col) const {
    return col < end ? row[col] : -1;
  }
  __device__ __forceinline__ void start(const int32_t* row, int first,
                                        int last, int lane) {
    base = first;
    end = last;
    cur = get(row, base + lane);
    next = get(row, base + 32 + lane);
  }
  __device__ __forceinline__ void move_to(const int32_t* row, int col,
                                          int lane) {
    while (col >= base + 32) {
      base += 32;
      cur = next;
      next = get(row, base + 32 + lane);
    }
  }
  __device__ __forceinline__ int at(int col) const {   // base ≤ col < base + 64
    const int a = __shfl_sync(0xffffffffu, cur, col - base);
    const int b = __shfl_sync(0xffffffffu, next, col - base);
    return col - base < 32 ? a : b;
  }
};

// A segment: blocks [blk0, blk1) of a unit.  Units take nb + EXTRA slots of
// the CTAs' pieces, so that many short ones weigh what they cost; the blocks
// lie behind the extra ones.
struct Segment {
  int seq, kvh, tile;
  int len, n;            // the sequence's tokens, those that are followed
  int nb, blk0, blk1;
  int first;             // slot of the unit's first block
  int there;             // 0: the piece ended before
};

// Walks a CTA's piece, slots [at, stop) of all.
struct Walk {
  int at, stop, before, seq;   // before: slots in front of the sequence
};
// The next segment with blocks of the piece (one thread).  Whatever the lengths
// are (they are read again here, and may have been changed under the call), it
// names a sequence of the batch, a kv head and tokens that its table lists.
template <class C>
__device__ __forceinline__ void next_segment(const Params& p, Walk* walk,
                                             Segment* out) {
  Walk w = *walk;
  Segment s = {};
#pragma unroll 1
  while (w.at < w.stop && w.seq < p.c.b && !s.there) {
    s.len = max(p.c.lens[w.seq], 0);
    s.n = tokens_of(p, w.seq);
    s.nb = blocks_of<C::BLOCK>(s.n);
    s.seq = w.seq;
    const int extra = p.whole ? 0 : C::EXTRA;
    const int weight = p.whole ? 1 : s.nb + extra;
    const int in_seq = w.at - w.before;
    const int unit = min(max(in_seq, 0) / weight, p.units - 1);
    const int x0 = min(max(in_seq - unit * weight, 0), weight - 1);
    const int x1 = min(weight, x0 + (w.stop - w.at));
    s.kvh = p.tiles == 1 ? unit : unit / p.tiles;
    s.tile = unit - s.kvh * p.tiles;
    s.first = w.before + unit * weight + extra;
    s.blk0 = max(0, x0 - extra);
    s.blk1 = p.whole ? s.nb : max(0, x1 - extra);
    s.there = s.blk1 > s.blk0;
    w.at += x1 - x0;
    if (unit == p.units - 1 && x1 == weight) {
      w.before += weight * p.units;
      ++w.seq;
    }
  }
  *walk = w;
  *out = s;
}

template <int CACHE, int D, int NT>
__global__ void __launch_bounds__(Conf<CACHE, D, NT>::THREADS, CTAS)
    decode_kernel(const Params p) {
  using C = Conf<CACHE, D, NT>;
  constexpr bool FP8 = CACHE == TP_FP8, BF = CACHE == TP_BF16;
  constexpr int WARPS = C::WARPS, THREADS = C::THREADS, STAGES = C::STAGES;
  constexpr int STEP = C::STEP, BLOCK = C::BLOCK;
  constexpr int PART = C::PART, MT = PART / 16;
  constexpr int KS = D / 16;          // steps of 16 elements
  constexpr int ROW = C::ROW, CHUNKS = ROW / 16;
  extern __shared__ unsigned char smem_raw[];
  __shared__ Walk s_walk;
  __shared__ Segment segs[3];   // the one computed, the next, the one after it
  __shared__ uint32_t valid_of[WARPS][STAGES];
  __shared__ float s_qf[C::ROWS];
  __shared__ float s_top[WARPS][C::ROWS], s_l[WARPS][C::ROWS];
  __shared__ float s_ref[C::ROWS], s_out[C::ROWS];
  const tp_kv_cache& c = p.c;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t4 = lane & 3;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- this CTA's piece of all slots, and the sequence in which it begins
  // (each warp for itself: lane l has sequences [l·span, (l + 1)·span))
  Pieces pieces;
  {
    const int span = (c.b + 31) / 32;
    const int i0 = lane * span, i1 = min(i0 + span, c.b);
    auto slots = [&](int i) {
      return p.whole
                 ? p.units
                 : (blocks_of<BLOCK>(tokens_of(p, i)) + C::EXTRA) * p.units;
    };
    int sum = 0;
#pragma unroll 4
    for (int i = i0; i < i1; ++i) sum += slots(i);
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += v;
    }
    pieces.total = __shfl_sync(0xffffffffu, inc, 31);
    pieces.ctas = min(pieces.total, (int)gridDim.x);
    pieces.share = pieces.total / pieces.ctas;
    pieces.more = pieces.total - pieces.share * pieces.ctas;
    const int cta = blockIdx.x;
    if (tid == 0) p.cuts[cta].tile = -1;
    // (read if this warp leaves and, lengths having changed, others do not)
    if (tid == 32) segs[0].there = segs[1].there = segs[2].there = 0;
    if (cta >= pieces.ctas) return;
    const int at = pieces.begin(cta);
    int before = inc - sum;
    if (warp == 1 && before <= at && at < inc) {   // one lane
      int i = i0;
#pragma unroll 1
      for (; i + 1 < i1; ++i) {
        const int w = slots(i);
        if (at < before + w) break;
        before += w;
      }
      s_walk = Walk{at, pieces.begin(cta + 1), before, i};
    }
    __syncwarp();
  }

  const float scale = p.a.scale * LOG2E;
  const char* const kpool = static_cast<const char*>(c.k);
  const int64_t to_v = static_cast<const char*>(c.v) - kpool;
  const bool whole_pages = p.page % STEP == 0;
  unsigned char* const smem =
      smem_raw + (-smem_u32(smem_raw) & (C::ALIGN - 1));
  float* const join = reinterpret_cast<float*>(smem + WARPS * C::RING);
  unsigned char* const ring = smem + warp * C::RING;
  constexpr int LANES = CHUNKS, PER = 32 / LANES;   // of a row, rows a copy
  const int sub = lane / LANES, ch = lane % LANES;
  const int64_t copy_bytes = mul(PER, p.token_s) * C::SIZE;

  // ---- loads: the warp's steps of a segment, and of the one after it
  struct Load {
    int left;              // steps that are still to be issued
    int t0, col, off;      // the next one's first token and its place
  };
  Load now = {}, then;
  Pages pages, pages2;     // of `now` and of `then`
  int cur = 1, next = 2, find = 0;   // places in segs: turns below
  int loads = 2;           // that of `now`
  bool moved = true;       // `now` is the segment after the computed one
  auto row_of = [&](const Segment& s) {
    return c.table + (int64_t)s.seq * c.table_stride;
  };
  int issued = 0, slot = 0;   // steps, and the ring's place of the next one
  auto issue = [&]() {
    const Segment& sg = segs[loads];
    pages.move_to(row_of(sg), now.col, lane);
    const int kvh = sg.kvh;
    const int rest = sg.n - now.t0;   // ≥ 1
    const int tok = lane % STEP;
    constexpr uint32_t ALL = 0xffffffffu >> (32 - STEP);
    const uint32_t dst = smem_u32(ring) + slot * C::STAGE;
    // the page and the offset of the lane's token
    bool in = tok < rest;
    int off = now.off + tok, ahead = 0;
    if (!whole_pages && in) ahead = p.col_of(off);
    off -= ahead * p.page;
    const int page = pages.at(now.col + ahead);
    if (in && (page < 0 || page >= p.pages)) {
      in = false;
      record_error(p.status, kDevPage, 44);
    }
    const uint32_t valid = __ballot_sync(0xffffffffu, in) & ALL;
    if constexpr (FP8) {
      static_assert(STEP == 32, "a lane for each token's scales");
      const int64_t at = in ? mul(page, p.s_page_s) + mul(off, p.s_token_s) +
                                  mul(kvh, p.s_head_s)
                            : 0;
      float* d = reinterpret_cast<float*>(ring + slot * C::STAGE + 2 * C::TILE);
      cp_async4(d + lane, c.ks + at, in);
      cp_async4(d + STEP + lane, c.vs + at, in);
    }
    if (whole_pages && valid == ALL) {   // one page
      const char* src = kpool +
                        (mul(page, p.page_s) + mul(now.off + sub, p.token_s) +
                         mul(kvh, p.head_s)) *
                            C::SIZE +
                        16 * ch;
#pragma unroll
      for (int k = 0; k < STEP / PER; ++k) {
        const uint32_t d = dst + spread<ROW>(k * PER + sub, ch);
        cp_async16(d, src);
        cp_async16(d + C::TILE, src + to_v);
        src += copy_bytes;
      }
    } else {
      const int64_t place = in ? (mul(page, p.page_s) + mul(off, p.token_s) +
                                  mul(kvh, p.head_s)) *
                                     C::SIZE
                               : 0;
#pragma unroll 4
      for (int k = 0; k < STEP / PER; ++k) {
        const int r = k * PER + sub;
        const char* src = kpool + __shfl_sync(0xffffffffu, place, r) + 16 * ch;
        const uint32_t d = dst + spread<ROW>(r, ch);
        cp_async16(d, src, (valid >> r) & 1);
        cp_async16(d + C::TILE, src + to_v, (valid >> r) & 1);
      }
    }
    cp_async_commit();
    if (lane == 0) valid_of[warp][slot] = valid;
    if (++slot == STAGES) slot = 0;
    ++issued;
    --now.left;
    now.t0 += BLOCK;
    now.col += p.skip_cols;
    now.off += p.skip_off;
    if (now.off >= p.page) {
      now.off -= p.page;
      ++now.col;
    }
  };

  int done = 0, stage = 0;   // steps that are computed, the next one's place
  // Issues what there is until the ring is full; the slot of the step before
  // `done` is free.
  auto fill = [&]() {
#pragma unroll 1
    while (issued < done + STAGES) {
      if (now.left == 0) {
        if (moved || then.left == 0) break;   // one segment ahead, no further
        now = then;
        pages = pages2;
        loads = next;
        moved = true;
      }
      issue();
    }
  };

  // Turn k computes segment k; meanwhile the warps load on into segment k + 1
  // and one thread looks for segment k + 2.  Turns −2 and −1 have none yet.
  bool first_segment = true;
#pragma unroll 1
  for (int turn = -2;; turn = turn < 0 ? turn + 1 : 0) {
    if (tid == 32) next_segment<C>(p, &s_walk, &segs[find]);
    if (turn >= -1) {
      if (!moved) {
        now = then;
        pages = pages2;
        loads = cur;
      }
      moved = false;
      const Segment& s = segs[next];
      then = {};
      if (s.there) {
        then.t0 = s.blk0 * BLOCK + warp * STEP;
        const int end = min(s.n, s.blk1 * BLOCK) - 1;   // the last token
        if (then.t0 <= end) {
          then.left = (end - then.t0) / BLOCK + 1;
          then.col = p.col_of(then.t0);
          then.off = then.t0 - then.col * p.page;
          pages2.start(row_of(s), then.col, p.col_of(end) + 1, lane);
        }
      }
    }

    const Segment& seg = segs[cur];   // not read in the first two turns
    const int row0 = seg.tile * C::ROWS, rows = p.per_seq * p.group;
    const int len = seg.len, n = seg.n;
    const int64_t qrow = (int64_t)seg.seq * p.per_seq;
    const int last = turn < 0 ? 0 : min(n, seg.blk1 * BLOCK);
    // ---- Q: lane (g, t) holds elements of row 8·nt + g as the products take
    // them (over codes, four neighbours of a step instead of two and two)
    uint32_t q[C::QREG ? NT : 1][KS][2];
    float qf[C::QREG ? NT : 1][2];   // scale of rows 8·nt + 2·t4 (+ 1)
    float o[KS][NT][4];
    float top[NT][2], l[NT][2];   // running maxima of t, sums
    // tokens that row 8·nt + 2·t4 + h sees
    auto seen = [&](int nt, int h) {
      const int rr = row0 + 8 * nt + 2 * t4 + h;
      return rr < rows ? min(n, len - p.per_seq + 1 + rr / p.group) : n;
    };

    // ---- the warp's steps: 16·MT tokens from BLOCK·blk + STEP·warp on
    bool fresh = turn >= 0;
#pragma unroll 1
    for (int t0 = turn < 0 ? 0 : seg.blk0 * BLOCK + warp * STEP;;
         t0 += BLOCK) {
      if (turn >= -1) fill();
      if (fresh) {
        fresh = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int r = row0 + 8 * nt + g;
          const bool there = r < rows;
          const int j = there ? r / p.group : 0;
          const uint16_t* src =
              static_cast<const uint16_t*>(p.a.q) + (qrow + j) * p.a.q_row +
              (there ? (seg.kvh * p.group + r - j * p.group) * p.a.q_head : 0);
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
            auto pair = [&](uint32_t x) {
              return p.a.bf16 ? unpack_bf16x2(x) : unpack_f16x2(x);
            };
#pragma unroll
            for (int s = 0; s < KS; ++s)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float2 x = pair(u[s][h]);
                amax = fmaxf(amax, fmaxf(fabsf(x.x), fabsf(x.y)));
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
              for (int h = 0; h < 2; ++h) {
                const float2 x = pair(u[s][h]);
                u[s][h] = pack_f16x2(x.x * down, x.y * down);
              }
          }
          f *= scale;
          if constexpr (C::QREG) {
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              q[nt][s][0] = u[s][0];
              q[nt][s][1] = u[s][1];
            }
            qf[nt][0] = __shfl_sync(0xffffffffu, f, 8 * t4);
            qf[nt][1] = __shfl_sync(0xffffffffu, f, 8 * t4 + 4);
          } else if (nt % WARPS == warp) {   // [nt][s / 2][lane] four registers
            if (t4 == 0) s_qf[8 * nt + g] = f;
#pragma unroll
            for (int s = 0; s < KS; ++s)
              reinterpret_cast<uint2*>(
                  join)[((nt * KS + s) / 2 * 32 + lane) * 2 + s % 2] =
                  make_uint2(u[s][0], u[s][1]);
          }
        }
        if constexpr (!C::QREG) __syncthreads();

#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int s = 0; s < KS; ++s)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[s][nt][j] = 0.0f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            top[nt][h] = NOTHING;
            l[nt][h] = 0.0f;
          }
        }
      }
      if (t0 >= last) break;
      // this step's copies are done when those issued after it may not be
      switch (issued - done - 1) {
        case 0: cp_async_wait<0>(); break;
        case 1: cp_async_wait<1>(); break;
        case 2: cp_async_wait<2>(); break;
        case 3: cp_async_wait<3>(); break;
        default: cp_async_wait<4>();
      }
      static_assert(STAGES <= 5, "waits for the ring's steps");
      __syncwarp();
      const uint32_t valid_all = valid_of[warp][stage];
      // Over codes, a token a lane: makes the step's vectors without a value ones
      // of zeros with the scale NO_VALUE, and those whose scale is NaN or negative
      // ones of NaN (the scale itself would reach rows that do not see it through
      // the sums); whether there are any.
      auto mend_scales = [&]() {
        unsigned char* const v = ring + stage * C::STAGE + C::TILE;
        float* const sv = reinterpret_cast<float*>(v + C::TILE) + STEP + lane;
        auto codes = [&](int ch) -> uint4& {
          return *reinterpret_cast<uint4*>(v + spread<ROW>(lane, ch));
        };
        bool none = fabsf(*sv) < SMALLEST;   // (0: nothing was loaded)
        const bool bad = !none && !(*sv > 0.0f);
        const bool zeros = *sv == 1.0f && (codes(0).x & 0x7f7f7f7fu) == 0;
        if (!__any_sync(0xffffffffu, none || bad || zeros)) return false;
        if (zeros) {   // the first four are
          uint32_t any = 0;
#pragma unroll 1
          for (int ch = 0; ch < CHUNKS; ++ch) {
            const uint4 u = codes(ch);
            any |= u.x | u.y | u.z | u.w;
          }
          none = (any & 0x7f7f7f7fu) == 0;
        }
        if (none || bad) {
          *sv = none ? NO_VALUE : 1.0f;
          const uint32_t x = none ? 0u : 0x7f7f7f7fu;
#pragma unroll 1
          for (int ch = 0; ch < CHUNKS; ++ch) codes(ch) = make_uint4(x, x, x, x);
        }
        __syncwarp();
        return true;
      };
      // Looked for in front of every step of two parts; else only where the
      // scales, once they are read, give reason to (16x65536 with 4 new 364 and
      // 376 µs, 64x8192 46.1 and 44.3).
      if constexpr (FP8 && PART < STEP) mend_scales();
#pragma unroll 1
      for (int part = 0; part < STEP; part += PART) {
        const int t1 = t0 + part;   // the part's first token
        unsigned char* const rows_at = ring + stage * C::STAGE + part * ROW;
        const uint32_t kt = smem_u32(rows_at), vt = kt + C::TILE;
        constexpr uint32_t FULL = 0xffffffffu >> (32 - PART);
        const uint32_t valid = valid_all >> part & FULL;

        // ---- Sᵀ = K·Qᵀ
        float sc[MT][NT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) sc[mt][nt][j] = 0.0f;
        {
          // rows 0–7 and 8–15 of a chunk of 16 bytes, then of the next: over
          // codes that is all of steps s and s + 1, else of one step
          const uint32_t at = kt + spread<ROW>(lane & 15, lane >> 4);
#pragma unroll
          for (int s = 0; s < KS; s += 2) {
            uint4 b[NT];   // both steps' operands
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              if constexpr (C::QREG)
                b[nt] = make_uint4(q[nt][s][0], q[nt][s][1], q[nt][s + 1][0],
                                   q[nt][s + 1][1]);
              else
                b[nt] = reinterpret_cast<const uint4*>(
                    join)[(nt * KS + s) / 2 * 32 + lane];
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              uint32_t u[4];
              if constexpr (FP8)
                ldmatrix((at ^ (s << 4)) + mt * 16 * ROW, u);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                uint32_t a[4];
                if constexpr (FP8) {
                  codes_f16(u[2 * h], a[0], a[2]);
                  codes_f16(u[2 * h + 1], a[1], a[3]);
                } else {
                  ldmatrix((at ^ ((s + h) << 5)) + mt * 16 * ROW, a);
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma<BF>(sc[mt][nt], a, h ? b[nt].z : b[nt].x,
                          h ? b[nt].w : b[nt].y);
              }
            }
          }
        }

        // ---- softmax of the lane's rows 2·t4, 2·t4 + 1 at tokens 16·mt + g
        // and 16·mt + g + 8: t into sc
        float sk[MT][2], lv[MT][2], back[MT][2];   // s_k, log₂ s_v, 2^-RAISE / s_v
        if constexpr (FP8) {
          const float* ss = reinterpret_cast<const float*>(
                                ring + stage * C::STAGE + 2 * C::TILE) +
                            part;
          bool odd = false;
          auto scales = [&]() {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const float sv = ss[STEP + 16 * mt + g + 8 * h];
                sk[mt][h] = ss[16 * mt + g + 8 * h];
                lv[mt][h] = lg2_approx(sv);
                back[mt][h] = rcp_approx(sv) * C::LOWER;
                odd |= !(sv >= SMALLEST) || sv == 1.0f;
              }
          };
          scales();
          if constexpr (PART == STEP)
            if (__any_sync(0xffffffffu, odd) && mend_scales()) scales();
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float f;
              if constexpr (C::QREG)
                f = qf[nt][j & 1];
              else
                f = s_qf[8 * nt + 2 * t4 + (j & 1)];
              float& x = sc[mt][nt][j];
              x = FP8 ? fmaf(x * sk[mt][j >> 1], f, lv[mt][j >> 1]) : x * f;
            }
        const bool mixed = p.per_seq > 1 && t1 > len - p.per_seq + 1 - PART;
        if (valid != FULL || mixed) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int end = seen(nt, h) - t1;
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int k = 16 * mt + g + 8 * i;
                  if (!((valid >> k) & 1) || k >= end)
                    sc[mt][nt][2 * i + h] = -INFINITY;
                }
            }
        }
        float high[NT][2];
        bool rise = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float x = fmaxf(sc[0][nt][h], sc[0][nt][2 + h]);
#pragma unroll
            for (int mt = 1; mt < MT; ++mt)
              x = fmaxf(x, fmaxf(sc[mt][nt][h], sc[mt][nt][2 + h]));
            high[nt][h] = x;
            // (the difference: of far scores M + 15 may be rounded to M + 16)
            rise |= x - top[nt][h] > C::BELOW + C::SLACK;
          }
        if (__any_sync(0xffffffffu, rise)) {   // maxima of all rows anew
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float x = high[nt][h];
#pragma unroll
              for (int z = 4; z < 32; z <<= 1)
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, z));
              x = fmaxf(x - C::BELOW, top[nt][h]);
              const float f = ex2_approx(top[nt][h] - x);
              top[nt][h] = x;
              l[nt][h] *= f;
#pragma unroll
              for (int s = 0; s < KS; ++s) {
                o[s][nt][h] *= f;
                o[s][nt][2 + h] *= f;
              }
            }
        }
        // weights
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float& x = sc[mt][nt][2 * k + h];
                x = ex2_approx(x - top[nt][h]);
                l[nt][h] = FP8 ? fmaf(x, back[mt][k], l[nt][h]) : l[nt][h] + x;
              }
        if (mixed) {
          // Rows of several new tokens see different ends of this step.  What
          // a later token's v holds (NaN, say) must not reach a row that does
          // not see it through a weight of 0: the last tokens' products are
          // added one by one, and their v then cleared.
          const int k1 = min(PART, n - t1);
#pragma unroll 1
          for (int k = max(0, len - p.per_seq + 1 - t1); k < k1; ++k) {
            float w[NT][2];
            uint32_t sees = 0;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (t1 + k < seen(nt, h)) sees |= 1u << (2 * nt + h);
                w[nt][h] = 0.0f;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                  for (int i = 0; i < 2; ++i) {
                    const float x = __shfl_sync(
                        0xffffffffu, sc[mt][nt][2 * i + h], 4 * (k & 7) + t4);
                    if (k >> 3 == 2 * mt + i) w[nt][h] = x;
                  }
              }
            unsigned char* const vrow = rows_at + C::TILE;
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              float2 v;
              if constexpr (FP8) {
                v = pair_to_f32<TP_FP8>(*reinterpret_cast<const uint16_t*>(
                    vrow + spread<ROW>(k, s) + 2 * g));
              } else {
                const uint32_t a = *reinterpret_cast<const uint16_t*>(
                    vrow + spread<ROW>(k, 2 * s) + 2 * g);
                const uint32_t b = *reinterpret_cast<const uint16_t*>(
                    vrow + spread<ROW>(k, 2 * s + 1) + 2 * g);
                v = pair_to_f32<CACHE>(a | b << 16);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                  if (sees >> (2 * nt + h) & 1) {
                    o[s][nt][h] = fmaf(w[nt][h], v.x, o[s][nt][h]);
                    o[s][nt][2 + h] = fmaf(w[nt][h], v.y, o[s][nt][2 + h]);
                  }
            }
            __syncwarp();
            if (lane < CHUNKS)
              *reinterpret_cast<uint4*>(vrow + spread<ROW>(k, lane)) =
                  make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
        uint32_t b[MT][NT][2], b2[MT][NT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float w0 = sc[mt][nt][2 * h], w1 = sc[mt][nt][2 * h + 1];
              if (BF) {
                const uint32_t x = pack_bf16x2(w0, w1);
                const float2 f = unpack_bf16x2(x);
                b[mt][nt][h] = movmatrix(x);
                b2[mt][nt][h] = movmatrix(pack_bf16x2(w0 - f.x, w1 - f.y));
              } else {
                b[mt][nt][h] = movmatrix(pack_f16x2(w0, w1));
              }
            }

        // ---- Oᵀ += Vᵀ·Pᵀ
        auto add_values = [&](const uint32_t(&a)[4], int s, int mt) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma<BF>(o[s][nt], a, b[mt][nt][0], b[mt][nt][1]);
            if (BF) mma<BF>(o[s][nt], a, b2[mt][nt][0], b2[mt][nt][1]);
          }
        };
        if constexpr (FP8) {
          const uint32_t at = vt + spread<ROW>(lane & 15, lane >> 4);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int s = 0; s < KS; s += 2) {
              uint32_t u[4];
              ldmatrix_trans((at ^ (s << 4)) + mt * 16 * ROW, u);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                // elements 2g, 2g + 1 of tokens 2t, 2t + 1 to pairs of tokens
                uint32_t a[4];
                codes_f16(__byte_perm(u[2 * h], 0, 0x3120), a[0], a[1]);
                codes_f16(__byte_perm(u[2 * h + 1], 0, 0x3120), a[2], a[3]);
                add_values(a, s + h, mt);
              }
            }
        } else {
          const uint32_t at =
              vt + spread<ROW>((lane & 7) + ((lane >> 1) & 8), (lane >> 3) & 1);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int s = 0; s < KS; ++s) {
              uint32_t a[4];
              ldmatrix_trans((at ^ (s << 5)) + mt * 16 * ROW, a);
              add_values(a, s, mt);
            }
        }
      }
      if (++stage == STAGES) stage = 0;
      ++done;
      __syncwarp();   // its place in the ring is free
    }
    const int old = cur;
    cur = next;
    next = find;
    find = old;
    if (turn < 0) {
      __syncthreads();   // the segment that was found
      if (turn == -1 && !segs[cur].there) return;
      continue;
    }

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
          s_top[warp][r] = top[nt][h];
          s_l[warp][r] = l[nt][h];
        }
      }
    const bool part = seg.blk0 > 0 || seg.blk1 < seg.nb;
    const int64_t part_at = 2 * (int64_t)blockIdx.x + !first_segment;
    __syncthreads();   // and Q is read
    if (tid < C::ROWS) {
      const int r = tid;
      float all = s_top[0][r], sum = 0.0f;
#pragma unroll
      for (int w = 1; w < WARPS; ++w) all = fmaxf(all, s_top[w][r]);
#pragma unroll
      for (int w = 0; w < WARPS; ++w)
        sum = fmaf(s_l[w][r], ex2_approx(s_top[w][r] - all), sum);
      const bool none = sum == 0.0f;
      s_ref[r] = all;
      s_out[r] = none ? 0.0f : 1.0f / sum;
      const int rr = row0 + r, j = rr / p.group;
      if (rr >= rows) {
      } else if (part) {
        p.part_l[part_at * C::ROWS + r] = make_float2(all + C::RAISE, sum);
      } else if (p.a.lse != nullptr) {
        p.a.lse[(qrow + j) * p.a.n_q + seg.kvh * p.group + rr -
                j * p.group] =
            none ? -INFINITY : (all + C::RAISE + log2f(sum)) * LN2;
      }
    }
    if (tid == THREADS - 1) {
      if (len > n) record_error(p.status, kDevPage, 43);
      if (seg.blk0 == 0 && seg.blk1 < seg.nb) {
        Cut cut;
        cut.seq = seg.seq;
        cut.head = seg.kvh;
        cut.tile = seg.tile;
        cut.first_slot = (int)part_at;
        const int end =
            min(pieces.cta_of(seg.first + seg.nb - 1), pieces.ctas - 1);
        cut.parts = end - (int)blockIdx.x + 1;
        p.cuts[blockIdx.x] = cut;
      }
    }
    __syncthreads();
    // Half of the warps take the other half's in, eight rows at a time, then
    // all threads add what is left.
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float f[2];
#pragma unroll
      for (int h = 0; h < 2; ++h)
        f[h] = ex2_approx(top[nt][h] - s_ref[8 * nt + 2 * t4 + h] - C::RAISE);
      float* const mine =
          join + ((warp % (WARPS / 2)) * 8 + 2 * t4) * (D + 4) +
          (FP8 ? 2 * g : g);
      constexpr int PAIR = FP8 ? 1 : 8;
      if (warp >= WARPS / 2) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            mine[h * (D + 4) + 16 * s] = o[s][nt][h] * f[h];
            mine[h * (D + 4) + 16 * s + PAIR] = o[s][nt][2 + h] * f[h];
          }
      }
      __syncthreads();
      if (warp < WARPS / 2) {
#pragma unroll
        for (int s = 0; s < KS; ++s)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float* const d = mine + h * (D + 4) + 16 * s;
            d[0] = fmaf(o[s][nt][h], f[h], d[0]);
            d[PAIR] = fmaf(o[s][nt][2 + h], f[h], d[PAIR]);
          }
      }
      __syncthreads();
      constexpr int QUADS = D / 4;
#pragma unroll 1
      for (int i = tid; i < 8 * QUADS; i += THREADS) {
        const int r8 = i / QUADS, e = 4 * (i - r8 * QUADS);
        const int r = 8 * nt + r8, rr = row0 + r;
        if (rr >= rows) break;
        const float y = s_out[r];
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < WARPS / 2; ++w) {
          const float4 x = *reinterpret_cast<const float4*>(
              join + (w * 8 + r8) * (D + 4) + e);
          v.x += x.x;
          v.y += x.y;
          v.z += x.z;
          v.w += x.w;
        }
        v.x *= y;
        v.y *= y;
        v.z *= y;
        v.w *= y;
        if (part) {
          *reinterpret_cast<float4*>(p.part_o +
                                     (part_at * C::ROWS + r) * D + e) = v;
        } else {
          const int j = rr / p.group;
          store4<!BF>(p, qrow + j, seg.kvh * p.group + rr - j * p.group, e,
                      v);
        }
      }
      __syncthreads();   // the sums, and `seg`, are read
    }
    if (!segs[cur].there) return;
    first_segment = false;
  }
}

// Joins the parts of the units that were cut: CTA (i, j) rows j·cta_rows up to
// (j + 1)·cta_rows of the one that CTA i of the first kernel begins, if there
// is one.  A warp has a row, D/4 lanes of it a part each time; with more than
// FEW parts all eight warps share a row, one after the other.  What bounds it
// is a launch and a chain of two loads, the cut and then its parts (2.7 µs; 4
// with 38 parts a row).
constexpr int JOIN_WARPS = 8;
constexpr int FEW = 8;
template <int D>
__global__ void __launch_bounds__(32 * JOIN_WARPS)
    join_kernel(const Params p, int tile_rows, int cta_rows) {
  constexpr int LANES = D / 4, SIDE = 32 / LANES;   // of a part, parts a load
  constexpr int U = 4;
  __shared__ float s_top[JOIN_WARPS], s_sum[JOIN_WARPS];
  __shared__ float4 s_o[JOIN_WARPS][LANES];
  // launched while the first kernel runs: everything is read after this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Cut cut = p.cuts[blockIdx.x];
  const int r0 = cta_rows * blockIdx.y, warp = threadIdx.x >> 5;
  const int r1 = min(min(tile_rows, r0 + cta_rows),
                     p.per_seq * p.group - cut.tile * tile_rows);
  if (cut.tile < 0 || r0 >= r1) return;
  const int lane = threadIdx.x & 31, e = 4 * (lane % LANES);
  const bool few = cut.parts <= FEW;
  const int stride = SIDE * (few ? 1 : JOIN_WARPS);
  // o and the sum of parts side, side + stride, … of row r, relative to top
  float top = NOTHING, sum = 0.0f;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add_parts = [&](int r) {
    top = NOTHING;
    sum = 0.0f;
    v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i0 = lane / LANES + (few ? 0 : SIDE * warp); i0 < cut.parts;
         i0 += U * stride) {
      float2 x[U];
      float4 u[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = i0 + k * stride;
        x[k] = make_float2(NOTHING, 0.0f);
        u[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (i < cut.parts) {
          const int64_t slot =
              i == 0 ? cut.first_slot : 2 * ((int64_t)blockIdx.x + i);
          const int64_t at = slot * tile_rows + r;
          x[k] = p.part_l[at];
          u[k] = *reinterpret_cast<const float4*>(p.part_o + at * D + e);
        }
      }
      float high = top;
#pragma unroll
      for (int k = 0; k < U; ++k) high = fmaxf(high, x[k].x);
      const float f = ex2_approx(top - high);
      top = high;
      sum *= f;
      v.x *= f;
      v.y *= f;
      v.z *= f;
      v.w *= f;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float w = x[k].y * ex2_approx(x[k].x - high);
        sum += w;
        v.x = fmaf(w, u[k].x, v.x);
        v.y = fmaf(w, u[k].y, v.y);
        v.z = fmaf(w, u[k].z, v.z);
        v.w = fmaf(w, u[k].w, v.w);
      }
    }
  };
  // another set of parts, with its top, sum and v, joins them
  auto merge = [&](float top2, float sum2, float4 v2) {
    const float high = fmaxf(top, top2);
    const float f = ex2_approx(top - high), f2 = ex2_approx(top2 - high);
    top = high;
    sum = sum * f + sum2 * f2;
    v.x = v.x * f + v2.x * f2;
    v.y = v.y * f + v2.y * f2;
    v.z = v.z * f + v2.z * f2;
    v.w = v.w * f + v2.w * f2;
  };
  auto sides = [&]() {   // D = 64: the half-warps' parts
    if constexpr (SIDE == 2) {
      float4 v2;
      const float top2 = __shfl_xor_sync(0xffffffffu, top, 16);
      const float sum2 = __shfl_xor_sync(0xffffffffu, sum, 16);
      v2.x = __shfl_xor_sync(0xffffffffu, v.x, 16);
      v2.y = __shfl_xor_sync(0xffffffffu, v.y, 16);
      v2.z = __shfl_xor_sync(0xffffffffu, v.z, 16);
      v2.w = __shfl_xor_sync(0xffffffffu, v.w, 16);
      merge(top2, sum2, v2);
    }
  };
  auto finish = [&](int r) {
    const bool none = sum == 0.0f;
    const float f = none ? 0.0f : 1.0f / sum;
    const int rr = cut.tile * tile_rows + r, j = rr / p.group;
    const int head = cut.head * p.group + rr - j * p.group;
    const int64_t row = (int64_t)cut.seq * p.per_seq + j;
    v.x *= f;
    v.y *= f;
    v.z *= f;
    v.w *= f;
    if (lane < LANES) store4<true>(p, row, head, e, v);
    if (lane == 0 && p.a.lse != nullptr)
      p.a.lse[row * p.a.n_q + head] =
          none ? -INFINITY : (top + log2f(sum)) * LN2;
  };
  if (few) {
    const int r = r0 + warp;
    if (r >= r1) return;
    add_parts(r);
    sides();
    finish(r);
    return;
  }
  for (int r = r0; r < r1; ++r) {
    add_parts(r);
    sides();
    if (lane < LANES) s_o[warp][lane] = v;
    if (lane == 0) {
      s_top[warp] = top;
      s_sum[warp] = sum;
    }
    __syncthreads();
    if (warp == 0) {
#pragma unroll 1
      for (int w = 1; w < JOIN_WARPS; ++w)
        merge(s_top[w], s_sum[w], s_o[w][lane % LANES]);
      finish(r);
    }
    __syncthreads();
  }
}

// Rows of a unit's tile: as few as hold them, 32 at most.
int tile_rows_of(int64_t rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : 32; }

struct Layout {
  size_t o, l, cuts, bytes;
};
Layout layout_of(int ctas, int tile_rows, int d) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  Layout l;
  l.o = 0;
  l.l = up((size_t)2 * ctas * tile_rows * d * 4);
  l.cuts = l.l + up((size_t)2 * ctas * tile_rows * 8);
  l.bytes = l.cuts + up((size_t)ctas * sizeof(Cut));
  return l;
}

// Where no sequence can have more than a few blocks its units are left whole:
// that spares the join and its launch, at the price of the blocks that idle CTAs
// would have taken.  Measured whole / cut (µs, 8 kv heads, sequences of all the
// blocks they can have; a block is 64 tokens of 256 bytes or 128 shorter ones):
//   8 units of 3 and 4 blocks: bf16 7.0 / 7.2 and 7.8 / 7.4, with 32 rows 16.1 /
//     15.6 and 17.3 / 15.9, E4M3 7.8 / 7.7 and 8.6 / 7.8
//   32 units of 3, 4 and 6: bf16 7.2 / 8.3, 8.0 / 8.8, 10.0 / 9.5
//   64 units of 8 and 12: bf16 11.9 / 12.0 and 14.9 / 13.4, E4M3 13.4 / 13.2 and
//     16.9 / 15.1, with 32 rows 29.0 / 29.7 and 35.5 / 32.8, fp16 heads of 64
//     11.4 / 11.7 and 14.1 / 13.2
//   256 units of 8 and 16: bf16 15.6 / 19.1 and 24.9 / 29.4
// Where lengths differ the border lies lower (64 units of up to 8: E4M3 12.7 /
// 11.6).  Over 8 to 512 units of up to 16 blocks and 8, 16 and 32 rows in all of
// these types the rule costs 1.3 % against the better of both in the mean.
bool left_whole(int64_t units, int blocks) {
  return blocks <= (units < 64 ? 3 : 8);
}

// `sms` SMs' worth of CTAs.
template <int CACHE, int D, int NT>
int launch(Params& p, int sms, cudaStream_t s) {
  using C = Conf<CACHE, D, NT>;
  static std::atomic<uint64_t> ready{0};   // devices whose attribute is set
  int dev = 0;
  int err = cudaGetDevice(&dev);
  if (err) return err;
  const uint64_t bit = 1ull << (dev & 63);
  if (!(ready.load() & bit)) {
    err = cudaFuncSetAttribute(decode_kernel<CACHE, D, NT>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                               C::SMEM);
    if (err) return err;
    ready.fetch_or(bit);
  }
  // no more CTAs than there are slots if every sequence is as long as it can be
  const int64_t units = (int64_t)p.c.b * p.units;
  const int blocks = (p.cap - 1) / C::BLOCK + 1;
  p.whole = left_whole(units, blocks);
  const int ctas = (int)std::min<int64_t>(
      CTAS * sms, p.whole ? units : units * (blocks + C::EXTRA));
  p.skip_cols = C::BLOCK / p.page;
  p.skip_off = C::BLOCK % p.page;
  decode_kernel<CACHE, D, NT><<<ctas, C::THREADS, C::SMEM, s>>>(p);
  count_launch(1);
  err = cudaGetLastError();
  if (err || p.whole) return err;
  const int64_t unit = (int64_t)p.per_seq * p.group;
  cudaLaunchConfig_t cfg = {};
  // With fewer units than CTAs / 4 a unit has more than FEW parts, whose rows
  // go to CTAs of their own (1x131072 with 8 units: 88 µs a call, else 99).
  const int cta_rows = 4 * units < ctas ? 1 : 8;
  const int rows = (int)std::min<int64_t>(unit, 8 * NT);
  cfg.gridDim = dim3(ctas, (rows + cta_rows - 1) / cta_rows);
  cfg.blockDim = dim3(32 * JOIN_WARPS);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  count_launch(1);
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, p, 8 * NT, cta_rows);
}
template <int CACHE, int D>
int launch_rows(Params& p, int tile_rows, int sms, cudaStream_t s) {
  return tile_rows == 8    ? launch<CACHE, D, 1>(p, sms, s)
         : tile_rows == 16 ? launch<CACHE, D, 2>(p, sms, s)
                           : launch<CACHE, D, 4>(p, sms, s);
}
template <int CACHE>
int launch_d(Params& p, int tile_rows, int sms, cudaStream_t s) {
  return p.c.d == 128 ? launch_rows<CACHE, 128>(p, tile_rows, sms, s)
                      : launch_rows<CACHE, 64>(p, tile_rows, sms, s);
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
  p.page = c.page;
  p.units = c.n_kv * p.tiles;
  p.cap = c.table_cols * c.page;
  p.page_shift = 30;
  while (1 << (p.page_shift - 30) < c.page) ++p.page_shift;
  p.page_mul =
      (uint32_t)((((uint64_t)1 << p.page_shift) + c.page - 1) / c.page);
  p.pages = (int)c.pages;
  p.page_s = (int)c.page_stride;
  p.token_s = (int)c.token_stride;
  p.head_s = (int)c.head_stride;
  p.s_page_s = (int)c.s_page_stride;
  p.s_token_s = (int)c.s_token_stride;
  p.s_head_s = (int)c.s_head_stride;
  const int sms = device_sm_count();
  const Layout l = layout_of(CTAS * sms, tile_rows, c.d);
  char* ws = static_cast<char*>(a.ws);
  p.part_o = reinterpret_cast<float*>(ws + l.o);
  p.part_l = reinterpret_cast<float2*>(ws + l.l);
  p.cuts = reinterpret_cast<Cut*>(ws + l.cuts);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the lengths, and with them the work, are known on the device alone
  ProfScope prof(stream, KF_ATTN_DECODE, 0.0, 0.0);
  return c.dtype == TP_BF16  ? launch_d<TP_BF16>(p, tile_rows, sms, s)
         : c.dtype == TP_F16 ? launch_d<TP_F16>(p, tile_rows, sms, s)
                             : launch_d<TP_FP8>(p, tile_rows, sms, s);
}

}  // namespace tp
