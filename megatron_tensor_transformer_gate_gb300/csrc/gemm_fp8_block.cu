// gemm_fp8_block.cu — C[M, N] = Σ_b sa[b]·sb[b]·Σ_{k in block b} qa·qb over
// K blocks of 128, E4M3 codes with fp32 scales, C in bf16 or fp32.
//
// The tensor cores give the plain sum of one K block (four tcgen05.mma
// kind::f8f6f4 of K = 32 into fresh TMEM columns); the epilogue warps read it
// back while the next block runs, multiply it by sa·sb and add it to the
// output tile, which stays in their registers over the whole K loop.  Two
// forms here (up to eight rows of A have a third, gemm_fp8_block_thin.cu):
//  * wide: persistent pairs of CTAs, each with 128×256 of a 256×256 tile and
//    half of its B (cta_group::2), for products that fill the card with such
//    tiles;
//  * narrow: one CTA per 128×BN tile with B's rows (the weight) on the
//    instruction's M side, BN = 16 to 128 rows of A, and K split over a
//    cluster whose CTAs add up their parts through distributed shared memory
//    in rank order: the form for few rows of A, which reads the weight once.
// Neither keeps anything between calls or needs a workspace, and no sum's
// order is left open: it is the form's, which the sizes choose.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>
#include <type_traits>

#include "common.cuh"
#include "fp8_block.h"
#include "gemm.h"
#include "profile.h"

namespace tp {
namespace {

constexpr int BM = 128;             // rows of an operand tile
constexpr int BK = 128;             // a K block: 128 bytes per row
constexpr int TILE_BYTES = BM * BK;

struct Params {
  CUtensorMap ma, mb;
  const float *sa, *sb;
  int64_t ldsa, ldsb;
  int a_row;               // sa: a scale for each row (1) or for 128 rows (0)
  int M, N, kblocks;
  int m_tiles, n_tiles, total_tiles, group_m;
  void* c;
  int64_t ldc;
  int vec;                 // rows of C start on 16 bytes
  unsigned* status;
};

// ==================================================================== wide ==
constexpr int BN = 256;
constexpr int BNH = BN / 2;                    // B rows loaded by each CTA
constexpr int STAGES = 6;                      // even: two threads take turns
constexpr int STAGE_BYTES = 2 * TILE_BYTES;    // 128 rows of A, 128 of B
constexpr int TMEM_COLS = 512;                 // two K blocks × 256
constexpr int WIDE_THREADS = 384;
// Scales of the tile's 128 rows and of its columns (two blocks', or 256) for
// one K block; staged this many blocks deep.
constexpr int SLOT = BM + BN;                  // floats
constexpr int SLOTS = 8;
constexpr int STAGING = 2048;                  // bytes an epilogue warp
constexpr int WIDE_SMEM = STAGES * STAGE_BYTES + SLOTS * SLOT * 4 +
                          8 * STAGING + 1024 + 256;

__device__ __forceinline__ void decode_tile(const Params& p, int t, int& mt,
                                            int& nt) {
  const int gsz = p.group_m * p.n_tiles;
  const int g = t / gsz;
  const int first_m = g * p.group_m;
  const int gm = min(p.group_m, p.m_tiles - first_m);
  const int rr = t - g * gsz;
  mt = first_m + rr % gm;
  nt = rr / gm;
}

// 16 TMEM lanes × 32 columns: the layout of tmem_ld16x256b_x8, four units.
__device__ __forceinline__ void tmem_ld16x256b_x4(uint32_t taddr,
                                                  uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(taddr));
}

// One output tile's part of an epilogue warp: 32 rows × 128 columns.
//
// RowAcc: a scale for each row (sa) times one for the columns.  A thread has
// one row and all 128 columns, so one multiplier serves them all.
struct RowAcc {
  static constexpr int CHUNKS = 4;        // of 32 columns
  static constexpr int SCALES_READ = 0;   // before this chunk all have been
  using Chunk = uint32_t[32];
  uint64_t acc[64];
  float s, sn;   // this block's multiplier, the next one's
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0;
  }
  __device__ __forceinline__ static void load(uint32_t taddr, int c,
                                              Chunk& r) {
    tmem_ld32(taddr + 32 * c, r);
  }
  __device__ __forceinline__ static void wait(Chunk& r) { tmem_ld_wait(r); }
  __device__ __forceinline__ void scales(const float* rows, const float* cols,
                                         int half, int lane) {
    sn = rows[lane] * cols[half];
  }
  __device__ __forceinline__ void next() { s = sn; }
  __device__ __forceinline__ void columns(const float*, int, int) {}
  __device__ __forceinline__ void add(const Chunk& r, int c) {
    const uint64_t s2 = pack_f32x2(__float_as_uint(s), __float_as_uint(s));
#pragma unroll
    for (int i = 0; i < 16; ++i)
      fma_f32x2(acc[c * 16 + i], pack_f32x2(r[2 * i], r[2 * i + 1]), s2);
  }
  // Stores go through 2 KB of shared memory, 64 bytes of each row at a time
  // (16-byte piece k of row r at k ^ (r / 2 mod 4)): a warp's store then
  // writes 64 bytes in each of eight rows instead of 16 in each of 32, or,
  // where rows are not 16-byte aligned or end inside the tile, one row's
  // elements side by side (2000×2500×4096 43 µs; by each thread into its own
  // row 95).
  template <int OUT_F32>
  __device__ __forceinline__ void store(const Params& p, uint4* stage, int m0,
                                        int n0, int lane) const {
    const bool whole = p.vec && n0 + BNH <= p.N;
    constexpr int W = OUT_F32 ? 16 : 32;   // columns in 64 bytes
    constexpr int ES = OUT_F32 ? 4 : 2;
#pragma unroll
    for (int c = 0; c < BNH / W; ++c) {
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (OUT_F32) {
            const float2 x = unpack_f32x2(acc[c * 8 + k * 2 + (j >> 1)]);
            w[j] = __float_as_uint(j & 1 ? x.y : x.x);
          } else {
            const float2 x = unpack_f32x2(acc[c * 16 + k * 4 + j]);
            w[j] = pack_bf16x2(x.x, x.y);
          }
        }
        stage[lane * 4 + (k ^ ((lane >> 1) & 3))] =
            make_uint4(w[0], w[1], w[2], w[3]);
      }
      __syncwarp();
      if (whole) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = i * 8 + (lane >> 2), k = lane & 3;
          if (m0 + r < p.M)
            *reinterpret_cast<uint4*>(
                static_cast<uint8_t*>(p.c) +
                ((int64_t)(m0 + r) * p.ldc + n0 + c * W) * ES + k * 16) =
                stage[r * 4 + (k ^ ((r >> 1) & 3))];
        }
      } else {
        rows_out<OUT_F32>(p, stage, m0, n0 + c * W, lane);
      }
    }
  }
  // 32 staged rows of 64 bytes, a row's elements side by side.
  template <int OUT_F32>
  __device__ __forceinline__ static void rows_out(const Params& p,
                                                  const uint4* stage, int m0,
                                                  int n0, int lane) {
    constexpr int W = OUT_F32 ? 16 : 32, EACH = W / 4;   // EACH: of a piece
    using T = typename std::conditional<OUT_F32 != 0, float, __nv_bfloat16>::type;
    const int col = lane & (W - 1), up = lane / W;
    const T* from = reinterpret_cast<const T*>(stage) + (col & (EACH - 1));
    T* to = static_cast<T*>(p.c) + (int64_t)(m0 + up) * p.ldc + n0 + col;
    const int rows = n0 + col < p.N ? p.M - m0 - up : 0;
#pragma unroll 8
    for (int r = 0; r < 32; r += 32 / W) {
      const T v = from[((r + up) * 4 + ((col / EACH) ^ (((r + up) >> 1) & 3))) *
                       EACH];
      if (r < rows) *to = v;
      to += 32 / W * p.ldc;
    }
  }
  template <int OUT_F32>
  __device__ __forceinline__ static void put(void* c, int64_t at, float v) {
    if (OUT_F32)
      static_cast<float*>(c)[at] = v;
    else
      static_cast<__nv_bfloat16*>(c)[at] = __float2bfloat16_rn(v);
  }
};

// GridAcc: a scale for each row and each column.  Chunks of 16 rows × 32
// columns in which a thread has rows lane/4 and lane/4 + 8 and in each unit of
// eight columns 2·(lane mod 4) and the next: four rows and 32 columns in all,
// so that a column pair's scales, read once from shared memory, serve four
// products.  Chunk c: rows 16·(c mod 2), columns 32·(c / 2).
struct GridAcc {
  static constexpr int CHUNKS = 8;
  static constexpr int SCALES_READ = 6;
  using Chunk = uint32_t[16];
  uint64_t acc[64];   // [chunk][unit][row]
  float s[4], sn[4];
  uint64_t w2[2][4];   // the columns' of the pair of chunks added, of the next
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 64; ++i) acc[i] = 0;
  }
  __device__ __forceinline__ static void load(uint32_t taddr, int c,
                                              Chunk& r) {
    tmem_ld16x256b_x4(
        taddr + (static_cast<uint32_t>(16 * (c & 1)) << 16) + 32 * (c >> 1), r);
  }
  __device__ __forceinline__ static void wait(Chunk& r) { tmem_ld_wait16(r); }
  __device__ __forceinline__ void scales(const float* rows, const float*, int,
                                         int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) sn[j] = rows[(lane >> 2) + 8 * j];
  }
  __device__ __forceinline__ void next() {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = sn[j];
  }
  // cols: the half's 128 scales, column 16g + 8u + 2q + e at 16g + 4q + 2u + e
  __device__ __forceinline__ void columns(const float* cols, int pair,
                                          int lane) {
#pragma unroll
    for (int u = 0; u < 4; u += 2)   // in order: hoisted loads cost spills
      asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                   : "=l"(w2[pair & 1][u]), "=l"(w2[pair & 1][u + 1])
                   : "r"(smem_u32(cols + 32 * pair + 8 * u +
                                  (lane & 3) * 4)));
  }
  __device__ __forceinline__ void add(const Chunk& r, int c) {
    uint64_t s2[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t v = __float_as_uint(s[(c & 1) * 2 + i]);
      s2[i] = pack_f32x2(v, v);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        fma_f32x2(acc[c * 8 + u * 2 + i],
                  pack_f32x2(r[4 * u + 2 * i], r[4 * u + 2 * i + 1]),
                  mul_f32x2(s2[i], w2[(c >> 1) & 1][u]));
  }
  // The four lanes of a row exchange what makes 16 bytes in each: 64 bytes of
  // a row a store.  Rows that are not 16-byte aligned or end inside the tile
  // go through shared memory, as in RowAcc (2000×2500×4096 53 µs; when it was
  // put in 59, and 64 without).
  template <int OUT_F32>
  __device__ __forceinline__ void store(const Params& p, uint4* stage, int m0,
                                        int n0, int lane) const {
    const int q = lane & 3;
    if (!p.vec || n0 + BNH > p.N) {
      constexpr int W = OUT_F32 ? 16 : 32;   // columns in 64 bytes
#pragma unroll
      for (int g = 0; g < BNH / W; ++g) {
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 4; ++h) {   // rows 8h + lane / 4
          const int r = 8 * h + (lane >> 2);
#pragma unroll
          for (int v = 0; v < W / 8; ++v) {
            const int col = g * W + 8 * v;   // and 2q
            const float2 x = unpack_f32x2(
                acc[(col / 32 * 2 + (h >> 1)) * 8 + col % 32 / 8 * 2 +
                    (h & 1)]);
            const int piece = OUT_F32 ? 2 * v + (q >> 1) : v;
            uint4* to = stage + r * 4 + (piece ^ ((r >> 1) & 3));
            if (OUT_F32)
              reinterpret_cast<float2*>(to)[q & 1] = x;
            else
              reinterpret_cast<uint32_t*>(to)[q] = pack_bf16x2(x.x, x.y);
          }
        }
        __syncwarp();
        RowAcc::rows_out<OUT_F32>(p, stage, m0, n0 + g * W, lane);
      }
      return;
    }
#pragma unroll
    for (int c = 0; c < CHUNKS; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int m = m0 + 16 * (c & 1) + 8 * i + (lane >> 2);
        const int nc = n0 + 32 * (c >> 1);
        const int64_t at = (int64_t)m * p.ldc + nc;
        if (OUT_F32) {
#pragma unroll
          for (int u = 0; u < 4; u += 2) {
            // even lanes: four columns of unit u, odd lanes: of unit u + 1
            const float2 x = unpack_f32x2(acc[c * 8 + u * 2 + i]);
            const float2 y = unpack_f32x2(acc[c * 8 + u * 2 + 2 + i]);
            const bool odd = q & 1;
            const float sx = __shfl_xor_sync(0xffffffffu, odd ? x.x : y.x, 1);
            const float sy = __shfl_xor_sync(0xffffffffu, odd ? x.y : y.y, 1);
            if (m < p.M)
              *reinterpret_cast<float4*>(static_cast<float*>(p.c) + at +
                                         8 * (u + (q & 1)) + 4 * (q >> 1)) =
                  odd ? make_float4(sx, sy, y.x, y.y)
                      : make_float4(x.x, x.y, sx, sy);
          }
        } else {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x = unpack_f32x2(acc[c * 8 + j * 2 + i]);
            w[j] = pack_bf16x2(x.x, x.y);
          }
          // 4×4 transpose over the row's lanes: lane q gets unit q
          const bool o1 = q & 1, o2 = q & 2;
          uint32_t a = __shfl_xor_sync(0xffffffffu, o1 ? w[0] : w[1], 1);
          uint32_t b = __shfl_xor_sync(0xffffffffu, o1 ? w[2] : w[3], 1);
          if (o1) w[0] = a, w[2] = b; else w[1] = a, w[3] = b;
          a = __shfl_xor_sync(0xffffffffu, o2 ? w[0] : w[2], 2);
          b = __shfl_xor_sync(0xffffffffu, o2 ? w[1] : w[3], 2);
          if (o2) w[0] = a, w[1] = b; else w[2] = a, w[3] = b;
          if (m < p.M)
            *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.c) + at +
                                      8 * q) =
                make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
  }
};

// Two CTAs, each with 128 rows of a 256×256 tile: every CTA loads its A rows
// and half of B, and rank 0 (the leader) issues MMAs of M = 256 that read both
// halves (cta_group::2).  No load is multicast: such a load is for one GPU's own
// memory, and one library serves every rank of a run on several (with it, and
// MMAs of each CTA's own, 8192×8192×4096 took 237 µs where the pair's took 242
// on the same GPU, with row scales 315 both).  Roles:
//   warp 0      TMA producer, a ring of six K blocks;
//   warps 1, 2  of the leader: MMA issue, every other K block and one TMEM
//               buffer each: beside eight busy epilogue warps one thread's
//               waits and commits for a K block take about 400 cycles, in which
//               the other's MMAs (512) run;
//   warp 3      the scales, by asynchronous copies four K blocks ahead; its
//               arrival joins the MMAs' commit on the epilogue's barrier;
//   warps 4–11  epilogue, warp w on TMEM lanes 32·(w mod 4) of half (w − 4)/4.
// The epilogue's 128 sums a thread need more than the 168 registers that 384
// threads can have, so the first warpgroup hands some over (128·40 + 256·232
// = 384·168).
//
// Measured: 8192×8192×4096 with a scale for 128×128 of B 242 µs (2270 TFLOP/s),
// with one for each of its rows 318 (1730); 8192×8192×28672 1490 µs alone (2580,
// SM clock at 2070 MHz), 1578 in a loop at the power limit (1942 MHz).  What
// bounds it is the chain of a K block: its MMAs (512 cycles on an idle SM, nearer
// 700 while the epilogue reads TMEM), the read back and the hand-over both ways
// take some 1900 cycles together, and the two halves of TMEM hide one block's
// behind another's, so that one ends every 980 to 1100; the tensor pipe is
// active 53 % of the cycles, the tcgen05 pipe 59 %.  With scales for rows of
// both sides the epilogue multiplies twice as often and a block ends every 1400
// to 1450 (39 and 44 %).  Removing the epilogue's additions altogether gains
// 10 %, the scales' products 10 % of the second kind (both measured with MMAs
// of each CTA's own).
template <int B_ROW, int OUT_F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(WIDE_THREADS, 1)
    gemm_fp8_block_wide(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smA = smem;
  uint8_t* smB = smem + STAGES * TILE_BYTES;
  float* scales = reinterpret_cast<float*>(smB + STAGES * TILE_BYTES);
  uint8_t* staging = reinterpret_cast<uint8_t*>(scales + SLOTS * SLOT);
  uint64_t* full = reinterpret_cast<uint64_t*>(staging + 8 * STAGING);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* sread = tempty + 2;
  uint64_t* drain = sread + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank() & 1u;
  const bool leader = rank == 0;
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  const int64_t blocks =
      (int64_t)((p.total_tiles - cid + ncl - 1) / ncl) * p.kblocks;

  if (threadIdx.x == 0) {
    // full: the leader's counts both CTAs' bytes; empty: the leader's commits
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 2);        // the MMAs and the CTA's own scales
      mbar_init(&tempty[b], 2 * 8);   // the leader's: a lane of each epilogue
      mbar_init(&sread[b], 8);        // warp of both; sread: of this CTA
      mbar_init(&drain[b], 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.ma);
    tma_prefetch_desc(&p.mb);
  }
  if (warp == 1) tmem_alloc_pair(tmem_slot, TMEM_COLS);
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // barriers of both CTAs initialised before any remote use
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 40;");
    if (warp == 0 && lane == 0) {
      // ---------------------------------------------------- TMA producer --
      const uint32_t full0 = cluster_addr(full, 0);   // the leader's full[0]
      uint32_t stage = 0, phase = 0, armed = 0, armed_par = 0;
      bool ok = true;
      for (int t = cid; ok && t < p.total_tiles; t += ncl) {
        int mt, nt;
        decode_tile(p, t, mt, nt);
        const int m0 = mt * 2 * BM + (int)rank * BM;
        const int n0 = nt * BN + (int)rank * BNH;
        for (int kb = 0; kb < p.kblocks; ++kb) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status, 41)) {
            ok = false;
            break;
          }
          if (leader) {
            mbar_arrive_expect_tx(&full[stage], 2 * STAGE_BYTES);
            armed |= 1u << stage;
            armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
          }
          const uint32_t fb = full0 + stage * 8;
          tma_load_3d_pair(smA + stage * TILE_BYTES, &p.ma, fb, kb * BK, 0, m0);
          tma_load_3d_pair(smB + stage * TILE_BYTES, &p.mb, fb, kb * BK, 0, n0);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (ok) {
        // the leader's last commits land on this CTA's empty barriers before
        // it may exit
        for (int i = 0; i < STAGES; ++i) {
          if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status, 42))
            break;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (*abort_flag && leader) {
        // let every copy counted on this CTA's barriers land
        volatile int no_abort = 0;
        for (int s = 0; s < STAGES; ++s)
          if (armed & (1u << s))
            mbar_wait(&full[s], (armed_par >> s) & 1u, &no_abort, nullptr, 0);
      }
    } else if (leader && (warp == 1 || warp == 2)) {
      // -------------------------------------------------------- MMA issue --
      // The warp waits as one and elects the issuing thread, whose operands
      // then sit in uniform registers (8192×8192×4096 242 µs, by one thread
      // that waits alone 248; with row scales 319 / 320).
      constexpr uint32_t IDESC = idesc_e4m3_f32(2 * BM, BN);
      const int buf = __shfl_sync(0xffffffffu, warp, 0) - 1;
      const uint64_t ad0 = smem_desc_sw128(smem_u32(smA), 16, 1024);
      const uint64_t bd0 = smem_desc_sw128(smem_u32(smB), 16, 1024);
      auto wait = [&](uint64_t* bar, uint32_t par, unsigned site) {
        return mbar_wait_warp(bar, par, abort_flag, p.status, site);
      };
      uint32_t stage = buf, phase = 0, tphase = 1;
      for (int64_t it = buf; it < blocks; it += 2) {
        if (!wait(&full[stage], phase, 43)) break;
        const uint64_t ad = ad0 + stage * (TILE_BYTES >> 4);
        const uint64_t bd = bd0 + stage * (TILE_BYTES >> 4);
        if (!wait(&tempty[buf], tphase, 44)) break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * BN;
        if (elect_one()) {
          tc_mma_f8_pair(d, ad, bd, IDESC, 0);
          tc_mma_f8_pair(d, ad + 2, bd + 2, IDESC, 1);
          tc_mma_f8_pair(d, ad + 4, bd + 4, IDESC, 1);
          tc_mma_f8_pair(d, ad + 6, bd + 6, IDESC, 1);
          tc_commit_pair(&tfull[buf], 3);
          tc_commit_pair(&empty[stage], 3);
        }
        __syncwarp();
        stage += 2;
        if (stage >= STAGES) {
          stage -= STAGES;
          phase ^= 1;
        }
        tphase ^= 1;
      }
      const bool gave_up = __any_sync(0xffffffffu, *abort_flag);
      if (gave_up && elect_one()) {   // the thread of the MMAs
        volatile int no_abort = 0;
        tc_commit_pair(&drain[buf], 1);
        mbar_wait(&drain[buf], 0, &no_abort, nullptr, 0);
      }
    } else if (warp == 3) {
      // ----------------------------------------------------------- scales --
      constexpr int AHEAD = 4;
      static_assert(AHEAD + 2 <= SLOTS, "slots are read when reused");
      int ft = cid, fk = 0, fslot = 0;
      int m0 = 0, n0 = 0;
      auto fetch = [&]() {
        if (ft < p.total_tiles) {
          if (fk == 0) {
            int mt, nt;
            decode_tile(p, ft, mt, nt);
            m0 = mt * 2 * BM + (int)rank * BM;
            n0 = nt * BN;
          }
          float* rows = scales + fslot * SLOT;
          float* cols = rows + BM;
          const float* pa = p.sa + fk * p.ldsa;
          const float* pb = p.sb + fk * p.ldsb;
#pragma unroll
          for (int j = 0; j < BM / 32; ++j) {
            const int m = m0 + 32 * j + lane;
            const bool in = m < p.M;
            cp_async4(rows + 32 * j + lane,
                      pa + (in ? (p.a_row ? m : m / BM) : 0), in);
          }
          if (B_ROW) {
            // column 16g + 8u + 2q + e is kept at 16g + 4q + 2u + e
            const int at = (lane & 16) + ((lane >> 1) & 3) * 4 +
                           ((lane >> 3) & 1) * 2 + (lane & 1);
#pragma unroll
            for (int j = 0; j < BN / 32; ++j) {
              const int n = n0 + 32 * j + lane;
              const bool in = n < p.N;
              cp_async4(cols + 32 * j + at, pb + (in ? n : 0), in);
            }
          } else if (lane < 2) {
            const int n = n0 + BNH * lane;
            const bool in = n < p.N;
            cp_async4(cols + lane, pb + (in ? n / BM : 0), in);
          }
          if (++fk == p.kblocks) {
            fk = 0;
            ft += ncl;
          }
        }
        cp_async_commit();
        fslot = (fslot + 1) & (SLOTS - 1);
      };
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) fetch();
      for (int64_t it = 0; it < blocks; ++it) {
        const int buf = it & 1;
        // The epilogue has read the scales of block it − 2: its MMAs are
        // complete, so that this block's phase is open, and the slot that the
        // next copies go to, of block it − 4, is free.
        if (it >= 2) {
          const uint32_t par = ((it - 2) >> 1) & 1;
          if (!mbar_wait_warp(&sread[buf], par, abort_flag, p.status, 46))
            break;
        }
        fetch();
        cp_async_wait<AHEAD>();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tfull[buf]);
      }
      cp_async_wait<0>();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 232;");
    // ------------------------------------------------------------ epilogue --
    using Acc = typename std::conditional<B_ROW != 0, GridAcc, RowAcc>::type;
    const int quarter = warp & 3;          // TMEM lanes this warp may read
    const int half = (warp - 4) >> 2;      // its 128 of the 256 columns
    uint4* stage = reinterpret_cast<uint4*>(staging + (warp - 4) * STAGING);
    const uint32_t taddr0 = tmem_base +
                            (static_cast<uint32_t>(quarter * 32) << 16) +
                            half * BNH;
    const uint32_t tempty0 = cluster_addr(tempty, 0);   // the leader's
    int64_t it = 0;
    bool ok = true, ready = false;
    typename Acc::Chunk r[2];   // a chunk being added, the next on its way
    Acc a;
    auto slot = [&](int64_t i) { return scales + (i & (SLOTS - 1)) * SLOT; };
    auto begin = [&](int64_t i) {   // block i is there: its first chunk, scales
      tc_fence_after();
      Acc::load(taddr0 + (i & 1) * BN, 0, r[0]);
      a.scales(slot(i) + quarter * 32, slot(i) + BM, half, lane);
      a.columns(slot(i) + BM + half * BNH, 0, lane);
    };
    // The warp's reads of a block's scales come before the copies into their
    // slot.  The buffer's arrival below orders TMEM alone: a release to the
    // leader's SM for each block would double the kernel's time.  Placed where
    // little is in flight this one costs 1 to 2 % (242 against 239 µs, with row
    // scales 319 / 313; at the block's end 248, 326).
    auto slot_read = [&](int buf) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sread[buf]);
    };
    for (int t = cid; ok && t < p.total_tiles; t += ncl) {
      a.clear();
      for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
        const int buf = it & 1;
        const uint32_t taddr = taddr0 + buf * BN;
        if (!ready) {
          if (!mbar_wait_warp(&tfull[buf], (it >> 1) & 1, abort_flag, p.status,
                              45)) {
            ok = false;
            break;
          }
          begin(it);
        }
        a.next();
        const float* cols = slot(it) + BM + half * BNH;
#pragma unroll
        for (int c = 0; c < Acc::CHUNKS; ++c) {
          if ((c & 1) == 1 && c + 1 < Acc::CHUNKS)
            a.columns(cols, c / 2 + 1, lane);
          // whether the next block is there is asked in the shadow of a load
          if (c + 1 == Acc::CHUNKS)
            ready = mbar_test_warp(&tfull[buf ^ 1], ((it + 1) >> 1) & 1);
          if (B_ROW && c == Acc::SCALES_READ) slot_read(buf);
          Acc::wait(r[c & 1]);
          if (!B_ROW && c == Acc::SCALES_READ) slot_read(buf);
          if (c + 1 < Acc::CHUNKS) {
            Acc::load(taddr, c + 1, r[(c + 1) & 1]);
          } else {
            // the buffer is read (by all lanes: the wait is the warp's): the
            // MMAs may have it back
            tc_fence_before();
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + buf * 8);
            if (ready) begin(it + 1);
          }
          a.add(r[c & 1], c);
        }
      }
      if (!ok) break;
      int mt, nt;
      decode_tile(p, t, mt, nt);
      const int n0 = nt * BN + half * BNH;
      if (n0 < p.N)
        a.template store<OUT_F32>(p, stage,
                                  mt * 2 * BM + (int)rank * BM + quarter * 32,
                                  n0, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA leaves while the pair still uses it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// ================================================================== narrow ==
// BNT rows of A against 128 rows of B.  Up to 64 rows two CTAs share an SM
// (four epilogue warps of 32 × BNT); 128 rows take eight epilogue warps of
// 32 × 64 and the SM's shared memory for themselves.
constexpr int NSLOTS = 16;   // K blocks of scales kept; a power of two
constexpr int NAHEAD = 8;    // and loaded ahead of the epilogue
template <int BNT>
struct Narrow {
  static constexpr int EWARPS = BNT <= 64 ? 4 : 8;
  static constexpr int THREADS = 96 + 32 * EWARPS;
  static constexpr int CTAS = BNT <= 64 ? 2 : 1;
  static constexpr int NC = BNT <= 64 ? BNT : 64;      // columns of a warp
  static constexpr int UNITS = NC <= 16 ? 2 : 4;       // of 8 columns a chunk
  static constexpr int CHUNKS = 2 * NC / (8 * UNITS);  // 16 rows × 8·UNITS
  static constexpr int T_BYTES = BNT * BK;
  static constexpr int STAGE = TILE_BYTES + T_BYTES;
  static constexpr int STAGES = BNT <= 32 ? 5 : BNT <= 64 ? 4 : 6;
  static constexpr int BUFS = 4;
  static constexpr int COLS = BUFS * BNT;    // TMEM: 64, 128, 256, 512
  static_assert(COLS >= 32 && COLS <= 512 && (COLS & (COLS - 1)) == 0,
                "what TMEM is handed out in");
  static constexpr int SLOT = BM + BNT;                        // floats
  static constexpr int SCALES = NSLOTS * SLOT;
  static constexpr int SMEM = STAGES * STAGE + SCALES * 4 + 1024 + 256;
};

struct NarrowParams {
  CUtensorMap mr, mt;      // the 128-row side (B), the BNT-row side (A)
  const float *sr, *st;
  int64_t ldsr, ldst;
  int r_row, t_row;
  int R, T, kblocks;
  int t_tiles, split;
  void* c;
  int64_t ldc;
  int vec;                 // four outputs of a row start on 4·(their size)
  unsigned* status;
};

// 16 TMEM lanes × 16 columns (two units).
__device__ __forceinline__ void tmem_ld16x256b_x2(uint32_t taddr,
                                                  uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]),
        "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait8(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]),
                 "+r"(r[5]), "+r"(r[6]), "+r"(r[7])::"memory");
}

// Warp 0: TMA producer.  Warp 1: MMA issue and TMEM.  Warp 2: the scales, far
// enough ahead for their latency from DRAM (three blocks ahead: 0.47 µs a K
// block, whatever the tile).  The others: epilogue, in the layout of GridAcc
// (four rows and a quarter of the columns a thread).
//
// Bound by the read of B: 48×8192×28672 45 µs (5.3 TB/s, 79 % of a copy's
// rate; 16 rows 42), and where that is short by a K block's latency through
// the ring, the MMAs and TMEM: 16×4096×4096 8.5 µs.
template <int BNT, int OUT_F32>
__global__ void __launch_bounds__(Narrow<BNT>::THREADS, Narrow<BNT>::CTAS)
    gemm_fp8_block_narrow(const __grid_constant__ NarrowParams p) {
  using L = Narrow<BNT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smR = smem;
  uint8_t* smT = smem + L::STAGES * TILE_BYTES;
  float* scales = reinterpret_cast<float*>(smT + L::STAGES * L::T_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + L::SCALES);
  uint64_t* empty = full + L::STAGES;
  uint64_t* tfull = empty + L::STAGES;
  uint64_t* tempty = tfull + L::BUFS;
  uint64_t* drain = tempty + L::BUFS;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int part = blockIdx.x % p.split;    // rank in the cluster
  const int tile = blockIdx.x / p.split;
  const int r0 = tile / p.t_tiles * BM, t0 = tile % p.t_tiles * BNT;
  const int kb0 = (int)((int64_t)p.kblocks * part / p.split);
  const int kb1 = (int)((int64_t)p.kblocks * (part + 1) / p.split);

  auto copy = [&](int kb, uint32_t stage) {
    mbar_arrive_expect_tx(&full[stage], L::STAGE);
    tma_load_3d(smR + stage * TILE_BYTES, &p.mr, &full[stage], kb * BK, 0, r0);
    tma_load_3d(smT + stage * L::T_BYTES, &p.mt, &full[stage], kb * BK, 0, t0);
  };
  const int primed = min(kb1 - kb0, L::STAGES);
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < L::BUFS; ++b) {
      mbar_init(&tfull[b], 2);   // the MMAs and the scales
      mbar_init(&tempty[b], L::EWARPS);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    // the ring is filled while TMEM is allocated and the warps meet
    for (int s = 0; s < primed; ++s) copy(kb0 + s, s);
  }
  if (warp == 1) tmem_alloc(tmem_slot, L::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  // epilogue warps: rows 32·(warp mod 4), columns NC·((warp − 3) / 4)
  const int quarter = warp & 3;
  const int colw = warp >= 3 ? (warp - 3) / 4 * L::NC : 0;
  uint64_t acc[L::NC / 2];   // [chunk][unit][row]
#pragma unroll
  for (int i = 0; i < L::NC / 2; ++i) acc[i] = 0;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 1, armed = (1u << primed) - 1, armed_par = 0;
      for (int kb = kb0 + primed; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status, 51))
          break;
        armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
        copy(kb, stage);
        if (++stage == L::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (*abort_flag) {
        volatile int no_abort = 0;
        for (int s = 0; s < L::STAGES; ++s)
          if (armed & (1u << s))
            mbar_wait(&full[s], (armed_par >> s) & 1u, &no_abort, nullptr, 0);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t IDESC = idesc_e4m3_f32(BM, BNT);
      const uint64_t rd0 = smem_desc_sw128(smem_u32(smR), 16, 1024);
      const uint64_t td0 = smem_desc_sw128(smem_u32(smT), 16, 1024);
      uint32_t stage = 0, phase = 0, buf = 0, tphase = 1;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&full[stage], phase, abort_flag, p.status, 52) ||
            !mbar_wait(&tempty[buf], tphase, abort_flag, p.status, 53))
          break;
        tc_fence_after();
        const uint32_t d = tmem_base + buf * BNT;
        const uint64_t rd = rd0 + stage * (TILE_BYTES >> 4);
        const uint64_t td = td0 + stage * (L::T_BYTES >> 4);
        tc_mma_f8(d, rd, td, IDESC, 0);
        tc_mma_f8(d, rd + 2, td + 2, IDESC, 1);
        tc_mma_f8(d, rd + 4, td + 4, IDESC, 1);
        tc_mma_f8(d, rd + 6, td + 6, IDESC, 1);
        tc_commit(&tfull[buf]);
        tc_commit(&empty[stage]);
        if (++stage == L::STAGES) {
          stage = 0;
          phase ^= 1;
        }
        if (++buf == L::BUFS) {
          buf = 0;
          tphase ^= 1;
        }
      }
      // every commit lands before the ring's memory is used again
      volatile int no_abort = 0;
      tc_commit(drain);
      mbar_wait(drain, 0, &no_abort, nullptr, 0);
    }
  } else if (warp == 2) {
    // the 128 rows' scales, then the columns' (column 16g + 8u + 2q + e at
    // 16g + 4q + 2u + e, so that a thread reads its four of 16 at once)
    static_assert(NAHEAD + 2 * L::BUFS <= NSLOTS, "slots are read when reused");
    const int at = (lane & 16) + ((lane >> 1) & 3) * 4 + ((lane >> 3) & 1) * 2 +
                   (lane & 1);
    const float* pr = p.sr + kb0 * p.ldsr;
    const float* pt = p.st + kb0 * p.ldst;
    int fkb = kb0, fslot = 0;
    auto fetch = [&]() {
      if (fkb < kb1) {
        float* rows = scales + fslot * L::SLOT;
#pragma unroll
        for (int j = 0; j < BM / 32; ++j) {
          const int r = r0 + 32 * j + lane;
          cp_async4(rows + 32 * j + lane,
                    pr + (r < p.R ? (p.r_row ? r : r / BM) : 0), r < p.R);
        }
#pragma unroll
        for (int j = 0; j < (BNT + 31) / 32; ++j) {
          const int t = t0 + 32 * j + lane;
          if (32 * j + lane < BNT)
            cp_async4(rows + BM + 32 * j + at,
                      pt + (t < p.T ? (p.t_row ? t : t / BM) : 0), t < p.T);
        }
        pr += p.ldsr;
        pt += p.ldst;
        ++fkb;
        fslot = (fslot + 1) & (NSLOTS - 1);
      }
      cp_async_commit();
    };
#pragma unroll 1
    for (int i = 0; i < NAHEAD; ++i) fetch();
    int buf = 0;
    uint32_t par = 1;   // of the phase before this block's on its barrier
    for (int kb = kb0; kb < kb1; ++kb) {
      // the epilogue is done with block kb − BUFS: this block's phase is open,
      // and the slot that the next copies go to (of kb − BUFS·2 or before) is
      // free
      if (kb - kb0 >= L::BUFS &&
          !mbar_wait_warp(&tempty[buf], par, abort_flag, p.status, 55))
        break;
      fetch();
      cp_async_wait<NAHEAD>();
      __syncwarp();
      if (lane == 0) mbar_arrive(&tfull[buf]);
      if (++buf == L::BUFS) {
        buf = 0;
        par ^= 1;
      }
    }
    cp_async_wait<0>();
  } else {
    const uint32_t taddr0 =
        tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + colw;
    constexpr int W = 8 * L::UNITS;   // columns of a chunk
    auto load = [&](int buf, int c, uint32_t (&x)[4 * L::UNITS]) {
      const uint32_t ta = taddr0 + buf * BNT + W * (c >> 1) +
                          (static_cast<uint32_t>(16 * (c & 1)) << 16);
      if constexpr (L::UNITS == 2)
        tmem_ld16x256b_x2(ta, x);
      else
        tmem_ld16x256b_x4(ta, x);
    };
    auto wait = [&](uint32_t (&x)[4 * L::UNITS]) {
      if constexpr (L::UNITS == 2)
        tmem_ld_wait8(x);
      else
        tmem_ld_wait16(x);
    };
    int buf = 0, slot = 0;
    uint32_t par = 0;
    uint32_t x[2][4 * L::UNITS];
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_warp(&tfull[buf], par, abort_flag, p.status, 54)) break;
      tc_fence_after();
      load(buf, 0, x[0]);
      const float* rs = scales + slot * L::SLOT + quarter * 32 + (lane >> 2);
      const float* cs = scales + slot * L::SLOT + BM + colw;
      uint64_t s2[4], w2[L::UNITS];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = __float_as_uint(rs[8 * j]);
        s2[j] = pack_f32x2(v, v);
      }
#pragma unroll
      for (int c = 0; c < L::CHUNKS; ++c) {
        if ((c & 1) == 0) {
#pragma unroll
          for (int u = 0; u < L::UNITS; u += 2)
            asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];"
                         : "=l"(w2[u]), "=l"(w2[u + 1])
                         : "r"(smem_u32(cs + W * (c >> 1) + 8 * u +
                                        (lane & 3) * 4)));
        }
        wait(x[c & 1]);
        if (c + 1 < L::CHUNKS) {
          load(buf, c + 1, x[(c + 1) & 1]);
        } else {
          // a release: the scales' reads are ordered before the copies that
          // reuse their slot as well
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[buf]);
        }
#pragma unroll
        for (int u = 0; u < L::UNITS; ++u)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            fma_f32x2(acc[(c * L::UNITS + u) * 2 + i],
                      pack_f32x2(x[c & 1][4 * u + 2 * i],
                                 x[c & 1][4 * u + 2 * i + 1]),
                      mul_f32x2(s2[(c & 1) * 2 + i], w2[u]));
      }
      slot = (slot + 1) & (NSLOTS - 1);
      if (++buf == L::BUFS) {
        buf = 0;
        par ^= 1;
      }
    }
  }

  tc_fence_before();
  __syncthreads();   // copies, MMAs and TMEM reads of this CTA are done
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, L::COLS);

  // Every CTA leaves its sums in its own shared memory, [column][row] over the
  // operand ring (pitch 132: the lanes' rows and columns fall on 32 banks);
  // rank j of the cluster adds up columns [j·w, (j + 1)·w) in rank order.
  constexpr int PITCH = BM + 4;
  float* out = reinterpret_cast<float*>(smem);
  if (warp >= 3) {
#pragma unroll
    for (int c = 0; c < L::CHUNKS; ++c)
#pragma unroll
      for (int u = 0; u < L::UNITS; ++u) {
        float* d = out + (colw + 8 * L::UNITS * (c >> 1) + 8 * u +
                          2 * (lane & 3)) * PITCH +
                   quarter * 32 + 16 * (c & 1) + (lane >> 2);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float2 v = unpack_f32x2(acc[(c * L::UNITS + u) * 2 + i]);
          d[8 * i] = v.x;
          d[PITCH + 8 * i] = v.y;
        }
      }
  }
  if (p.split > 1)
    cluster_sync();
  else
    __syncthreads();
  if (warp >= 3) {
    // a warp per column, four rows a lane
    const int w = (BNT + p.split - 1) / p.split;
    const int end = min(min((part + 1) * w, BNT), p.T - t0);
    const int row = r0 + 4 * lane;
    uint32_t from[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < p.split) from[k] = cluster_addr(out + 4 * lane, k);
#pragma unroll 2
    for (int col = part * w + warp - 3; col < end; col += L::EWARPS) {
      float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
      if (p.split == 1) {
        const float4 x = *reinterpret_cast<const float4*>(out + 4 * lane +
                                                          col * PITCH);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      } else {
        float x[8][4];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < p.split)
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(x[k][0]), "=f"(x[k][1]), "=f"(x[k][2]),
                           "=f"(x[k][3])
                         : "r"(from[k] + col * PITCH * 4));
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < p.split) {
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] += x[k][j];
          }
      }
      const int64_t at = (int64_t)(t0 + col) * p.ldc + row;
      if (p.vec && row + 4 <= p.R) {
        if (OUT_F32)
          *reinterpret_cast<float4*>(static_cast<float*>(p.c) + at) =
              make_float4(v[0], v[1], v[2], v[3]);
        else
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.c) + at) =
              make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (row + j < p.R) RowAcc::put<OUT_F32>(p.c, at + j, v[j]);
      }
    }
  }
  if (p.split > 1) cluster_sync();   // no CTA leaves while it is read
}

// ==================================================================== host ==
bool operand_map(CUtensorMap* m, const uint8_t* q, int64_t rows, int64_t K,
                 int64_t ld, uint32_t box_rows) {
  return encode_tmap_3d_u8(m, q, K, 1, rows, ld, ld, BK, 1, box_rows);
}

constexpr int kMaxDevices = 64;

int current_device(int& dev) {
  const cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  return dev < 0 || dev >= kMaxDevices ? cudaErrorInvalidDevice : cudaSuccess;
}

// Clusters of the wide kernel that the device holds at once; the first call on
// a device sets the kernel's attributes.
template <int B_ROW, int OUT_F32>
int launch_wide(const Params& prm, cudaStream_t s) {
  static std::atomic<int> clusters[kMaxDevices];
  auto kernel = gemm_fp8_block_wide<B_ROW, OUT_F32>;
  int dev = 0, err = current_device(dev);
  if (err) return err;
  int ncl = clusters[dev].load();
  if (ncl == 0) {
    if ((err = cudaFuncSetAttribute(kernel,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    WIDE_SMEM)))
      return err;
    // the register hand-over sums to 384·168: refuse a build with fewer
    cudaFuncAttributes fa;
    if ((err = cudaFuncGetAttributes(&fa, kernel))) return err;
    if (fa.numRegs < 168) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)(device_sm_count() & ~1));
    cfg.blockDim = dim3(WIDE_THREADS);
    cfg.dynamicSmemBytes = WIDE_SMEM;
    if ((err = cudaOccupancyMaxActiveClusters(&ncl, kernel, &cfg))) return err;
    if (ncl < 1) return cudaErrorInvalidConfiguration;
    clusters[dev].store(ncl);
  }
  const int grid = 2 * std::min(prm.total_tiles, ncl);
  kernel<<<grid, WIDE_THREADS, WIDE_SMEM, s>>>(prm);
  return cudaGetLastError();
}

template <int BNT, int OUT_F32>
int launch_narrow(const NarrowParams& prm, unsigned grid, cudaStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  auto kernel = gemm_fp8_block_narrow<BNT, OUT_F32>;
  int dev = 0, err = current_device(dev);
  if (err) return err;
  if (!done[dev].load()) {
    if ((err = cudaFuncSetAttribute(kernel,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    Narrow<BNT>::SMEM)))
      return err;
    done[dev].store(true);
  }
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(Narrow<BNT>::THREADS);
  cfg.dynamicSmemBytes = Narrow<BNT>::SMEM;
  cfg.stream = s;
  cudaLaunchAttribute at;
  memset(&at, 0, sizeof(at));
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = (unsigned)prm.split;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, prm);
}

int wide(const GemmFp8Block& g, cudaStream_t s, unsigned* status) {
  Params p;
  memset(&p, 0, sizeof(p));
  if (!operand_map(&p.ma, g.qa, g.M, g.K, g.lda, BM) ||
      !operand_map(&p.mb, g.qb, g.N, g.K, g.ldb, BNH))
    return cudaErrorInvalidValue;
  p.sa = g.sa;
  p.sb = g.sb;
  p.ldsa = g.ldsa;
  p.ldsb = g.ldsb;
  p.a_row = g.a_group == kFp8Row;
  p.M = (int)g.M;
  p.N = (int)g.N;
  p.kblocks = (int)((g.K + BK - 1) / BK);
  p.m_tiles = (int)((g.M + 2 * BM - 1) / (2 * BM));
  p.n_tiles = (int)((g.N + BN - 1) / BN);
  p.total_tiles = p.m_tiles * p.n_tiles;
  p.group_m = 8;
  p.c = g.c;
  p.ldc = g.ldc;
  const int es = g.out_f32 ? 4 : 2;
  p.vec = (reinterpret_cast<uintptr_t>(g.c) & 15u) == 0 && g.ldc * es % 16 == 0;
  p.status = status;
  const bool b_row = g.b_group == kFp8Row;
  if (g.out_f32)
    return b_row ? launch_wide<1, 1>(p, s) : launch_wide<0, 1>(p, s);
  return b_row ? launch_wide<1, 0>(p, s) : launch_wide<0, 0>(p, s);
}

int narrow(const GemmFp8Block& g, cudaStream_t s, unsigned* status, int bn,
           int split) {
  NarrowParams p;
  memset(&p, 0, sizeof(p));
  if (!operand_map(&p.mr, g.qb, g.N, g.K, g.ldb, BM) ||
      !operand_map(&p.mt, g.qa, g.M, g.K, g.lda, (uint32_t)bn))
    return cudaErrorInvalidValue;
  p.sr = g.sb;
  p.st = g.sa;
  p.ldsr = g.ldsb;
  p.ldst = g.ldsa;
  p.r_row = g.b_group == kFp8Row;
  p.t_row = g.a_group == kFp8Row;
  p.R = (int)g.N;
  p.T = (int)g.M;
  p.kblocks = (int)((g.K + BK - 1) / BK);
  p.t_tiles = (int)((g.M + bn - 1) / bn);
  p.split = split;
  p.c = g.c;
  p.ldc = g.ldc;
  const uintptr_t four = g.out_f32 ? 16 : 8;
  p.vec = reinterpret_cast<uintptr_t>(g.c) % four == 0 && g.ldc % 4 == 0;
  p.status = status;
  const int64_t grid =
      (g.N + BM - 1) / BM * (int64_t)p.t_tiles * split;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned n = (unsigned)grid;
  switch (bn * 2 + (g.out_f32 ? 1 : 0)) {
    case 32: return launch_narrow<16, 0>(p, n, s);
    case 33: return launch_narrow<16, 1>(p, n, s);
    case 64: return launch_narrow<32, 0>(p, n, s);
    case 65: return launch_narrow<32, 1>(p, n, s);
    case 128: return launch_narrow<64, 0>(p, n, s);
    case 129: return launch_narrow<64, 1>(p, n, s);
    case 256: return launch_narrow<128, 0>(p, n, s);
    default: return launch_narrow<128, 1>(p, n, s);
  }
}

// Which form, and the narrow one's rows of A a tile and split of K, by an
// estimate in µs from what both were measured to take on 152 SMs:
//  * narrow: 4 a wave of CTAs, and the K blocks' time (0.34 to 0.40 each,
//    latency of the ring) beside the bytes at 6.4 TB/s, 0.3 of the shorter of
//    the two not hidden.  Estimated / measured: 16×4096×4096 split 8 7.0 / 8.5,
//    48×8192×28672 split 4 47 / 45, split 1 98 / 90;
//    128×8192×28672 split 2 60 / 56, split 4 64 / 62; 512×4096×4096 18 / 19;
//  * wide: 5, and for each round of tiles 2 and 0.46 a K block (0.66 with a
//    scale for each row of B).  512×4096×4096 22 / 21, 1024×8192×8192 68 / 70,
//    256×8192×28672 110 / 111 (narrow, split 1: 105 / 97),
//    8192×8192×4096 239 / 242.
// Clusters of more than four CTAs leave SMs of a GPC empty.
Fp8BlockPlan choose(int64_t M, int64_t N, int64_t K, bool b_row, int sms) {
  auto up = [](int64_t a, int64_t b) { return (a + b - 1) / b; };
  const int64_t kblocks = up(K, BK);
  const int64_t tiles = up(M, 2 * BM) * up(N, BN);
  Fp8BlockPlan best;
  double least = 5.0 + up(tiles, std::max(sms / 2, 1)) *
                           (2.0 + kblocks * (b_row ? 0.66 : 0.46));
  const double bytes = ((double)M + (double)N) * (double)K / 6.4e6;
  const int bn = M <= 16 ? 16 : M <= 32 ? 32 : M <= 64 ? 64 : 128;
  const double kb_us = bn <= 32 ? 0.34 : bn <= 64 ? 0.37 : 0.40;
  const int64_t t = up(N, BM) * up(M, bn);
  for (int split = 1; split <= 8 && split <= kblocks; ++split) {
    const double slots = sms * (bn <= 64 ? 2 : 1) * (split > 4 ? 0.85 : 1.0);
    const double waves = std::max(1.0, std::ceil(t * split / slots));
    const double work = waves * up(kblocks, split) * kb_us;
    const double us = 4.0 * waves + std::max(work, bytes) +
                      0.3 * std::min(work, bytes);
    if (us < least) {
      least = us;
      best.form = kFp8Narrow;
      best.rows = bn;
      best.split = split;
    }
  }
  return best;
}

}  // namespace

Fp8BlockPlan plan_fp8_block(int64_t M, int64_t N, int64_t K, int b_group,
                            int sms) {
  if (M > 8) return choose(M, N, K, b_group == kFp8Row, sms);
  Fp8BlockPlan p;   // measured in gemm_fp8_block_thin.cu
  p.form = kFp8Thin;
  p.rows = 8;
  return p;
}

int gemm_fp8_block(const GemmFp8Block& g, void* stream, unsigned* status) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const Fp8BlockPlan pl =
      plan_fp8_block(g.M, g.N, g.K, g.b_group, device_sm_count());
  int err;
  {
    ProfScope ps(s, KF_GEMM_TC_FP8, 2.0 * g.M * g.N * g.K,
                 (double)(g.M + g.N) * g.K + (g.out_f32 ? 4.0 : 2.0) * g.M * g.N);
    if (pl.form == kFp8Thin)
      err = gemm_fp8_block_thin(g, s);
    else if (pl.form == kFp8Narrow)
      err = narrow(g, s, status, pl.rows, pl.split);
    else
      err = wide(g, s, status);
  }
  if (err) return err;
  count_launch();
  return cudaSuccess;
}

}  // namespace tp
