// gemm_fp8_block.cu — C[M, N] = Σ_b sa[b]·sb[b]·Σ_{k in block b} qa·qb over
// K blocks of 128, E4M3 codes with fp32 scales, C in bf16 or fp32.
//
// The tensor cores give the plain sum of one K block (four tcgen05.mma
// kind::f8f6f4 of K = 32 into fresh TMEM columns); the epilogue warps read it
// back while the next block runs, multiply it by sa·sb and add it to the
// output tile, which stays in their registers over the whole K loop.  Two
// forms:
//  * wide: persistent clusters of two CTAs, 256×256 tiles (cta_group::2),
//    for products that fill the card with such tiles;
//  * narrow: one CTA per 128×BN tile with B's rows (the weight) on the
//    instruction's M side, BN = 16 to 128 rows of A, and K split over a
//    cluster whose CTAs add up their parts through distributed shared memory
//    in rank order: the form for few rows of A, which reads the weight once.
// Neither keeps anything between calls or needs a workspace, and no sum's
// order is left open.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

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
  int a_row, b_row;        // a scale for each row (1) or for 128 rows (0)
  int M, N, kblocks;
  int m_tiles, n_tiles, total_tiles, group_m;
  void* c;
  int64_t ldc;
  int vec;                 // rows of C start on 16 bytes
  unsigned* status;
};

// ==================================================================== wide ==
constexpr int BN = 256;
constexpr int BNH = BN / 2;                    // B rows held by each CTA
constexpr int STAGES = 6;
constexpr int STAGE_BYTES = 2 * TILE_BYTES;
constexpr int TMEM_COLS = 512;
constexpr int WIDE_THREADS = 384;
// Scales reach the epilogue through shared memory by asynchronous copies
// SLOTS − 1 K blocks ahead, each warp's apart: 32 row scales and up to 128
// column scales a block.  (Loads into registers that are handed on from block
// to block stall on the hand-over: 480 instead of ... µs.)
constexpr int SLOTS = 4;   // a power of two
constexpr int WIDE_SCALES = 8 * SLOTS * (32 + BNH);   // floats
constexpr int WIDE_SMEM = STAGES * STAGE_BYTES + WIDE_SCALES * 4 + 1024 + 256;

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

// The K blocks of this CTA's tiles in order.
struct Cursor {
  int t, kb, mt, nt;
  __device__ void start(const Params& p, int cid) {
    t = cid;
    kb = 0;
    if (t < p.total_tiles) decode_tile(p, t, mt, nt);
  }
  __device__ void next(const Params& p, int ncl) {
    if (++kb == p.kblocks) {
      kb = 0;
      t += ncl;
      if (t < p.total_tiles) decode_tile(p, t, mt, nt);
    }
  }
};

// Warp 0: TMA producer.  Warp 1: MMA issue (leader) and TMEM.  Warps 4–11:
// epilogue, warp w on TMEM lanes 32·(w mod 4) and on 128 of the 256 columns.
// The epilogue's 128 sums a thread need more than the 168 registers that 384
// threads can have, so the first warpgroup hands some over (128·88 + 256·208
// = 384·168).
template <int B_ROW, int OUT_F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(WIDE_THREADS, 1)
    gemm_fp8_block_wide(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* smA = smem;
  uint8_t* smB = smem + STAGES * TILE_BYTES;
  float* scales = reinterpret_cast<float*>(smB + STAGES * TILE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(scales + WIDE_SCALES);
  uint64_t* empty = full + STAGES;
  uint64_t* tfull = empty + STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank() & 1u;
  const bool leader = rank == 0;
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 2 * 8);   // a lane of each epilogue warp, both CTAs
    }
    mbar_init(drain, 1);
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
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
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
        // the CTA may exit
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
    } else if (warp == 1 && leader && lane == 0) {
      // -------------------------------------------------------- MMA issue --
      constexpr uint32_t IDESC = idesc_e4m3_f32(2 * BM, BN);
      uint32_t stage = 0, phase = 0;
      bool ok = true;
      int it = 0;   // K blocks so far: TMEM buffer it & 1
      for (int t = cid; ok && t < p.total_tiles; t += ncl) {
        for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
          const int buf = it & 1;
          if (!mbar_wait(&tempty[buf], ((it >> 1) & 1) ^ 1, abort_flag,
                         p.status, 43) ||
              !mbar_wait(&full[stage], phase, abort_flag, p.status, 44)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a0 = smem_u32(smA + stage * TILE_BYTES);
          const uint32_t b0 = smem_u32(smB + stage * TILE_BYTES);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f8_pair(tmem_base + buf * BN,
                           smem_desc_sw128(a0 + kk * 32, 16, 1024),
                           smem_desc_sw128(b0 + kk * 32, 16, 1024), IDESC,
                           kk != 0);
          tc_commit_pair(&empty[stage], 3);
          tc_commit_pair(&tfull[buf], 3);
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (*abort_flag) {
        volatile int no_abort = 0;
        tc_commit_pair(drain, 1);
        mbar_wait(drain, 0, &no_abort, nullptr, 0);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------ epilogue --
    const int quarter = warp & 3;          // TMEM lanes this warp may read
    const int half = (warp - 4) >> 2;      // its 128 of the 256 columns
    const int row = (int)rank * BM + quarter * 32 + lane;   // in the pair tile
    float* myrows = scales + (warp - 4) * SLOTS * (32 + BNH);  // [SLOTS][32]
    float* mycols = myrows + SLOTS * 32;                       // [SLOTS][BNH]
    const uint32_t tempty0 = cluster_addr(tempty, 0);   // the leader's
    const uint32_t taddr0 =
        tmem_base + (static_cast<uint32_t>(quarter * 32) << 16) + half * BNH;

    // one group of copies per K block: the lane's row scale, and the column
    // block's scale (lane 0) or four columns' (B_ROW)
    Cursor ahead;
    ahead.start(p, cid);
    int slot_in = 0;
    auto fetch = [&]() {
      if (ahead.t < p.total_tiles) {
        const int m = ahead.mt * 2 * BM + row;
        const int n = ahead.nt * BN + half * BNH;
        const float* pa = p.sa + ahead.kb * p.ldsa;
        const float* pb = p.sb + ahead.kb * p.ldsb;
        cp_async4(myrows + slot_in * 32 + lane,
                  pa + (m < p.M ? (p.a_row ? m : m / BM) : 0), m < p.M);
        if (B_ROW) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int nj = n + 32 * j + lane;
            cp_async4(mycols + slot_in * BNH + 32 * j + lane,
                      pb + (nj < p.N ? nj : 0), nj < p.N);
          }
        } else if (lane == 0) {
          cp_async4(mycols + slot_in * BNH, pb + (n < p.N ? n / BM : 0),
                    n < p.N);
        }
        ahead.next(p, ncl);
      }
      cp_async_commit();
      slot_in = (slot_in + 1) & (SLOTS - 1);
    };
#pragma unroll
    for (int i = 0; i < SLOTS - 1; ++i) fetch();

    int it = 0;
    bool ok = true;
    for (int t = cid; ok && t < p.total_tiles; t += ncl) {
      uint64_t acc[BNH / 2];
#pragma unroll
      for (int i = 0; i < BNH / 2; ++i) acc[i] = 0;
      for (int kb = 0; kb < p.kblocks; ++kb, ++it) {
        const int buf = it & 1;
        cp_async_wait<SLOTS - 2>();   // this block's group is complete
        __syncwarp();   // for every lane's, and the last block's are read
        const float a0 = myrows[(it & (SLOTS - 1)) * 32 + lane];
        const float* cs = mycols + (it & (SLOTS - 1)) * BNH;
        fetch();
        if (!mbar_wait_warp(&tfull[buf], (it >> 1) & 1, abort_flag, p.status,
                            45)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t sb = __float_as_uint(B_ROW ? a0 : a0 * cs[0]);
        const uint64_t s2 = pack_f32x2(sb, sb);
        const uint32_t taddr = taddr0 + buf * BN;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          tmem_ld32(taddr + c * 32, r);
          tmem_ld_wait(r);
          if (c == 3) {   // the buffer is read: the MMAs may have it back
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster_relaxed(tempty0 + buf * 8);
          }
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            uint64_t x0 = s2, x1 = s2;
            if (B_ROW) {
              const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(
                  cs + c * 32 + 2 * i);
              x0 = mul_f32x2(s2, w.x);
              x1 = mul_f32x2(s2, w.y);
            }
            fma_f32x2(acc[c * 16 + i], pack_f32x2(r[2 * i], r[2 * i + 1]), x0);
            fma_f32x2(acc[c * 16 + i + 1],
                      pack_f32x2(r[2 * i + 2], r[2 * i + 3]), x1);
          }
        }
      }
      if (!ok) break;
      int mt, nt;
      decode_tile(p, t, mt, nt);
      const int m = mt * 2 * BM + row;
      const int n0 = nt * BN + half * BNH;
      if (m < p.M && n0 < p.N) {
        const int valid = min(BNH, p.N - n0);
        if (OUT_F32) {
          float* dst = static_cast<float*>(p.c) + (int64_t)m * p.ldc + n0;
#pragma unroll
          for (int i = 0; i < BNH / 2; i += 2) {
            const float2 x = unpack_f32x2(acc[i]), y = unpack_f32x2(acc[i + 1]);
            if (p.vec && 2 * i + 4 <= valid) {
              *reinterpret_cast<float4*>(dst + 2 * i) =
                  make_float4(x.x, x.y, y.x, y.y);
            } else {
              if (2 * i < valid) dst[2 * i] = x.x;
              if (2 * i + 1 < valid) dst[2 * i + 1] = x.y;
              if (2 * i + 2 < valid) dst[2 * i + 2] = y.x;
              if (2 * i + 3 < valid) dst[2 * i + 3] = y.y;
            }
          }
        } else {
          __nv_bfloat16* dst =
              static_cast<__nv_bfloat16*>(p.c) + (int64_t)m * p.ldc + n0;
#pragma unroll
          for (int i = 0; i < BNH / 2; i += 4) {
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 x = unpack_f32x2(acc[i + j]);
              w[j] = pack_bf16x2(x.x, x.y);
            }
            if (p.vec && 2 * i + 8 <= valid) {
              *reinterpret_cast<uint4*>(dst + 2 * i) =
                  make_uint4(w[0], w[1], w[2], w[3]);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (2 * i + j < valid)
                  reinterpret_cast<uint16_t*>(dst)[2 * i + j] =
                      (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync();   // neither CTA leaves while the pair still uses it
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// ================================================================== narrow ==
constexpr int NARROW_THREADS = 192;

// BN rows of A against 128 rows of B; shared memory for two CTAs on an SM.
template <int BNT>
struct Narrow {
  static constexpr int T_BYTES = BNT * BK;
  static constexpr int STAGE = TILE_BYTES + T_BYTES;
  static constexpr int STAGES = BNT <= 16 ? 6 : BNT <= 32 ? 5 : BNT <= 64 ? 4 : 3;
  static constexpr int BUFS = BNT <= 64 ? 4 : 2;
  static constexpr int COLS = BUFS * BNT;    // TMEM: 64, 128, 256, 256
  static constexpr int SCALES = 4 * SLOTS * (32 + BNT);   // floats
  static constexpr int SMEM = STAGES * STAGE + SCALES * 4 + 1024 + 256;
};

struct NarrowParams {
  CUtensorMap mr, mt;      // the 128-row side, the BN-row side
  const float *sr, *st;
  int64_t ldsr, ldst;
  int r_row, t_row;
  int R, T, kblocks;
  int t_tiles, split;
  void* c;
  int64_t cr, ct;          // element strides of C along R and T
  unsigned* status;
};

// Warp 0: TMA producer.  Warp 1: MMA issue and TMEM.  Warps 2–5: epilogue, a
// row of the 128 each thread.
template <int BNT, int OUT_F32>
__global__ void __launch_bounds__(NARROW_THREADS, 2)
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

  if (threadIdx.x == 0) {
    for (int s = 0; s < L::STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < L::BUFS; ++b) {
      mbar_init(&tfull[b], 1);
      mbar_init(&tempty[b], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.mr);
    tma_prefetch_desc(&p.mt);
  }
  if (warp == 1) tmem_alloc(tmem_slot, L::COLS);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;

  float acc[BNT];
#pragma unroll
  for (int i = 0; i < BNT; ++i) acc[i] = 0.0f;
  const int ctid = (warp & 3) * 32 + lane;

  if (warp == 0) {
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, armed = 0, armed_par = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(&empty[stage], phase ^ 1, abort_flag, p.status, 51))
          break;
        mbar_arrive_expect_tx(&full[stage], L::STAGE);
        armed |= 1u << stage;
        armed_par = (armed_par & ~(1u << stage)) | (phase << stage);
        tma_load_3d(smR + stage * TILE_BYTES, &p.mr, &full[stage], kb * BK, 0,
                    r0);
        tma_load_3d(smT + stage * L::T_BYTES, &p.mt, &full[stage], kb * BK, 0,
                    t0);
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
      uint32_t stage = 0, phase = 0;
      int it = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++it) {
        const int buf = it % L::BUFS;
        if (!mbar_wait(&tempty[buf], ((it / L::BUFS) & 1) ^ 1, abort_flag,
                       p.status, 52) ||
            !mbar_wait(&full[stage], phase, abort_flag, p.status, 53))
          break;
        tc_fence_after();
        const uint32_t a0 = smem_u32(smR + stage * TILE_BYTES);
        const uint32_t b0 = smem_u32(smT + stage * L::T_BYTES);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          tc_mma_f8(tmem_base + buf * BNT,
                    smem_desc_sw128(a0 + kk * 32, 16, 1024),
                    smem_desc_sw128(b0 + kk * 32, 16, 1024), IDESC, kk != 0);
        tc_commit(&empty[stage]);
        tc_commit(&tfull[buf]);
        if (++stage == L::STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
      // every commit lands before the barriers' memory is used again
      volatile int no_abort = 0;
      tc_commit(drain);
      mbar_wait(drain, 0, &no_abort, nullptr, 0);
    }
  } else {
    const int r = r0 + ctid;
    float* myrows = scales + (warp - 2) * SLOTS * (32 + BNT);   // [SLOTS][32]
    float* mycols = myrows + SLOTS * 32;                        // [SLOTS][BNT]
    auto fetch = [&](int kb) {
      if (kb < kb1) {
        const int slot = (kb - kb0) & (SLOTS - 1);
        const float* pr = p.sr + kb * p.ldsr;
        const float* pt = p.st + kb * p.ldst;
        cp_async4(myrows + slot * 32 + lane,
                  pr + (r < p.R ? (p.r_row ? r : r / BM) : 0), r < p.R);
#pragma unroll
        for (int j = 0; j < (BNT + 31) / 32; ++j) {
          const int t = t0 + 32 * j + lane;
          if (32 * j + lane < BNT)
            cp_async4(mycols + slot * BNT + 32 * j + lane,
                      pt + (t < p.T ? (p.t_row ? t : t / BM) : 0), t < p.T);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < SLOTS - 1; ++i) fetch(kb0 + i);
    const uint32_t taddr0 =
        tmem_base + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    int it = 0;
    for (int kb = kb0; kb < kb1; ++kb, ++it) {
      const int buf = it % L::BUFS;
      cp_async_wait<SLOTS - 2>();   // this block's group is complete
      __syncwarp();   // for every lane's, and the last block's are read
      const float a0 = myrows[(it & (SLOTS - 1)) * 32 + lane];
      const float* cs = mycols + (it & (SLOTS - 1)) * BNT;
      fetch(kb + SLOTS - 1);
      if (!mbar_wait_warp(&tfull[buf], (it / L::BUFS) & 1, abort_flag,
                          p.status, 54))
        break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < BNT / 16; ++c) {
        uint32_t v[16];
        tmem_ld16(taddr0 + buf * BNT + c * 16, v);
        tmem_ld_wait16(v);
        if (c == BNT / 16 - 1) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&tempty[buf]);
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
          const float4 w = *reinterpret_cast<const float4*>(cs + c * 16 + i);
          float* d = acc + c * 16 + i;
          d[0] = fmaf(__uint_as_float(v[i]), a0 * w.x, d[0]);
          d[1] = fmaf(__uint_as_float(v[i + 1]), a0 * w.y, d[1]);
          d[2] = fmaf(__uint_as_float(v[i + 2]), a0 * w.z, d[2]);
          d[3] = fmaf(__uint_as_float(v[i + 3]), a0 * w.w, d[3]);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, L::COLS);

  auto store = [&](int r, int t, float v) {
    const int64_t at = r * p.cr + t * p.ct;
    if (OUT_F32)
      static_cast<float*>(p.c)[at] = v;
    else
      static_cast<__nv_bfloat16*>(p.c)[at] = __float2bfloat16_rn(v);
  };
  if (p.split == 1) {
    if (warp >= 2 && r0 + ctid < p.R) {
#pragma unroll
      for (int i = 0; i < BNT; ++i)
        if (t0 + i < p.T) store(r0 + ctid, t0 + i, acc[i]);
    }
    return;
  }
  // The cluster's parts: rank j adds up columns [j·w, (j + 1)·w) of the tile;
  // every CTA hands it its own through j's shared memory, [rank][column][row]
  // over the operand ring, which is free once every CTA's copies and MMAs are
  // done (the barrier).
  const int w = (BNT + p.split - 1) / p.split;
  cluster_sync();
  if (warp >= 2) {
    const uint32_t mine = smem_u32(smem);
#pragma unroll
    for (int i = 0; i < BNT; ++i) {
      const int j = i / w;
      if (t0 + i < p.T) {
        uint32_t dst;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(dst)
                     : "r"(mine), "r"(j));
        dst += ((uint32_t)(part * w + i - j * w) * BM + ctid) * 4;
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst), "f"(acc[i])
                     : "memory");
      }
    }
  }
  cluster_sync();
  if (warp >= 2 && r0 + ctid < p.R) {
    const float* in = reinterpret_cast<const float*>(smem);
    for (int i = 0; i < w; ++i) {
      const int col = part * w + i;
      if (col >= BNT || t0 + col >= p.T) break;
      float v = 0.0f;
      for (int k = 0; k < p.split; ++k) v += in[(k * w + i) * BM + ctid];
      store(r0 + ctid, t0 + col, v);
    }
  }
}

// ==================================================================== host ==
bool operand_map(CUtensorMap* m, const uint8_t* q, int64_t rows, int64_t K,
                 int64_t ld, uint32_t box_rows) {
  return encode_tmap_3d_u8(m, q, K, 1, rows, ld, ld, BK, 1, box_rows);
}

constexpr int kMaxDevices = 64;

// Attributes of a kernel, set once per device.
template <typename K>
int prepare_kernel(K kernel, int smem, bool (&done)[kMaxDevices]) {
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev >= 0 && dev < kMaxDevices && done[dev]) return cudaSuccess;
  err = cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[dev] = true;
  return err;
}

template <int B_ROW, int OUT_F32>
int launch_wide(const Params& prm, cudaStream_t s) {
  static bool done[kMaxDevices];
  static int clusters[kMaxDevices];
  auto kernel = gemm_fp8_block_wide<B_ROW, OUT_F32>;
  int err = prepare_kernel(kernel, WIDE_SMEM, done);
  if (err) return err;
  int dev = 0;
  if ((err = cudaGetDevice(&dev))) return err;
  int ncl = dev < kMaxDevices ? clusters[dev] : 0;
  if (ncl == 0) {
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
    if (dev < kMaxDevices) clusters[dev] = ncl;
  }
  const int grid = 2 * std::min(prm.total_tiles, ncl);
  kernel<<<grid, WIDE_THREADS, WIDE_SMEM, s>>>(prm);
  return cudaGetLastError();
}

template <int BNT, int OUT_F32>
int launch_narrow(const NarrowParams& prm, unsigned grid, cudaStream_t s) {
  static bool done[kMaxDevices];
  auto kernel = gemm_fp8_block_narrow<BNT, OUT_F32>;
  const int err = prepare_kernel(kernel, Narrow<BNT>::SMEM, done);
  if (err) return err;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(NARROW_THREADS);
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
  p.b_row = g.b_group == kFp8Row;
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
  if (g.out_f32)
    return p.b_row ? launch_wide<1, 1>(p, s) : launch_wide<0, 1>(p, s);
  return p.b_row ? launch_wide<1, 0>(p, s) : launch_wide<0, 0>(p, s);
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
  p.cr = 1;
  p.ct = g.ldc;
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

}  // namespace

int gemm_fp8_block(const GemmFp8Block& g, void* stream, unsigned* status) {
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t kblocks = (g.K + BK - 1) / BK;
  int err;
  {
    ProfScope ps(s, KF_GEMM_TC_FP8, 2.0 * g.M * g.N * g.K,
                 (double)(g.M + g.N) * g.K + (g.out_f32 ? 4.0 : 2.0) * g.M * g.N);
    if (g.M <= 128) {
      const int bn = g.M <= 16 ? 16 : g.M <= 32 ? 32 : g.M <= 64 ? 64 : 128;
      const int64_t tiles = (g.N + BM - 1) / BM;
      int split = 1;
      while (split < 8 && split * 2 <= kblocks &&
             tiles * split * 2 <= 2 * device_sm_count())
        split *= 2;
      err = narrow(g, s, status, bn, split);
    } else {
      err = wide(g, s, status);
    }
  }
  if (err) return err;
  count_launch();
  return cudaSuccess;
}

}  // namespace tp
