// block_gemm.cuh -- products of e4m3 codes whose scales change every 128 terms of the sum, on
// the 5th-generation tensor cores, for batches of many rows:
//
//   C[m,n] = sum_b SA[b, m] * SB[b, n/128] * ( sum_{r in block b} A(m,r) * B(n,r) )
//
// with b the blocks of 128 along the reduction.  Uses of it (codes q, scales S of
// block_quant.cuh):
//   y  = x W^T       A = row codes of x [T,K]       B = tile codes of W [N,K]   both K-major
//   dx = dy W        A = row codes of dy [T,N]      B = tile codes of W [N,K]   B MN-major
//   dW = dy^T x      A = tile codes of dy [T,N]     B = tile codes of x [T,K]   both MN-major
// so a weight is read in its one stored layout in both directions, and nothing is transposed.
// The rows of A may be split into groups, each with its own B (the experts of a layer).
//
// The scales do not commute with the sum, and they are arbitrary fp32 numbers, so the tensor
// cores' accumulator holds one block (128 terms) at a time: while the MMAs of block b+1 fill
// one of the two 256-column TMEM accumulators, the eight epilogue warps read block b out of
// the other (tcgen05.ld) and add it, times its scale, to fp32 sums in registers (128 a thread).
// A sum of 128 e4m3 products and the fp32 sum over the blocks are the only accumulations.
//
// Design (sm_100a): persistent clusters of two CTAs, 256 x 256 output tiles,
// tcgen05.mma.cta_group::2 kind::f8f6f4 (M = 256, N = 256, K = 32), a ring of four 32 KB stages
// filled by TMA (no multicast).  Warps: 0 loads A and B and arms the leader's barrier,
// 1 lays out the groups' tiles, allocates TMEM and (leader lane 0) issues the MMAs, 3 holds the
// products of the scales ready in shared memory, 4..11 are the
// epilogue: warp w reads TMEM lanes 32*(w%4).. and columns 128*((w-4)/4)...
// A thread's row is fixed and its 128 columns share one B scale, so a block costs it 64 packed
// FMAs (fma.rn.f32x2) with one scalar factor.  The registers are split 72 / 208 between the first
// four warps and the epilogue (setmaxnreg): 128 * 72 + 256 * 208 = 62,464 of the 64,512 that the
// CTA starts with.  With 128 sums a thread, 32 values on their way out of TMEM spilled in the
// loop; two sets of 16, one loading while the other is added, do not.
//
// Gated form (kOut = kOutGated, an expert's first product): a tile holds 128 hidden features,
// each CTA's 128 rows of B being 64 rows of the gate weight and the same 64 of the up weight,
// so that a thread ends with g and u of the same 64 features of its row.  h = silu(g) * u is
// formed in fp32, the row's maximum over the 128 features joined between the two threads that
// hold it, and h leaves as e4m3 row codes and scales.  g and u go to memory (fp32) only for a
// backward that will read them.
#pragma once

#include "block_quant.cuh"
#include "common.cuh"
#include "gemm.cuh"

namespace i8 {
namespace blk {

constexpr int TM = 256, TN = 256, HM = 128, HN = 128;
constexpr int BK = 128;                       // reduction terms (bytes) per stage = one block
constexpr int STAGES = 4;
constexpr int A_BYTES = HM * BK;
constexpr int STAGE_BYTES = A_BYTES + HN * BK;
constexpr int THREADS = 384;
constexpr int EPI_WARP0 = 4;
constexpr int REGS_LOW = 72, REGS_EPI = 208;
constexpr int REGS_NEEDED = (128 * REGS_LOW + 256 * REGS_EPI + THREADS - 1) / THREADS;
constexpr uint32_t TMEM_COLS = 512;
constexpr int GROUP_M = 16;                   // m-tiles per raster group
constexpr int MAX_GROUPS = 512;
constexpr int CST_WARP = 4 * 32 * 64;         // output staging of a warp: 32 rows x 128 16-bit columns
constexpr int CST_BYTES = 8 * CST_WARP;
constexpr int AUX_BYTES = 2 * 2 * 128 * 4;    // bias of the tile's columns, or row maxima
constexpr int PRE_BYTES = 2064;               // m-tiles before each group
constexpr int SLOTS = 8;                      // blocks whose scales are held ready
constexpr int SCALE_BYTES = SLOTS * 2 * HM * 4;
constexpr int BAR_BYTES = 512;
constexpr size_t SMEM_BYTES = static_cast<size_t>(STAGES) * STAGE_BYTES + CST_BYTES + AUX_BYTES +
                              PRE_BYTES + SCALE_BYTES + BAR_BYTES + 1024;
static_assert(SMEM_BYTES <= 232448, "shared memory per CTA");
static_assert(PRE_BYTES >= (MAX_GROUPS + 1) * 4, "group prefix");

enum { kOutF16 = 0, kOutBf16 = 1, kOutF32 = 2, kOutGated = 3 };

struct GemmArgs {
  int M, Nc;                    // rows of A in all groups; output columns
  int k_blocks, n_tiles;
  int groups;                   // 1 with offsets NULL: one group of all M rows
  const int32_t* offsets;       // [groups + 1] first row of each group
  int blocks_per_z, z_per_group;   // B's third coordinate: group * z_per_group + block / blocks_per_z
  const float* SA;              // SA[block * sa_pitch + (row >> sa_shift)]
  int64_t sa_pitch;
  int sa_shift;
  const float* SB;              // SB[group * sb_group + block * sb_block + (col / 128) * sb_col]
  int64_t sb_group, sb_block, sb_col;
  const uint16_t* bias;         // [Nc] in the output's type, or NULL
  void* C;
  int64_t ldc;
  bool c_tma;                   // 16-bit output whose rows start on 16 bytes: written by TMA
  // gated form: codes [M][h_pitch] and scales [ceil(Nc/128)][M] of h; g and u in fp32,
  // [M][2][Nc], when GU is not NULL.  Nc = hidden features.
  uint8_t* H;
  int64_t h_pitch;
  float* SH;
  float* GU;
  uint64_t wait_limit_ns;
};

struct SmemBars {
  uint64_t full[STAGES];
  uint64_t empty[STAGES];     // a block's MMAs are done: its stage is free, its sums are in TMEM
  uint64_t tmem_empty[2];
  uint64_t scaled[SLOTS];     // the block's scales are in its slot
  uint64_t unscaled[SLOTS];   // the epilogue is done with them
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};
static_assert(sizeof(SmemBars) <= BAR_BYTES, "barrier block");

__device__ __forceinline__ void epi_bar256() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

// Arrive on the pair leader's barrier, ordered as the reads of TMEM before it are (they have
// completed: tcgen05.wait::ld, then the tcgen05 fence).  The release is at CTA scope: nothing in
// memory is handed over, and a release at cluster scope waits for the thread's outstanding
// memory operations every time (it was the warps' largest stall: 2.78 ms against 1.71 at
// 2048 x 12288 x 49152).
__device__ __forceinline__ void arrive_leader(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns of TMEM into 16 registers; and the wait for it,
// declared to produce them, so that no use comes before it.
__device__ __forceinline__ void tmem_ld_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld_x16_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
        "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
      :
      : "memory");
}

// two fp32 numbers in a register pair: the same value twice, and d * s + a of each
__device__ __forceinline__ uint64_t pair2(float v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint32_t d0, uint32_t d1, uint64_t s, uint64_t a) {
  uint64_t r;
  asm("{\n\t.reg .b64 d;\n\t"
      "mov.b64 d, {%1, %2};\n\t"
      "fma.rn.f32x2 %0, d, %3, %4;\n\t}"
      : "=l"(r) : "r"(d0), "r"(d1), "l"(s), "l"(a));
  return r;
}

__device__ __forceinline__ uint4 lds_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint16_t lds_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
}

// every bulk store of this thread has read its shared-memory source
__device__ __forceinline__ void bulk_wait_read_0() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

// sigmoid(g) for silu(g) = g * sigmoid(g), within a few units in the last place of fp32.  Below g =
// -87.3, where the sigmoid is smaller than 2^-126, it comes out as 0 (the quick division gives 0
// for divisors above 2^126, an infinite exp(-g) among them): g * 0 = -0, the limit.
__device__ __forceinline__ float fast_sigmoid(float g) { return __fdividef(1.0f, 1.0f + expf(-g)); }

// 64 bytes a thread (16 fp32 or 32 16-bit columns of its row) of a warp's 32 rows through 2 KB of
// shared memory, so that four lanes write 64 bytes of one row; written by themselves, a thread's 16
// bytes lie a row apart from the next thread's.  base: row 0, first column; of a row's 64 bytes the
// first `valid` exist (a multiple of 16, or none), of the 32 rows the first `rows`.
__device__ __forceinline__ void store_rows(uint32_t stage, const uint32_t (&o)[16], void* base, int64_t ld_bytes, int valid,
                                           int rows) {
  const int lane = lane_id();
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 4; ++j)
    gemm::sts_v4(stage + static_cast<uint32_t>(lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)), o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
  __syncwarp();
  const int j = lane & 3;
  uint4 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2);
    x[i] = lds_v4(stage + static_cast<uint32_t>(r * 64 + ((j ^ ((r >> 1) & 3)) << 4)));
  }
  uint8_t* dst = static_cast<uint8_t*>(base) + (lane >> 2) * ld_bytes + 16 * j;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (i * 8 + (lane >> 2) < rows && 16 * j < valid) *reinterpret_cast<uint4*>(dst + i * 8 * ld_bytes) = x[i];
}
__device__ __forceinline__ void store16_f32(uint32_t stage, const float* v, float* base, int64_t ld, int col, int n, int rows) {
  uint32_t o[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(v[j]);
  store_rows(stage, o, base + col, ld * 4, (n - col) * 4, rows);
}

// position of tile t of a group of m_tiles x n_tiles: GROUP_M m-tiles, then the next n-tile
__device__ __forceinline__ void raster(int t, int m_tiles, int n_tiles, int& mt, int& nt) {
  const int G = m_tiles < GROUP_M ? m_tiles : GROUP_M;
  const int group = t / (G * n_tiles);
  const int r = t - group * (G * n_tiles);
  const int mb = group * G;
  const int rows = (m_tiles - mb) < G ? (m_tiles - mb) : G;
  mt = mb + r % rows;
  nt = r / rows;
}

// Shared-memory descriptors of the 128-byte-swizzled operand tiles (K-major, and MN-major with
// 128 elements of m or n in a row): the low word holds the address, the high word is the same
// for every tile: 1024 bytes between groups of 8 rows, version 1, 128-byte swizzle.
constexpr uint32_t DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
template <bool kMN>
__device__ __forceinline__ uint32_t desc_lo(uint32_t smem_addr) {
  return ((smem_addr & 0x3FFFFu) >> 4) | ((kMN ? (8192u >> 4) : 1u) << 16);
}

// D[tmem] (+)= A[smem] B[smem]^T over the CTA pair, issued by the lane with lead != 0.
__device__ __forceinline__ void umma_lead(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                          uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %6};\n\t"
      "mov.b64 db, {%2, %6};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(lead), "r"(DESC_HI)
      : "memory");
}
// The lead lane's MMAs so far done: one arrival on the barrier at `bar` of both CTAs.
__device__ __forceinline__ void commit_lead(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;\n\t}" ::"r"(bar),
      "h"(gemm::PAIR_MASK), "r"(lead)
      : "memory");
}

template <bool kAMN, bool kBMN, int kOut>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    block_gemm_kernel(const __grid_constant__ CUtensorMap tmA,
                      const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmC, const GemmArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t ring = raw_s + pad;
  const uint32_t cstage = ring + static_cast<uint32_t>(STAGES * STAGE_BYTES);
  float* aux = reinterpret_cast<float*>(smem + static_cast<size_t>(STAGES) * STAGE_BYTES + CST_BYTES);
  int* pre = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(aux) + AUX_BYTES);
  float* slots = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(pre) + PRE_BYTES);
  SmemBars* bars = reinterpret_cast<SmemBars*>(reinterpret_cast<uint8_t*>(slots) + SCALE_BYTES);
  // the warp's number as one value for the warp: what follows from it stays in uniform registers
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);
  const int lane = threadIdx.x & 31;
  const uint32_t rank = gemm::cluster_rank();
  volatile int* abort_flag = &bars->abort_flag;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&bars->full[s]), 1);
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(smem_u32(&bars->tmem_empty[b]), 16);   // 8 epilogue warps x 2 CTAs
    }
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(smem_u32(&bars->scaled[i]), 1);
      mbar_init(smem_u32(&bars->unscaled[i]), 8);    // this CTA's epilogue warps
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (a.c_tma) tma_prefetch_desc(&tmC);
  }
  if (warp == 1) {
    gemm::tmem_alloc_pair(smem_u32(&bars->tmem_base), TMEM_COLS);
    gemm::tmem_relinquish_pair();
  }
  grid_dep_wait();
  grid_dep_launch();
  if (warp == 1) {
    // m-tiles before each group: every lane sums its run of groups, then a scan over lanes
    if (a.offsets == nullptr) {
      if (lane == 0) {
        pre[0] = 0;
        pre[1] = (a.M + TM - 1) / TM;
      }
    } else {
      const int per = (a.groups + 31) / 32;
      const int g0 = min(lane * per, a.groups), g1 = min(g0 + per, a.groups);
      int sum = 0;
      for (int g = g0; g < g1; ++g) sum += (__ldg(a.offsets + g + 1) - __ldg(a.offsets + g) + TM - 1) / TM;
      int run = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += x;
      }
      if (lane == 31) pre[a.groups] = run;
      run -= sum;
      for (int g = g0; g < g1; ++g) {
        pre[g] = run;
        run += (__ldg(a.offsets + g + 1) - __ldg(a.offsets + g) + TM - 1) / TM;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  gemm::cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, bars->tmem_base, 0);

  const int KB = a.k_blocks;
  const int num_tiles = __shfl_sync(0xffffffffu, pre[a.groups] * a.n_tiles, 0);
  const int cluster_id = blockIdx.x >> 1;
  const int num_clusters = gridDim.x >> 1;
  const uint64_t lim = a.wait_limit_ns;
  // tile t: its group, first row, the end of the group's rows, and its n-tile
  auto tile_at = [&](int t, int& g, int& row0, int& row_end, int& nt) {
    int lo = 0, hi = a.groups - 1;                // the last group whose first tile is <= t
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] * a.n_tiles <= t) lo = mid; else hi = mid - 1;
    }
    g = lo;
    const int m_tiles = pre[g + 1] - pre[g];
    int mt;
    raster(t - pre[g] * a.n_tiles, m_tiles, a.n_tiles, mt, nt);
    row0 = mt * TM;
    row_end = a.M;
    if (a.offsets != nullptr) {
      row0 += __ldg(a.offsets + g);
      row_end = __ldg(a.offsets + g + 1);
    }
  };

  if (warp < EPI_WARP0) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_LOW));
    if (warp == 0) {
      if (lane == 0) {
        // -------------------------------------------------------------- TMA producer
        const uint32_t full_leader0 = gemm::map_to_rank(smem_u32(&bars->full[0]), 0);
        int s = 0;
        uint32_t ph = 0, issued = 0;
        bool ok = true;
        for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
          int g, row0, row_end, nt;
          tile_at(t, g, row0, row_end, nt);
          const int m0 = row0 + static_cast<int>(rank) * HM;
          const int n0 = nt * TN + static_cast<int>(rank) * HN;
          const int z0 = g * a.z_per_group;
          int zb = 0, kz = 0;                       // block / blocks_per_z, block % blocks_per_z
          for (int kb = 0; kb < KB; ++kb) {
            if (!mbar_wait(smem_u32(&bars->empty[s]), ph ^ 1u, abort_flag, lim)) {
              ok = false;
              break;
            }
            const uint32_t da = ring + s * STAGE_BYTES, db = da + A_BYTES;
            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&bars->full[s]), 2 * STAGE_BYTES);
            const uint32_t fb = full_leader0 + static_cast<uint32_t>(s) * 8u;
            if (kAMN)
              gemm::tma_load_2d_pair(da, &tmA, fb, m0, kb * BK);
            else
              gemm::tma_load_2d_pair(da, &tmA, fb, kb * BK, m0);
            if (kOut == kOutGated) {
              const int i0 = nt * HN + static_cast<int>(rank) * 64;
              gemm::tma_load_3d_pair(db, &tmB, fb, kb * BK, i0, z0);
              gemm::tma_load_3d_pair(db + 8192u, &tmB, fb, kb * BK, i0, z0 + 1);
            } else if (kBMN) {
              gemm::tma_load_3d_pair(db, &tmB, fb, n0, kz * BK, z0 + zb);
              if (++kz == a.blocks_per_z) {
                kz = 0;
                ++zb;
              }
            } else {
              gemm::tma_load_3d_pair(db, &tmB, fb, kb * BK, n0, z0);
            }
            ++issued;
            if (++s == STAGES) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
        if (!ok && rank == 0) {
          // wind down: wait (bounded, ignoring the abort flag) for the copies in flight
          int no_abort = 0;
          const uint32_t inflight = issued < STAGES ? issued : STAGES;
          for (uint32_t i = 0; i < inflight; ++i) {
            const uint32_t u = issued - 1 - i;
            mbar_wait(smem_u32(&bars->full[u % STAGES]), (u / STAGES) & 1u, &no_abort, lim);
          }
        }
      }
    } else if (warp == 1) {
      if (rank == 0) {
        // -------------------------------------------------------------- MMA issuer
        // The whole warp walks the loop, so that descriptors and addresses are uniform values;
        // lane 0 alone issues.  (With one lane in the loop every MMA and commit took about 70
        // cycles to issue, 600 to 780 a block against the 512 that its MMAs run.)
        constexpr uint32_t ID = idesc_e4m3_f32(TM, TN) | (kAMN ? (1u << 15) : 0u) | (kBMN ? (1u << 16) : 0u);
        const uint32_t lead = lane == 0 ? 1u : 0u;
        const uint32_t a0 = desc_lo<kAMN>(ring), b0 = desc_lo<kBMN>(ring + A_BYTES);
        int s = 0;
        uint32_t ph = 0, n = 0;                     // n: blocks issued so far
        bool ok = true;
        for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
          for (int kb = 0; kb < KB; ++kb, ++n) {
            const uint32_t b = n & 1u;
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->tmem_empty[b]), ((n >> 1) & 1u) ^ 1u, abort_flag, lim) &&
                                             mbar_wait(smem_u32(&bars->full[s]), ph, abort_flag, lim))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t so = static_cast<uint32_t>(s) * (STAGE_BYTES >> 4);
#pragma unroll
            for (int kk = 0; kk < BK / 32; ++kk)
              // 32 terms further: 32 bytes along a K-major row, 32 rows of 128 bytes otherwise
              umma_lead(tmem_base + b * TN, a0 + so + kk * (kAMN ? 256 : 2), b0 + so + kk * (kBMN ? 256 : 2), ID,
                        kk != 0, lead);
            commit_lead(smem_u32(&bars->empty[s]), lead);
            if (++s == STAGES) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
        int no_abort = 0;
        commit_lead(smem_u32(&bars->drain), lead);
        mbar_wait(smem_u32(&bars->drain), 0u, &no_abort, lim);
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------------- scales
      // SA * SB of every block, for the 128 rows of this CTA and both halves of the columns (gate
      // and up in the gated form), into one of SLOTS slots.  The epilogue has no load of its own
      // in its loop: with the loads there, one block ahead, it took 888 cycles a block, with
      // constants in their place 740.
      constexpr int AHEAD = 4;                      // blocks loaded together
      uint32_t n = 0;                               // blocks so far
      bool ok = true;
      for (int t = cluster_id; t < num_tiles && ok; t += num_clusters) {
        int g, row0, row_end, nt;
        tile_at(t, g, row0, row_end, nt);
        const int r0 = row0 + static_cast<int>(rank) * HM + lane;
        const float* sb0 = a.SB + g * a.sb_group;
        const float* sb1;
        if (kOut == kOutGated) {
          sb0 += nt * a.sb_col;
          sb1 = sb0 + (a.sb_group >> 1);
        } else {
          const int c1 = nt * TN + HN < a.Nc ? 2 * nt + 1 : 2 * nt;   // a half past the last column: any scale
          sb1 = sb0 + c1 * a.sb_col;
          sb0 += 2 * nt * a.sb_col;
        }
        int64_t ra[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) ra[i] = min(r0 + 32 * i, a.M - 1) >> a.sa_shift;
        for (int k0 = 0; k0 < KB && ok; k0 += AHEAD) {
          float va[AHEAD][4], vb[AHEAD][2];
#pragma unroll
          for (int u = 0; u < AHEAD; ++u)
            if (k0 + u < KB) {
              const float* p = a.SA + static_cast<int64_t>(k0 + u) * a.sa_pitch;
#pragma unroll
              for (int i = 0; i < 4; ++i) va[u][i] = __ldg(p + ra[i]);
              vb[u][0] = __ldg(sb0 + (k0 + u) * a.sb_block);
              vb[u][1] = __ldg(sb1 + (k0 + u) * a.sb_block);
            }
#pragma unroll
          for (int u = 0; u < AHEAD; ++u) {
            if (k0 + u >= KB || !ok) break;
            const uint32_t slot = n & (SLOTS - 1);
            ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->unscaled[slot]), ((n / SLOTS) & 1u) ^ 1u, abort_flag, lim));
            if (!ok) break;
            float* dst = slots + slot * (2 * HM) + lane;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              dst[32 * i] = va[u][i] * vb[u][0];
              dst[HM + 32 * i] = va[u][i] * vb[u][1];
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bars->scaled[slot]));
            ++n;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_EPI));
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int half = (warp - EPI_WARP0) >> 2;       // which 128 columns
    const int et = threadIdx.x - EPI_WARP0 * 32;    // 0..255
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(half * HN);
    const uint32_t cst = cstage + static_cast<uint32_t>((warp - EPI_WARP0) * CST_WARP);
    const uint32_t empty_leader0 = gemm::map_to_rank(smem_u32(&bars->tmem_empty[0]), 0);
    uint32_t n = 0;
    int s = 0;                                      // the block's ring stage, as the issuer's
    uint32_t ph = 0;
    int parity = 0;
    // after a wait that ran out, a warp keeps walking the tiles (it must meet the others at
    // the named barrier) but touches TMEM and memory no more
    bool dead = false;
    for (int t = cluster_id; t < num_tiles; t += num_clusters, parity ^= 1) {
      int g, row0, row_end, nt;
      tile_at(t, g, row0, row_end, nt);
      const int wrow0 = row0 + static_cast<int>(rank) * HM + q * 32;   // the warp's first row
      const int row = wrow0 + lane;
      const bool row_ok = row < row_end;
      const int n0 = nt * TN + half * HN;
      if (kOut != kOutGated) {
        const int c = nt * TN + et;
        float bv = 0.0f;
        if (a.bias != nullptr && c < a.Nc)
          bv = kOut == kOutBf16 ? load16<true>(a.bias + c) : load16<false>(a.bias + c);
        aux[parity * 256 + et] = bv;
        epi_bar256();
      }
      // sums of the thread's 128 columns, two to a register pair (fma.rn.f32x2)
      uint64_t acc2[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) acc2[j] = 0ull;
      for (int kb = 0; kb < KB && !dead; ++kb, ++n) {
        const uint32_t b = n & 1u;
        const bool got = mbar_wait(smem_u32(&bars->scaled[n & (SLOTS - 1)]), (n / SLOTS) & 1u, abort_flag, lim) &&
                         mbar_wait(smem_u32(&bars->empty[s]), ph, abort_flag, lim);
        const float* sc = slots + (n & (SLOTS - 1)) * (2 * HM) + q * 32 + lane;
        const uint64_t s0 = pair2(sc[kOut == kOutGated ? 0 : half * HM]);
        const uint64_t s1 = kOut == kOutGated ? pair2(sc[HM]) : s0;
        if (!__all_sync(0xffffffffu, got)) {
          dead = true;
          break;
        }
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
        tc_fence_after();
        const uint32_t tb = lane_base + b * TN;
        // 16 columns at a time: the next 16 are on their way while these are added
        uint32_t r[2][16];
        tmem_ld_x16(tb, r[0]);
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          tmem_ld_x16_wait(r[c & 1]);
          if (c < 7) tmem_ld_x16(tb + static_cast<uint32_t>((c + 1) * 16), r[(c + 1) & 1]);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            acc2[c * 8 + j] = fma2(r[c & 1][2 * j], r[c & 1][2 * j + 1], c >= 4 ? s1 : s0, acc2[c * 8 + j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          arrive_leader(empty_leader0 + b * 8u);
          mbar_arrive(smem_u32(&bars->unscaled[n & (SLOTS - 1)]));
        }
      }
      float acc[128];
#pragma unroll
      for (int j = 0; j < 64; ++j) {
        acc[2 * j] = __uint_as_float(static_cast<uint32_t>(acc2[j]));
        acc[2 * j + 1] = __uint_as_float(static_cast<uint32_t>(acc2[j] >> 32));
      }
      if (kOut == kOutGated) {
        // acc[0..63] = g, acc[64..127] = u of features i0 .. i0 + 63
        const int i0 = nt * HN + half * 64;
        float am = 0.0f;
        if (a.GU != nullptr && !dead) {
#pragma unroll
          for (int j = 0; j < 128; j += 16)
            store16_f32(cst, &acc[j], a.GU + static_cast<int64_t>(wrow0) * 2 * a.Nc + (j >> 6) * a.Nc, 2 * static_cast<int64_t>(a.Nc),
                        i0 + (j & 63), a.Nc, row_end - wrow0);
        }
#pragma unroll
        for (int j = 0; j < 64; ++j) {
          const float gv = acc[j];
          acc[j] = gv * fast_sigmoid(gv) * acc[64 + j];
          am = fmaxf(am, fabsf(acc[j]));
        }
        float* mx = aux + parity * 256;              // [half][128 rows of this CTA]
        mx[half * 128 + q * 32 + lane] = am;
        epi_bar256();
        am = fmaxf(fmaxf(am, mx[(half ^ 1) * 128 + q * 32 + lane]), kScaleFloor);
        if (row_ok && !dead) {
          const float up = block_up(am);
          uint4* dst = reinterpret_cast<uint4*>(a.H + static_cast<int64_t>(row) * a.h_pitch + i0);
#pragma unroll
          for (int j = 0; j < 64; j += 16) {
            const float f0[8] = {acc[j], acc[j + 1], acc[j + 2], acc[j + 3], acc[j + 4], acc[j + 5], acc[j + 6], acc[j + 7]};
            const float f1[8] = {acc[j + 8], acc[j + 9], acc[j + 10], acc[j + 11], acc[j + 12], acc[j + 13], acc[j + 14], acc[j + 15]};
            const uint2 x = codes8_scaled(f0, up), y = codes8_scaled(f1, up);
            dst[j >> 4] = make_uint4(x.x, x.y, y.x, y.y);
          }
          if (half == 0) a.SH[static_cast<int64_t>(nt) * a.M + row] = block_down(am);
        }
      } else if (!dead && n0 < a.Nc && wrow0 < row_end) {
        const float* bs = aux + parity * 256 + half * HN;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int c0 = n0 + c * 32;
          if (c0 >= a.Nc) continue;
          if constexpr (kOut == kOutF32) {
#pragma unroll
            for (int w = 0; w < 2; ++w)
              store16_f32(cst, &acc[c * 32 + w * 16], static_cast<float*>(a.C) + static_cast<int64_t>(wrow0) * a.ldc, a.ldc,
                          c0 + w * 16, a.Nc, row_end - wrow0);
          } else {
            uint32_t o[16];
#pragma unroll
            for (int j = 0; j < 16; ++j)
              o[j] = pack2<kOut == kOutBf16>(acc[c * 32 + 2 * j] + bs[c * 32 + 2 * j], acc[c * 32 + 2 * j + 1] + bs[c * 32 + 2 * j + 1]);
            if (a.c_tma) {
              // The warp's 32 x 128 columns wait in shared memory, four TMA stores of 32 x 32 (clipped by
              // the map) take them out while the next tile runs.  Stores that the warp waits for go at
              // the rate of all the SMs' tiles at once, 3500 cycles a tile.
              const uint32_t box = cst + static_cast<uint32_t>(c * 2048);
              if (c == 0) {
                if (lane == 0) bulk_wait_read_0();    // the last tile's have left
                __syncwarp();
              }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                gemm::sts_v4(box + static_cast<uint32_t>(lane * 64 + j * 16), o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
              gemm::fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                gemm::tma_store_2d(&tmC, box, c0, wrow0);
                gemm::bulk_commit();
              }
            } else {
              // rows that do not start on 16 bytes: the warp writes them one by one, a column a lane
              uint16_t* dst = static_cast<uint16_t*>(a.C) + static_cast<int64_t>(wrow0) * a.ldc + c0;
              const int rows = min(32, row_end - wrow0);
              __syncwarp();
#pragma unroll
              for (int j = 0; j < 4; ++j)
                gemm::sts_v4(cst + static_cast<uint32_t>(lane * 64 + j * 16), o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
              __syncwarp();
              if (c0 + lane < a.Nc)
#pragma unroll 8
                for (int r = 0; r < rows; ++r)
                  dst[static_cast<int64_t>(r) * a.ldc + lane] = lds_u16(cst + static_cast<uint32_t>(r * 64 + lane * 2));
            }
          }
        }
      }
    }
    if (lane == 0) gemm::bulk_wait_all();           // the stores are complete before the CTA ends
  }

  tc_fence_before();
  __syncthreads();
  gemm::cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    gemm::tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
  gemm::cluster_sync();
}

}  // namespace blk
}  // namespace i8
