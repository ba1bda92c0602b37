// block_skinny.cuh -- the forward product of block_gemm.cuh for batches of few rows (a decode
// batch, or the few tokens of each expert), where streaming the weight is all the time:
//
//   C[t,n] = sum_b SA[b, t] * SB[b, n/128] * ( sum_{r in block b} A(t,r) * B(n,r) )
//
// The roles of the operands are swapped: 128 rows of the weight are the tensor cores' M, and
// NT = 16..64 tokens their N, so that one token costs an MMA of N = 16 and not of M = 128.
// TMEM lanes are then output features and columns tokens; the weight's scale is one number for
// a whole tile and block, the tokens' scales differ by column and come through shared memory.
//
// The bound is HBM: each weight byte is read once.  To keep all SMs reading to the end, the
// (tile, block) units of the whole product are dealt out in equal contiguous runs, one run a
// CTA, whatever tile they fall in.  A tile that one CTA ran alone is written at once; the
// others leave fp32 partial sums in the workspace, and the CTA that arrives last (a counter)
// adds the parts of the tile in the order of the CTAs and writes it: the order of arrival
// changes nothing in the result, and no CTA waits for another.  Where whole tiles fill the SMs
// well enough by themselves, none is split.
//
// Design (sm_100a): one CTA an SM; warp 0 fills a ring of [128 x 128 weight | NT x 128 token]
// stages by TMA, warp 1 issues tcgen05.mma (cta_group::1, kind::f8f6f4, M = 128, N = NT), one
// block to one of NBUF small TMEM accumulators, warps 2..5 add them, scaled, to fp32 sums in
// registers, warp 6 holds the scales of the units ahead ready in shared memory (loaded by the
// epilogue itself, one unit ahead, they kept it waiting for memory every unit).  The weight does
// not depend on the kernel before (the quantiser of the tokens), so with a tile order known from
// the start the ring fills with weights while that kernel runs.  Measured: 4096 -> 16384, one
// token, 16 us (67 MB); 14336 -> 28672 75 us (411 MB, 5.5 TB/s).
#pragma once

#include "block_gemm.cuh"

namespace i8 {
namespace skinny {

using blk::BK;
using blk::MAX_GROUPS;
constexpr int ROWS = 128;                    // weight rows of a tile
constexpr int W_BYTES = ROWS * BK;
constexpr int X_WARPS = 8;                   // warps that form the tokens' codes (direct input)
__host__ __device__ constexpr int threads(int in) { return in == 0 ? 224 : (6 + X_WARPS) * 32; }
constexpr int PRE_BYTES = blk::PRE_BYTES;
constexpr int BAR_BYTES = 1024;
constexpr int MAX_STAGES = 12;
constexpr int NBUF = 4;                      // TMEM accumulators
constexpr int MIN_UNITS = 8;                 // units of a CTA: joining a tile's parts costs about as much
                                             // (4096 -> 4096, one token: 12.7 us; with 4: 15.0)
constexpr int RING_BUDGET = 210 * 1024;

__host__ __device__ constexpr int stage_bytes(int nt) { return W_BYTES + nt * BK; }
__host__ __device__ constexpr int stages(int nt) {
  return RING_BUDGET / stage_bytes(nt) < MAX_STAGES ? RING_BUDGET / stage_bytes(nt) : MAX_STAGES;
}
constexpr int SLOTS = 16;                    // units whose scales are held ready
__host__ __device__ constexpr int scale_bytes(int nt) { return SLOTS * nt * 4; }
__host__ __device__ constexpr size_t smem_bytes(int nt) {
  return static_cast<size_t>(stages(nt)) * stage_bytes(nt) + scale_bytes(nt) + PRE_BYTES + BAR_BYTES + 1024;
}
static_assert(smem_bytes(16) <= 232448 && smem_bytes(32) <= 232448 && smem_bytes(64) <= 232448, "shared memory per CTA");

// Where the tokens' codes come from: the quantiser's, by TMA; or, for tiles of 16 tokens, formed in
// the kernel by eight warps that take the units in turn and write codes and scales straight into
// the stage (128-byte swizzle): from the 16-bit rows of X, or from g and u as h = silu(g) * u.
// Every CTA forms the codes of its own units again, a few hundred instructions beside a weight
// tile that takes about 600 cycles to arrive, and the kernel that would have formed them once
// falls away: 5.5 us and its launch.
enum { kInCodes = 0, kInF16 = 1, kInBf16 = 2, kInGated = 3 };

struct Args {
  // direct input: rows [tokens][k_cols] of X, 16-bit, or GU [M][2][k_cols] fp32.  With groups, row
  // p of X is the token row_at[p] / copies; GU's rows are in order.
  const void* X;
  int64_t k_cols;
  const int32_t* row_at;
  int copies;
  int M;                        // rows (tokens) in all groups
  int k_blocks;
  int n_tiles, n_per_z;         // weight tiles of a group; of one z slice of it
  int z_cols;                   // output columns of one z slice
  int groups;
  const int32_t* offsets;       // as in GemmArgs
  int z_per_group;
  const float* SA;              // [k_blocks][M]: the scales of the quantiser's codes
  const float* SB;              // [z][n_per_z][k_blocks]
  const uint16_t* bias;         // [z_cols] in the output's type, or NULL (one z slice)
  void* C;                      // [M][ldc]
  int64_t ldc;
  float* parts;                 // [2 * grid][NT][128]
  unsigned int* arrived;        // [grid], zero at the start
  uint64_t wait_limit_ns;
};

struct SmemBars {
  uint64_t full[MAX_STAGES];
  uint64_t empty[MAX_STAGES];
  uint64_t tmem_full[NBUF];
  uint64_t tmem_empty[NBUF];
  uint64_t scaled[SLOTS];      // the unit's scales are in its slot
  uint64_t unscaled[SLOTS];    // the epilogue is done with them
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  unsigned int last;
};
static_assert(sizeof(SmemBars) <= BAR_BYTES, "barrier block");

// as blk::umma_lead and blk::commit_lead, for one CTA
__device__ __forceinline__ void umma_lead(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                          uint32_t accumulate, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 da, db;\n\t"
      "mov.b64 da, {%1, %6};\n\t"
      "mov.b64 db, {%2, %6};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], da, db, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(lead), "r"(blk::DESC_HI)
      : "memory");
}
__device__ __forceinline__ void commit_lead(uint32_t bar, uint32_t lead) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(lead)
      : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns of TMEM into 16 registers, and the wait for them.
__device__ __forceinline__ void tmem_ld_x16_wait(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void epi_bar128() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// clears the counters of a product that no other kernel goes before
__global__ void clear_kernel(unsigned int* zero) {
  grid_dep_launch();
  zero[threadIdx.x] = 0u;
}

template <int NT, int kOut, int kIn>
__global__ void __launch_bounds__(threads(kIn), 1)
    block_skinny_kernel(const __grid_constant__ CUtensorMap tmW,
                        const __grid_constant__ CUtensorMap tmX, const Args a) {
  static_assert(kIn == kInCodes ? NT > 16 && kOut != blk::kOutF32 : NT == 16, "forms that are launched");
  constexpr int STAGES = stages(NT);
  constexpr int SBYTES = stage_bytes(NT);
  constexpr uint32_t TMEM_COLS = NBUF * NT < 32 ? 32 : NBUF * NT;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t ring = raw_s + pad;
  float* sscale = reinterpret_cast<float*>(smem + static_cast<size_t>(STAGES) * SBYTES);
  int* pre = reinterpret_cast<int*>(reinterpret_cast<uint8_t*>(sscale) + scale_bytes(NT));
  SmemBars* bars = reinterpret_cast<SmemBars*>(reinterpret_cast<uint8_t*>(pre) + PRE_BYTES);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // uniform in the warp
  const int lane = threadIdx.x & 31;
  volatile int* abort_flag = &bars->abort_flag;
  const uint64_t lim = a.wait_limit_ns;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(smem_u32(&bars->full[s]), kIn == kInCodes ? 1 : 2);   // TMA, and the unit's x warp
      mbar_init(smem_u32(&bars->empty[s]), 1);
    }
    for (int b = 0; b < NBUF; ++b) {
      mbar_init(smem_u32(&bars->tmem_full[b]), 1);
      mbar_init(smem_u32(&bars->tmem_empty[b]), 4);
    }
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(smem_u32(&bars->scaled[i]), 1);
      mbar_init(smem_u32(&bars->unscaled[i]), 4);
    }
    mbar_init(smem_u32(&bars->drain), 1);
    bars->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmW);
    if (kIn == kInCodes) tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&bars->tmem_base), TMEM_COLS);
    tmem_relinquish();
  }
  const bool grouped = kIn != kInCodes && a.offsets != nullptr;
  if (grouped) {
    grid_dep_wait();
    grid_dep_launch();
  }
  if (warp == 2) {
    // token tiles before each group
    if (!grouped) {
      if (lane == 0) {
        pre[0] = 0;
        pre[1] = (a.M + NT - 1) / NT;
      }
    } else {
      const int per = (a.groups + 31) / 32;
      const int g0 = min(lane * per, a.groups), g1 = min(g0 + per, a.groups);
      int sum = 0;
      for (int g = g0; g < g1; ++g) sum += (__ldg(a.offsets + g + 1) - __ldg(a.offsets + g) + NT - 1) / NT;
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
        run += (__ldg(a.offsets + g + 1) - __ldg(a.offsets + g) + NT - 1) / NT;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, bars->tmem_base, 0);

  const int KB = a.k_blocks;
  const int64_t units = static_cast<int64_t>(__shfl_sync(0xffffffffu, pre[a.groups], 0)) * a.n_tiles * KB;
  // How many units there are is known only here, by the groups' sizes.  Where whole tiles, dealt out
  // to the CTAs in turn, keep at least 85 in 100 of them busy to the end, no tile is split;
  // otherwise G CTAs share the units, each at least MIN_UNITS unless there are fewer in all.  One
  // token, 16384 features, whole / split in us: 118 tiles (80 in 100) 50.3 / 49.5, 126 (85) 50.2 /
  // 52.6, 148 52.2 / 52.6; in two rounds 250 (84) 96.3 / 89.3, 280 (95) 96.1 / 98.9.  With 4096
  // features joining weighs more: 74 (50) 16.4 / 16.2, 104 (70) 17.5 / 21.6, 126 16.9 / 22.6.
  // CTAs past the last take no part in any tile.
  const int64_t tiles = units / KB, grid = gridDim.x;
  const bool whole = tiles > 0 && tiles * 100 >= (tiles + grid - 1) / grid * grid * 85;
  const int64_t most = whole ? tiles : units / MIN_UNITS > 0 ? units / MIN_UNITS : (units > 0 ? 1 : 0);
  const int64_t G = most < grid ? most : grid;
  auto first_unit = [&](int64_t c) -> int64_t { return whole ? tiles * c / G * KB : units * c / G; };
  const bool idle = static_cast<int64_t>(blockIdx.x) >= G;
  const int64_t u0 = idle ? 0 : first_unit(blockIdx.x);
  const int64_t u1 = idle ? 0 : first_unit(static_cast<int64_t>(blockIdx.x) + 1);
  // tile: its group, first token, end of the group's tokens, z slice and weight tile in it
  auto tile_at = [&](int tile, int& row0, int& row_end, int& z, int& nz) {
    int lo = 0, hi = a.groups - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (pre[mid] * a.n_tiles <= tile) lo = mid; else hi = mid - 1;
    }
    const int tt = pre[lo + 1] - pre[lo];
    const int r = tile - pre[lo] * a.n_tiles;
    const int nt = r / tt;                        // the token tiles of one weight tile in turn
    row0 = (r - nt * tt) * NT;
    row_end = a.M;
    if (grouped) {
      row0 += __ldg(a.offsets + lo);
      row_end = __ldg(a.offsets + lo + 1);
    }
    const int zz = nt / a.n_per_z;
    z = lo * a.z_per_group + zz;
    nz = nt - zz * a.n_per_z;
  };

  if (warp == 0) {
    if (lane == 0) {
      // ---------------------------------------------------------------- TMA producer
      // One pass over the run.  While the kernel before may still write the tokens' codes
      // (kInCodes), the first STAGES units get their weight half only; then the wait, their
      // token halves, and the rest of the run whole.
      const int64_t head = kIn != kInCodes ? 0 : (u1 - u0 < STAGES ? u1 - u0 : STAGES);
      auto issue = [&](int64_t u, int s, bool w, bool x, int& row0, int& z, int& nz, int& last_tile) {
        const int tile = static_cast<int>(u / KB);
        const int kb = static_cast<int>(u - static_cast<int64_t>(tile) * KB);
        if (tile != last_tile) {
          int row_end;
          tile_at(tile, row0, row_end, z, nz);
          last_tile = tile;
        }
        const uint32_t dst = ring + s * SBYTES;
        const uint32_t fb = smem_u32(&bars->full[s]);
        if (w) {
          mbar_arrive_expect_tx(fb, kIn == kInCodes ? SBYTES : W_BYTES);
          tma_load_3d(dst, &tmW, fb, kb * BK, nz * ROWS, z);
        }
        if (x && kIn == kInCodes) tma_load_2d(dst + W_BYTES, &tmX, fb, kb * BK, row0);
      };
      int row0 = 0, z = 0, nz = 0, last_tile = -1;
      for (int64_t i = 0; i < head; ++i) issue(u0 + i, static_cast<int>(i), true, false, row0, z, nz, last_tile);
      if (!grouped) {
        if (kIn == kInCodes) grid_dep_wait();
        grid_dep_launch();
      }
      last_tile = -1;
      for (int64_t i = 0; i < head; ++i) issue(u0 + i, static_cast<int>(i), false, true, row0, z, nz, last_tile);
      int s = static_cast<int>(head % STAGES);
      uint32_t ph = head == STAGES ? 1u : 0u;
      uint32_t issued = static_cast<uint32_t>(head);
      bool ok = true;
      for (int64_t u = u0 + head; u < u1; ++u) {
        if (!mbar_wait(smem_u32(&bars->empty[s]), ph ^ 1u, abort_flag, lim)) {
          ok = false;
          break;
        }
        issue(u, s, true, true, row0, z, nz, last_tile);
        ++issued;
        if (++s == STAGES) {
          s = 0;
          ph ^= 1u;
        }
      }
      if (!ok) {
        int no_abort = 0;
        const uint32_t inflight = issued < STAGES ? issued : STAGES;
        for (uint32_t i = 0; i < inflight; ++i) {
          const uint32_t u = issued - 1 - i;
          mbar_wait(smem_u32(&bars->full[u % STAGES]), (u / STAGES) & 1u, &no_abort, lim);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    // the whole warp walks the loop (uniform descriptors), lane 0 issues
    constexpr uint32_t ID = idesc_e4m3_f32(ROWS, NT);
    const uint32_t lead = lane == 0 ? 1u : 0u;
    const uint32_t w0 = blk::desc_lo<false>(ring), x0 = blk::desc_lo<false>(ring + W_BYTES);
    int s = 0;
    uint32_t ph = 0, n = 0;
    for (int64_t u = u0; u < u1; ++u, ++n) {
      const uint32_t b = n % NBUF;
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->tmem_empty[b]), ((n / NBUF) & 1u) ^ 1u, abort_flag, lim) &&
                                       mbar_wait(smem_u32(&bars->full[s]), ph, abort_flag, lim)))
        break;
      tc_fence_after();
      const uint32_t so = static_cast<uint32_t>(s) * (SBYTES >> 4);
#pragma unroll
      for (int kk = 0; kk < BK / 32; ++kk)
        umma_lead(tmem_base + b * NT, w0 + so + kk * 2, x0 + so + kk * 2, ID, kk != 0, lead);
      commit_lead(smem_u32(&bars->empty[s]), lead);
      commit_lead(smem_u32(&bars->tmem_full[b]), lead);
      if (++s == STAGES) {
        s = 0;
        ph ^= 1u;
      }
    }
    int no_abort = 0;
    commit_lead(smem_u32(&bars->drain), lead);
    mbar_wait(smem_u32(&bars->drain), 0u, &no_abort, lim);
  } else if (warp >= 6 && kIn != kInCodes) {
    // ------------------------------------------------------------------ token codes
    // Unit i of the run belongs to warp 6 + i % X_WARPS.  Eight lanes hold a token's block, 16
    // features each; the warp takes four tokens at a time, as many times as the tile has tokens.
    // Rows past the tile's tokens keep what the stage held: their columns are never read.
    const int xw = warp - 6;
    const int c = lane & 7;                         // 16-byte chunk of the token's codes
    int tile = -1, row0 = 0, row_end = 0, z = 0, nz = 0;
    uint32_t n = static_cast<uint32_t>(xw);
    for (int64_t u = u0 + xw; u < u1; u += X_WARPS, n += X_WARPS) {
      const int t = static_cast<int>(u / KB);
      const int kb = static_cast<int>(u - static_cast<int64_t>(t) * KB);
      if (t != tile) {
        tile_at(t, row0, row_end, z, nz);
        tile = t;
      }
      const float w = __ldg(a.SB + (static_cast<int64_t>(z) * a.n_per_z + nz) * KB + kb);
      const int64_t col = static_cast<int64_t>(kb) * BK + c * 16;
      const bool in = col < a.k_cols;               // k_cols % 16 == 0: a chunk is whole or absent
      const int turns = (min(row_end - row0, NT) + 3) >> 2;
      const int s = static_cast<int>(n % STAGES);
      const uint32_t xs = ring + s * SBYTES + W_BYTES;
      bool ok = true;
      uint4 raw[4][2];                              // X: every turn's values, loaded together
      if (kIn != kInGated) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int p = row0 + i * 4 + (lane >> 3);
          if (i < turns && p < row_end && in) {
            const int64_t token = a.row_at != nullptr ? __ldg(a.row_at + p) / a.copies : p;
            const uint16_t* x = static_cast<const uint16_t*>(a.X) + token * a.k_cols + col;
            raw[i][0] = ldg_v4(x);
            raw[i][1] = ldg_v4(x + 8);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= turns) break;
        const int r = i * 4 + (lane >> 3);
        const bool live = row0 + r < row_end;
        float f[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] = 0.0f;
        if (live && in) {
          if (kIn == kInGated) {
            const float* g = static_cast<const float*>(a.X) + static_cast<int64_t>(row0 + r) * 2 * a.k_cols + col;
            float4 gv[4], uv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              gv[j] = __ldg(reinterpret_cast<const float4*>(g) + j);
              uv[j] = __ldg(reinterpret_cast<const float4*>(g + a.k_cols) + j);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              f[4 * j] = gv[j].x * blk::fast_sigmoid(gv[j].x) * uv[j].x;
              f[4 * j + 1] = gv[j].y * blk::fast_sigmoid(gv[j].y) * uv[j].y;
              f[4 * j + 2] = gv[j].z * blk::fast_sigmoid(gv[j].z) * uv[j].z;
              f[4 * j + 3] = gv[j].w * blk::fast_sigmoid(gv[j].w) * uv[j].w;
            }
          } else {
            float lo[8], hi[8];
            blk::unpack8<kIn == kInBf16>(raw[i][0], lo);
            blk::unpack8<kIn == kInBf16>(raw[i][1], hi);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              f[j] = lo[j];
              f[8 + j] = hi[j];
            }
          }
        }
        float am = 0.0f;
#pragma unroll
        for (int j = 0; j < 16; ++j) am = fmaxf(am, fabsf(f[j]));
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        am = fmaxf(am, blk::kScaleFloor);
        const float up = blk::block_up(am);
        if (i == 0) {
          // the stage is free, and with it the slot: its last unit's MMAs are done, so TMEM was free
          // for them, so the epilogue is past unit n - STAGES - NBUF >= n - SLOTS
          static_assert(kIn == kInCodes || SLOTS >= STAGES + NBUF, "slot reuse");
          ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->empty[s]), ((n / STAGES) & 1u) ^ 1u, abort_flag, lim));
          if (!ok) break;
        }
        if (live) {
          const float f0[8] = {f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]};
          const float f1[8] = {f[8], f[9], f[10], f[11], f[12], f[13], f[14], f[15]};
          const uint2 x = blk::codes8_scaled(f0, up), y = blk::codes8_scaled(f1, up);
          gemm::sts_v4(xs + static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4)), x.x, x.y, y.x, y.y);
          if (c == 0) sscale[(n % SLOTS) * NT + r] = blk::block_down(am) * w;
        }
      }
      if (!ok) break;
      gemm::fence_proxy_async_smem();               // the tensor cores read what these lanes wrote
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&bars->scaled[n % SLOTS]));
        mbar_arrive(smem_u32(&bars->full[s]));
      }
    }
  } else if (warp == 6) {
    // ------------------------------------------------------------------ scales
    // SA * SB of each unit's tokens, AHEAD units loaded together
    grid_dep_wait();
    constexpr int SL = (NT + 31) / 32;              // tokens of a lane
    constexpr int AHEAD = SL > 2 ? 4 : 8;
    uint32_t n = 0;
    int tile = -1, row0 = 0, row_end = 0, z = 0, nz = 0;
    bool ok = true;
    for (int64_t u = u0; u < u1 && ok; u += AHEAD) {
      float v[AHEAD][SL], w[AHEAD];
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (u + i >= u1) break;
        const int t = static_cast<int>((u + i) / KB);
        const int kb = static_cast<int>(u + i - static_cast<int64_t>(t) * KB);
        if (t != tile) {
          tile_at(t, row0, row_end, z, nz);
          tile = t;
        }
        w[i] = __ldg(a.SB + (static_cast<int64_t>(z) * a.n_per_z + nz) * KB + kb);
#pragma unroll
        for (int l = 0; l < SL; ++l) {
          const int r = row0 + lane + 32 * l;
          v[i][l] = __ldg(a.SA + static_cast<int64_t>(kb) * a.M + (r < a.M ? r : a.M - 1));
        }
      }
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) {
        if (u + i >= u1) break;
        const uint32_t slot = n % SLOTS;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars->unscaled[slot]), ((n / SLOTS) & 1u) ^ 1u, abort_flag, lim));
        if (!ok) break;
#pragma unroll
        for (int l = 0; l < SL; ++l)
          if (lane + 32 * l < NT) sscale[slot * NT + lane + 32 * l] = v[i][l] * w[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bars->scaled[slot]));
        ++n;
      }
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int q = warp & 3;
    const int nl = q * 32 + lane;                   // the thread's weight row in the tile
    const uint32_t lane_base = tmem_base + (static_cast<uint32_t>(q * 32) << 16);
    uint32_t n = 0;
    bool dead = false;
    for (int64_t u = u0; u < u1;) {
      const int tile = static_cast<int>(u / KB);
      const int64_t t0 = static_cast<int64_t>(tile) * KB;
      const int kb0 = static_cast<int>(u - t0);
      const int kb1 = static_cast<int>((t0 + KB < u1 ? t0 + KB : u1) - t0);
      int row0, row_end, z, nz;
      tile_at(tile, row0, row_end, z, nz);
      float acc[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) acc[j] = 0.0f;
      for (int kb = kb0; kb < kb1 && !dead; ++kb, ++n) {
        const uint32_t b = n % NBUF;
        const float* row = sscale + (n % SLOTS) * NT;
        const bool got = mbar_wait(smem_u32(&bars->scaled[n % SLOTS]), (n / SLOTS) & 1u, abort_flag, lim) &&
                         mbar_wait(smem_u32(&bars->tmem_full[b]), (n / NBUF) & 1u, abort_flag, lim);
        if (!__all_sync(0xffffffffu, got)) {
          dead = true;
          break;
        }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < NT / 16; ++c) {
          uint32_t r[16];
          tmem_ld_x16_wait(lane_base + b * NT + c * 16, r);
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 s4 = *reinterpret_cast<const float4*>(row + c * 16 + j);
            acc[c * 16 + j] = fmaf(__uint_as_float(r[j]), s4.x, acc[c * 16 + j]);
            acc[c * 16 + j + 1] = fmaf(__uint_as_float(r[j + 1]), s4.y, acc[c * 16 + j + 1]);
            acc[c * 16 + j + 2] = fmaf(__uint_as_float(r[j + 2]), s4.z, acc[c * 16 + j + 2]);
            acc[c * 16 + j + 3] = fmaf(__uint_as_float(r[j + 3]), s4.w, acc[c * 16 + j + 3]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(smem_u32(&bars->tmem_empty[b]));
          if (kIn == kInCodes) mbar_arrive(smem_u32(&bars->unscaled[n % SLOTS]));
        }
      }
      u = t0 + kb1;
      bool write = !dead;
      if (kb0 != 0 || kb1 != KB) {
        if (!grouped) grid_dep_wait();              // the counters are cleared by the kernel before
        // the CTAs that share this tile, and this one's part of it
        const int64_t me = blockIdx.x;
        int64_t c0 = t0 * G / units, c1 = (t0 + KB - 1) * G / units;   // estimates, then exact
        while (c0 > 0 && first_unit(c0) > t0) --c0;
        while (first_unit(c0 + 1) <= t0) ++c0;
        while (c1 > 0 && first_unit(c1) > t0 + KB - 1) --c1;
        while (first_unit(c1 + 1) <= t0 + KB - 1) ++c1;
        auto slot = [&](int64_t c) { return 2 * c + (first_unit(c) / KB == tile ? 0 : 1); };
        float* part = a.parts + slot(me) * (NT * ROWS) + nl;
        if (!dead) {
#pragma unroll
          for (int j = 0; j < NT; ++j)
            if (row0 + j < row_end) part[j * ROWS] = acc[j];
        }
        __threadfence();
        epi_bar128();
        if (threadIdx.x == 64) bars->last = dead ? 0u : atomicAdd(a.arrived + c0, 1u);
        epi_bar128();
        write = !dead && bars->last == static_cast<unsigned int>(c1 - c0);
        epi_bar128();                               // `last` is free for the next tile
        if (write) {
          __threadfence();
#pragma unroll
          for (int j = 0; j < NT; ++j) acc[j] = 0.0f;
          // in the order of the CTAs; JOIN parts' loads in flight
          constexpr int JOIN = NT <= 16 ? 4 : NT <= 32 ? 2 : 1;
          for (int64_t c = c0; c <= c1; c += JOIN) {
            float v[JOIN][NT];
#pragma unroll
            for (int i = 0; i < JOIN; ++i) {
              const float* p = a.parts + slot(c + i <= c1 ? c + i : c1) * (NT * ROWS) + nl;
#pragma unroll
              for (int j = 0; j < NT; ++j) v[i][j] = row0 + j < row_end ? __ldcg(p + j * ROWS) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < JOIN; ++i)
              if (c + i <= c1) {
#pragma unroll
                for (int j = 0; j < NT; ++j) acc[j] += v[i][j];
              }
          }
        }
      }
      const int col_z = nz * ROWS + nl;
      if (write && col_z < a.z_cols) {
        const int zz = z % a.z_per_group;
        const int64_t col = static_cast<int64_t>(zz) * a.z_cols + col_z;
        float bv = 0.0f;
        if (a.bias != nullptr)
          bv = kOut == blk::kOutBf16 ? blk::load16<true>(a.bias + col) : blk::load16<false>(a.bias + col);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const int64_t t = row0 + j;
          if (t < row_end) {
            if (kOut == blk::kOutF32)
              static_cast<float*>(a.C)[t * a.ldc + col] = acc[j] + bv;
            else
              static_cast<uint16_t*>(a.C)[t * a.ldc + col] =
                  static_cast<uint16_t>(blk::pack2<kOut == blk::kOutBf16>(acc[j] + bv, 0.0f) & 0xffffu);
          }
        }
      }
    }
  }

  grid_dep_wait();                                  // no CTA ends before the kernel before it
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

}  // namespace skinny
}  // namespace i8
