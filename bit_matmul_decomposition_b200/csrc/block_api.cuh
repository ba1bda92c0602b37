// block_api.cuh -- host side of the block-scaled e4m3 calls: argument checks, workspace layout,
// tensor maps and launches.  Included by api.cu inside its anonymous namespace (checks, device
// information and launch helpers are defined there).
#pragma once

constexpr int kPartGrid = 160;                // CTAs that the workspace of a split product allows for

bool dtype16(int32_t dt) { return dt == I8_DTYPE_F16 || dt == I8_DTYPE_BF16; }
bool fits_int(int64_t v) { return v > 0 && v <= 0x7fffffffLL; }
int64_t blocks128(int64_t n) { return (n + 127) / 128; }
// Sizes of a product.  The kernels number rows and columns with 32 bits, in tiles of up to 256: the
// last tile has to end below 2^31.
bool tiles_ok(int64_t v) { return v > 0 && v <= 0x80000000LL - 256; }
bool product_ok(int64_t T, int64_t N, int64_t K) { return tiles_ok(T) && tiles_ok(N) && tiles_ok(K) && K % 16 == 0; }

// ------------------------------------------------------------------ kernels' attributes
using BlockGemmFn = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, blk::GemmArgs);
using SkinnyFn = void (*)(CUtensorMap, CUtensorMap, skinny::Args);

BlockGemmFn block_gemm_fn(bool amn, bool bmn, int out) {
  if (!amn && !bmn) {
    switch (out) {
      case blk::kOutF16: return blk::block_gemm_kernel<false, false, blk::kOutF16>;
      case blk::kOutBf16: return blk::block_gemm_kernel<false, false, blk::kOutBf16>;
      case blk::kOutF32: return blk::block_gemm_kernel<false, false, blk::kOutF32>;
      default: return blk::block_gemm_kernel<false, false, blk::kOutGated>;
    }
  }
  if (!amn) {
    switch (out) {
      case blk::kOutF16: return blk::block_gemm_kernel<false, true, blk::kOutF16>;
      case blk::kOutBf16: return blk::block_gemm_kernel<false, true, blk::kOutBf16>;
      default: return blk::block_gemm_kernel<false, true, blk::kOutF32>;
    }
  }
  return out == blk::kOutF16 ? blk::block_gemm_kernel<true, true, blk::kOutF16>
                             : blk::block_gemm_kernel<true, true, blk::kOutBf16>;
}

// the streaming product: tiles of 16 tokens form their codes themselves, larger ones (of a layer,
// so with 16-bit outputs) take the quantiser's
template <int NT>
SkinnyFn skinny_fn_nt(int out) {
  using namespace skinny;
  return out == blk::kOutBf16 ? block_skinny_kernel<NT, blk::kOutBf16, kInCodes> : block_skinny_kernel<NT, blk::kOutF16, kInCodes>;
}

SkinnyFn skinny_fn(int nt, int out, int in) {
  using namespace skinny;
  if (in == kInGated) return block_skinny_kernel<16, blk::kOutF32, kInGated>;
  if (in == kInF16)
    return out == blk::kOutF32 ? block_skinny_kernel<16, blk::kOutF32, kInF16> : block_skinny_kernel<16, blk::kOutF16, kInF16>;
  if (in == kInBf16)
    return out == blk::kOutF32 ? block_skinny_kernel<16, blk::kOutF32, kInBf16> : block_skinny_kernel<16, blk::kOutBf16, kInBf16>;
  return nt == 32 ? skinny_fn_nt<32>(out) : skinny_fn_nt<64>(out);
}

struct BlockInfo {
  bool init = false;
  int clusters = 0;             // co-resident CTA pairs of block_gemm_kernel
};
BlockInfo g_block[kMaxDevices];

i8_status block_info(const DeviceInfo& d, BlockInfo** out) {
  int dev = 0;
  if (!cuda_ok(cudaGetDevice(&dev), "cudaGetDevice")) return I8_ERR_CUDA;
  std::lock_guard<std::mutex> lk(g_mu);
  BlockInfo& b = g_block[dev];
  if (!b.init) {
    const auto smem_attr = cudaFuncAttributeMaxDynamicSharedMemorySize;
    const struct { bool a, b; int out; } kinds[] = {
        {false, false, blk::kOutF16}, {false, false, blk::kOutBf16}, {false, false, blk::kOutF32},
        {false, false, blk::kOutGated}, {false, true, blk::kOutF16}, {false, true, blk::kOutBf16},
        {false, true, blk::kOutF32}, {true, true, blk::kOutF16}, {true, true, blk::kOutBf16}};
    int clusters = 0;
    for (const auto& k : kinds) {
      const BlockGemmFn f = block_gemm_fn(k.a, k.b, k.out);
      if (!cuda_ok(cudaFuncSetAttribute(f, smem_attr, static_cast<int>(blk::SMEM_BYTES)),
                   "cudaFuncSetAttribute(block gemm)"))
        return I8_ERR_CUDA;
      // the epilogue's registers come out of those that the CTA starts with: with fewer, its
      // setmaxnreg would wait for good
      cudaFuncAttributes fa;
      if (!cuda_ok(cudaFuncGetAttributes(&fa, f), "cudaFuncGetAttributes(block gemm)")) return I8_ERR_CUDA;
      if (fa.numRegs < blk::REGS_NEEDED) {
        note_cuda("register split of the block product", fa.numRegs, "too few registers");
        return I8_ERR_CUDA;
      }
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(2 * d.sms, 1, 1);
      cfg.blockDim = dim3(blk::THREADS, 1, 1);
      cfg.dynamicSmemBytes = blk::SMEM_BYTES;
      int c = 0;
      if (!cuda_ok(cudaOccupancyMaxActiveClusters(&c, f, &cfg), "cudaOccupancyMaxActiveClusters(block gemm)"))
        return I8_ERR_CUDA;
      if (c < 1) return I8_ERR_UNSUPPORTED;
      clusters = clusters == 0 || c < clusters ? c : clusters;
    }
    for (int o = blk::kOutF16; o <= blk::kOutF32; ++o) {
      for (int nt = 32; nt <= 64 && o != blk::kOutF32; nt *= 2)
        if (!cuda_ok(cudaFuncSetAttribute(skinny_fn(nt, o, skinny::kInCodes), smem_attr, static_cast<int>(skinny::smem_bytes(nt))),
                     "cudaFuncSetAttribute(block skinny)"))
          return I8_ERR_CUDA;
      for (int in = skinny::kInF16; in <= skinny::kInGated; ++in)
        if (!cuda_ok(cudaFuncSetAttribute(skinny_fn(16, o, in), smem_attr, static_cast<int>(skinny::smem_bytes(16))),
                     "cudaFuncSetAttribute(block skinny)"))
          return I8_ERR_CUDA;
    }
    b.clusters = clusters;
    b.init = true;
  }
  *out = &b;
  return I8_OK;
}

// codes [z][rows][cols] with rows `pitch` bytes apart, 128-byte-swizzled boxes of [box_rows][128]
bool map_codes(CUtensorMap* m, const void* base, int64_t cols, int64_t rows, int64_t z, int64_t pitch,
               uint32_t box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) {
    note_cuda("cudaGetDriverEntryPoint(cuTensorMapEncodeTiled)", 0, "not found");
    return false;
  }
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(z)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(pitch), static_cast<cuuint64_t>(pitch) * static_cast<cuuint64_t>(rows)};
  cuuint32_t box[3] = {128, box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return encoded(enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, z > 0 ? 3 : 2, const_cast<void*>(base), dims, strides,
                     box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                     CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE));
}

// ------------------------------------------------------------------ stage launchers
// after: launched with programmatic serialization (its kernel waits for the one before)
i8_status run_block_quant(int32_t dtype, blk::QuantArgs a, int64_t Z, bool after, cudaStream_t s) {
  const bool rows = a.Qr != nullptr, tiles = a.Qt != nullptr, bf = dtype == I8_DTYPE_BF16;
  const bool thin = rows && !tiles && a.colsum == nullptr;    // row codes alone: 32 rows a CTA
  if (thin) a.row_blocks = static_cast<int>((a.R + 31) / 32);
  const int64_t grid = Z * a.row_blocks * a.col_blocks;
  if (!fits_int(grid)) return I8_ERR_INVALID_ARG;
  using Fn = void (*)(blk::QuantArgs);
  const Fn fns[10] = {blk::block_quant_kernel<false, false, false, 4>, blk::block_quant_kernel<false, false, true, 4>,
                      blk::block_quant_kernel<false, true, false, 4>, blk::block_quant_kernel<false, true, true, 4>,
                      blk::block_quant_kernel<true, false, false, 4>, blk::block_quant_kernel<true, false, true, 4>,
                      blk::block_quant_kernel<true, true, false, 4>, blk::block_quant_kernel<true, true, true, 4>,
                      blk::block_quant_kernel<false, true, false, 1>, blk::block_quant_kernel<true, true, false, 1>};
  const Fn f = fns[thin ? 8 + (bf ? 1 : 0) : (bf ? 4 : 0) + (rows ? 2 : 0) + (tiles ? 1 : 0)];
  if (after) {
    const cudaError_t e = launch_overlapped(f, dim3(static_cast<unsigned>(grid)), dim3(blk::kQuantThreads), 0, s, a);
    return cuda_ok(e, "kernel launch") ? launch_status() : I8_ERR_CUDA;
  }
  f<<<static_cast<unsigned>(grid), blk::kQuantThreads, 0, s>>>(a);
  return launch_status();
}

blk::QuantArgs quant_args(const void* X, int64_t R, int64_t C) {
  blk::QuantArgs a = {};
  a.X = static_cast<const uint16_t*>(X);
  a.R = R;
  a.C = C;
  a.row_blocks = static_cast<int>(blocks128(R));
  a.col_blocks = static_cast<int>(blocks128(C));
  return a;
}

// one launch of block_gemm_kernel; m_tiles: at most this many tiles of 256 rows
i8_status run_block_gemm(bool amn, bool bmn, int out, const CUtensorMap& tA, const CUtensorMap& tB,
                         blk::GemmArgs a, int64_t m_tiles, const BlockInfo& b, cudaStream_t s) {
  CUtensorMap tC = tA;
  a.c_tma = (out == blk::kOutF16 || out == blk::kOutBf16) && a.offsets == nullptr && (a.Nc % 8) == 0;
  if (a.c_tma && !map_c(&tC, a.C, static_cast<uint64_t>(a.Nc), static_cast<uint64_t>(a.M))) return I8_ERR_CUDA;
  a.wait_limit_ns = kWaitLimitNs;
  const int64_t tiles = m_tiles * a.n_tiles;
  if (tiles > 0x7fffffffLL) return I8_ERR_INVALID_ARG;
  const int clusters = static_cast<int>(tiles < b.clusters ? tiles : b.clusters);
  const cudaError_t e = launch_overlapped(block_gemm_fn(amn, bmn, out), dim3(2 * clusters), dim3(blk::THREADS),
                                          blk::SMEM_BYTES, s, tA, tB, tC, a);
  return cuda_ok(e, "kernel launch") ? launch_status() : I8_ERR_CUDA;
}

i8_status run_skinny(int nt, int out, int in, const CUtensorMap& tW, const CUtensorMap& tX, skinny::Args a,
                     int64_t token_tiles, const DeviceInfo& d, cudaStream_t s) {
  a.wait_limit_ns = kWaitLimitNs;
  const int64_t tiles = token_tiles * a.n_tiles;
  if (tiles > 0x7fffffffLL) return I8_ERR_INVALID_ARG;
  const int64_t units = tiles * a.k_blocks;
  int64_t grid = d.sms < kPartGrid ? d.sms : kPartGrid;
  if (units < grid) grid = units;
  const cudaError_t e = launch_overlapped(skinny_fn(nt, out, in), dim3(static_cast<unsigned>(grid)), dim3(skinny::threads(in)),
                                          skinny::smem_bytes(nt), s, tW, tX, a);
  return cuda_ok(e, "kernel launch") ? launch_status() : I8_ERR_CUDA;
}

int skinny_tokens(int64_t rows) { return rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// Whether a linear layer streams its weight (block_skinny.cuh) or takes the 256 x 256 tiles: up to
// 16 tokens always; up to 64 when the weight has more tiles of 256 outputs than there are CTA
// pairs, so that the tiles would leave SMs idle in their last round.  T = 32: 4096 -> 16384 (64
// tiles) 26 us streaming, 21 us in tiles; 14336 -> 28672 (112 tiles) 83 and 105 us; T = 96 there:
// 116 and 114 us.
bool streams(int64_t T, int64_t N) { return T <= 16 || (T <= 64 && (N + blk::TN - 1) / blk::TN > kPartGrid / 2); }
size_t parts_bytes(int nt) { return static_cast<size_t>(2 * kPartGrid) * static_cast<size_t>(nt) * 128u * 4u; }

struct Taker {
  size_t off = 0;
  size_t operator()(int64_t bytes) {
    const size_t o = off;
    off = align_up(off + static_cast<size_t>(bytes), 256);
    return o;
  }
};

// ------------------------------------------------------------------ the linear layer
struct LinearWs {
  size_t xq, sx, arrived, parts, total;
};
LinearWs linear_ws(int64_t T, int64_t N, int64_t K) {
  LinearWs w{};
  Taker take;
  if (T > 16) {
    w.xq = take(T * K);
    w.sx = take(blocks128(K) * T * 4);
  }
  if (streams(T, N)) {
    w.arrived = take(kPartGrid * 4);
    w.parts = take(static_cast<int64_t>(parts_bytes(skinny_tokens(T))));
  }
  w.total = take.off;
  return w;
}

i8_status block_linear_forward(const void* X, int32_t dtype, int64_t T, int64_t K, const uint8_t* CB,
                               const float* SCB, const void* bias, int64_t N, void* Y, uint8_t* ws,
                               const DeviceInfo& d, cudaStream_t s) {
  BlockInfo* b;
  i8_status st = block_info(d, &b);
  if (st != I8_OK) return st;
  const LinearWs w = linear_ws(T, N, K);
  const bool few = streams(T, N), direct = T <= 16;
  const bool bf = dtype == I8_DTYPE_BF16;
  blk::QuantArgs q = quant_args(X, T, K);
  q.Qr = ws + w.xq;
  q.qr_pitch = K;
  q.Sr = reinterpret_cast<float*>(ws + w.sx);
  q.rows_out = T;
  if (few) {
    q.zero = reinterpret_cast<unsigned int*>(ws + w.arrived);
    q.zero_words = kPartGrid;
  }
  // Neither kernel is launched with programmatic serialization: the product that follows may
  // read the weight (and, direct, X) from its start, so what wrote them has to be done by then.
  if (direct) {
    skinny::clear_kernel<<<1, kPartGrid, 0, s>>>(q.zero);
    st = launch_status();
  } else {
    st = run_block_quant(dtype, q, 1, false, s);
  }
  if (st != I8_OK) return st;
  const int out = bf ? blk::kOutBf16 : blk::kOutF16;
  const int KB = static_cast<int>(blocks128(K));
  CUtensorMap tX, tW;
  if (few) {
    const int nt = skinny_tokens(T);
    const int in = !direct ? skinny::kInCodes : bf ? skinny::kInBf16 : skinny::kInF16;
    if (!map_codes(&tW, CB, K, N, 1, K, skinny::ROWS)) return I8_ERR_CUDA;
    tX = tW;
    if (!direct && !map_codes(&tX, ws + w.xq, K, T, 0, K, nt)) return I8_ERR_CUDA;
    skinny::Args a = {};
    a.X = X;
    a.k_cols = K;
    a.M = static_cast<int>(T);
    a.k_blocks = KB;
    a.n_tiles = a.n_per_z = static_cast<int>(blocks128(N));
    a.z_cols = static_cast<int>(N);
    a.groups = 1;
    a.z_per_group = 1;
    a.SA = q.Sr;
    a.SB = SCB;
    a.bias = static_cast<const uint16_t*>(bias);
    a.C = Y;
    a.ldc = N;
    a.parts = reinterpret_cast<float*>(ws + w.parts);
    a.arrived = reinterpret_cast<unsigned int*>(ws + w.arrived);
    return run_skinny(nt, out, in, tW, tX, a, 1, d, s);
  }
  if (!map_codes(&tW, CB, K, N, 1, K, blk::HN) || !map_codes(&tX, ws + w.xq, K, T, 0, K, blk::HM)) return I8_ERR_CUDA;
  blk::GemmArgs a = {};
  a.M = static_cast<int>(T);
  a.Nc = static_cast<int>(N);
  a.k_blocks = KB;
  a.n_tiles = static_cast<int>((N + blk::TN - 1) / blk::TN);
  a.groups = 1;
  a.blocks_per_z = KB;
  a.z_per_group = 1;
  a.SA = q.Sr;
  a.sa_pitch = T;
  a.SB = SCB;
  a.sb_block = 1;
  a.sb_col = KB;
  a.bias = static_cast<const uint16_t*>(bias);
  a.C = Y;
  a.ldc = N;
  return run_block_gemm(false, false, out, tX, tW, a, (T + blk::TM - 1) / blk::TM, *b, s);
}

struct LinearBwdWs {
  size_t yr, syr, yt, syt, xt, sxt, sums, total;
};
LinearBwdWs linear_bwd_ws(int64_t T, int64_t N, int64_t K) {
  LinearBwdWs w{};
  Taker take;
  const int64_t Np = (N + 15) / 16 * 16;
  w.yr = take(T * Np);
  w.syr = take(blocks128(N) * T * 4);
  w.yt = take(T * Np);
  w.syt = take(blocks128(T) * blocks128(N) * 4);
  w.xt = take(T * K);
  w.sxt = take(blocks128(T) * blocks128(K) * 4);
  w.sums = take(blocks128(T) * N * 4);
  w.total = take.off;
  return w;
}

i8_status block_linear_backward(const void* dY, const void* X, int32_t dtype, int64_t T, int64_t N, int64_t K,
                                const uint8_t* CB, const float* SCB, void* dX, void* dW, void* db, uint8_t* ws,
                                const DeviceInfo& d, cudaStream_t s) {
  BlockInfo* b;
  i8_status st = block_info(d, &b);
  if (st != I8_OK) return st;
  const LinearBwdWs w = linear_bwd_ws(T, N, K);
  const int64_t Np = (N + 15) / 16 * 16;
  const int out = dtype == I8_DTYPE_BF16 ? blk::kOutBf16 : blk::kOutF16;
  const int KB = static_cast<int>(blocks128(K)), NB = static_cast<int>(blocks128(N)), TB = static_cast<int>(blocks128(T));
  blk::QuantArgs q = quant_args(dY, T, N);
  if (dX != nullptr) {
    q.Qr = ws + w.yr;
    q.qr_pitch = Np;
    q.Sr = reinterpret_cast<float*>(ws + w.syr);
    q.rows_out = T;
  }
  if (dW != nullptr) {
    q.Qt = ws + w.yt;
    q.qt_pitch = Np;
    q.St = reinterpret_cast<float*>(ws + w.syt);
  }
  if (db != nullptr) q.colsum = reinterpret_cast<float*>(ws + w.sums);
  st = run_block_quant(dtype, q, 1, false, s);
  if (st != I8_OK) return st;
  if (db != nullptr) {
    const dim3 grid(static_cast<unsigned>((N + 255) / 256)), block(256);
    const cudaError_t e =
        dtype == I8_DTYPE_BF16
            ? launch_overlapped(blk::colsum_join_kernel<true>, grid, block, 0, s, static_cast<const float*>(q.colsum), TB, N, static_cast<uint16_t*>(db))
            : launch_overlapped(blk::colsum_join_kernel<false>, grid, block, 0, s, static_cast<const float*>(q.colsum), TB, N, static_cast<uint16_t*>(db));
    if (!cuda_ok(e, "kernel launch") || launch_status() != I8_OK) return I8_ERR_CUDA;
  }
  blk::GemmArgs a = {};
  a.groups = 1;
  a.z_per_group = 1;
  a.Nc = static_cast<int>(K);
  a.n_tiles = static_cast<int>((K + blk::TN - 1) / blk::TN);
  a.ldc = K;
  a.sb_block = KB;
  a.sb_col = 1;
  if (dX != nullptr) {
    CUtensorMap tA, tB;
    if (!map_codes(&tA, ws + w.yr, N, T, 0, Np, blk::HM) || !map_codes(&tB, CB, K, N, 1, K, blk::BK)) return I8_ERR_CUDA;
    blk::GemmArgs x = a;
    x.M = static_cast<int>(T);
    x.k_blocks = x.blocks_per_z = NB;
    x.SA = q.Sr;
    x.sa_pitch = T;
    x.SB = SCB;
    x.C = dX;
    st = run_block_gemm(false, true, out, tA, tB, x, (T + blk::TM - 1) / blk::TM, *b, s);
    if (st != I8_OK) return st;
  }
  if (dW != nullptr) {
    blk::QuantArgs qx = quant_args(X, T, K);
    qx.Qt = ws + w.xt;
    qx.qt_pitch = K;
    qx.St = reinterpret_cast<float*>(ws + w.sxt);
    st = run_block_quant(dtype, qx, 1, true, s);
    if (st != I8_OK) return st;
    CUtensorMap tA, tB;
    if (!map_codes(&tA, ws + w.yt, N, T, 0, Np, blk::BK) || !map_codes(&tB, ws + w.xt, K, T, 1, K, blk::BK)) return I8_ERR_CUDA;
    blk::GemmArgs x = a;
    x.M = static_cast<int>(N);
    x.k_blocks = x.blocks_per_z = TB;
    x.SA = q.St;
    x.sa_pitch = NB;
    x.sa_shift = 7;
    x.SB = qx.St;
    x.C = dW;
    st = run_block_gemm(true, true, out, tA, tB, x, (N + blk::TM - 1) / blk::TM, *b, s);
    if (st != I8_OK) return st;
  }
  return I8_OK;
}

// ------------------------------------------------------------------ routing
template <int PER>
void route_launch(const moe::RouteArgs& a, int32_t dtype, bool backward, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((a.T + moe::kRouteWarps - 1) / moe::kRouteWarps);
  const dim3 block(moe::kRouteWarps * 32);
  if (backward) {
    if (dtype == I8_DTYPE_F32) moe::route_backward_kernel<moe::kInF32, PER><<<grid, block, 0, s>>>(a);
    else if (dtype == I8_DTYPE_BF16) moe::route_backward_kernel<moe::kInBf16, PER><<<grid, block, 0, s>>>(a);
    else moe::route_backward_kernel<moe::kInF16, PER><<<grid, block, 0, s>>>(a);
  } else {
    if (dtype == I8_DTYPE_F32) moe::route_kernel<moe::kInF32, PER><<<grid, block, 0, s>>>(a);
    else if (dtype == I8_DTYPE_BF16) moe::route_kernel<moe::kInBf16, PER><<<grid, block, 0, s>>>(a);
    else moe::route_kernel<moe::kInF16, PER><<<grid, block, 0, s>>>(a);
  }
}

i8_status run_route(const moe::RouteArgs& a, int32_t dtype, bool backward, cudaStream_t s) {
  const int per = (a.E + 31) / 32;
  if (per <= 1) route_launch<1>(a, dtype, backward, s);
  else if (per <= 2) route_launch<2>(a, dtype, backward, s);
  else if (per <= 4) route_launch<4>(a, dtype, backward, s);
  else if (per <= 8) route_launch<8>(a, dtype, backward, s);
  else route_launch<16>(a, dtype, backward, s);
  return launch_status();
}

bool route_shape_ok(int32_t dtype, int64_t T, int64_t E, int64_t k, int32_t score, float scale) {
  return dtype >= I8_DTYPE_F16 && dtype <= I8_DTYPE_F32 && fits_int(T) && E > 0 && E <= moe::MAX_EXPERTS && k > 0 &&
         k <= E && k <= moe::MAX_CHOICES && (score == I8_SCORE_SOFTMAX || score == I8_SCORE_SIGMOID) &&
         scale == scale && fits_int(T * k);
}

// ------------------------------------------------------------------ experts
struct ExpertsShape {
  int64_t T, K, I, E, k, R, Ip;
  int KB, IB;
};

bool experts_shape(int64_t T, int64_t K, int64_t I, int64_t E, int64_t k, ExpertsShape* o) {
  if (T <= 0 || !product_ok(1, I, K) || I % 16 != 0 || E <= 0 || E > moe::MAX_EXPERTS || k <= 0 || k > moe::MAX_CHOICES)
    return false;
  if (T > 0x7fffffffLL || !tiles_ok(T * k) || !fits_int(2 * E) || I > 0x3fffffffLL) return false;
  *o = ExpertsShape{T, K, I, E, k, T * k, blocks128(I) * 128, static_cast<int>(blocks128(K)), static_cast<int>(blocks128(I))};
  return true;
}

// Whether the experts' rows are so few on average that their products stream the weights in tiles
// of 16 rows.  64 experts of 4096 x 1024, 8 a token, in us streaming / in 256-row tiles: 4 rows an
// expert 169 / 214, 8 rows 210 / 226, 16 rows 296 / 237.
bool experts_stream(const ExpertsShape& x) { return x.R <= 8 * x.E; }

struct ExpertsWs {
  size_t offsets, place, row_at, xq, sx, arrived, parts, gu, h, sh, y, total;
};
ExpertsWs experts_ws(const ExpertsShape& x, bool backward) {
  ExpertsWs w{};
  Taker take;
  const bool direct = !backward && experts_stream(x);
  w.offsets = take((x.E + 1) * 4);
  w.place = take(x.R * 4);
  w.row_at = take(x.R * 4);
  if (!direct) {
    w.xq = take(x.R * x.K);                    // rows of x, or of dy, by expert
    w.sx = take(static_cast<int64_t>(x.KB) * x.R * 4);
  }
  w.arrived = take(2 * kPartGrid * 4);
  if (direct) {
    w.parts = take(static_cast<int64_t>(parts_bytes(16)));
    w.gu = take(x.R * 2 * x.I * 4);
  }
  if (backward) w.gu = take(x.R * x.I * 4);    // dy W2
  if (!direct) {
    w.h = take(x.R * x.Ip * (backward ? 2 : 1));
    w.sh = take(static_cast<int64_t>(x.IB) * x.R * 4 * (backward ? 2 : 1));
  }
  w.y = take(x.R * x.K * 4);
  w.total = take.off;
  return w;
}

// groups the rows by expert and lays the codes of X's rows out in that order
i8_status experts_rows(const void* X, int32_t dtype, const int32_t* idx, const ExpertsShape& x, const ExpertsWs& w,
                       uint8_t* ws, float* dw, bool codes, cudaStream_t s) {
  int32_t* place = reinterpret_cast<int32_t*>(ws + w.place);
  moe::sort_rows_kernel<<<static_cast<unsigned>(x.E), moe::kSortThreads, 0, s>>>(
      idx, x.R, static_cast<int>(x.E), reinterpret_cast<int32_t*>(ws + w.offsets), place,
      reinterpret_cast<int32_t*>(ws + w.row_at), dw, reinterpret_cast<unsigned int*>(ws + w.arrived), 2 * kPartGrid);
  i8_status st = launch_status();
  if (st != I8_OK || !codes) return st;
  blk::QuantArgs q = quant_args(X, x.T, x.K);
  q.Qr = ws + w.xq;
  q.qr_pitch = x.K;
  q.Sr = reinterpret_cast<float*>(ws + w.sx);
  q.rows_out = x.R;
  q.dest = place;
  q.copies = static_cast<int>(x.k);
  return run_block_quant(dtype, q, 1, true, s);
}

i8_status run_combine(int32_t dtype, const float* V, const int32_t* place, const float* weights, const ExpertsShape& x,
                      void* out, cudaStream_t s) {
  const int64_t grid = (x.T * (x.K / 8) + 255) / 256;
  if (!fits_int(grid)) return I8_ERR_INVALID_ARG;
  const auto f = dtype == I8_DTYPE_BF16 ? moe::combine_kernel<true> : moe::combine_kernel<false>;
  const cudaError_t e = launch_overlapped(f, dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, V, place, weights, x.T,
                                          static_cast<int>(x.k), x.K, static_cast<uint16_t*>(out));
  return cuda_ok(e, "kernel launch") ? launch_status() : I8_ERR_CUDA;
}

i8_status experts_forward(const void* X, int32_t dtype, const int32_t* idx, const float* weights, const uint8_t* CB13,
                          const float* S13, const uint8_t* CB2, const float* S2, const ExpertsShape& x, void* Y,
                          float* GU, uint8_t* ws, const DeviceInfo& d, cudaStream_t s) {
  BlockInfo* b;
  i8_status st = block_info(d, &b);
  if (st != I8_OK) return st;
  const ExpertsWs w = experts_ws(x, false);
  const bool direct = experts_stream(x);      // the products form the codes of their rows
  st = experts_rows(X, dtype, idx, x, w, ws, nullptr, !direct, s);
  if (st != I8_OK) return st;
  const int32_t* offsets = reinterpret_cast<const int32_t*>(ws + w.offsets);
  const int M = static_cast<int>(x.R), E = static_cast<int>(x.E);
  float* SX = reinterpret_cast<float*>(ws + w.sx);
  float* SH = reinterpret_cast<float*>(ws + w.sh);
  float* Y2 = reinterpret_cast<float*>(ws + w.y);
  unsigned int* arrived = reinterpret_cast<unsigned int*>(ws + w.arrived);
  CUtensorMap tX, tW13, tH, tW2;
  if (direct) {
    float* gu = GU != nullptr ? GU : reinterpret_cast<float*>(ws + w.gu);
    const int64_t token_tiles = x.R / 16 + (x.R < x.E ? x.R : x.E);   // at most
    if (!map_codes(&tW13, CB13, x.K, x.I, 2 * x.E, x.K, skinny::ROWS) || !map_codes(&tW2, CB2, x.I, x.K, x.E, x.I, skinny::ROWS))
      return I8_ERR_CUDA;
    skinny::Args a = {};
    a.X = X;
    a.k_cols = x.K;
    a.row_at = reinterpret_cast<const int32_t*>(ws + w.row_at);
    a.copies = static_cast<int>(x.k);
    a.M = M;
    a.groups = E;
    a.offsets = offsets;
    a.k_blocks = x.KB;
    a.n_per_z = x.IB;
    a.n_tiles = 2 * x.IB;
    a.z_cols = static_cast<int>(x.I);
    a.z_per_group = 2;
    a.SB = S13;
    a.C = gu;
    a.ldc = 2 * x.I;
    a.parts = reinterpret_cast<float*>(ws + w.parts);
    a.arrived = arrived;
    st = run_skinny(16, blk::kOutF32, dtype == I8_DTYPE_BF16 ? skinny::kInBf16 : skinny::kInF16, tW13, tW13, a, token_tiles, d, s);
    if (st != I8_OK) return st;
    a.X = gu;
    a.k_cols = x.I;
    a.k_blocks = x.IB;
    a.n_tiles = a.n_per_z = x.KB;
    a.z_cols = static_cast<int>(x.K);
    a.z_per_group = 1;
    a.SB = S2;
    a.C = Y2;
    a.ldc = x.K;
    a.arrived = arrived + kPartGrid;
    st = run_skinny(16, blk::kOutF32, skinny::kInGated, tW2, tW2, a, token_tiles, d, s);
  } else {
    const int64_t m_tiles = x.R / blk::TM + (x.R < x.E ? x.R : x.E);
    if (!map_codes(&tX, ws + w.xq, x.K, x.R, 0, x.K, blk::HM) || !map_codes(&tW13, CB13, x.K, x.I, 2 * x.E, x.K, 64) ||
        !map_codes(&tH, ws + w.h, x.Ip, x.R, 0, x.Ip, blk::HM) || !map_codes(&tW2, CB2, x.I, x.K, x.E, x.I, blk::HN))
      return I8_ERR_CUDA;
    blk::GemmArgs a = {};
    a.M = M;
    a.groups = E;
    a.offsets = offsets;
    a.Nc = static_cast<int>(x.I);
    a.k_blocks = a.blocks_per_z = x.KB;
    a.n_tiles = x.IB;
    a.z_per_group = 2;
    a.SA = SX;
    a.sa_pitch = x.R;
    a.SB = S13;
    a.sb_group = 2LL * x.IB * x.KB;
    a.sb_block = 1;
    a.sb_col = x.KB;
    a.H = ws + w.h;
    a.h_pitch = x.Ip;
    a.SH = SH;
    a.GU = GU;
    st = run_block_gemm(false, false, blk::kOutGated, tX, tW13, a, m_tiles, *b, s);
    if (st != I8_OK) return st;
    a.Nc = static_cast<int>(x.K);
    a.k_blocks = a.blocks_per_z = x.IB;
    a.n_tiles = static_cast<int>((x.K + blk::TN - 1) / blk::TN);
    a.z_per_group = 1;
    a.SA = SH;
    a.SB = S2;
    a.sb_group = static_cast<int64_t>(x.KB) * x.IB;
    a.sb_col = x.IB;
    a.C = Y2;
    a.ldc = x.K;
    st = run_block_gemm(false, false, blk::kOutF32, tH, tW2, a, m_tiles, *b, s);
  }
  if (st != I8_OK) return st;
  return run_combine(dtype, Y2, reinterpret_cast<const int32_t*>(ws + w.place), weights, x, Y, s);
}

i8_status experts_backward(const void* dY, int32_t dtype, const int32_t* idx, const float* weights, const uint8_t* CB13,
                           const float* S13, const uint8_t* CB2, const float* S2, const ExpertsShape& x, const float* GU,
                           void* dX, float* dw, uint8_t* ws, const DeviceInfo& d, cudaStream_t s) {
  BlockInfo* b;
  i8_status st = block_info(d, &b);
  if (st != I8_OK) return st;
  const ExpertsWs w = experts_ws(x, true);
  st = experts_rows(dY, dtype, idx, x, w, ws, dw, true, s);
  if (st != I8_OK) return st;
  const int32_t* offsets = reinterpret_cast<const int32_t*>(ws + w.offsets);
  const int64_t m_tiles = x.R / blk::TM + (x.R < x.E ? x.R : x.E);
  float* dH = reinterpret_cast<float*>(ws + w.gu);
  float* SQ = reinterpret_cast<float*>(ws + w.sh);
  float* dXr = reinterpret_cast<float*>(ws + w.y);
  CUtensorMap tY, tW2, tQ, tW13;
  if (!map_codes(&tY, ws + w.xq, x.K, x.R, 0, x.K, blk::HM) || !map_codes(&tW2, CB2, x.I, x.K, x.E, x.I, blk::BK) ||
      !map_codes(&tQ, ws + w.h, 2 * x.Ip, x.R, 0, 2 * x.Ip, blk::HM) || !map_codes(&tW13, CB13, x.K, x.I, 2 * x.E, x.K, blk::BK))
    return I8_ERR_CUDA;
  blk::GemmArgs a = {};
  a.M = static_cast<int>(x.R);
  a.groups = static_cast<int>(x.E);
  a.offsets = offsets;
  a.Nc = static_cast<int>(x.I);
  a.k_blocks = a.blocks_per_z = x.KB;
  a.n_tiles = static_cast<int>((x.I + blk::TN - 1) / blk::TN);
  a.z_per_group = 1;
  a.SA = reinterpret_cast<const float*>(ws + w.sx);
  a.sa_pitch = x.R;
  a.SB = S2;
  a.sb_group = static_cast<int64_t>(x.KB) * x.IB;
  a.sb_block = x.IB;
  a.sb_col = 1;
  a.C = dH;
  a.ldc = x.I;
  st = run_block_gemm(false, true, blk::kOutF32, tY, tW2, a, m_tiles, *b, s);
  if (st != I8_OK) return st;
  const cudaError_t e = launch_overlapped(moe::gated_backward_kernel, dim3(static_cast<unsigned>(x.R)), dim3(256), 0, s,
                                          static_cast<const float*>(dH), GU, offsets + x.E,
                                          reinterpret_cast<const int32_t*>(ws + w.row_at), weights, x.R,
                                          static_cast<int>(x.I), ws + w.h, x.Ip, SQ, dw);
  if (!cuda_ok(e, "kernel launch") || launch_status() != I8_OK) return I8_ERR_CUDA;
  a.Nc = static_cast<int>(x.K);
  a.k_blocks = 2 * x.IB;
  a.blocks_per_z = x.IB;
  a.n_tiles = static_cast<int>((x.K + blk::TN - 1) / blk::TN);
  a.z_per_group = 2;
  a.SA = SQ;
  a.SB = S13;
  a.sb_group = 2LL * x.IB * x.KB;
  a.sb_block = x.KB;
  a.C = dXr;
  a.ldc = x.K;
  st = run_block_gemm(false, true, blk::kOutF32, tQ, tW13, a, m_tiles, *b, s);
  if (st != I8_OK) return st;
  return run_combine(dtype, dXr, reinterpret_cast<const int32_t*>(ws + w.place), nullptr, x, dX, s);
}
