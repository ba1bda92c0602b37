// block_quant.cuh -- e4m3 codes with one fp32 scale for each block of 128.
//
// A block is 128 consecutive features of one row ("row blocks": activations and gradients of
// outputs) or a 128 x 128 tile ("tiles": weights, and both operands of a weight gradient).
// With a = max(max |v| over the block, 2^-100):
//   code  = e4m3(fl32(v * fl32(448 / a)))     nearest, ties to even; |v| = a gives 448
//   scale = fl32(a * fl32(1 / 448))           code * scale stands for v
// The floor 2^-100 keeps 448 / a finite for bf16 inputs down to their smallest value and makes
// an all-zero block need no branch (its codes are 0).  The maximum is taken over the values
// that are not NaN; a NaN becomes the NaN code 0x7f, and an infinity makes a infinite, so its
// own code is inf * 0 = NaN: whatever is not finite reaches every output of its row (or
// tile), and no other.
//
// One CTA of 256 threads holds a 128 x 128 tile of the input in registers (eight 16-byte groups a
// thread, all in flight at once; 32 rows where only row codes are wanted), so one read of the
// input gives any of: its row codes, its tile codes, its column sums.  The bound is HBM, 2 bytes
// read and 1 written per value and code set.  In a row of such calls a 16384 x 4096 weight takes 35
// us, 5.8 TB/s, and row codes of 2048 x 16384 25 us, 4.0 TB/s; behind a flush of the L2 39 and 31.
#pragma once

#include <cuda_bf16.h>

#include "common.cuh"
#include "quant.cuh"

namespace i8 {
namespace blk {

constexpr int QB = 128;                      // block edge
constexpr float kScaleFloor = 7.888609052210118e-31f;   // 2^-100
constexpr int kQuantThreads = 256;

__device__ __forceinline__ float block_up(float a) { return __fdiv_rn(448.0f, a); }
__device__ __forceinline__ float block_down(float a) { return __fmul_rn(a, 1.0f / 448.0f); }

template <bool kBf16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
  if (kBf16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

template <bool kBf16>
__device__ __forceinline__ float load16(const uint16_t* p) {
  const uint32_t w = *p;
  return unpack2<kBf16>(w).x;
}

template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if (kBf16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// largest |v| of 8 packed values (two at a time; a NaN gives way to the other operand)
template <bool kBf16>
__device__ __forceinline__ float absmax8(const uint4& v) {
  const uint32_t w[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
  if (kBf16) {
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(w);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
  }
  const __half2* h = reinterpret_cast<const __half2*>(w);
  const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  return fmaxf(__low2float(m), __high2float(m));
}

struct QuantArgs {
  const uint16_t* X;       // [Z][R][C], 16-bit values
  int64_t R, C;
  int row_blocks, col_blocks;
  // row codes [*][q_pitch] and scales [col_blocks][rows_out]; NULL = not wanted.  Row t goes
  // to row t, or with `dest` (copies > 0) to the rows dest[t * copies + j] that are >= 0.
  uint8_t* Qr;
  int64_t qr_pitch;
  float* Sr;
  int64_t rows_out;
  const int32_t* dest;
  int copies;
  // tile codes [Z][R][qt_pitch] and scales [Z][row_blocks][col_blocks]
  uint8_t* Qt;
  int64_t qt_pitch;
  float* St;
  float* colsum;           // [row_blocks][C] column sums of each row block (Z = 1)
  unsigned int* zero;      // words cleared for the product that follows
  int zero_words;
};

// 8 codes of 8 values (as floats) times `up`
__device__ __forceinline__ uint2 codes8_scaled(const float (&f)[8], float up) {
  uint2 o;
  o.x = e4m3x2(__fmul_rn(f[0], up), __fmul_rn(f[1], up)) |
        (static_cast<uint32_t>(e4m3x2(__fmul_rn(f[2], up), __fmul_rn(f[3], up))) << 16);
  o.y = e4m3x2(__fmul_rn(f[4], up), __fmul_rn(f[5], up)) |
        (static_cast<uint32_t>(e4m3x2(__fmul_rn(f[6], up), __fmul_rn(f[7], up))) << 16);
  return o;
}

template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p = unpack2<kBf16>(w[i]);
    f[2 * i] = p.x;
    f[2 * i + 1] = p.y;
  }
}

// 16 codes of 16 packed values times `up`
template <bool kBf16>
__device__ __forceinline__ uint4 codes16_scaled(const uint4& lo, const uint4& hi, float up) {
  float f[8];
  unpack8<kBf16>(lo, f);
  const uint2 x = codes8_scaled(f, up);
  unpack8<kBf16>(hi, f);
  const uint2 y = codes8_scaled(f, up);
  return make_uint4(x.x, x.y, y.x, y.y);
}

// Eight lanes hold a row's 128 features, 16 each, and the CTA 32 rows at a time.  PASSES: how many
// times; 4 for tiles, 1 when row codes alone are wanted (four times the CTAs: 333 x 4112 takes 3.3
// us, with 128 rows a CTA 6.3).
template <bool kBf16, bool kRows, bool kTiles, int PASSES>
__global__ void __launch_bounds__(kQuantThreads, PASSES == 1 ? 6 : kRows && kTiles ? 3 : 4)
    block_quant_kernel(const QuantArgs a) {
  static_assert(PASSES == 4 || !kTiles, "a tile has 128 rows");
  __shared__ float s_max[kQuantThreads / 32];
  __shared__ float s_sum[32][QB];
  grid_dep_wait();
  grid_dep_launch();
  if (a.zero != nullptr && blockIdx.x == 0)
    for (int i = threadIdx.x; i < a.zero_words; i += kQuantThreads) a.zero[i] = 0u;
  int64_t b = blockIdx.x;
  const int cb = static_cast<int>(b % a.col_blocks);
  b /= a.col_blocks;
  const int rb = static_cast<int>(b % a.row_blocks);
  const int64_t z = b / a.row_blocks;
  const int r_in = threadIdx.x >> 3;                 // 32 rows a pass, 8 threads a row
  const int lane8 = threadIdx.x & 7;
  const int64_t c0 = static_cast<int64_t>(cb) * QB + lane8 * 16;
  const int64_t row0 = static_cast<int64_t>(rb) * (PASSES * 32) + r_in;
  const uint16_t* X = a.X + z * a.R * a.C;
  const bool vec = (a.C & 7) == 0;                   // rows start on 16 bytes
  uint4 v[PASSES][2];
#pragma unroll
  for (int p = 0; p < PASSES; ++p) {
    const int64_t r = row0 + p * 32;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t c = c0 + 8 * h;
      v[p][h] = make_uint4(0u, 0u, 0u, 0u);
      if (r < a.R && c < a.C) {
        const uint16_t* src = X + r * a.C + c;
        if (vec) {
          v[p][h] = ldg_v4(src);
        } else {
          uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (c + i < a.C) w[i >> 1] |= static_cast<uint32_t>(src[i]) << (16 * (i & 1));
          v[p][h] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
  }
  float m[PASSES];                                   // the row's maximum over this thread's 16
#pragma unroll
  for (int p = 0; p < PASSES; ++p) m[p] = fmaxf(absmax8<kBf16>(v[p][0]), absmax8<kBf16>(v[p][1]));
  if (kRows) {
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int64_t r = row0 + p * 32;
      float am = m[p];
#pragma unroll
      for (int o = 4; o > 0; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
      am = fmaxf(am, kScaleFloor);
      if (r >= a.R) continue;
      const uint4 q = codes16_scaled<kBf16>(v[p][0], v[p][1], block_up(am));
      const float down = block_down(am);
      const int n = a.dest != nullptr ? a.copies : 1;
      for (int j0 = 0; j0 < n; j0 += 4) {            // four places' loads in flight
        int64_t t[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          t[j] = j0 + j >= n ? -1 : a.dest != nullptr ? __ldg(a.dest + r * a.copies + j0 + j) : r;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (t[j] < 0) continue;
          if (c0 < a.qr_pitch) *reinterpret_cast<uint4*>(a.Qr + t[j] * a.qr_pitch + c0) = q;
          if (lane8 == 0) a.Sr[cb * a.rows_out + t[j]] = down;
        }
      }
    }
  }
  if (kTiles) {
    float am = m[0];
#pragma unroll
    for (int p = 1; p < PASSES; ++p) am = fmaxf(am, m[p]);
    am = warp_max(am);
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = am;
    __syncthreads();
    am = s_max[0];
#pragma unroll
    for (int i = 1; i < kQuantThreads / 32; ++i) am = fmaxf(am, s_max[i]);
    am = fmaxf(am, kScaleFloor);
    const float up = block_up(am);
#pragma unroll
    for (int p = 0; p < PASSES; ++p) {
      const int64_t r = row0 + p * 32;
      if (r >= a.R || c0 >= a.qt_pitch) continue;
      *reinterpret_cast<uint4*>(a.Qt + (z * a.R + r) * a.qt_pitch + c0) = codes16_scaled<kBf16>(v[p][0], v[p][1], up);
    }
    if (threadIdx.x == 0) a.St[blockIdx.x] = block_down(am);
  }
  if (a.colsum != nullptr) {
    // column sums in a fixed order: each thread its rows from the top, then the 32 threads of
    // a column in turn
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int p = 0; p < PASSES; ++p) {
        float f[8];
        unpack8<kBf16>(v[p][h], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) sum[i] += f[i];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) s_sum[r_in][lane8 * 16 + 8 * h + i] = sum[i];
    }
    __syncthreads();
    const int64_t c = static_cast<int64_t>(cb) * QB + threadIdx.x;
    if (threadIdx.x < QB && c < a.C) {
      float t = s_sum[0][threadIdx.x];
#pragma unroll
      for (int i = 1; i < 32; ++i) t += s_sum[i][threadIdx.x];
      a.colsum[static_cast<int64_t>(rb) * a.C + c] = t;
    }
  }
}

// out[c] = 16-bit rounding of the sum of part[0..blocks)[c], added in fp32 from the first
template <bool kBf16>
__global__ void __launch_bounds__(256)
    colsum_join_kernel(const float* __restrict__ part, int blocks, int64_t C,
                       uint16_t* __restrict__ out) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t c = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (c >= C) return;
  float s = 0.0f;
  for (int b = 0; b < blocks; ++b) s += part[static_cast<int64_t>(b) * C + c];
  out[c] = static_cast<uint16_t>(pack2<kBf16>(s, 0.0f) & 0xffffu);
}

}  // namespace blk
}  // namespace i8
