// experts.cuh -- what stands around the experts' products (block_gemm.cuh, block_skinny.cuh):
// the routing of tokens and its gradient, the grouping of rows by expert, the gated
// activation with its quantisation, and the weighted sum of a token's experts.
#pragma once

#include "block_gemm.cuh"
#include "block_quant.cuh"
#include "common.cuh"

namespace i8 {
namespace moe {

constexpr int MAX_EXPERTS = blk::MAX_GROUPS;
constexpr int MAX_CHOICES = 32;
constexpr int MAX_ROUTE_GROUPS = 32;

// ------------------------------------------------------------------ routing
// One warp a token; expert e is held by lane e % 32.  Steps:
//   score p_e = softmax or sigmoid of the logits; key_e = p_e + balance_e, or -inf for a masked
//   expert (logit -inf); with groups, a group's total is the sum of its best 2 keys (1 without
//   balance) among its live members and only the experts of the top_groups best groups stay;
//   the k largest keys in order, the lower index first among equals; weight = p (without
//   balance), over the sum of the chosen p's when renormalised, times `scale`.
// Choices that find no live expert get index -1 and weight 0.
// Scores, keys and sums are fp64: which expert is chosen hangs on the order of keys that may be
// equal to within an fp32 rounding, and a user's check of the choice has to find the same ones.
// A NaN logit is never chosen, and makes every weight of its token NaN; so does +inf under
// softmax (its score has no value).
struct RouteArgs {
  const void* logits;          // [T][E]
  int64_t T;
  int E, k, groups, top_groups;
  const float* balance;        // [E] or NULL
  bool softmax, renorm;
  float scale;
  float* weights;              // [T][k]
  int32_t* idx;                // [T][k]
  // backward
  const float* dweights;       // [T][k]
  void* dlogits;               // [T][E]
};

enum { kInF16 = 0, kInBf16 = 1, kInF32 = 2 };
constexpr int kRouteWarps = 4;

template <int kIn>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  if (kIn == kInF32) return __ldg(static_cast<const float*>(p) + i);
  return blk::load16<kIn == kInBf16>(static_cast<const uint16_t*>(p) + i);
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// scores of a token's experts; returns whether the token's weights have a value
template <int kIn, int PER>
__device__ __forceinline__ bool route_scores(const RouteArgs& a, int64_t t, float (&x)[PER],
                                             double (&p)[PER]) {
  const int lane = lane_id();
  const float ninf = __int_as_float(0xff800000);
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    x[i] = e < a.E ? load_logit<kIn>(a.logits, t * a.E + e) : ninf;
    if (x[i] != x[i]) {
      bad = true;
      x[i] = ninf;
    }
  }
  if (a.softmax) {
    float m = ninf;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = fmaxf(m, x[i]);
    m = warp_max(m);
    const bool top = m == __int_as_float(0x7f800000);
    bad |= top;
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (x[i] == ninf) p[i] = 0.0;
      else if (top) p[i] = x[i] == m ? 1.0 : 0.0;
      else p[i] = exp(static_cast<double>(x[i]) - static_cast<double>(m));
      sum += p[i];
    }
    sum = warp_sum(sum);
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i] *= inv;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) p[i] = x[i] == ninf ? 0.0 : 1.0 / (1.0 + exp(-static_cast<double>(x[i])));
  }
  return !__any_sync(0xffffffffu, bad);
}

__device__ __forceinline__ double neg_inf_d() { return __longlong_as_double(0xfff0000000000000ll); }

// the largest (key, lowest index) of the warp
__device__ __forceinline__ void warp_best(double& key, int& e) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double ok = __shfl_xor_sync(0xffffffffu, key, o);
    const int oe = __shfl_xor_sync(0xffffffffu, e, o);
    if (ok > key || (ok == key && oe < e)) {
      key = ok;
      e = oe;
    }
  }
}

template <int kIn, int PER>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_kernel(const RouteArgs a) {
  __shared__ double s_key[kRouteWarps][PER * 32];
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  if (t >= a.T) return;
  float x[PER];
  double p[PER], key[PER];
  const bool good = route_scores<kIn, PER>(a, t, x, p);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    key[i] = neg_inf_d();
    if (x[i] != __int_as_float(0xff800000))
      key[i] = p[i] + (a.balance != nullptr ? static_cast<double>(__ldg(a.balance + e)) : 0.0);
    if (!(key[i] == key[i])) key[i] = neg_inf_d();      // a NaN balance: never chosen
  }
  if (a.groups > 1) {
#pragma unroll
    for (int i = 0; i < PER; ++i) s_key[warp][i * 32 + lane] = key[i];
    __syncwarp();
    const int size = a.E / a.groups;
    double total = neg_inf_d();
    if (lane < a.groups) {
      double b1 = neg_inf_d(), b2 = neg_inf_d();
      for (int j = 0; j < size; ++j) {
        const double v = s_key[warp][lane * size + j];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
      total = b1;
      if (a.balance != nullptr && b2 > neg_inf_d()) total += b2;
    }
    // a lane past the last group takes no part: its index loses every tie, its key is -inf
    unsigned kept = 0u;
    double mine = total;
    int id = lane < a.groups ? lane : 64 + lane;
    for (int j = 0; j < a.top_groups; ++j) {
      double b = mine;
      int g = id;
      warp_best(b, g);
      if (g < 32) kept |= 1u << g;
      if (g == id) {
        mine = neg_inf_d();
        id = 64 + lane;                                 // taken
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = i * 32 + lane;
      if (e < a.E && !((kept >> (e / size)) & 1u)) key[i] = neg_inf_d();
    }
  }
  double mine_p = 0.0, sum = 0.0;                       // lane j keeps choice j
  int mine_e = -1;
  for (int j = 0; j < a.k; ++j) {
    double b = neg_inf_d(), pb = 0.0;
    int e = 0x7fffffff;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] > b) {
        b = key[i];
        e = i * 32 + lane;
        pb = p[i];
      }
    const int own = e;
    warp_best(b, e);
    const bool found = b > neg_inf_d();
    const double pw = __shfl_sync(0xffffffffu, pb, e & 31);
    if (found && own == e) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i * 32 + lane == e) key[i] = neg_inf_d();
    }
    if (found) sum += pw;
    if (lane == j) {
      mine_e = found ? e : -1;
      mine_p = found ? pw : 0.0;
    }
  }
  if (lane < a.k) {
    double w = mine_p;
    if (a.renorm) w = sum > 0.0 ? mine_p / sum : 0.0;
    w *= static_cast<double>(a.scale);
    a.weights[t * a.k + lane] = good || mine_e < 0 ? static_cast<float>(w) : __int_as_float(0x7fc00000);
    a.idx[t * a.k + lane] = mine_e;
  }
}

// Gradient of the weights with respect to the logits; the choice itself and the balance have
// none.  With s the chosen scores, S their sum, g = dweights:
//   ds_j = scale * (g_j - [renorm] sum_i g_i s_i / S) / ([renorm] S, else 1), 0 elsewhere
//   softmax: dx_e = p_e (ds_e - sum_j ds_j p_j)      sigmoid: dx_e = ds_e p_e (1 - p_e)
template <int kIn, int PER>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_backward_kernel(const RouteArgs a) {
  __shared__ double s_val[kRouteWarps][PER * 32];
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  if (t >= a.T) return;
  float x[PER];
  double p[PER];
  const bool good = route_scores<kIn, PER>(a, t, x, p);
  double* val = s_val[warp];
#pragma unroll
  for (int i = 0; i < PER; ++i) val[i * 32 + lane] = p[i];
  __syncwarp();
  int e = -1;
  double g = 0.0, s = 0.0;
  if (lane < a.k) {
    e = __ldg(a.idx + t * a.k + lane);
    if (e >= a.E) {
      raise_error(kErrBounds);
      e = -1;
    }
    if (e >= 0) {
      g = static_cast<double>(__ldg(a.dweights + t * a.k + lane)) * static_cast<double>(a.scale);
      s = val[e];
    }
  }
  double ds = g;
  if (a.renorm) {
    const double S = warp_sum(s), gs = warp_sum(g * s);
    ds = S > 0.0 && e >= 0 ? (g - gs / S) / S : 0.0;
  }
  const double dot = warp_sum(ds * s);
  __syncwarp();
#pragma unroll
  for (int i = 0; i < PER; ++i) val[i * 32 + lane] = 0.0;
  __syncwarp();
  // an index may be given twice: its terms add up, in the order of the choices
  for (int j = 0; j < a.k; ++j) {
    if (lane == j && e >= 0) val[e] += ds;
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int ei = i * 32 + lane;
    if (ei >= a.E) continue;
    const double d = val[ei];
    double dx = a.softmax ? p[i] * (d - dot) : d * p[i] * (1.0 - p[i]);
    if (!good) dx = __longlong_as_double(0x7ff8000000000000ll);
    const int64_t at = t * a.E + ei;
    if (kIn == kInF32)
      static_cast<float*>(a.dlogits)[at] = static_cast<float>(dx);
    else if (kIn == kInBf16)
      static_cast<__nv_bfloat16*>(a.dlogits)[at] = __double2bfloat16(dx);
    else
      static_cast<__half*>(a.dlogits)[at] = __double2half(dx);
  }
}

// ------------------------------------------------------------------ rows by expert
// Row r = (token r / k, choice r % k).  CTA e counts the rows of the experts below e and its
// own, then numbers its own in order: offsets[e], place[r] (the row's position, -1 without an
// expert) and row_at[position].  Positions are a stable sort by expert: no atomics, so the same
// on every run.  An index outside [0, E) that is not negative sets the error word and counts as
// none.  With `dw`, the entries of rows without an expert are cleared; CTA 0 clears `zero`, the
// counters of the products that follow.
constexpr int kSortThreads = 512;

__global__ void __launch_bounds__(kSortThreads)
    sort_rows_kernel(const int32_t* __restrict__ idx, int64_t R, int E, int32_t* __restrict__ offsets,
                     int32_t* __restrict__ place, int32_t* __restrict__ row_at,
                     float* __restrict__ dw, unsigned int* __restrict__ zero, int zero_words) {
  __shared__ int s_less[kSortThreads / 32], s_eq[kSortThreads / 32];
  const int e = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = lane_id();
  grid_dep_launch();
  if (e == 0)
    for (int i = threadIdx.x; i < zero_words; i += kSortThreads) zero[i] = 0u;
  int less = 0, eq = 0;
  for (int64_t r = threadIdx.x; r < R; r += kSortThreads) {
    const int v = __ldg(idx + r);
    const bool in = v >= 0 && v < E;
    less += in && v < e;
    eq += v == e;
    if (e == 0 && !in) {
      place[r] = -1;
      if (dw != nullptr) dw[r] = 0.0f;
      if (v >= E) raise_error(kErrBounds);
    }
  }
  less = __reduce_add_sync(0xffffffffu, less);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    s_less[warp] = less;
    s_eq[warp] = eq;
  }
  __syncthreads();
  int base = 0, total = 0;
  for (int w = 0; w < kSortThreads / 32; ++w) {
    base += s_less[w];
    total += s_eq[w];
  }
  if (threadIdx.x == 0) {
    offsets[e] = base;
    if (e == E - 1) offsets[E] = base + total;
  }
  if (total == 0) return;
  for (int64_t r0 = 0; r0 < R; r0 += kSortThreads) {
    const int64_t r = r0 + threadIdx.x;
    const bool hit = r < R && __ldg(idx + r) == e;
    const unsigned bits = __ballot_sync(0xffffffffu, hit);
    __syncthreads();                                    // the counts of the round before are read
    if (lane == 0) s_eq[warp] = __popc(bits);
    __syncthreads();
    int before = 0, round = 0;
    for (int w = 0; w < kSortThreads / 32; ++w) {
      if (w < warp) before += s_eq[w];
      round += s_eq[w];
    }
    if (hit) {
      const int at = base + before + __popc(bits & ((1u << lane) - 1u));
      place[r] = at;
      row_at[at] = static_cast<int32_t>(r);
    }
    base += round;
  }
}

// ------------------------------------------------------------------ gated activation
// h = silu(g) * u of GU [R][2][I] (fp32) as row codes [R][h_pitch] and scales [ceil(I/128)][R];
// one warp a block of 128 features.  Rows past the last expert's are left alone.
__global__ void __launch_bounds__(256)
    gated_quant_kernel(const float* __restrict__ GU, const int32_t* __restrict__ rows_end, int64_t R, int I,
                       uint8_t* __restrict__ H, int64_t h_pitch, float* __restrict__ SH) {
  grid_dep_wait();
  grid_dep_launch();
  const int blocks = (I + blk::QB - 1) / blk::QB;
  const int64_t w = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) >> 5;
  const int64_t row = w / blocks;
  const int b = static_cast<int>(w - row * blocks);
  if (row >= __ldg(rows_end)) return;
  const int i = b * blk::QB + lane_id() * 4;
  float h[4] = {0.f, 0.f, 0.f, 0.f};
  if (i < I) {
    const float4 g = __ldg(reinterpret_cast<const float4*>(GU + (row * 2) * I + i));
    const float4 u = __ldg(reinterpret_cast<const float4*>(GU + (row * 2 + 1) * I + i));
    h[0] = g.x * blk::fast_sigmoid(g.x) * u.x;
    h[1] = g.y * blk::fast_sigmoid(g.y) * u.y;
    h[2] = g.z * blk::fast_sigmoid(g.z) * u.z;
    h[3] = g.w * blk::fast_sigmoid(g.w) * u.w;
  }
  float am = fmaxf(fmaxf(fabsf(h[0]), fabsf(h[1])), fmaxf(fabsf(h[2]), fabsf(h[3])));
  am = fmaxf(warp_max(am), blk::kScaleFloor);
  const float up = blk::block_up(am);
  const uint32_t q = e4m3x2(h[0] * up, h[1] * up) | (static_cast<uint32_t>(e4m3x2(h[2] * up, h[3] * up)) << 16);
  *reinterpret_cast<uint32_t*>(H + row * h_pitch + i) = q;
  if (lane_id() == 0) SH[static_cast<int64_t>(b) * R + row] = blk::block_down(am);
}

// Gradient of a row's activation.  dH [R][I] is dy W2 without the row's weight w:
//   dw = sum_i dH_i h_i;   dg = w dH u s (1 + g (1 - s)),  du = w dH g s,  s = sigmoid(g)
// dg and du leave as row codes [R][2 * h_pitch] and scales [2 * ceil(I/128)][R].  One CTA a row;
// its warps take blocks of 128 features in turn and the sum of dw is joined in a fixed order.
__global__ void __launch_bounds__(256)
    gated_backward_kernel(const float* __restrict__ dH, const float* __restrict__ GU,
                          const int32_t* __restrict__ rows_end, const int32_t* __restrict__ row_at,
                          const float* __restrict__ weights, int64_t R, int I, uint8_t* __restrict__ Q,
                          int64_t h_pitch, float* __restrict__ SQ, float* __restrict__ dw) {
  __shared__ float s_part[8];
  grid_dep_wait();
  grid_dep_launch();
  const int64_t row = blockIdx.x;
  if (row >= __ldg(rows_end)) return;
  const int r = __ldg(row_at + row);
  const float w = __ldg(weights + r);
  const int blocks = (I + blk::QB - 1) / blk::QB;
  float part = 0.0f;
  for (int b = threadIdx.x >> 5; b < blocks; b += 8) {
    const int i = b * blk::QB + lane_id() * 4;
    float dg[4] = {0.f, 0.f, 0.f, 0.f}, du[4] = {0.f, 0.f, 0.f, 0.f};
    if (i < I) {
      const float4 g4 = __ldg(reinterpret_cast<const float4*>(GU + (row * 2) * I + i));
      const float4 u4 = __ldg(reinterpret_cast<const float4*>(GU + (row * 2 + 1) * I + i));
      const float4 d4 = __ldg(reinterpret_cast<const float4*>(dH + row * I + i));
      const float g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
      const float d[4] = {d4.x, d4.y, d4.z, d4.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float s = blk::fast_sigmoid(g[j]);
        const float gs = g[j] * s;
        part += d[j] * (gs * u[j]);
        const float wd = w * d[j];
        du[j] = wd * gs;
        dg[j] = wd * u[j] * s * (1.0f + g[j] * (1.0f - s));
      }
    }
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      const float* v = which ? du : dg;
      float am = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
      am = fmaxf(warp_max(am), blk::kScaleFloor);
      const float up = blk::block_up(am);
      const uint32_t q = e4m3x2(v[0] * up, v[1] * up) | (static_cast<uint32_t>(e4m3x2(v[2] * up, v[3] * up)) << 16);
      *reinterpret_cast<uint32_t*>(Q + row * 2 * h_pitch + which * h_pitch + i) = q;
      if (lane_id() == 0) SQ[static_cast<int64_t>(which * blocks + b) * R + row] = blk::block_down(am);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(0xffffffffu, part, o);
  if (lane_id() == 0) s_part[threadIdx.x >> 5] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    float s = s_part[0];
    for (int i = 1; i < 8; ++i) s += s_part[i];
    dw[r] = s;
  }
}

// ------------------------------------------------------------------ sum over a token's experts
// out[t] = sum_j w[t,j] * V[place[t*k+j]] over the choices that have an expert, in the order of
// the choices, in fp32, rounded once; weights NULL: all 1.  A thread holds 8 columns.
template <bool kBf16>
__global__ void __launch_bounds__(256)
    combine_kernel(const float* __restrict__ V, const int32_t* __restrict__ place,
                   const float* __restrict__ weights, int64_t T, int k, int64_t K, uint16_t* __restrict__ out) {
  grid_dep_wait();
  const int64_t per = K / 8;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  const int64_t t = at / per;
  if (t >= T) return;
  const int64_t c = (at - t * per) * 8;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < k; ++j) {
    const int p = __ldg(place + t * k + j);
    if (p < 0) continue;
    const float w = weights != nullptr ? __ldg(weights + t * k + j) : 1.0f;
    const float4 x = __ldg(reinterpret_cast<const float4*>(V + static_cast<int64_t>(p) * K + c));
    const float4 y = __ldg(reinterpret_cast<const float4*>(V + static_cast<int64_t>(p) * K + c + 4));
    s[0] = fmaf(w, x.x, s[0]);
    s[1] = fmaf(w, x.y, s[1]);
    s[2] = fmaf(w, x.z, s[2]);
    s[3] = fmaf(w, x.w, s[3]);
    s[4] = fmaf(w, y.x, s[4]);
    s[5] = fmaf(w, y.y, s[5]);
    s[6] = fmaf(w, y.z, s[6]);
    s[7] = fmaf(w, y.w, s[7]);
  }
  *reinterpret_cast<uint4*>(out + t * K + c) =
      make_uint4(blk::pack2<kBf16>(s[0], s[1]), blk::pack2<kBf16>(s[2], s[3]), blk::pack2<kBf16>(s[4], s[5]), blk::pack2<kBf16>(s[6], s[7]));
}

}  // namespace moe
}  // namespace i8
