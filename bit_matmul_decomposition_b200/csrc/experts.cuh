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

// An fp64 key as an unsigned number of the same order (0 below all of them: no live expert).
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v + 0.0));   // -0 as +0
  return (b >> 63) ? ~b : b | 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered(uint64_t k) {
  return __longlong_as_double(static_cast<long long>((k >> 63) ? k & 0x7fffffffffffffffull : ~k));
}

// The warp's largest key and the lowest index that has it.  The high words decide unless two lanes
// share the largest; one hardware reduction in place of five exchanges of key and index.
__device__ __forceinline__ void warp_best(uint64_t& key, int& e) {
  const uint32_t hi = static_cast<uint32_t>(key >> 32);
  const uint32_t mh = __reduce_max_sync(0xffffffffu, hi);
  unsigned who = __ballot_sync(0xffffffffu, hi == mh);
  if (who & (who - 1)) {
    const uint32_t lo = hi == mh ? static_cast<uint32_t>(key) : 0u;
    const uint32_t ml = __reduce_max_sync(0xffffffffu, lo);
    const bool mine = hi == mh && lo == ml;
    const int me = __reduce_min_sync(0xffffffffu, mine ? e : 0x7fffffff);
    key = (static_cast<uint64_t>(mh) << 32) | ml;
    e = me;
    return;
  }
  const int src = __ffs(who) - 1;
  key = __shfl_sync(0xffffffffu, key, src);
  e = __shfl_sync(0xffffffffu, e, src);
}

template <int kIn, int PER>
__global__ void __launch_bounds__(kRouteWarps * 32)
    route_kernel(const RouteArgs a) {
  __shared__ uint64_t s_key[kRouteWarps][PER * 32 + MAX_ROUTE_GROUPS];
  const int warp = threadIdx.x >> 5, lane = lane_id();
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRouteWarps + warp;
  if (t >= a.T) return;
  float x[PER];
  double p[PER];
  uint64_t key[PER];
  const bool good = route_scores<kIn, PER>(a, t, x, p);
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = i * 32 + lane;
    key[i] = 0ull;
    if (x[i] != __int_as_float(0xff800000)) {
      const double v = p[i] + (a.balance != nullptr ? static_cast<double>(__ldg(a.balance + e)) : 0.0);
      if (v > __longlong_as_double(0xfff0000000000000ll)) key[i] = ordered(v);   // a NaN or -inf key: never chosen
    }
  }
  if (a.groups > 1) {
    const int size = a.E / a.groups;
    // one word of padding a group, so that the lanes, one a group, read different banks
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = i * 32 + lane;
      if (e < a.E) s_key[warp][e + e / size] = key[i];
    }
    __syncwarp();
    uint64_t total = 0ull;
    if (lane < a.groups) {
      uint64_t b1 = 0ull, b2 = 0ull;
      for (int j = 0; j < size; ++j) {
        const uint64_t v = s_key[warp][lane * (size + 1) + j];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
      total = b1;
      if (a.balance != nullptr && b2 > 0ull) total = ordered(unordered(b1) + unordered(b2));
      total = total > 1ull ? total : 1ull;              // a group of masked experts: below all others
    }
    unsigned kept = 0u;
    int id = lane < a.groups ? lane : 64 + lane;        // a lane without a group: key 0, loses every tie
    for (int j = 0; j < a.top_groups; ++j) {
      uint64_t b = total;
      int g = id;
      warp_best(b, g);
      if (g < 32) kept |= 1u << g;
      if (g == id) {
        total = 0ull;                                   // taken
        id = 64 + lane;
      }
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = i * 32 + lane;
      if (e < a.E && !((kept >> (e / size)) & 1u)) key[i] = 0ull;
    }
  }
  // The scores by expert, for the lanes that will hold the choices; and the high words of the keys,
  // which decide the order by themselves unless two are equal (keys within 2^-20 of one another).
  __syncwarp();
  double* score = reinterpret_cast<double*>(s_key[warp]);
  uint32_t hi[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    score[i * 32 + lane] = p[i];
    hi[i] = static_cast<uint32_t>(key[i] >> 32);
  }
  int mine_e = -1;                                      // lane j keeps choice j
  for (int j = 0; j < a.k; ++j) {
    uint32_t m = 0u;
#pragma unroll
    for (int i = 0; i < PER; ++i) m = max(m, hi[i]);
    m = __reduce_max_sync(0xffffffffu, m);
    if (m == 0u) {                                      // no key with a high word is left: dead, or the 1 of a dead group
      break;
    }
    int at = 0, have = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (hi[i] == m) {
        at = i;
        ++have;
      }
    const unsigned who = __ballot_sync(0xffffffffu, have > 0);
    int e;
    if ((who & (who - 1)) == 0u && __ballot_sync(0xffffffffu, have > 1) == 0u) {
      e = __shfl_sync(0xffffffffu, at * 32 + lane, __ffs(who) - 1);
    } else {                                            // equal high words: the low ones, then the index
      uint32_t lo = 0u;
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (hi[i] == m) lo = max(lo, static_cast<uint32_t>(key[i]));
      lo = __reduce_max_sync(0xffffffffu, lo);
      int first = 0x7fffffff;
#pragma unroll
      for (int i = PER - 1; i >= 0; --i)
        if (hi[i] == m && static_cast<uint32_t>(key[i]) == lo) first = i * 32 + lane;
      e = __reduce_min_sync(0xffffffffu, first);
    }
    if (lane == (e & 31)) {
#pragma unroll
      for (int i = 0; i < PER; ++i)
        if (i == (e >> 5)) hi[i] = 0u;
    }
    if (lane == j) mine_e = e;
  }
  __syncwarp();
  const double mine_p = mine_e >= 0 ? score[mine_e] : 0.0;
  double sum = 0.0;                                     // in the order of the choices
  for (int j = 0; j < a.k; ++j) sum += __shfl_sync(0xffffffffu, mine_p, j);
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
  // every warp its own run of rows: counts, then positions, with one meeting of the CTA between
  const int64_t per = ((R + kSortThreads - 1) / kSortThreads) * 32;
  const int64_t r0 = warp * per, r1 = r0 + per < R ? r0 + per : R;
  int less = 0, eq = 0;
#pragma unroll 4
  for (int64_t r = r0 + lane; r < r1; r += 32) {
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
  int first = 0, total = 0, at = 0;
  for (int w = 0; w < kSortThreads / 32; ++w) {
    first += s_less[w];
    total += s_eq[w];
    if (w < warp) at += s_eq[w];
  }
  if (threadIdx.x == 0) {
    offsets[e] = first;
    if (e == E - 1) offsets[E] = first + total;
  }
  if (eq == 0) return;
  at += first;
#pragma unroll 4
  for (int64_t r = r0; r < r1; r += 32) {
    const bool hit = r + lane < r1 && __ldg(idx + r + lane) == e;
    const unsigned bits = __ballot_sync(0xffffffffu, hit);
    if (hit) {
      const int to = at + __popc(bits & ((1u << lane) - 1u));
      place[r + lane] = to;
      row_at[to] = static_cast<int32_t>(r + lane);
    }
    at += __popc(bits);
  }
}

// ------------------------------------------------------------------ gated activation
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
  for (int j0 = 0; j0 < k; j0 += 4) {               // four rows' loads in flight
    int p[4];
    float w[4];
    float4 x[4], y[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      p[u] = j0 + u < k ? __ldg(place + t * k + j0 + u) : -1;
      w[u] = p[u] < 0 ? 0.0f : weights != nullptr ? __ldg(weights + t * k + j0 + u) : 1.0f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (p[u] >= 0) {
        x[u] = __ldg(reinterpret_cast<const float4*>(V + static_cast<int64_t>(p[u]) * K + c));
        y[u] = __ldg(reinterpret_cast<const float4*>(V + static_cast<int64_t>(p[u]) * K + c + 4));
      }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (p[u] >= 0) {
        s[0] = fmaf(w[u], x[u].x, s[0]);
        s[1] = fmaf(w[u], x[u].y, s[1]);
        s[2] = fmaf(w[u], x[u].z, s[2]);
        s[3] = fmaf(w[u], x[u].w, s[3]);
        s[4] = fmaf(w[u], y[u].x, s[4]);
        s[5] = fmaf(w[u], y[u].y, s[5]);
        s[6] = fmaf(w[u], y[u].z, s[6]);
        s[7] = fmaf(w[u], y[u].w, s[7]);
      }
  }
  *reinterpret_cast<uint4*>(out + t * K + c) =
      make_uint4(blk::pack2<kBf16>(s[0], s[1]), blk::pack2<kBf16>(s[2], s[3]), blk::pack2<kBf16>(s[4], s[5]), blk::pack2<kBf16>(s[6], s[7]));
}

}  // namespace moe
}  // namespace i8
