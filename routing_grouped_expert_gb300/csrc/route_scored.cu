// Scored routing and its gradient.
//
// Forward, per token: scores s_e = 1 / (1 + exp(-l_e)) or softmax(l)_e; the
// choice ranks r_e = s_e + b_e with a balance bias b, and by the logits
// themselves without one (s rises with l); with groups of E / G consecutive
// experts, only the experts of the best groups are candidates, a group being
// worth its largest r or the sum of its two largest s + b; the k best
// candidates are taken, equal values going to the lower index; the weights are
// scale * s_j, or scale * s_j / sum of the chosen s.  The bias takes part in the
// choice only.
//
// Everything that decides the choice is plain fp32 arithmetic, each operation
// rounded to nearest (1 / (1 + expf(-l)), e / S with S the sum of the e rounded
// once, s + b, the sum of two group members): the picks are a function of the
// inputs, not of a reduction order.  S is accumulated as an unevaluated pair
// of floats (error-free additions), so it is the correctly rounded sum for any
// order of the lanes.
#include <math.h>

#include "route_token.cuh"

namespace moe {
namespace {

constexpr int kMaxWarps = 8;

// hi + lo += x without losing bits (Knuth's two-sum).
__device__ __forceinline__ void pair_add(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x);
  const float b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
  hi = s;
}
// The sum over the warp of a pair of floats per lane, rounded once.
__device__ __forceinline__ float warp_sum_rounded(float hi, float lo) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float ohi = __shfl_xor_sync(0xffffffffu, hi, off);
    const float olo = __shfl_xor_sync(0xffffffffu, lo, off);
    lo = __fadd_rn(lo, olo);
    pair_add(hi, lo, ohi);
  }
  return __fadd_rn(hi, lo);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
  return route_key_value(__reduce_max_sync(0xffffffffu, route_key(v)));
}

__device__ __forceinline__ float sigmoid_rn(float l) {
  return __fdiv_rn(1.f, __fadd_rn(1.f, expf(-l)));
}

// Weight of the pick that lane j < k holds (logit l; `on` false: no pick, or
// an expert switched off by its bias).  m, S: the row's largest logit and the
// sum of exp(l_e - m) (softmax without renormalisation only).
__device__ __forceinline__ float pick_weight(const RouteCfg& c, float l, bool on, float m,
                                             float S) {
  float s = 0.f;
  if (!c.renorm) {
    if (on) s = c.softmax ? __fdiv_rn(expf(l - m), S) : sigmoid_rn(l);
    return c.scale * s;
  }
  // Renormalised: a common factor of the chosen scores cancels.  Softmax scores
  // are exp(l - mx) up to one; sigmoid scores are exp(l) to 2^-57 where every
  // chosen logit is below -40, which keeps very low scores from vanishing.
  const float mx = warp_max(on ? l : -INFINITY);
  if (on) s = (c.softmax || mx < -40.f) ? expf(l - mx) : sigmoid_rn(l);
  const float sum = warp_sum(s);
  return sum > 0.f ? c.scale * (s / sum) : 0.f;
}

// One warp per token.  kPerLane logits per lane (expert lane + 32 i).
template <int kPerLane, bool kGroups>
__global__ void __launch_bounds__(32 * kMaxWarps)
route_scored_kernel(const float* __restrict__ logits, const float* __restrict__ bias, RouteCfg c,
                    int T, int E, int k, int tpc, int group_pad, int32_t* __restrict__ topk_idx,
                    float* __restrict__ topk_w, int32_t* __restrict__ chunk_hist,
                    int* __restrict__ status) {
  extern __shared__ float stage[];   // [warps][n_group * (group size + pad)] when grouped
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= T) return;
  const float* row = logits + (size_t)t * E;
  float v[kPerLane];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 32 * i;
    v[i] = e < E ? __ldg(row + e) : -INFINITY;
    bad |= e < E && !isfinite(v[i]);
  }
  // softmax: the row's maximum and the sum of exp(l - m)
  const bool two = kGroups && c.group_top == 2;
  const bool scored = bias != nullptr || two;   // the scores take part in the choice
  float m = 0.f, S = 1.f;
  if (c.softmax && (scored || !c.renorm)) {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) mx = fmaxf(mx, v[i]);
    m = warp_max(mx);
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      if (lane + 32 * i < E) pair_add(hi, lo, expf(v[i] - m));
    S = warp_sum_rounded(hi, lo);
  }
  // b: score (+ bias), the value that the two best of a group add up;
  // r: the value that ranks
  uint32_t key[kPerLane];
  const int gsz = kGroups ? E / c.n_group : E;
  float* st = kGroups ? stage + (size_t)warp * c.n_group * (gsz + group_pad) : nullptr;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + 32 * i;
    float r = v[i], b = v[i];
    if (scored && e < E) {
      b = c.softmax ? __fdiv_rn(expf(v[i] - m), S) : sigmoid_rn(v[i]);
      if (bias != nullptr) {
        const float be = __ldg(bias + e);
        bad |= !(be < INFINITY);   // NaN or +inf: -inf switches an expert off
        b = __fadd_rn(b, be);
        r = b;
      }
    }
    if (isnan(r)) r = -INFINITY;   // keep the order total; the status reports it
    key[i] = e < E ? route_key(r) : 0u;
    if (kGroups && e < E) {
      const int g = (int)((uint32_t)e * c.group_magic >> 20);
      st[e + g * group_pad] = two ? (isnan(b) ? -INFINITY : b) : r;
    }
  }
  if constexpr (kGroups) {
    __syncwarp();
    // lanes_per_group lanes scan one group: its two largest values
    const int lpg = c.lanes_per_group, sub = lane & (lpg - 1), g = lane / lpg;
    float a1 = -INFINITY, a2 = -INFINITY;
    if (g < c.n_group) {
      const float* gs = st + g * (gsz + group_pad);
      for (int j = sub; j < gsz; j += lpg) {
        const float x = gs[j];
        a2 = fmaxf(a2, fminf(a1, x));
        a1 = fmaxf(a1, x);
      }
    }
    for (int off = 1; off < lpg; off <<= 1) {
      const float o1 = __shfl_xor_sync(0xffffffffu, a1, off);
      const float o2 = __shfl_xor_sync(0xffffffffu, a2, off);
      a2 = fmaxf(fmaxf(a2, o2), fminf(a1, o1));
      a1 = fmaxf(a1, o1);
    }
    const uint32_t gk = route_key(two ? __fadd_rn(a1, a2) : a1);
    // a group's place among the groups: how many come before it
    int before = 0;
    for (int o = 0; o < c.n_group; ++o) {
      const uint32_t ok = __shfl_sync(0xffffffffu, gk, o * lpg);
      before += ok > gk || (ok == gk && o < g);
    }
    // bit l set: lane l's group is kept
    const unsigned kept = __ballot_sync(0xffffffffu, g < c.n_group && before < c.topk_group);
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + 32 * i;
      const int ge = (int)((uint32_t)e * c.group_magic >> 20);
      if (e < E && !((kept >> (ge * lpg)) & 1u)) key[i] = 0u;   // no candidate
    }
  }
  uint32_t my_key;
  int my_idx;
  route_select<kPerLane>(key, k, lane, &my_key, &my_idx);
  // the picks' logits, and whether the bias switched the expert off
  const bool have = lane < k;
  const int idx = have ? my_idx : 0;
  const float l = have ? __ldg(row + idx) : 0.f;
  const bool on = have && (bias == nullptr || __ldg(bias + idx) != -INFINITY);
  const float w = pick_weight(c, l, on, m, S);
  if (have) {
    topk_idx[(size_t)t * k + lane] = idx;
    topk_w[(size_t)t * k + lane] = w;
    if (chunk_hist) atomicAdd(&chunk_hist[(size_t)(t / tpc) * E + idx], 1);
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(status, MOE_ERR_NONFINITE);
}

// Gradient of the weights with respect to the logits, one warp per token.
//   sigmoid, renormalised:  dl_j = scale w_j (dw_j - sum_i w_i dw_i) (1 - s_j), w = s / sum s
//   sigmoid:                dl_j = scale dw_j s_j (1 - s_j)
//   softmax, renormalised:  dl_j = scale w_j (dw_j - sum_i w_i dw_i)
//   softmax (kDense):       dl_e = s_e (scale dw_e - D), D = sum_j scale dw_j s_j
// The first three are zero at every expert that was not chosen.
template <bool kDense>
__global__ void __launch_bounds__(32 * kMaxWarps)
route_scored_backward_kernel(const float* __restrict__ dw, const int32_t* __restrict__ topk_idx,
                             const float* __restrict__ logits, const float* __restrict__ bias,
                             RouteCfg c, int T, int E, int k, float* __restrict__ dlogits,
                             int* __restrict__ status) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * (blockDim.x >> 5) + warp;
  if (t >= T) return;
  const float* row = logits + (size_t)t * E;
  float* out = dlogits + (size_t)t * E;
  const int idx = lane < k ? __ldg(topk_idx + (size_t)t * k + lane) : 0;
  const bool in = idx >= 0 && idx < E;
  const bool on = lane < k && in && (bias == nullptr || __ldg(bias + idx) != -INFINITY);
  const float l = on ? __ldg(row + idx) : 0.f;
  const float g = on ? c.scale * __ldg(dw + (size_t)t * k + lane) : 0.f;
  bool bad = on && !isfinite(l);
  float d;
  if constexpr (kDense) {
    float mx = -INFINITY;
    for (int e = lane; e < E; e += 32) {
      const float x = __ldg(row + e);
      bad |= !isfinite(x);
      mx = fmaxf(mx, x);
    }
    const float m = warp_max(mx);
    float sum = 0.f;
    for (int e = lane; e < E; e += 32) sum += expf(__ldg(row + e) - m);
    const float S = warp_sum(sum);
    const float s = on ? __fdiv_rn(expf(l - m), S) : 0.f;
    const float D = warp_sum(g * s);
    for (int e = lane; e < E; e += 32) out[e] = -D * __fdiv_rn(expf(__ldg(row + e) - m), S);
    d = s * (g - D);
  } else {
    for (int e = lane; e < E; e += 32) out[e] = 0.f;
    const float rest = c.softmax ? 1.f : __fdiv_rn(1.f, 1.f + expf(l));   // 1 - s, no cancellation
    if (c.renorm) {
      RouteCfg unit = c;
      unit.scale = 1.f;
      const float w = pick_weight(unit, l, on, 0.f, 1.f);
      d = w * (g - warp_sum(w * g)) * rest;
    } else {
      d = g * sigmoid_rn(l) * rest;
    }
  }
  __syncwarp();   // the row's first values before the picks' own
  if (on) out[idx] = d;
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(status, MOE_ERR_NONFINITE);
  if (__any_sync(0xffffffffu, lane < k && !in) && lane == 0) set_status(status, MOE_ERR_INVALID_ARG);
}

template <int kPerLane>
cudaError_t launch_t(const float* logits, const float* bias, const RouteCfg& c, int T, int E, int k,
                     int32_t* topk_idx, float* topk_w, int32_t* chunk_hist, int* status,
                     cudaStream_t s) {
  const int tpc = tokens_per_chunk(k);
  if (c.n_group > 1) {
    // a group starts lanes_per_group banks after the one before it, so the
    // lanes that scan the groups read different banks
    const int gsz = E / c.n_group;
    const int pad = (c.lanes_per_group - gsz % 32 + 32) % 32;
    const size_t per_warp = (size_t)c.n_group * (gsz + pad) * 4;
    const int warps = per_warp * kMaxWarps <= 48 * 1024 ? kMaxWarps : kMaxWarps / 2;
    route_scored_kernel<kPerLane, true><<<(T + warps - 1) / warps, 32 * warps, per_warp * warps,
                                          s>>>(logits, bias, c, T, E, k, tpc, pad, topk_idx,
                                               topk_w, chunk_hist, status);
  } else {
    route_scored_kernel<kPerLane, false><<<(T + kMaxWarps - 1) / kMaxWarps, 32 * kMaxWarps, 0,
                                           s>>>(logits, bias, c, T, E, k, tpc, 0, topk_idx,
                                                topk_w, chunk_hist, status);
  }
  return cudaGetLastError();
}

}  // namespace

RouteCfg make_route_cfg(const moe_route_config& a, int E) {
  RouteCfg c{};
  c.softmax = a.score == MOE_SCORE_SOFTMAX;
  c.renorm = a.renormalize != 0;
  c.scale = a.scale;
  c.n_group = a.n_group;
  c.topk_group = a.topk_group;
  c.group_top = a.group_top;
  int lanes = 32;
  while (lanes * a.n_group > 32) lanes >>= 1;
  c.lanes_per_group = lanes;
  // e / (E / n_group) = e * magic >> 20 for every e < 1024
  c.group_magic = (1u << 20) / (uint32_t)(E / a.n_group) + 1;
  return c;
}

cudaError_t launch_route_scored(const float* logits, const float* bias, const RouteCfg& c, int T,
                                int E, int k, int32_t* topk_idx, float* topk_w,
                                int32_t* chunk_hist, int* status, cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  if (E <= 32)
    return launch_t<1>(logits, bias, c, T, E, k, topk_idx, topk_w, chunk_hist, status, s);
  if (E <= 64)
    return launch_t<2>(logits, bias, c, T, E, k, topk_idx, topk_w, chunk_hist, status, s);
  if (E <= 128)
    return launch_t<4>(logits, bias, c, T, E, k, topk_idx, topk_w, chunk_hist, status, s);
  if (E <= 256)
    return launch_t<8>(logits, bias, c, T, E, k, topk_idx, topk_w, chunk_hist, status, s);
  if (E <= 512)
    return launch_t<16>(logits, bias, c, T, E, k, topk_idx, topk_w, chunk_hist, status, s);
  return launch_t<32>(logits, bias, c, T, E, k, topk_idx, topk_w, chunk_hist, status, s);
}

cudaError_t launch_route_scored_backward(const float* dw, const int32_t* topk_idx,
                                         const float* logits, const float* bias, const RouteCfg& c,
                                         int T, int E, int k, float* dlogits, int* status,
                                         cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const int grid = (T + kMaxWarps - 1) / kMaxWarps;
  if (c.softmax && !c.renorm)
    route_scored_backward_kernel<true><<<grid, 32 * kMaxWarps, 0, s>>>(dw, topk_idx, logits, bias,
                                                                       c, T, E, k, dlogits, status);
  else
    route_scored_backward_kernel<false><<<grid, 32 * kMaxWarps, 0, s>>>(
        dw, topk_idx, logits, bias, c, T, E, k, dlogits, status);
  return cudaGetLastError();
}

}  // namespace moe
