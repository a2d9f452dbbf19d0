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

// Lanes per token L: 8 or 16 where the experts fit (a warp then routes four or
// two tokens), else 32.  Reductions over a token's lanes:
template <int L>
__device__ __forceinline__ uint32_t seg_max(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_max_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
  }
}
template <int L>
__device__ __forceinline__ uint32_t seg_min(uint32_t v) {
  if constexpr (L == 32) {
    return __reduce_min_sync(0xffffffffu, v);
  } else {
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1) v = min(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
  }
}
template <int L>
__device__ __forceinline__ float seg_sum(float v) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
template <int L>
__device__ __forceinline__ float seg_max(float v) {
  return route_key_value(seg_max<L>(route_key(v)));
}
// This token's bits of a warp-wide ballot.
template <int L>
__device__ __forceinline__ unsigned seg_ballot(bool p) {
  const unsigned m = __ballot_sync(0xffffffffu, p);
  if constexpr (L == 32) return m;
  else return (m >> (threadIdx.x & 31 & ~(L - 1))) & ((1u << L) - 1u);
}

// hi + lo += x without losing bits (Knuth's two-sum).
__device__ __forceinline__ void pair_add(float& hi, float& lo, float x) {
  const float s = __fadd_rn(hi, x);
  const float b = __fsub_rn(s, hi);
  lo = __fadd_rn(lo, __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)));
  hi = s;
}
// The sum over a token's lanes of a pair of floats per lane, rounded once.
template <int L>
__device__ __forceinline__ float seg_sum_rounded(float hi, float lo) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) {
    const float ohi = __shfl_xor_sync(0xffffffffu, hi, off);
    const float olo = __shfl_xor_sync(0xffffffffu, lo, off);
    lo = __fadd_rn(lo, olo);
    pair_add(hi, lo, ohi);
  }
  return __fadd_rn(hi, lo);
}

// 1 / (1 + exp(-l)); the reciprocal is the correctly rounded quotient, in
// fewer instructions than a division.
__device__ __forceinline__ float sigmoid_rn(float l) {
  return __frcp_rn(__fadd_rn(1.f, expf(-l)));
}

// Weight of the pick that lane j < k of a token holds (logit l; `on` false: no
// pick, or an expert switched off by its bias).  m, S: the row's largest logit
// and the sum of exp(l_e - m) (softmax without renormalisation only).
template <int L>
__device__ __forceinline__ float pick_weight(bool softmax, bool renorm, float scale, float l,
                                             bool on, float m, float S) {
  float s = 0.f;
  if (!renorm) {
    if (on) s = softmax ? __fdiv_rn(expf(l - m), S) : sigmoid_rn(l);
    return scale * s;
  }
  // Renormalised: a common factor of the chosen scores cancels.  Softmax scores
  // are exp(l - mx) up to one; sigmoid scores are exp(l) to 2^-57 where every
  // chosen logit is below -40, which keeps very low scores from vanishing.
  const float mx = seg_max<L>(on ? l : -INFINITY);
  if (on) s = (softmax || mx < -40.f) ? expf(l - mx) : sigmoid_rn(l);
  const float sum = seg_sum<L>(s);
  return sum > 0.f ? scale * (s / sum) : 0.f;
}

// The k largest of a token's candidates: lane i's keys are those of candidates
// lane + L i (0: none); lane j < k returns slot j's candidate.  A larger key wins,
// equal keys go to the lower candidate.  Up to eight keys per lane are sorted
// once (route_select); with more, each round rescans the winner's keys instead:
// 4 n instructions a round against 5 n (n - 1) / 2 for the sort.
template <int kPerLane, int L>
__device__ __forceinline__ int select_best(uint32_t (&key)[kPerLane], int k, int lane) {
  if constexpr (L == 32 && kPerLane <= 8) {
    uint32_t sel_key;
    int sel;
    route_select<kPerLane>(key, k, lane, &sel_key, &sel);
    return sel;
  } else {
    uint32_t best = 0u;
    int slot = 0, mine = 0;
    auto scan = [&]() {
      best = key[0];
      slot = 0;
#pragma unroll
      for (int i = 1; i < kPerLane; ++i)
        if (key[i] > best) {
          best = key[i];
          slot = i;
        }
    };
    scan();
    for (int j = 0; j < k; ++j) {
      const uint32_t m = seg_max<L>(best);
      const uint32_t win =
          seg_min<L>(best == m && m != 0u ? (uint32_t)(lane + L * slot) : ~0u);
      if (lane == j) mine = (int)win;
      if (m != 0u && (int)(win & (L - 1)) == lane) {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
          if (i == slot) key[i] = 0u;
        scan();
      }
    }
    return mine;
  }
}

// One token per L lanes, kPerLane logits per lane (expert lane + L i).  Bound by
// instruction issue, not memory: about 25 instructions per score (exp and a
// correctly rounded reciprocal or quotient) and 25 per selection round; so a
// token's candidates are compacted to the kept groups before the selection
// (8 groups of 32, 4 kept: four keys per lane to sort instead of eight).
template <int kPerLane, int L, bool kGroups>
__global__ void __launch_bounds__(32 * kMaxWarps)
route_scored_kernel(const float* __restrict__ logits, const float* __restrict__ bias, RouteCfg c,
                    int T, int E, int k, int tpc, int group_pad, int32_t* __restrict__ topk_idx,
                    float* __restrict__ topk_w, int32_t* __restrict__ chunk_hist,
                    int* __restrict__ status, bool whole) {
  // per token of the block: n_group * (group size + pad) values, n_group kept groups
  extern __shared__ float stage[];
  pdl_trigger();
  const int lane = threadIdx.x & (L - 1), seg = threadIdx.x / L;   // seg: the block's token
  const int t0 = blockIdx.x * (blockDim.x / L) + seg;
  const bool live = t0 < T;
  // a warp without a token leaves, unless the grid reports together
  if (!whole && !__any_sync(0xffffffffu, live)) return;
  const int t = live ? t0 : T - 1;
  const float* row = logits + (size_t)t * E;
  float v[kPerLane];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + L * i;
    v[i] = e < E ? __ldg(row + e) : -INFINITY;
    bad |= e < E && !isfinite(v[i]);
  }
  // softmax: the row's maximum and the sum of exp(l - m)
  const bool two = kGroups && c.group_top == 2;
  const bool scored = bias != nullptr || two;   // the scores take part in the choice
  float m = 0.f, S = 1.f;
  float ex[kPerLane];
  if (c.softmax && (scored || !c.renorm)) {
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) mx = fmaxf(mx, v[i]);
    m = seg_max<L>(mx);
    float hi = 0.f, lo = 0.f;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      ex[i] = lane + L * i < E ? expf(v[i] - m) : 0.f;
      pair_add(hi, lo, ex[i]);
    }
    S = seg_sum_rounded<L>(hi, lo);
  }
  // b: score (+ bias), the value that the two best of a group add up;
  // r: the value that ranks
  uint32_t key[kPerLane];
  const int gsz = kGroups ? E / c.n_group : E;
  float* st = kGroups ? stage + (size_t)seg * c.n_group * (gsz + group_pad + 1) : nullptr;
#pragma unroll
  for (int i = 0; i < kPerLane; ++i) {
    const int e = lane + L * i;
    float r = v[i], b = v[i];
    if (scored && e < E) {
      b = c.softmax ? __fdiv_rn(ex[i], S) : sigmoid_rn(v[i]);
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
  int idx;
  if constexpr (!kGroups) {
    idx = select_best<kPerLane, L>(key, k, lane);
  } else {
    __syncwarp();
    // lpg lanes scan one group: its two largest values
    const int lpg = c.lanes_per_group / (32 / L), sub = lane & (lpg - 1), g = lane / lpg;
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
      const uint32_t ok = __shfl_sync(0xffffffffu, gk, o * lpg, L);
      before += ok > gk || (ok == gk && o < g);
    }
    // the kept groups, ascending
    const bool keep = sub == 0 && g < c.n_group && before < c.topk_group;
    const unsigned kept = seg_ballot<L>(keep);
    __syncwarp();   // every lane has scanned its group
    int* list = reinterpret_cast<int*>(st) + c.n_group * (gsz + group_pad);
    if (keep) list[__popc(kept & ((1u << lane) - 1u))] = g;
    // The keys of all experts take the place of the group values: candidate j,
    // the j-th expert of the kept groups in ascending order, is read from them.
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + L * i;
      const int ge = (int)((uint32_t)e * c.group_magic >> 20);
      if (e < E) reinterpret_cast<uint32_t*>(st)[e + ge * group_pad] = key[i];
    }
    __syncwarp();
    const int n_cand = c.topk_group * gsz;
    auto expert_of = [&](int j) {
      const int cg = (int)((uint32_t)j * c.group_magic >> 20);
      return list[cg] * gsz + (j - cg * gsz);
    };
    auto load = [&](int j) {
      if (j >= n_cand) return 0u;
      const int cg = (int)((uint32_t)j * c.group_magic >> 20);
      return reinterpret_cast<const uint32_t*>(st)[list[cg] * (gsz + group_pad) + j - cg * gsz];
    };
    int pick;
    if (kPerLane > 1 && n_cand <= L * (kPerLane / 2)) {
      constexpr int kHalf = kPerLane > 1 ? kPerLane / 2 : 1;
      uint32_t half[kHalf];
#pragma unroll
      for (int i = 0; i < kHalf; ++i) half[i] = load(lane + L * i);
      pick = select_best<kHalf, L>(half, k, lane);
    } else {
#pragma unroll
      for (int i = 0; i < kPerLane; ++i) key[i] = load(lane + L * i);
      pick = select_best<kPerLane, L>(key, k, lane);
    }
    idx = lane < k ? expert_of(pick) : 0;
  }
  // the picks' logits, and whether the bias switched the expert off
  const bool have = lane < k;
  if (!have) idx = 0;
  const float l = have ? __ldg(row + idx) : 0.f;
  const bool on = have && (bias == nullptr || __ldg(bias + idx) != -INFINITY);
  const float w = pick_weight<L>(c.softmax, c.renorm, c.scale, l, on, m, S);
  if (have && live) {
    topk_idx[(size_t)t * k + lane] = idx;
    topk_w[(size_t)t * k + lane] = w;
    if (chunk_hist) atomicAdd(&chunk_hist[(size_t)(t / tpc) * E + idx], 1);
  }
  if (whole) {
    // a batch that one block routes: it writes the status itself
    const int any = __syncthreads_or(bad);
    if (threadIdx.x < 2) status[threadIdx.x] = threadIdx.x == 0 && any ? MOE_ERR_NONFINITE : 0;
  } else if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) {
    set_status(status, MOE_ERR_NONFINITE);
  }
}

// Gradient of the weights with respect to the logits, one warp per token.
//   sigmoid, renormalised:  dl_j = scale w_j (dw_j - sum_i w_i dw_i) (1 - s_j), w = s / sum s
//   sigmoid:                dl_j = scale dw_j s_j (1 - s_j)
//   softmax, renormalised:  dl_j = scale w_j (dw_j - sum_i w_i dw_i)
//   softmax (kDense):       dl_e = s_e (scale dw_e - D), D = sum_j scale dw_j s_j
// The first three are zero at every expert that was not chosen; they are bound
// by writing dlogits.  kDense > 0: that many logits per lane are kept from the
// first read to the last write.
template <int kDense>
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
  if constexpr (kDense > 0) {
    float v[kDense];
    float mx = -INFINITY;
#pragma unroll
    for (int i = 0; i < kDense; ++i) {
      const int e = lane + 32 * i;
      v[i] = e < E ? __ldg(row + e) : -INFINITY;
      bad |= e < E && !isfinite(v[i]);
      mx = fmaxf(mx, v[i]);
    }
    const float m = seg_max<32>(mx);
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kDense; ++i) {
      v[i] = lane + 32 * i < E ? expf(v[i] - m) : 0.f;
      sum += v[i];
    }
    const float inv = 1.f / seg_sum<32>(sum);
    const float s = on ? expf(l - m) * inv : 0.f;
    const float D = seg_sum<32>(g * s);
#pragma unroll
    for (int i = 0; i < kDense; ++i)
      if (lane + 32 * i < E) out[lane + 32 * i] = -D * (v[i] * inv);
    d = s * (g - D);
  } else {
    if ((E & 3) == 0) {   // rows are 16-byte aligned
      for (int e = lane; e < E / 4; e += 32)
        reinterpret_cast<float4*>(out)[e] = make_float4(0.f, 0.f, 0.f, 0.f);
    } else {
      for (int e = lane; e < E; e += 32) out[e] = 0.f;
    }
    const float rest = c.softmax ? 1.f : __frcp_rn(1.f + expf(l));   // 1 - s, no cancellation
    if (c.renorm) {
      const float w = pick_weight<32>(c.softmax, true, 1.f, l, on, 0.f, 1.f);
      d = w * (g - seg_sum<32>(w * g)) * rest;
    } else {
      d = g * sigmoid_rn(l) * rest;
    }
  }
  __syncwarp();   // the row's first values before the picks' own
  if (on) out[idx] = d;
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(status, MOE_ERR_NONFINITE);
  if (__any_sync(0xffffffffu, lane < k && !in) && lane == 0) set_status(status, MOE_ERR_INVALID_ARG);
}

template <int kPerLane, int L>
cudaError_t launch_t(const float* logits, const float* bias, const RouteCfg& c, int T, int E, int k,
                     int32_t* topk_idx, float* topk_w, int32_t* chunk_hist, int* status, bool whole,
                     cudaStream_t s) {
  const int tpc = tokens_per_chunk(k);
  const int per_warp = 32 / L;
  if (c.n_group > 1) {
    // a group starts as many banks after the one before it as lanes scan it, so
    // the lanes that scan the groups of a token read different banks
    const int gsz = E / c.n_group, lpg = c.lanes_per_group / per_warp;
    const int pad = (lpg - gsz % 32 + 32) % 32;
    const size_t bytes = (size_t)c.n_group * (gsz + pad + 1) * 4 * per_warp;
    const int warps = bytes * kMaxWarps <= 48 * 1024 ? kMaxWarps : kMaxWarps / 2;
    const int per_block = warps * per_warp;
    route_scored_kernel<kPerLane, L, true>
        <<<(T + per_block - 1) / per_block, 32 * warps, bytes * warps, s>>>(
            logits, bias, c, T, E, k, tpc, pad, topk_idx, topk_w, chunk_hist, status,
            whole && T <= per_block);
  } else {
    const int per_block = kMaxWarps * per_warp;
    route_scored_kernel<kPerLane, L, false>
        <<<(T + per_block - 1) / per_block, 32 * kMaxWarps, 0, s>>>(
            logits, bias, c, T, E, k, tpc, 0, topk_idx, topk_w, chunk_hist, status,
            whole && T <= per_block);
  }
  return cudaGetLastError();
}

// Lanes per token for E experts (k <= E, and at most E groups).
int lanes_of(int E) { return E <= 8 ? 8 : E <= 16 ? 16 : 32; }

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

// Tokens that one block routes: the block writes the status itself.
bool route_scored_whole(int T, int E) {
  const int per_warp = 32 / lanes_of(E);
  return T <= kMaxWarps / 2 * per_warp;
}

cudaError_t launch_route_scored(const float* logits, const float* bias, const RouteCfg& c, int T,
                                int E, int k, int32_t* topk_idx, float* topk_w,
                                int32_t* chunk_hist, int* status, cudaStream_t s, bool whole) {
  if (T == 0) return cudaSuccess;
#define MOE_ROUTE_CASE(most, n, lanes) \
  if (E <= most)                       \
    return launch_t<n, lanes>(logits, bias, c, T, E, k, topk_idx, topk_w, chunk_hist, status, whole, s)
  MOE_ROUTE_CASE(8, 1, 8);
  MOE_ROUTE_CASE(16, 1, 16);
  MOE_ROUTE_CASE(32, 1, 32);
  MOE_ROUTE_CASE(64, 2, 32);
  MOE_ROUTE_CASE(96, 3, 32);
  MOE_ROUTE_CASE(128, 4, 32);
  MOE_ROUTE_CASE(160, 5, 32);
  MOE_ROUTE_CASE(192, 6, 32);
  MOE_ROUTE_CASE(256, 8, 32);
  MOE_ROUTE_CASE(384, 12, 32);
  MOE_ROUTE_CASE(512, 16, 32);
  MOE_ROUTE_CASE(MOE_MAX_EXPERTS, 32, 32);
#undef MOE_ROUTE_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_route_scored_backward(const float* dw, const int32_t* topk_idx,
                                         const float* logits, const float* bias, const RouteCfg& c,
                                         int T, int E, int k, float* dlogits, int* status,
                                         cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const int grid = (T + kMaxWarps - 1) / kMaxWarps;
#define MOE_ROUTE_BWD(n)                                                                       \
  route_scored_backward_kernel<n><<<grid, 32 * kMaxWarps, 0, s>>>(dw, topk_idx, logits, bias, c, T, \
                                                                  E, k, dlogits, status)
  if (!c.softmax || c.renorm) MOE_ROUTE_BWD(0);
  else if (E <= 32) MOE_ROUTE_BWD(1);
  else if (E <= 64) MOE_ROUTE_BWD(2);
  else if (E <= 128) MOE_ROUTE_BWD(4);
  else if (E <= 256) MOE_ROUTE_BWD(8);
  else if (E <= 512) MOE_ROUTE_BWD(16);
  else MOE_ROUTE_BWD(32);
#undef MOE_ROUTE_BWD
  return cudaGetLastError();
}

}  // namespace moe
