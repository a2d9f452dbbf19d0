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

// As route_key, in fewer instructions: -0 + 0 is +0, and the sign spread over
// the word flips the rest of a negative number.  A NaN gets a key like any
// other, which keeps the order total (the status reports it).
__device__ __forceinline__ uint32_t rank_key(float x) {
  const int b = __float_as_int(__fadd_rn(x, 0.f));
  return (uint32_t)(b ^ ((b >> 31) | (int)0x80000000));
}

// One token per L lanes, kPerLane logits per lane (expert lane + L i); the warps
// go through the tokens in strides, the next token's logits on their way.
// Bound by instruction issue, not memory (8192 tokens of 256 experts read 8.4
// MB, 1.3 us): about 25 instructions per score (exp and a correctly rounded
// reciprocal or quotient) and 20 per selection round.  So a token's candidates
// are compacted to the kept groups before the selection (8 groups of 32, 4
// kept: four keys per lane to sort instead of eight), everything but the scores
// is done on integer keys, and what depends on the expert alone (bias, place
// in shared memory) is worked out once per warp.
template <int kPerLane, int L, bool kGroups>
__global__ void __launch_bounds__(32 * kMaxWarps)
route_scored_kernel(const float* __restrict__ logits, const float* __restrict__ bias, RouteCfg c,
                    int T, int E, int k, int tpc, int group_pad, int32_t* __restrict__ topk_idx,
                    float* __restrict__ topk_w, int32_t* __restrict__ chunk_hist,
                    int* __restrict__ status, bool whole) {
  // per token of the block: n_group * (group size + pad) keys, n_group kept groups
  extern __shared__ uint32_t stage[];
  pdl_trigger();
  const int lane = threadIdx.x & (L - 1), seg = threadIdx.x / L;   // seg: the block's token
  const int per_block = blockDim.x / L, stride = gridDim.x * per_block;
  const bool two = kGroups && c.group_top == 2;
  const bool scored = bias != nullptr;       // all scores take part in the choice
  const bool need_s = scored || (two && c.softmax);   // the scores' exact sum decides
  const int gsz = kGroups ? E / c.n_group : E, pitch = gsz + group_pad;
  uint32_t* st = kGroups ? stage + (size_t)seg * c.n_group * (pitch + 1) : nullptr;
  int* list = kGroups ? reinterpret_cast<int*>(st) + c.n_group * pitch : nullptr;
  // kept in registers across tokens: this lane's biases
  constexpr bool kKeep = kPerLane <= 8;
  float be[kKeep ? kPerLane : 1];
  float nan = 0.f;     // turns NaN with the first value that is not finite
  bool bad = false;
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      be[i] = scored && lane + L * i < E ? __ldg(bias + lane + L * i) : 0.f;
      bad |= !(be[i] < INFINITY);   // NaN or +inf: -inf switches an expert off
    }
  }
  float next[kPerLane];
  auto fetch = [&](int t) {
    const float* row = logits + (size_t)(t < T ? t : T - 1) * E;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i)
      next[i] = lane + L * i < E ? __ldg(row + lane + L * i) : -INFINITY;
  };
  // the warp's tokens stay together: its first one decides
  const int first = blockIdx.x * per_block + (seg & ~(32 / L - 1)), own = seg & (32 / L - 1);
  if (first < T) fetch(first + own);
  for (int tw = first; tw < T; tw += stride) {
    const bool live = tw + own < T;
    const int t = live ? tw + own : T - 1;
    const float* row = logits + (size_t)t * E;
    float v[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      v[i] = next[i];
      if (lane + L * i < E) nan = fmaf(v[i], 0.f, nan);
    }
    if (tw + stride < T) fetch(tw + stride + own);
    // softmax: the row's maximum and the sum of exp(l - m), rounded once where
    // the scores decide
    float m = 0.f, S = 1.f;
    if (c.softmax && (need_s || !c.renorm)) {
      float mx = v[0];
#pragma unroll
      for (int i = 1; i < kPerLane; ++i) mx = fmaxf(mx, v[i]);
      m = seg_max<L>(mx);
      if (need_s) {
        float hi = 0.f, lo = 0.f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i)
          pair_add(hi, lo, lane + L * i < E ? expf(v[i] - m) : 0.f);
        S = seg_sum_rounded<L>(hi, lo);
      } else {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) sum += lane + L * i < E ? expf(v[i] - m) : 0.f;
        S = seg_sum<L>(sum);
      }
    }
    auto score = [&](float l) { return c.softmax ? __fdiv_rn(expf(l - m), S) : sigmoid_rn(l); };
    uint32_t key[kPerLane];
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
      const int e = lane + L * i;
      float r = v[i];
      if (scored && e < E) {
        float b;
        if constexpr (kKeep) {
          b = be[i];
        } else {
          b = __ldg(bias + e);
          bad |= !(b < INFINITY);
        }
        r = __fadd_rn(score(r), b);
      }
      key[i] = e < E ? rank_key(r) : 0u;
      if constexpr (kGroups) {
        const int g = (int)((uint32_t)e * c.group_magic >> 20);
        if (e < E) st[e + g * group_pad] = key[i];
      }
    }
    int idx;
    if constexpr (!kGroups) {
      idx = select_best<kPerLane, L>(key, k, lane);
    } else {
      __syncwarp();
      // lpg lanes scan one group: its two largest keys
      const int lpg = c.lanes_per_group / (32 / L), sub = lane & (lpg - 1), g = lane / lpg;
      uint32_t a1 = 0u, a2 = 0u;
      if (g < c.n_group) {
        const uint32_t* gs = st + g * pitch;
#pragma unroll 4
        for (int j = sub; j < gsz; j += lpg) {
          const uint32_t x = gs[j];
          a2 = max(a2, min(a1, x));
          a1 = max(a1, x);
        }
      }
      for (int off = 1; off < lpg; off <<= 1) {
        const uint32_t o1 = __shfl_xor_sync(0xffffffffu, a1, off);
        const uint32_t o2 = __shfl_xor_sync(0xffffffffu, a2, off);
        a2 = max(max(a2, o2), min(a1, o1));
        a1 = max(a1, o1);
      }
      uint32_t gk = a1;
      if (two) {   // the sum of two values: of the biased scores, or of the scores themselves
        float x1 = route_key_value(a1), x2 = route_key_value(a2);
        if (!scored) {
          x1 = score(x1);
          x2 = score(x2);
        }
        gk = rank_key(__fadd_rn(x1, x2));
      }
      if (sub != 0 || g >= c.n_group) gk = 0u;
      // the best groups, one after the other (equal ones: the lower first)
      unsigned kept = 0u;
      for (int j = 0; j < c.topk_group; ++j) {
        const uint32_t top = seg_max<L>(gk);
        const uint32_t win = seg_min<L>(gk == top && top != 0u ? (uint32_t)lane : 31u);
        kept |= 1u << win;
        if ((int)win == lane) gk = 0u;
      }
      if ((kept >> lane) & 1u) list[__popc(kept & ((1u << lane) - 1u))] = g * pitch;
      __syncwarp();
      // candidate j: the j-th expert of the kept groups in ascending order
      const int n_cand = c.topk_group * gsz;
      auto place_of = [&](int j) {
        const int cg = (int)((uint32_t)j * c.group_magic >> 20);
        return list[cg] + (j - cg * gsz);
      };
      int pick;
      if (kPerLane > 1 && n_cand <= L * (kPerLane / 2)) {
        constexpr int kHalf = kPerLane > 1 ? kPerLane / 2 : 1;
        uint32_t half[kHalf];
#pragma unroll
        for (int i = 0; i < kHalf; ++i) {
          const int j = lane + L * i;
          half[i] = j < n_cand ? st[place_of(j)] : 0u;
        }
        pick = select_best<kHalf, L>(half, k, lane);
      } else {
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
          const int j = lane + L * i;
          key[i] = j < n_cand ? st[place_of(j)] : 0u;
        }
        pick = select_best<kPerLane, L>(key, k, lane);
      }
      pick = (int)min((uint32_t)pick, (uint32_t)(n_cand - 1));
      const int cg = (int)((uint32_t)pick * c.group_magic >> 20);
      idx = lane < k ? list[cg] / pitch * gsz + (pick - cg * gsz) : 0;
      __syncwarp();   // the next token's keys take this one's place
    }
    // the picks' logits, and whether the bias switched the expert off
    const bool have = lane < k;
    idx = have ? (int)min((uint32_t)idx, (uint32_t)(E - 1)) : 0;
    const float l = have ? __ldg(row + idx) : 0.f;
    const bool on = have && (!scored || __ldg(bias + idx) != -INFINITY);
    const float w = pick_weight<L>(c.softmax, c.renorm, c.scale, l, on, m, S);
    if (have && live) {
      topk_idx[(size_t)t * k + lane] = idx;
      topk_w[(size_t)t * k + lane] = w;
      if (chunk_hist) atomicAdd(&chunk_hist[(size_t)(t / tpc) * E + idx], 1);
    }
  }
  bad |= isnan(nan);
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

// Four blocks of eight warps per SM, about what the registers allow at once.
int grid_of(int T, int per_block) {
  const int blocks = (T + per_block - 1) / per_block, most = 4 * device_sm_count();
  return blocks < most ? blocks : most;
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
        <<<grid_of(T, per_block), 32 * warps, bytes * warps, s>>>(
            logits, bias, c, T, E, k, tpc, pad, topk_idx, topk_w, chunk_hist, status,
            whole && T <= per_block);
  } else {
    const int per_block = kMaxWarps * per_warp;
    route_scored_kernel<kPerLane, L, false>
        <<<grid_of(T, per_block), 32 * kMaxWarps, 0, s>>>(
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
