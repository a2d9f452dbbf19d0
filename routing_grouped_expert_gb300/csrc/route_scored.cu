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
// order of the lanes, but for sums within 2^-15 ulp of a rounding boundary.
#include <math.h>

#include <atomic>
#include <chrono>

#include "ptx.cuh"
#include "route_token.cuh"
#include "status.cuh"

namespace moe {
namespace {

constexpr int kMaxWarps = 8;

// L lanes route one token, so a warp routes 32 / L.  Reductions over a token's
// lanes:
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

// The lanes of this token whose `p` holds, as bits of its lanes.
template <int L>
__device__ __forceinline__ unsigned seg_ballot(bool p) {
  const unsigned m = __ballot_sync(0xffffffffu, p);
  if constexpr (L == 32) return m;
  else return (m >> (threadIdx.x & 31 & ~(L - 1))) & ((1u << L) - 1u);
}

// The k largest of a token's candidates: lane i's keys are n candidates of it
// (key 0: none), id[] their numbers, ascending; lane j < k returns slot j's
// number.  A larger key wins, equal keys go to the lower number.  Up to eight
// keys per lane are sorted once; with more, each round rescans the winner's keys
// instead: 4 n instructions a round against 5 n (n - 1) / 2 for the sort.  A round
// finds the largest head by one reduction and its lane by a vote; only where
// several lanes hold the same key a second reduction finds the lowest number.
template <int n, int L>
__device__ __forceinline__ int select_best(uint32_t (&key)[n], int (&id)[n], int k, int lane) {
  constexpr bool kSort = n <= 8;
  if constexpr (kSort) {
    // odd-even transposition, swapping only on a strictly smaller key
#pragma unroll
    for (int pass = 0; pass < n; ++pass) {
#pragma unroll
      for (int i = pass & 1; i + 1 < n; i += 2) {
        const bool swap = key[i] < key[i + 1];
        const uint32_t hi = max(key[i], key[i + 1]), lo = min(key[i], key[i + 1]);
        const int x = swap ? id[i + 1] : id[i], y = swap ? id[i] : id[i + 1];
        key[i] = hi;
        key[i + 1] = lo;
        id[i] = x;
        id[i + 1] = y;
      }
    }
  }
  uint32_t best = 0u;
  int head = 0, mine = 0;
  auto scan = [&]() {   // this lane's largest key
    best = key[0];
    head = id[0];
    if constexpr (!kSort) {
#pragma unroll
      for (int i = 1; i < n; ++i)
        if (key[i] > best) {
          best = key[i];
          head = id[i];
        }
    }
  };
  scan();
  for (int j = 0; j < k; ++j) {
    const bool top = best == seg_max<L>(best);
    const unsigned who = seg_ballot<L>(top);
    int win = __ffs(who) - 1;   // the lane that holds it
    if (__any_sync(0xffffffffu, (who & (who - 1)) != 0u)) {
      const uint32_t low = seg_min<L>(top ? (uint32_t)head : ~0u);
      win = __ffs(seg_ballot<L>(top && (uint32_t)head == low)) - 1;
    }
    const int cand = __shfl_sync(0xffffffffu, head, win, L);
    if (lane == j) mine = cand;
    if (win == lane) {
      if constexpr (kSort) {
#pragma unroll
        for (int i = 0; i + 1 < n; ++i) {
          key[i] = key[i + 1];
          id[i] = id[i + 1];
        }
        key[n - 1] = 0u;
      } else {
#pragma unroll
        for (int i = 0; i < n; ++i)
          if (id[i] == head) key[i] = 0u;
      }
      scan();
    }
  }
  return mine;
}

// As route_key, in fewer instructions: -0 + 0 is +0, and the sign spread over
// the word flips the rest of a negative number.  A NaN gets a key like any
// other, which keeps the order total (the status reports it).
__device__ __forceinline__ uint32_t rank_key(float x) {
  const int b = __float_as_int(__fadd_rn(x, 0.f));
  return (uint32_t)(b ^ ((b >> 31) | (int)0x80000000));
}


// Blocks of eight warps per SM for n logits per lane: what hides the fixed
// latencies of a token's dependent steps.
template <int n>
constexpr int kBlocks = n <= 20 ? 4 : 1;

// V consecutive values of global or shared memory by one access.
template <int V, typename Tp>
__device__ __forceinline__ void load_chunk(Tp (&x)[V], const Tp* p, bool global) {
  if constexpr (V == 4) {
    const uint4 v = global ? __ldg(reinterpret_cast<const uint4*>(p)) : *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if constexpr (sizeof(Tp) == 4) x[c] = *reinterpret_cast<const Tp*>(&w[c]);
  } else {
    x[0] = global ? __ldg(p) : *p;
  }
}

// One token per L lanes; lane l holds kC chunks of V experts, chunk q = l + L i
// being experts V q .. V q + V - 1.  The warps go through the tokens in strides.
// Bound by the latency of a token's chain of dependent steps and the instructions in
// it, not by memory: 8192 tokens of 256 experts in 8 groups read 8.4 MB, 1.3 us, in
// 13.4 us by itself (DRAM 8% busy); the schedulers issue in 61% of their active cycles
// and 43% of the launch's, with 6 warps each that mostly wait out fixed latencies.  40001
// of 160: 25.6 MB, 3.8 us, in 20.8 us, 18.5 in calls one after the other, issue 65% and
// 51%; one token of 256, replayed from a graph: 4.1 us.
// So experts go in chunks of four wherever E and the groups allow it (one load, one
// check and one group index for four), everything but the scores is done on integer
// keys, a token's candidates are compacted to the kept groups before the selection,
// and in a large batch one warp routes two or four tokens, which share the
// instructions of the groups, the rounds and the weights.
template <int V, int kC, int L, bool kGroups>
__global__ void __launch_bounds__(32 * kMaxWarps, kBlocks<V * kC>)
route_scored_kernel(const float* __restrict__ logits, const float* __restrict__ bias, RouteCfg c,
                    int T, int E, int k, int tpc, int group_pad, int region,
                    int32_t* __restrict__ topk_idx, float* __restrict__ topk_w,
                    int32_t* __restrict__ chunk_hist, int* __restrict__ status, uint64_t launch,
                    bool whole) {
  // per token of the block `region` words: n_group * (group size + pad) keys, then
  // the kept groups
  extern __shared__ __align__(16) uint32_t stage[];
  pdl_trigger();
  status_begin(status, launch);
  constexpr int n = V * kC;
  const int lane = threadIdx.x & (L - 1), seg = threadIdx.x / L;   // seg: the block's token
  const int per_block = blockDim.x / L;
  const uint32_t stride = gridDim.x * per_block;   // token numbers stay below 2^32
  const bool two = kGroups && c.group_top == 2;
  const bool scored = bias != nullptr;                  // all scores take part in the choice
  const bool need_s = scored || (two && c.softmax);     // the scores' exact sum decides
  const int gsz = kGroups ? E / c.n_group : E, pitch = gsz + group_pad;
  const int nq = E / V;                                 // chunks of a row
  uint32_t* st = kGroups ? stage + (size_t)seg * region : nullptr;
  int* list = kGroups ? reinterpret_cast<int*>(st) + c.n_group * pitch : nullptr;
  // few logits per lane: this lane's biases are kept across tokens, and the
  // next token's logits are on their way while one is routed
  constexpr bool kKeep = n <= 8;
  float be[kKeep ? kC : 1][V];
  float nan = 0.f;     // turns NaN with the first value that is not finite
  bool bad = false;
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < kC; ++i) {
#pragma unroll
      for (int x = 0; x < V; ++x) be[i][x] = 0.f;
      if (scored && lane + L * i < nq) load_chunk<V>(be[i], bias + V * (lane + L * i), true);
#pragma unroll
      for (int x = 0; x < V; ++x) bad |= !(be[i][x] < INFINITY);   // -inf switches an expert off
    }
  }
  float next[kC][V];
  auto fetch = [&](uint32_t t) {
    const float* row = logits + (size_t)(t < (uint32_t)T ? t : T - 1) * E + V * lane;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
#pragma unroll
      for (int x = 0; x < V; ++x) next[i][x] = -INFINITY;
      if (lane + L * i < nq) load_chunk<V>(next[i], row + V * L * i, true);
    }
  };
  // the warp's tokens stay together: its first one decides
  const uint32_t first = blockIdx.x * per_block + (seg & ~(32 / L - 1)), own = seg & (32 / L - 1);
  if (kKeep && first < (uint32_t)T) fetch(first + own);
  for (uint32_t tw = first; tw < (uint32_t)T; tw += stride) {
    const bool live = tw + own < (uint32_t)T;
    const int t = live ? (int)(tw + own) : T - 1;
    const float* row = logits + (size_t)t * E;
    float v[kC][V];
    if (!kKeep) fetch(t);
#pragma unroll
    for (int i = 0; i < kC; ++i)
#pragma unroll
      for (int x = 0; x < V; ++x) v[i][x] = next[i][x];
    if (kKeep && tw + stride < (uint32_t)T) fetch(tw + stride + own);
    // softmax: the row's maximum and the sum of exp(l - m), rounded once where
    // the scores decide
    float m = 0.f, S = 1.f;
    if (c.softmax && (need_s || !c.renorm)) {
      float mx = -INFINITY;
#pragma unroll
      for (int i = 0; i < kC; ++i)
#pragma unroll
        for (int x = 0; x < V; ++x) mx = fmaxf(mx, v[i][x]);
      m = seg_max<L>(mx);
      if (need_s) {
        float hi = 0.f, lo = 0.f;
#pragma unroll
        for (int i = 0; i < kC; ++i)
#pragma unroll
          for (int x = 0; x < V; ++x) pair_add(hi, lo, expf(v[i][x] - m));   // exp(-inf) = 0
        S = seg_sum_rounded<L>(hi, lo);
      } else {
        // a factor of the weights only: the short exp, whose error of 2 ulp + |l - m|
        // 2^-23 stands on terms of size exp(l - m)
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < kC; ++i)
#pragma unroll
          for (int x = 0; x < V; ++x) sum += __expf(v[i][x] - m);
        S = seg_sum<L>(sum);
      }
    }
    auto score = [&](float l) { return c.softmax ? __fdiv_rn(expf(l - m), S) : sigmoid_rn(l); };
    uint32_t key[n];
    int id[n];
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int q = lane + L * i;
      const bool in = q < nq;
#pragma unroll
      for (int x = 0; x < V; ++x) {
        key[i * V + x] = 0u;
        id[i * V + x] = V * q + x;
      }
      if (in) {
        float b[V];
        if (scored) {
          if constexpr (kKeep) {
#pragma unroll
            for (int x = 0; x < V; ++x) b[x] = be[i][x];
          } else {
            load_chunk<V>(b, bias + V * q, true);
#pragma unroll
            for (int x = 0; x < V; ++x) bad |= !(b[x] < INFINITY);
          }
        }
        uint32_t kx[V];
#pragma unroll
        for (int x = 0; x < V; ++x) {
          nan = fmaf(v[i][x], 0.f, nan);
          const float r = scored ? __fadd_rn(score(v[i][x]), b[x]) : v[i][x];
          kx[x] = key[i * V + x] = rank_key(r);
        }
        if constexpr (kGroups) {
          const int g = (int)((uint32_t)(V * q) * c.group_magic >> 20);
          uint32_t* at = st + V * q + g * group_pad;
          if constexpr (V == 4)
            *reinterpret_cast<uint4*>(at) = make_uint4(kx[0], kx[1], kx[2], kx[3]);
          else
            *at = kx[0];
        }
      }
    }
    int idx;
    if constexpr (!kGroups) {
      idx = select_best<n, L>(key, id, k, lane);
    } else {
      __syncwarp();
      // lpg lanes scan one group: its two largest keys
      const int lpg = c.lanes_per_group / (32 / L), sub = lane & (lpg - 1), g = lane / lpg;
      uint32_t a1 = 0u, a2 = 0u;
      if (g < c.n_group) {
        const uint32_t* gs = st + g * pitch;
#pragma unroll 2
        for (int j = V * sub; j < gsz; j += V * lpg) {
          uint32_t x[V];
          load_chunk<V>(x, gs + j, false);
#pragma unroll
          for (int y = 0; y < V; ++y) {
            a2 = max(a2, min(a1, x[y]));
            a1 = max(a1, x[y]);
          }
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
        const int win = __ffs(seg_ballot<L>(gk == seg_max<L>(gk))) - 1;
        kept |= 1u << win;
        if (win == lane) gk = 0u;
      }
      if ((kept >> lane) & 1u) list[__popc(kept & ((1u << lane) - 1u))] = g * pitch;
      __syncwarp();
      // candidate j: the j-th expert of the kept groups in ascending order
      const int n_cand = c.topk_group * gsz;
      auto candidates = [&](auto& ck, auto& ci, int chunks) {
#pragma unroll
        for (int i = 0; i < chunks; ++i) {
          const int j = V * (lane + L * i);
          const int cg = (int)((uint32_t)j * c.group_magic >> 20);
          uint32_t x[V];
#pragma unroll
          for (int y = 0; y < V; ++y) x[y] = 0u;
          if (j < n_cand) load_chunk<V>(x, st + list[cg] + (j - cg * gsz), false);
#pragma unroll
          for (int y = 0; y < V; ++y) {
            ck[i * V + y] = x[y];
            ci[i * V + y] = j + y;
          }
        }
      };
      int pick;
      constexpr int kH = kC > 1 ? kC / 2 : 1;
      if (kC > 1 && n_cand <= L * kH * V) {
        uint32_t hk[kH * V];
        int hi[kH * V];
        candidates(hk, hi, kH);
        pick = select_best<kH * V, L>(hk, hi, k, lane);
      } else {
        candidates(key, id, kC);
        pick = select_best<n, L>(key, id, k, lane);
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
    status_report(status, launch, MOE_ERR_NONFINITE);
  }
}

// Gradient of the weights with respect to the logits, one warp per token.
//   sigmoid, renormalised:  dl_j = scale w_j (dw_j - sum_i w_i dw_i) (1 - s_j), w = s / sum s
//   sigmoid:                dl_j = scale dw_j s_j (1 - s_j)
//   softmax, renormalised:  dl_j = scale w_j (dw_j - sum_i w_i dw_i)
//   softmax (kDense):       dl_e = s_e (scale dw_e - D), D = sum_j scale dw_j s_j
// The first three are zero at every expert that was not chosen.  kDense > 0: that
// many logits per lane are kept from the first read to the last write.  Both are bound
// by the latency of one row's steps, each warp waiting on loads that depend on one
// another (8192 x 256: 7.0 us by itself for 9.2 MB, 1.35 at the copy rate; 40001 x 64,
// dense: 14.2 us, 12.0 in calls one after the other, for 22.4 MB, 3.3; the schedulers
// issue in 47 and 62% of their active cycles).  With one slot the renormalised weight is
// the constant `scale`: its gradient comes out exactly zero.
template <int kDense>
__global__ void __launch_bounds__(32 * kMaxWarps)
route_scored_backward_kernel(const float* __restrict__ dw, const int32_t* __restrict__ topk_idx,
                             const float* __restrict__ logits, const float* __restrict__ bias,
                             RouteCfg c, int T, int E, int k, float* __restrict__ dlogits,
                             int* __restrict__ status, uint64_t launch) {
  status_begin(status, launch);
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
  const bool nonfinite = __any_sync(0xffffffffu, bad);
  const bool outside = __any_sync(0xffffffffu, lane < k && !in);
  if ((nonfinite || outside) && lane == 0)
    status_report(status, launch, outside ? MOE_ERR_INVALID_ARG : MOE_ERR_NONFINITE);
}

// Blocks of `per` tokens each; T may be the largest int.
int blocks_of(int T, int per) { return T / per + (T % per != 0); }

// How a batch is routed: lanes per token, and experts per chunk.
struct Shape {
  int L, V;
};
// The slots and the groups need a lane each.  Up to 2048 tokens (three warps per
// scheduler) are routed one per warp, for the shortest chain of steps; above, the
// instructions bound, and a warp shares them among as many tokens as can be.
// One per warp against several, with 2 us of a memset ahead of each: 2048 x
// 256 in 8 groups 8.2 / 10.3 us, 8192 x 256 16.4 / 14.3, 8192 x 160 13.5 / 9.3,
// 40001 x 160 39.3 / 20.5, 40001 x 64 26.6 / 14.3.  Eight lanes hold up to 20 logits
// each and sixteen up to 16; with more a lane's registers leave one block per SM.  40001
// tokens by 8, 16 and 32 lanes, memset included: 128 experts in 8 groups 22.8, 28.8 and
// 39.3 us, 160 35.0, 37.3 and 49.3, 192 55.9, 37.1 and 49.2, 256 67.8, 41.1 and 47.5; without
// groups 160 25.1, 37.3 and 35.0, 192 35.0, 37.2 and 35.0.  Chunks of four where neither
// a row nor a group splits one: 40001 x 160 34.6 us by single experts.
constexpr int kFewTokens = 2048;
Shape shape_of(int T, int E, int k, int n_group) {
  const int need = k > n_group ? k : n_group;
  const int V = E % 4 == 0 && E / n_group % 4 == 0 && E > 16 ? 4 : 1;
  if (T > kFewTokens || E <= 16) {
    if (need <= 8 && E <= 160) return {8, V};
    if (need <= 16 && E <= 256) return {16, V};
  }
  return {32, V};
}

template <int V, int kC, int L>
cudaError_t launch_t(const float* logits, const float* bias, const RouteCfg& c, int T, int E, int k,
                     int32_t* topk_idx, float* topk_w, int32_t* chunk_hist, int* status,
                     uint64_t launch, bool whole, cudaStream_t s) {
  const int tpc = tokens_per_chunk(k);
  constexpr int per_warp = 32 / L;
  int warps = kMaxWarps;
  auto grid_of = [&]() {   // as many blocks as the SMs take at once
    const int blocks = blocks_of(T, warps * per_warp), most = kBlocks<V * kC> * device_sm_count();
    return blocks < most ? blocks : most;
  };
  if (c.n_group > 1) {
    // A group starts as many chunks' banks after the one before it as lanes scan
    // it, and a token L chunks after the one before it, so that a warp's lanes
    // read different banks; every group starts on a chunk.
    const int gsz = E / c.n_group, lpg = c.lanes_per_group / per_warp;
    const int pad = (V * lpg - gsz % 32 + 64) % 32;
    int region = c.n_group * (gsz + pad + 1);
    region += (V * L % 32 - region % 32 + 32) % 32;
    const size_t bytes = (size_t)region * 4 * per_warp;
    if (bytes * warps > 48 * 1024) warps /= 2;
    if (bytes * warps > 48 * 1024) warps /= 2;
    route_scored_kernel<V, kC, L, true><<<grid_of(), 32 * warps, bytes * warps, s>>>(
        logits, bias, c, T, E, k, tpc, pad, region, topk_idx, topk_w, chunk_hist, status, launch,
        whole);
  } else {
    route_scored_kernel<V, kC, L, false><<<grid_of(), 32 * warps, 0, s>>>(
        logits, bias, c, T, E, k, tpc, 0, 0, topk_idx, topk_w, chunk_hist, status, launch, whole);
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

// From the clock on, so that no number an earlier process left in memory comes again.
uint64_t unique_number() {
  static std::atomic<uint64_t> n{
      (uint64_t)std::chrono::system_clock::now().time_since_epoch().count() | 1};
  return n.fetch_add(2, std::memory_order_relaxed);
}
cudaError_t launch_number(cudaStream_t s, uint64_t* launch) {
  cudaStreamCaptureStatus cs = cudaStreamCaptureStatusNone;
  const cudaError_t err = cudaStreamIsCapturing(s, &cs);
  *launch = err == cudaSuccess && cs == cudaStreamCaptureStatusNone
                ? unique_number()
                : 0;
  return err;
}

cudaError_t launch_route_scored(const float* logits, const float* bias, const RouteCfg& c, int T,
                                int E, int k, int32_t* topk_idx, float* topk_w,
                                int32_t* chunk_hist, int* status, cudaStream_t s, bool clear) {
  if (T == 0) return cudaSuccess;
  const Shape f = shape_of(T, E, k, c.n_group);
  // A quarter of a block's tokens at most (the block may have two warps) are one
  // block's work, which writes the status itself at its end.
  const bool whole = clear && T <= kMaxWarps / 4 * (32 / f.L);
  uint64_t launch = 0;
  if (clear && !whole) {
    const cudaError_t err = begin_status(status, s, &launch);
    if (err != cudaSuccess) return err;
  }
#define MOE_ROUTE_CASE(v, n, lanes)                      \
  if (f.V == v && f.L == lanes && E <= v * n * lanes)    \
    return launch_t<v, n, lanes>(logits, bias, c, T, E, k, topk_idx, topk_w, chunk_hist, status, launch, \
                                 whole, s)
  MOE_ROUTE_CASE(1, 1, 8);
  MOE_ROUTE_CASE(1, 2, 8);
  MOE_ROUTE_CASE(1, 8, 8);
  MOE_ROUTE_CASE(1, 20, 8);
  MOE_ROUTE_CASE(1, 1, 16);
  MOE_ROUTE_CASE(1, 8, 16);
  MOE_ROUTE_CASE(1, 16, 16);
  MOE_ROUTE_CASE(1, 2, 32);
  MOE_ROUTE_CASE(1, 4, 32);
  MOE_ROUTE_CASE(1, 8, 32);
  MOE_ROUTE_CASE(1, 16, 32);
  MOE_ROUTE_CASE(1, 32, 32);
  MOE_ROUTE_CASE(4, 1, 8);
  MOE_ROUTE_CASE(4, 2, 8);
  MOE_ROUTE_CASE(4, 4, 8);
  MOE_ROUTE_CASE(4, 5, 8);
  MOE_ROUTE_CASE(4, 2, 16);
  MOE_ROUTE_CASE(4, 4, 16);
  MOE_ROUTE_CASE(4, 1, 32);
  MOE_ROUTE_CASE(4, 2, 32);
  MOE_ROUTE_CASE(4, 4, 32);
  MOE_ROUTE_CASE(4, 8, 32);
#undef MOE_ROUTE_CASE
  return cudaErrorInvalidValue;
}

cudaError_t launch_route_scored_backward(const float* dw, const int32_t* topk_idx,
                                         const float* logits, const float* bias, const RouteCfg& c,
                                         int T, int E, int k, float* dlogits, int* status,
                                         cudaStream_t s, bool clear) {
  if (T == 0) return cudaSuccess;
  uint64_t launch = 0;
  if (clear) {
    const cudaError_t err = begin_status(status, s, &launch);
    if (err != cudaSuccess) return err;
  }
  const int grid = blocks_of(T, kMaxWarps);
#define MOE_ROUTE_BWD(n)                                                                       \
  route_scored_backward_kernel<n><<<grid, 32 * kMaxWarps, 0, s>>>(dw, topk_idx, logits, bias, c, T, \
                                                                  E, k, dlogits, status, launch)
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
