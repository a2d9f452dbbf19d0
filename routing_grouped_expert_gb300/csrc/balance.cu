// The loss that keeps the experts' loads even, with the loads themselves, and its gradient.
//
// For each sequence s (tokens seq_offsets[s] .. seq_offsets[s + 1] - 1 whose mask is set; n of
// them), with p_t = softmax(l_t), or the sigmoid scores over their sum:
//
//   c_e = choices of expert e,  P_e = sum_t p_te
//   loss = alpha / S * sum_s E / (k n^2) sum_e c_e P_e      (a sequence of no token adds 0)
//   dl_te = g alpha E / (S k n^2) p_te f_te (c_e - sum_i p_ti c_i)
//
// with f = 1 (softmax) or 1 - sigmoid(l_te).  Since sum_i p_ti = 1, any constant can be taken
// from all c_e: the gradient subtracts the sequence's mean load, as an integer, which leaves
// exact zeros where the loads are even.
//
// Forward: blocks of consecutive tokens sum p in registers and count choices in shared
// memory; each (block, sequence) pair that meets has a slot of its own, number block +
// sequence (pairs that meet lie on a staircase, so their numbers differ).  One cluster then
// adds the slots in order.  No atomics on floats: results are the same from run to run.
#include <math.h>

#include <cooperative_groups.h>

#include "moe_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCluster = 8;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
  return v;
}

// Where sequence s starts: 0 <= start <= T whatever the offsets hold.
__device__ __forceinline__ int seq_start(const BalanceArgs& a, int s) {
  if (a.seq_offsets == nullptr) return s == 0 ? 0 : a.T;
  return min(max(__ldg(a.seq_offsets + s), 0), a.T);
}
// The first sequence that ends after token t (S: none).
__device__ __forceinline__ int seq_after(const BalanceArgs& a, int t) {
  int lo = 0, hi = a.S;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (seq_start(a, mid + 1) > t) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

// Lane l holds n / V chunks of V experts, chunk i being experts V (l + 32 i) ...
template <int V, int n>
__device__ __forceinline__ void load_row(const float* row, int E, int lane, float (&v)[n]) {
#pragma unroll
  for (int i = 0; i < n / V; ++i) {
    const int e = V * (lane + 32 * i);
    if constexpr (V == 4) {
      const float4 x = e < E ? __ldg(reinterpret_cast<const float4*>(row + e))
                             : make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
      v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
    } else {
      v[i] = e < E ? __ldg(row + e) : -INFINITY;
    }
  }
}

// v: the logits -> the probabilities; one: 1 - sigmoid(l), where asked for.  The sigmoid
// scores of a row whose logits are all below -40 are exp(l) to 2^-57 and could vanish:
// there their ratios are taken.  Places past the row hold -inf and come out as 0.
template <int n, bool kOne>
__device__ __forceinline__ void probabilities(bool softmax, float (&v)[n], float (&one)[kOne ? n : 1]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < n; ++i) m = fmaxf(m, v[i]);
  m = warp_max(m);
  float sum = 0.f;
  if (softmax || m < -40.f) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      v[i] = __expf(v[i] - m);
      sum += v[i];
      if constexpr (kOne) one[i] = 1.f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float e = __expf(-fabsf(v[i]));       // no overflow on either side
      const float r = __frcp_rn(1.f + e);
      const bool up = v[i] >= 0.f;
      if constexpr (kOne) one[i] = up ? e * r : r;
      v[i] = up ? r : e * r;
      sum += v[i];
    }
  }
  const float inv = 1.f / warp_sum(sum);
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] *= inv;
}

struct BalanceShared {
  int hist[MOE_MAX_EXPERTS];
  int tokens, bad;
  float loss[kWarps];
  float sums[kWarps][33];
  int cnts[kWarps][33];
  float total;
};

// One block of tokens: the sums and counts of each sequence that it meets, into their slots.
template <int V, int n>
__device__ __forceinline__ void sum_tokens(const BalanceArgs& a, int block, BalanceShared& sh,
                                           float* sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.E;
  const long long first = (long long)block * a.chunk;
  const int begin = (int)min(first, (long long)a.T);
  const int end = (int)min(first + a.chunk, (long long)a.T);
  if (threadIdx.x == 0) sh.bad = 0;
  bool nonfinite = false, outside = false;
  for (int s = seq_after(a, begin); s < a.S; ++s) {
    const int lo = max(begin, seq_start(a, s)), hi = min(end, seq_start(a, s + 1));
    if (lo >= end) break;
    if (lo >= hi) continue;
    for (int e = threadIdx.x; e < E; e += kThreads) sh.hist[e] = 0;
    if (threadIdx.x == 0) sh.tokens = 0;
    __syncthreads();
    float acc[n];
#pragma unroll
    for (int i = 0; i < n; ++i) acc[i] = 0.f;
    int mine = 0;
    for (int t = lo + warp; t < hi; t += kWarps) {
      if (a.mask != nullptr && __ldg(a.mask + t) == 0) continue;
      ++mine;
      float v[n];
      load_row<V, n>(a.logits + (size_t)t * E, E, lane, v);
      if (lane < a.k) {
        const int e = __ldg(a.topk_idx + (size_t)t * a.k + lane);
        if (e >= 0 && e < E) atomicAdd(&sh.hist[e], 1);
        else outside = true;
      }
      float none[1], nan = 0.f;
#pragma unroll
      for (int i = 0; i < n; ++i) nan = fmaf(V * (lane + 32 * (i / V)) < E ? v[i] : 0.f, 0.f, nan);
      nonfinite |= isnan(nan);
      probabilities<n, false>(a.softmax, v, none);
#pragma unroll
      for (int i = 0; i < n; ++i) acc[i] += v[i];
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const int e = V * (lane + 32 * (i / V)) + i % V;
      if (e < E) sums[warp * E + e] = acc[i];
    }
    if (lane == 0 && mine) atomicAdd(&sh.tokens, mine);
    __syncthreads();
    const size_t slot = (size_t)block + s;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += sums[w * E + e];
      a.part_p[slot * E + e] = v;
      a.part_c[slot * E + e] = sh.hist[e];
    }
    if (threadIdx.x == 0) a.part_n[slot] = sh.tokens;
    __syncthreads();
  }
  if (nonfinite) atomicOr(&sh.bad, 1);
  if (outside) atomicOr(&sh.bad, 2);
  __syncthreads();
  if (threadIdx.x == 0) a.flags[block] = sh.bad;
}

// The cluster's part: the slots' sums in order, the counts, the loss and the status.
__device__ __forceinline__ void add_slots(const BalanceArgs& a, BalanceShared& sh) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int E = a.E, groups = (E + 31) / 32;
  const long long units = (long long)a.S * groups;
  // several warps share a unit (a sequence's 32 experts) where there are few units
  int share = 1;
  while (share < kWarps && units * share < (long long)ranks * kWarps) share *= 2;
  const int per = kWarps / share;
  const long long rounds = (units + (long long)ranks * per - 1) / ((long long)ranks * per);
  float loss = 0.f;
  for (long long r = 0; r < rounds; ++r) {
    const long long u = (r * ranks + rank) * per + warp / share;
    const int s = (int)(u / groups), e = (int)(u % groups) * 32 + lane;
    float p = 0.f;
    int c = 0, tokens = 0;
    if (u < units) {
      const int lo = seq_start(a, s), hi = seq_start(a, s + 1);
      if (lo < hi) {
        const int b0 = lo / a.chunk, b1 = (hi - 1) / a.chunk;
        for (int b = b0 + lane; b <= b1; b += 32) tokens += a.part_n[(size_t)b + s];
        if (e < E) {
#pragma unroll 8
          for (int b = b0 + warp % share; b <= b1; b += share) {
            p += a.part_p[((size_t)b + s) * E + e];
            c += a.part_c[((size_t)b + s) * E + e];
          }
        }
      }
    }
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    if (share > 1) {
      sh.sums[warp][lane] = p;
      sh.cnts[warp][lane] = c;
      __syncthreads();
      if (warp % share == 0)
        for (int w = 1; w < share; ++w) {
          p += sh.sums[warp + w][lane];
          c += sh.cnts[warp + w][lane];
        }
      __syncthreads();
    }
    if (u < units && warp % share == 0) {
      if (e < E) a.counts[(size_t)s * E + e] = c;
      if (e == 0) a.tokens[s] = tokens;
      const float dot = warp_sum(e < E ? (float)c * p : 0.f);
      if (tokens > 0) loss += dot * (a.factor / ((float)tokens * (float)tokens));
    }
  }
  if (lane == 0) sh.loss[warp] = loss;
  __syncthreads();
  if (threadIdx.x == 0) {
    float v = 0.f;
    for (int w = 0; w < kWarps; ++w) v += sh.loss[w];
    sh.total = v;
  }
  cluster.sync();
  if (rank == 0) {
    int bad = 0;
    for (int b = threadIdx.x; b < a.blocks; b += kThreads) bad |= a.flags[b];
    if (a.seq_offsets != nullptr)
      for (int s = threadIdx.x; s <= a.S; s += kThreads) {
        const int o = __ldg(a.seq_offsets + s);
        if (o < 0 || o > a.T || (s > 0 && o < __ldg(a.seq_offsets + s - 1))) bad |= 2;
      }
    const int nonfinite = __syncthreads_or(bad & 1), outside = __syncthreads_or(bad & 2);
    if (threadIdx.x == 0) {
      float v = 0.f;
      for (int i = 0; i < ranks; ++i) v += *cluster.map_shared_rank(&sh.total, i);
      *a.loss = v;
      a.status[0] = outside ? MOE_ERR_INVALID_ARG : nonfinite ? MOE_ERR_NONFINITE : 0;
      a.status[1] = 0;
    }
  }
  cluster.sync();   // no block leaves while its total is read
}

template <int V, int n>
__global__ void __launch_bounds__(kThreads) balance_sum_kernel(BalanceArgs a) {
  __shared__ BalanceShared sh;
  extern __shared__ float sums[];   // [kWarps][E]
  sum_tokens<V, n>(a, blockIdx.x, sh, sums);
}

__global__ void __launch_bounds__(kThreads) balance_add_kernel(BalanceArgs a) {
  __shared__ BalanceShared sh;
  add_slots(a, sh);
}

// Both in one launch of one cluster, for batches of few tokens.
template <int V, int n>
__global__ void __launch_bounds__(kThreads) balance_small_kernel(BalanceArgs a) {
  __shared__ BalanceShared sh;
  extern __shared__ float sums[];
  if ((int)blockIdx.x < a.blocks) sum_tokens<V, n>(a, blockIdx.x, sh, sums);
  __threadfence();
  cooperative_groups::this_cluster().sync();
  add_slots(a, sh);
}

// dlogits: a block of consecutive tokens, a warp per token.  kOnto: added onto `out`.
template <int V, int n, bool kOnto>
__global__ void __launch_bounds__(kThreads)
balance_backward_kernel(BalanceArgs a, const float* __restrict__ dloss,
                        const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
                        float* out) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int E = a.E;
  const long long first = (long long)blockIdx.x * a.chunk;
  const int begin = (int)min(first, (long long)a.T);
  const int end = (int)min(first + a.chunk, (long long)a.T);
  const float g = a.factor * (dloss != nullptr ? __ldg(dloss) : 1.f);
  int s = seq_after(a, begin), at = -1;   // at: the sequence whose loads are held
  float load[n];
  for (int t = begin + warp; t < end; t += kWarps) {
    while (s < a.S && seq_start(a, s + 1) <= t) ++s;
    const bool in = s < a.S && seq_start(a, s) <= t && (a.mask == nullptr || __ldg(a.mask + t) != 0);
    float v[n];
    if (!in) {
      if constexpr (kOnto) continue;
#pragma unroll
      for (int i = 0; i < n; ++i) v[i] = 0.f;
    } else {
      load_row<V, n>(a.logits + (size_t)t * E, E, lane, v);
      if (at != s) {
        at = s;
        const int m = __ldg(tokens + s);
        const int mean = (int)((long long)a.k * m / E);
        const float f = m > 0 ? g / ((float)m * (float)m) : 0.f;
#pragma unroll
        for (int i = 0; i < n; ++i) {
          const int e = V * (lane + 32 * (i / V)) + i % V;
          load[i] = e < E ? (float)(__ldg(counts + (size_t)s * E + e) - mean) * f : 0.f;
        }
      }
      float one[n];
      probabilities<n, true>(a.softmax, v, one);
      float dot = 0.f;
#pragma unroll
      for (int i = 0; i < n; ++i) dot = fmaf(v[i], load[i], dot);
      dot = warp_sum(dot);
#pragma unroll
      for (int i = 0; i < n; ++i) v[i] *= one[i] * (load[i] - dot);
    }
    float* row = out + (size_t)t * E;
#pragma unroll
    for (int i = 0; i < n / V; ++i) {
      const int e = V * (lane + 32 * i);
      if (e >= E) continue;
      if constexpr (V == 4) {
        float4 x = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        if constexpr (kOnto) {
          const float4 y = *reinterpret_cast<const float4*>(row + e);
          x.x += y.x; x.y += y.y; x.z += y.z; x.w += y.w;
        }
        *reinterpret_cast<float4*>(row + e) = x;
      } else {
        row[e] = kOnto ? row[e] + v[i] : v[i];
      }
    }
  }
}

// Tokens per block: one block of 16 warps for each SM, twice where there are many.
int chunk_of(int T) {
  const int most = 2 * kSms;
  const long long c = ((long long)T + most - 1) / most;
  return (int)((c + kWarps - 1) / kWarps * kWarps);
}

#define MOE_BALANCE_SHAPE(E, CASE) \
  do {                             \
    if (E % 4 == 0 && E >= 64) {   \
      if (E <= 128) CASE(4, 4);    \
      else if (E <= 256) CASE(4, 8);   \
      else if (E <= 512) CASE(4, 16);  \
      else CASE(4, 32);            \
    } else if (E <= 32) CASE(1, 1);  \
    else if (E <= 64) CASE(1, 2);  \
    else if (E <= 128) CASE(1, 4); \
    else if (E <= 256) CASE(1, 8); \
    else if (E <= 512) CASE(1, 16); \
    else CASE(1, 32);              \
  } while (0)

template <typename K>
cudaError_t launch_cluster(K kern, const BalanceArgs& a, int ranks, size_t smem, bool pdl,
                           cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

}  // namespace

size_t balance_layout(int T, int E, int S, BalanceArgs* a, void* ws) {
  const int chunk = T > 0 ? chunk_of(T) : kWarps;
  const int blocks = (int)(((long long)T + chunk - 1) / chunk);
  const size_t slots = (size_t)blocks + S;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = align_up(o + bytes, 256); return at; };
  const size_t status = take(256), flags = take((size_t)blocks * 4), n = take(slots * 4);
  const size_t p = take(slots * E * 4), c = take(slots * E * 4);
  if (a != nullptr) {
    a->chunk = chunk;
    a->blocks = blocks;
    a->status = ws_ptr<int>(ws, status);
    a->flags = ws_ptr<int>(ws, flags);
    a->part_n = ws_ptr<int>(ws, n);
    a->part_p = ws_ptr<float>(ws, p);
    a->part_c = ws_ptr<int>(ws, c);
  }
  return o;
}

cudaError_t launch_balance(const BalanceArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)kWarps * a.E * 4;
  const int E = a.E;
  if (a.blocks <= kCluster) {
#define CASE(V, n)                                                                             \
  do {                                                                                         \
    cudaError_t e = cudaFuncSetAttribute(balance_small_kernel<V, n>,                           \
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem); \
    return e != cudaSuccess ? e : launch_cluster(balance_small_kernel<V, n>, a, kCluster, smem, false, s); \
  } while (0)
    MOE_BALANCE_SHAPE(E, CASE);
#undef CASE
  }
#define CASE(V, n)                                                                             \
  do {                                                                                         \
    cudaError_t e = cudaFuncSetAttribute(balance_sum_kernel<V, n>,                             \
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem); \
    if (e != cudaSuccess) return e;                                                            \
    balance_sum_kernel<V, n><<<a.blocks, kThreads, smem, s>>>(a);                              \
  } while (0)
  MOE_BALANCE_SHAPE(E, CASE);
#undef CASE
  const cudaError_t e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_cluster(balance_add_kernel, a, kCluster, 0, false, s);
}

cudaError_t launch_balance_backward(const BalanceArgs& a, const float* dloss, const int32_t* counts,
                                    const int32_t* tokens, bool onto, float* out, cudaStream_t s) {
  const int E = a.E;
#define CASE(V, n)                                                                              \
  do {                                                                                          \
    if (onto)                                                                                   \
      balance_backward_kernel<V, n, true><<<a.blocks, kThreads, 0, s>>>(a, dloss, counts, tokens, out); \
    else                                                                                        \
      balance_backward_kernel<V, n, false><<<a.blocks, kThreads, 0, s>>>(a, dloss, counts, tokens, out); \
  } while (0)
  MOE_BALANCE_SHAPE(E, CASE);
#undef CASE
  return cudaGetLastError();
}

}  // namespace moe
