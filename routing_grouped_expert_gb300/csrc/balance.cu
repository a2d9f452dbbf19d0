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
// sequence (pairs that meet lie on a staircase, so their numbers differ).  More blocks behind
// those then add the slots in order: a block announces its slots by the launch's own number,
// and the adding ones wait for all of them, the very last for the others' sums.  Blocks
// start in order, and a block waits only for blocks before it, which are running or done by
// then: it holds up none that it waits for, however few blocks fit the SMs beside other
// work.  Waits are bounded all the same.  No atomics on floats: results are the same from run to run.
//
// 40001 x 256 logits: 17.0 us in one sequence, 22.5 in 24 with a mask (42 MB, 6.2 us at the
// rate of a plain copy).  Of a call's time, rows are done after 11 us (median; memory from a
// cold start), announced by 14, the slots added by 17.4: the last part is a chain of loads
// through L2, each waiting for the one before.  131072 x 256: 34.2 us (0.60).  One token: 6.8.
// Two launches, the second one cluster: 24 and 33 us.
// The gradient: 40001 x 256 in 13.9 us (0.87), onto dlogits, 24 sequences, 22.5 (0.80),
// 131072 x 256 in 47.9 (0.83); 8192 x 64 in 3.5, latency.
#include <math.h>

#include "moe_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;

// Over the L lanes of a row, for R rows at once.
template <int L, int R>
__device__ __forceinline__ void rows_sum(float (&v)[R]) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1)
#pragma unroll
    for (int i = 0; i < R; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
}
template <int L, int R>
__device__ __forceinline__ void rows_max(float (&v)[R]) {
  if constexpr (L == 32) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      asm("redux.sync.max.f32 %0, %0, 0xffffffff;" : "+f"(v[i]));
  } else {
#pragma unroll
    for (int off = L / 2; off > 0; off >>= 1)
#pragma unroll
      for (int i = 0; i < R; ++i) v[i] = fmaxf(v[i], __shfl_xor_sync(0xffffffffu, v[i], off));
  }
}
__device__ __forceinline__ float warp_sum(float v) {
  float a[1] = {v};
  rows_sum<32>(a);
  return a[0];
}

// Where sequence s starts: 0 <= start <= T whatever the offsets hold.
__device__ __forceinline__ int seq_start(const BalanceArgs& a, int s) {
  if (a.seq_offsets == nullptr) return s == 0 ? 0 : a.T;
  return min(max(__ldg(a.seq_offsets + s), 0), a.T);
}
// The first sequence that ends after token t (S: none), found by the whole block: the
// ends are compared a stretch at a time, then those of the stretch in which the last one
// before t lies.
__device__ __forceinline__ int seq_after(const BalanceArgs& a, int t) {
  int lo = 0, n = a.S;   // it is among lo .. lo + n
  while (n > 0) {
    const int step = (n + kThreads - 1) / kThreads;
    const int i = (int)threadIdx.x * step;
    const int before = __syncthreads_count(i < n && seq_start(a, lo + min(i + step, n)) <= t);
    if (step == 1) return lo + before;
    lo += before * step;
    n = min(step, a.S - lo);
  }
  return a.S;
}
// The starts of the sequences from s0 on, kThreads of them at hand in shared memory.
struct Starts {
  const BalanceArgs& a;
  const int* held;
  int s0;
  __device__ __forceinline__ Starts(const BalanceArgs& a, int* held, int s0) : a(a), held(held), s0(s0) {
    held[threadIdx.x] = seq_start(a, min(s0 + (int)threadIdx.x, a.S));
    __syncthreads();
  }
  __device__ __forceinline__ int operator()(int s) const {
    return s - s0 < kThreads ? held[s - s0] : seq_start(a, s);
  }
};

// How a row is held: L lanes take one, lane l n / V chunks of V experts, chunk i being
// experts V (l + L i) ..., and a warp R rows of each of its 32 / L at once: a row's steps
// depend on each other, so the rows' loads and sums are in flight together.
template <int kV, int kN, int kL, int kR>
struct Shape {
  static constexpr int V = kV, n = kN, L = kL, R = kR;
  // The gradient holds more of a row, and most where it is added onto another.  Rows at once,
  // 256 experts: 40001 tokens 13.7 us by two, 14.5 by one; onto, 26.7 and 22.6.
  template <bool kOnto>
  using Backward = Shape<V, n, L, n <= 4 ? (R + 1) / 2 : n == 8 && !kOnto ? 2 : 1>;
  static constexpr int kRows = R * (32 / L);   // of a warp at once
  static __device__ __forceinline__ int expert(int lane, int i) {
    return V * (lane + L * (i / V)) + i % V;
  }
  // places past the row: `rest`
  static __device__ __forceinline__ void load(const float* row, int E, int lane, float rest,
                                              float (&v)[n]) {
#pragma unroll
    for (int i = 0; i < n; i += V) {
      const int e = expert(lane, i);
      if constexpr (V == 4) {
        const float4 x = e < E ? __ldg(reinterpret_cast<const float4*>(row + e))
                               : make_float4(rest, rest, rest, rest);
        v[i] = x.x; v[i + 1] = x.y; v[i + 2] = x.z; v[i + 3] = x.w;
      } else {
        v[i] = e < E ? __ldg(row + e) : rest;
      }
    }
  }
};

// Elementwise steps of a row, on pairs where there are some: a = a b + c, or with numbers in
// the place of b or c.
__device__ __forceinline__ float2 two(const float* p) { return make_float2(p[0], p[1]); }
__device__ __forceinline__ float2 two(float v) { return make_float2(v, v); }
template <int n, typename F, typename F2>
__device__ __forceinline__ void each(F&& one, F2&& pair) {
  if constexpr (n % 2 == 0) {
#pragma unroll
    for (int i = 0; i < n; i += 2) pair(i);
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) one(i);
  }
}
template <int n>
__device__ __forceinline__ void fma_into(float (&a)[n], const float (&b)[n], float c) {   // a += b c
  each<n>([&](int i) { a[i] = fmaf(b[i], c, a[i]); },
          [&](int i) {
            const float2 x = __ffma2_rn(two(b + i), two(c), two(a + i));
            a[i] = x.x;
            a[i + 1] = x.y;
          });
}
template <int n>
__device__ __forceinline__ void add_mul(float (&a)[n], float b, float c) {   // a = (a + b) c
  each<n>([&](int i) { a[i] = (a[i] + b) * c; },
          [&](int i) {
            const float2 x = __fmul2_rn(__fadd2_rn(two(a + i), two(b)), two(c));
            a[i] = x.x;
            a[i + 1] = x.y;
          });
}
template <int n>
__device__ __forceinline__ float dot(const float (&a)[n], const float (&b)[n]) {
  float2 s = two(0.f);
  each<n>([&](int i) { s.x = fmaf(a[i], b[i], s.x); },
          [&](int i) { s = __ffma2_rn(two(a + i), two(b + i), s); });
  return s.x + s.y;
}
template <int n>
__device__ __forceinline__ float total(const float (&a)[n]) {
  float2 s = two(0.f);
  each<n>([&](int i) { s.x += a[i]; }, [&](int i) { s = __fadd2_rn(two(a + i), s); });
  return s.x + s.y;
}
__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// v: the rows' logits -> weights that are the probabilities times a number of the row,
// whose reciprocal is inv; one: 1 - sigmoid(l), where asked for and not softmax (else
// as it was).  The sigmoid scores of a row whose logits are all below -40 are exp(l) to
// 2^-57 and could vanish: there their ratios are taken.  Places past the row hold -inf and
// come out as 0.
template <typename S, bool kOne>
__device__ __forceinline__ void weigh(bool softmax, float (&v)[S::R][S::n], float (&inv)[S::R],
                                      float (&one)[kOne ? S::R : 1][kOne ? S::n : 1]) {
  constexpr int R = S::R, n = S::n;
  constexpr float kLog2e = 1.44269504f;
  float m[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    m[r] = v[r][0];
#pragma unroll
    for (int i = 1; i < n; ++i) m[r] = fmaxf(m[r], v[r][i]);
  }
  rows_max<S::L>(m);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    if (softmax || m[r] < -40.f) {
      add_mul(v[r], -m[r], kLog2e);
#pragma unroll
      for (int i = 0; i < n; ++i) {
        v[r][i] = exp2_approx(v[r][i]);
        if constexpr (kOne)
          if (!softmax) one[r][i] = 1.f;
      }
    } else {
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float e = exp2_approx(-fabsf(v[r][i]) * kLog2e);       // no overflow on either side
        const float q = __fdividef(1.f, 1.f + e), o = e * q;
        const bool up = v[r][i] >= 0.f;
        if constexpr (kOne) one[r][i] = up ? o : q;
        v[r][i] = up ? q : o;
      }
    }
    inv[r] = total(v[r]);
  }
  rows_sum<S::L>(inv);
#pragma unroll
  for (int r = 0; r < R; ++r) inv[r] = __fdividef(1.f, inv[r]);
}

struct BalanceShared {
  int starts[kThreads];   // of the sequences from the block's first on
  int hist[MOE_MAX_EXPERTS];
  int tokens, bad;
  float loss[kWarps];
  float sums[kWarps][33];
  int cnts[kWarps][33];
};
static_assert(sizeof(BalanceShared) <= 12 * 1024, "allow_smem");

// One block of tokens: the sums and counts of each sequence that it meets, into their slots.
template <typename S>
__device__ __forceinline__ void sum_tokens(const BalanceArgs& a, int block, BalanceShared& sh,
                                           float* sums) {
  constexpr int R = S::R, n = S::n, per = 32 / S::L;
  const int warp = threadIdx.x >> 5, seg = (threadIdx.x & 31) / S::L, lane = threadIdx.x & (S::L - 1);
  const int E = a.E;
  const long long first = (long long)block * a.chunk;
  const int begin = (int)min(first, (long long)a.T);
  const int end = (int)min(first + a.chunk, (long long)a.T);
  if (threadIdx.x == 0) sh.bad = 0;
  bool outside = false;
  const bool full = E == n * S::L;
  float nan[n];   // turn NaN with the first logit that is not finite
#pragma unroll
  for (int i = 0; i < n; ++i) nan[i] = 0.f;
  const Starts starts(a, sh.starts, seq_after(a, begin));
  for (int s = starts.s0; s < a.S; ++s) {
    const int lo = max(begin, starts(s)), hi = min(end, starts(s + 1));
    if (lo >= end) break;
    if (lo >= hi) continue;
    for (int e = threadIdx.x; e < E; e += kThreads) sh.hist[e] = 0;
    if (threadIdx.x == 0) sh.tokens = 0;
    __syncthreads();
    // the first rows are on their way while the choices are counted, and then the next
    // ones while one is worked on
    float next[R][n];
    uint8_t next_on[R];
    auto fetch = [&](unsigned t) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const unsigned at = t + r * per + seg;
        next_on[r] = 0;
        if (at < (unsigned)hi) {
          S::load(a.logits + (size_t)at * E, E, lane, -INFINITY, next[r]);
          next_on[r] = a.mask == nullptr ? 1 : __ldg(a.mask + at);
        }
      }
    };
    const unsigned start = lo + warp * S::kRows;
    // the choices, in the order in which they lie, four of a thread on their way at once
    const size_t from = (size_t)lo * a.k;
    const unsigned choices = (unsigned)(hi - lo) * (unsigned)a.k;
    int pick[4];
    uint8_t pick_on[4];
    auto fetch_picks = [&](unsigned i0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const unsigned i = i0 + j * kThreads;
        pick_on[j] = 0;
        if (i < choices) {
          pick[j] = __ldg(a.topk_idx + from + i);
          pick_on[j] = a.mask == nullptr ? 1 : __ldg(a.mask + lo + i / (unsigned)a.k);
        }
      }
    };
    fetch_picks(threadIdx.x);
    fetch(start);
    for (unsigned i = threadIdx.x; i < choices; i += 4 * kThreads) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (pick_on[j] == 0) continue;
        if (pick[j] >= 0 && pick[j] < E) atomicAdd(&sh.hist[pick[j]], 1);
        else outside = true;
      }
      fetch_picks(i + 4 * kThreads);
    }
    float acc[n];
#pragma unroll
    for (int i = 0; i < n; ++i) acc[i] = 0.f;
    int mine = 0;
    for (unsigned t = start; t < (unsigned)hi; t += kWarps * S::kRows) {
      float v[R][n], inv[R], none[1][1];
      bool on[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        on[r] = next_on[r] != 0;
        mine += on[r] && lane == 0;
#pragma unroll
        for (int i = 0; i < n; ++i) v[r][i] = next[r][i];
        if (!on[r]) {   // whatever a masked row holds stays out
#pragma unroll
          for (int i = 0; i < n; ++i) v[r][i] = 0.f;
        }
      }
      fetch(t + kWarps * S::kRows);
      if (full) {
#pragma unroll
        for (int r = 0; r < R; ++r) fma_into(nan, v[r], 0.f);
      } else {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < n; ++i)
            if (S::expert(lane, i) < E) nan[i] = fmaf(v[r][i], 0.f, nan[i]);
      }
      weigh<S, false>(a.softmax, v, inv, none);
#pragma unroll
      for (int r = 0; r < R; ++r) fma_into(acc, v[r], on[r] ? inv[r] : 0.f);
    }
#pragma unroll
    for (int i = 0; i < n; ++i)
      if (S::expert(lane, i) < E) sums[(warp * per + seg) * E + S::expert(lane, i)] = acc[i];
    if (mine) atomicAdd(&sh.tokens, mine);
    __syncthreads();
    const size_t slot = (size_t)block + s;
    for (int e = threadIdx.x; e < E; e += kThreads) {
      float v = 0.f;
#pragma unroll 16
      for (int w = 0; w < kWarps * per; ++w) v += sums[w * E + e];
      a.part_p[slot * E + e] = v;
      a.part_c[slot * E + e] = sh.hist[e];
    }
    if (threadIdx.x == 0) a.part_n[slot] = sh.tokens;
    __syncthreads();
  }
  if (isnan(total(nan))) atomicOr(&sh.bad, 1);
  if (outside) atomicOr(&sh.bad, 2);
  __syncthreads();
}

// Wait for what other blocks write: until *at is `launch` but for its two lowest bits, which
// are returned; 4: the wait ran out.
__device__ __forceinline__ int wait_for(const uint64_t* at, uint64_t launch,
                                        uint64_t limit) {
  uint64_t v;
  const uint64_t t0 = ptx::globaltimer_ns();
  do {
    asm volatile("ld.acquire.gpu.global.b64 %0, [%1];" : "=l"(v) : "l"(at) : "memory");
    if ((v & ~3ull) == launch) return (int)(v & 3u);
  } while (ptx::globaltimer_ns() - t0 < limit);
  return 4;
}
// The words of a launch are cleared before it ends, since a captured one comes again under its
// number: by the last block, which has seen them all.  Where it gave up it exchanges them for
// `spent`, and a block that then finds that in its word clears it itself.
__device__ __forceinline__ uint64_t spent(uint64_t launch) { return launch ^ 4u; }   // no launch's
__device__ __forceinline__ void clear(uint64_t* at) {
  asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(at), "l"(0ull) : "memory");
}
__device__ __forceinline__ uint64_t exchange(uint64_t* at, uint64_t v) {
  uint64_t old;
  asm volatile("atom.exch.relaxed.gpu.global.b64 %0, [%1], %2;" : "=l"(old) : "l"(at), "l"(v) : "memory");
  return old;
}
__device__ __forceinline__ void announce(uint64_t* at, uint64_t launch, int bits) {
  uint64_t old;
  asm volatile("atom.exch.release.gpu.global.b64 %0, [%1], %2;"
               : "=l"(old) : "l"(at), "l"(launch | (uint64_t)bits) : "memory");
  if (old == spent(launch)) clear(at);
}
// A number handed to another block in the words that announce it, beside one half of the
// launch's number each: nothing else has to be visible with it, and a store that waits for
// none before it takes 1 us less of the launch's end.  kLate: the wait before it ran out.
constexpr uint32_t kLate = 0x7fc0dead;   // a NaN that no arithmetic makes
__device__ __forceinline__ void post(uint64_t* at, uint64_t launch, uint32_t bits) {
  const uint64_t w0 = (launch & ~0xffffffffull) | bits, w1 = launch << 32 | bits;
  asm volatile("st.relaxed.gpu.global.b64 [%0], %1;" ::"l"(at), "l"(w0) : "memory");
  if (exchange(at + 1, w1) == spent(launch)) {
    clear(at);
    clear(at + 1);
  }
}
__device__ __forceinline__ uint32_t wait_posted(const uint64_t* at, uint64_t launch,
                                                uint64_t limit) {
  const uint64_t t0 = ptx::globaltimer_ns();
  do {
    uint64_t w0, w1;
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(w0) : "l"(at) : "memory");
    asm volatile("ld.relaxed.gpu.global.b64 %0, [%1];" : "=l"(w1) : "l"(at + 1) : "memory");
    const uint32_t bits = (uint32_t)w0;
    if (w0 == ((launch & ~0xffffffffull) | bits) && w1 == (launch << 32 | bits)) return bits;
  } while (ptx::globaltimer_ns() - t0 < limit);
  return kLate;
}

// Adder `rank` of a.adders: its share of the slots' sums, in order, and of the counts, once
// `wait` has returned.  Returns the share's loss, in the first warp.
template <typename Wait>
__device__ __forceinline__ float add_slots(const BalanceArgs& a, int rank, BalanceShared& sh,
                                           Wait&& wait) {
  const unsigned lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const unsigned E = a.E, groups = (E + 31) / 32, units = (unsigned)a.S * groups;   // < 2^22
  const unsigned share = a.share, per = kWarps / share;   // warps of a unit: a sequence's 32 experts
  const unsigned part = warp % share;
  float loss = 0.f;
  // where a unit's sequence lies is known ahead
  int next_lo = 0, next_hi = 0;
  auto look_up = [&](unsigned u0) {
    const unsigned u = u0 + warp / share;
    next_lo = next_hi = 0;
    if (u < units) {
      next_lo = seq_start(a, u / groups);
      next_hi = seq_start(a, u / groups + 1);
    }
  };
  look_up((unsigned)rank * per);
  wait();
  for (unsigned u0 = (unsigned)rank * per; u0 < units; u0 += (unsigned)a.adders * per) {
    const unsigned u = u0 + warp / share;
    const unsigned s = u / groups, e = (u - s * groups) * 32 + lane;
    float p = 0.f;
    int c = 0, tokens = 0;
    const int lo = next_lo, hi = next_hi;
    look_up(u0 + (unsigned)a.adders * per);
    if (u < units) {
      if (lo < hi) {
        const unsigned b0 = (unsigned)lo / (unsigned)a.chunk, b1 = (unsigned)(hi - 1) / (unsigned)a.chunk;
        if (a.mask == nullptr) tokens = lane == 0 ? hi - lo : 0;
        else if (b0 + lane <= b1) tokens = __ldcg(a.part_n + b0 + lane + s);
        if (e < E) {
          const size_t step = (size_t)share * E;
          const float* fp = a.part_p + ((size_t)b0 + part + s) * E + e;
          const int* fc = a.part_c + ((size_t)b0 + part + s) * E + e;
          int left = (int)(b1 - b0) - (int)part;
          // twenty slots' values are on their way at once, and added in order
          for (; left >= 0; left -= 20 * (int)share) {
            float x[20];
            int y[20];
#pragma unroll
            for (int i = 0; i < 20; ++i) {
              const bool in = left - i * (int)share >= 0;
              x[i] = in ? __ldcg(fp + i * step) : 0.f;
              y[i] = in ? __ldcg(fc + i * step) : 0;
            }
#pragma unroll
            for (int i = 0; i < 20; ++i) {
              p += x[i];
              c += y[i];
            }
            fp += 20 * step;
            fc += 20 * step;
          }
        }
        if (a.mask != nullptr)
          for (unsigned b = b0 + 32 + lane; b <= b1; b += 32) tokens += __ldcg(a.part_n + b + s);
      }
    }
    tokens = __reduce_add_sync(0xffffffffu, tokens);
    if (share > 1) {
      sh.sums[warp][lane] = p;
      sh.cnts[warp][lane] = c;
      __syncthreads();
      if (part == 0) {
        p = 0.f;
        c = 0;
#pragma unroll
        for (unsigned w = 0; w < kWarps; ++w) {
          p += w < share ? sh.sums[(warp + w) % kWarps][lane] : 0.f;
          c += w < share ? sh.cnts[(warp + w) % kWarps][lane] : 0;
        }
      }
      __syncthreads();
    }
    if (u < units && part == 0) {
      if (e < E) a.counts[(size_t)s * E + e] = c;
      if (e == 0) a.tokens[s] = tokens;
      // every lane its own experts: the lanes are added at the end
      if (e < E && tokens > 0) loss += (float)c * p * (a.factor / ((float)tokens * (float)tokens));
    }
  }
  loss = warp_sum(loss);
  if (lane == 0) sh.loss[warp] = loss;
  __syncthreads();
  return warp == 0 ? warp_sum(lane < kWarps ? sh.loss[lane] : 0.f) : 0.f;
}

template <typename S>
__global__ void __launch_bounds__(kThreads, S::n <= 16 ? 2 : 1) balance_kernel(BalanceArgs a) {
  __shared__ BalanceShared sh;
  extern __shared__ float sums[];   // [kWarps * 32 / L][E]
  const int block = blockIdx.x, blocks = a.blocks;
  if (block < blocks) {
    if (block == 0 && threadIdx.x == 0) ptx::hold_up(a.hold.at);
    sum_tokens<S>(a, block, sh, sums);
    // the threads' slots, seen by this one past a barrier, are released with the word
    if (threadIdx.x == 0) announce(a.done + block, a.launch, sh.bad);
    return;
  }
  const int rank = block - blocks;
  const bool last = rank == a.adders - 1;
  int bad = 0;   // 1: not finite, 2: outside, 4: late
  if (last && a.seq_offsets != nullptr)
    for (int s = threadIdx.x; s <= a.S; s += kThreads) {
      const int o = __ldg(a.seq_offsets + s);
      if (o < 0 || o > a.T || (s > 0 && o < __ldg(a.seq_offsets + s - 1))) bad |= 2;
    }
  const float share = add_slots(a, rank, sh, [&]() {
    for (int b = threadIdx.x; b < blocks; b += kThreads) bad |= wait_for(a.done + b, a.launch, a.hold.limit);
    __syncthreads();
  });
  uint64_t* added = a.done + blocks;   // two words each
  const int late = __syncthreads_or(bad & 4);
  if (!last) {
    if (threadIdx.x == 0) post(added + 2 * rank, a.launch, late ? kLate : __float_as_uint(share));
    return;
  }
  // the last block: the shares in order, and what the blocks have to report
  if (threadIdx.x == 0) sh.bad = 0;
  __syncthreads();
  bad = __reduce_or_sync(0xffffffffu, (unsigned)bad);
  if (bad != 0 && (threadIdx.x & 31) == 0) atomicOr(&sh.bad, bad);
  float v = 0.f;
  if (threadIdx.x < 32)
    for (int r = threadIdx.x; r < a.adders - 1; r += 32) {
      const uint32_t bits = wait_posted(added + 2 * r, a.launch, a.hold.limit);
      if (bits == kLate) atomicOr(&sh.bad, 4);
      else v += __uint_as_float(bits);
    }
  __syncthreads();
  if (sh.bad & 4) {   // some are still to come
    for (int b = threadIdx.x; b < blocks; b += kThreads)
      if ((exchange(a.done + b, spent(a.launch)) & ~3ull) == a.launch) clear(a.done + b);
    for (int r = threadIdx.x; r < a.adders - 1; r += kThreads)
      if (exchange(added + 2 * r + 1, spent(a.launch)) >> 32 == (a.launch & 0xffffffffull)) {
        clear(added + 2 * r);
        clear(added + 2 * r + 1);
      }
  } else {
    for (int b = threadIdx.x; b < blocks + 2 * a.adders; b += kThreads) a.done[b] = 0;
  }
  if (threadIdx.x < 32) {
    v = warp_sum(v) + share;
    if (threadIdx.x == 0) {
      *a.loss = v;
      a.status[0] = sh.bad & 4 ? MOE_ERR_TIMEOUT : sh.bad & 2 ? MOE_ERR_INVALID_ARG
                    : sh.bad & 1 ? MOE_ERR_NONFINITE : 0;
      a.status[1] = 0;
    }
  }
}

// dlogits: a block of consecutive tokens.  kOnto: added onto `out`.
template <typename S, bool kOnto>
__global__ void __launch_bounds__(kThreads, S::n <= 16 ? 2 : 1)
balance_backward_kernel(BalanceArgs a, const float* __restrict__ dloss,
                        const int32_t* __restrict__ counts, const int32_t* __restrict__ tokens,
                        float* out) {
  constexpr int R = S::R, n = S::n, per = 32 / S::L;
  const int warp = threadIdx.x >> 5, seg = (threadIdx.x & 31) / S::L, lane = threadIdx.x & (S::L - 1);
  const int E = a.E;
  const long long first = (long long)blockIdx.x * a.chunk;
  const int begin = (int)min(first, (long long)a.T);
  const int end = (int)min(first + a.chunk, (long long)a.T);
  const float g = a.factor * (dloss != nullptr ? __ldg(dloss) : 1.f);
  // rows lo .. hi - 1 of sequence s; s < 0: rows of none
  auto rows = [&](int s, int lo, int hi) {
    float load[n];
    if (s >= 0) {
      const int m = __ldg(tokens + s);
      const int mean = (int)((long long)a.k * m / E);
      const float f = m > 0 ? g / ((float)m * (float)m) : 0.f;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const int e = S::expert(lane, i);
        load[i] = e < E ? (float)(__ldg(counts + (size_t)s * E + e) - mean) * f : 0.f;
      }
    } else if (kOnto) {
      return;
    }
    for (unsigned t = lo + warp * S::kRows; t < (unsigned)hi; t += kWarps * S::kRows) {
      float v[R][n], old[kOnto ? R : 1][kOnto ? n : 1];
      bool on[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const unsigned at = t + r * per + seg;   // past the last int at the most
        on[r] = s >= 0 && at < (unsigned)hi && (a.mask == nullptr || __ldg(a.mask + at) != 0);
        if (on[r]) {
          S::load(a.logits + (size_t)at * E, E, lane, -INFINITY, v[r]);
          if constexpr (kOnto) {
            // plain loads: the same rows are written below
#pragma unroll
            for (int i = 0; i < n; i += S::V) {
              const int e = S::expert(lane, i);
              if constexpr (S::V == 4) {
                const float4 x = e < E ? *reinterpret_cast<const float4*>(out + (size_t)at * E + e)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
                old[r][i] = x.x; old[r][i + 1] = x.y; old[r][i + 2] = x.z; old[r][i + 3] = x.w;
              } else {
                old[r][i] = e < E ? out[(size_t)at * E + e] : 0.f;
              }
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < n; ++i) v[r][i] = 0.f;
        }
      }
      if (s >= 0) {
        float one[R][n], inv[R], mean[R];
        weigh<S, true>(a.softmax, v, inv, one);
#pragma unroll
        for (int r = 0; r < R; ++r) mean[r] = dot(v[r], load);
        rows_sum<S::L>(mean);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          // p (load - sum p load), p = v inv
          const float shift = -inv[r] * (mean[r] * inv[r]);
          if (!a.softmax) {
#pragma unroll
            for (int i = 0; i < n; ++i) v[r][i] *= one[r][i];
          }
          each<n>(
              [&](int i) { v[r][i] = fmaf(v[r][i], fmaf(load[i], inv[r], shift), kOnto ? old[kOnto ? r : 0][kOnto ? i : 0] : 0.f); },
              [&](int i) {
                const float2 f = __ffma2_rn(two(load + i), two(inv[r]), two(shift));
                const float2 x = kOnto ? __ffma2_rn(two(v[r] + i), f, two(old[kOnto ? r : 0] + (kOnto ? i : 0)))
                                       : __fmul2_rn(two(v[r] + i), f);
                v[r][i] = x.x;
                v[r][i + 1] = x.y;
              });
          if (!on[r]) {
#pragma unroll
            for (int i = 0; i < n; ++i) v[r][i] = 0.f;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const unsigned at = t + r * per + seg;
        if (kOnto ? !on[r] : at >= (unsigned)hi) continue;
        float* row = out + (size_t)at * E;
#pragma unroll
        for (int i = 0; i < n; i += S::V) {
          const int e = S::expert(lane, i);
          if (e >= E) continue;
          if constexpr (S::V == 4)
            *reinterpret_cast<float4*>(row + e) = make_float4(v[r][i], v[r][i + 1], v[r][i + 2], v[r][i + 3]);
          else
            row[e] = v[r][i];
        }
      }
    }
  };
  __shared__ int held[kThreads];
  const Starts starts(a, held, seq_after(a, begin));
  int at = begin;
  for (int s = starts.s0; s < a.S; ++s) {
    const int lo = max(at, starts(s)), hi = min(end, starts(s + 1));
    if (lo >= end) break;
    if (lo > at) rows(-1, at, lo);
    at = lo;
    if (lo >= hi) continue;
    rows(s, lo, hi);
    at = hi;
  }
  if (at < end) rows(-1, at, end);
}

// Tokens per block: two blocks for each SM where there are many (three: 40001 x 256 23.6 us
// in the place of 20.6), at least 64 (8192 x 256 12.6 us, and 13.7 from 16 on).
constexpr int kMinChunk = 64, kRound = 4;
int chunk_of(int T) {
  const long long c = ((long long)T + 2 * kSms - 1) / (2 * kSms);
  return (int)(c < kMinChunk ? kMinChunk : (c + kRound - 1) / kRound * kRound);
}
// Warps that share a sequence's 32 experts, each adding up to 20 of their slots, and the
// blocks that this takes, half as many as sum tokens at most.
int share_of(int blocks, int S) {
  int share = 1;
  while (share < kWarps && 20 * share < blocks / S + 1) share *= 2;
  return share;
}
int adders_of(int blocks, int E, int S) {
  const long long units = (long long)S * ((E + 31) / 32);
  const long long want = (units * share_of(blocks, S) + kWarps - 1) / kWarps;
  const int most = blocks / 2 > 1 ? blocks / 2 : 1;
  return (int)(want < most ? want : most);
}

#define MOE_UNWRAP(...) __VA_ARGS__
#define MOE_BALANCE_SHAPE(E, CASE)                              \
  do {                                                          \
    if (E % 4 == 0 && E >= 16) {                                \
      if (E <= 32) CASE((Shape<4, 4, 8, 2>));                   \
      else if (E <= 64) CASE((Shape<4, 4, 16, 4>));             \
      else if (E <= 128) CASE((Shape<4, 4, 32, 4>));            \
      else if (E <= 256) CASE((Shape<4, 8, 32, 2>));            \
      else if (E <= 512) CASE((Shape<4, 16, 32, 1>));           \
      else CASE((Shape<4, 32, 32, 1>));                         \
    } else if (E <= 8) CASE((Shape<1, 1, 8, 4>));               \
    else if (E <= 32) CASE((Shape<1, 4, 8, 2>));                \
    else if (E <= 64) CASE((Shape<1, 2, 32, 4>));               \
    else if (E <= 128) CASE((Shape<1, 4, 32, 4>));              \
    else if (E <= 256) CASE((Shape<1, 8, 32, 2>));              \
    else if (E <= 512) CASE((Shape<1, 16, 32, 1>));             \
    else CASE((Shape<1, 32, 32, 1>));                           \
  } while (0)

}  // namespace

size_t balance_layout(int T, int E, int S, BalanceArgs* a, void* ws) {
  const int chunk = T > 0 ? chunk_of(T) : kWarps;
  const int blocks = (int)(((long long)T + chunk - 1) / chunk);
  const size_t slots = (size_t)blocks + S;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = align_up(o + bytes, 256); return at; };
  const int adders = adders_of(blocks, E, S);
  const size_t status = take(256), done = take((size_t)(blocks + 2 * adders) * 8);
  const size_t n = take(slots * 4), p = take(slots * E * 4), c = take(slots * E * 4);
  if (a != nullptr) {
    a->chunk = chunk;
    a->blocks = blocks;
    a->adders = adders;
    a->share = share_of(blocks, S);
    a->status = ws_ptr<int>(ws, status);
    a->done = ws_ptr<uint64_t>(ws, done);
    a->part_n = ws_ptr<int>(ws, n);
    a->part_p = ws_ptr<float>(ws, p);
    a->part_c = ws_ptr<int>(ws, c);
  }
  return o;
}

template <typename S>
cudaError_t launch_sum(const BalanceArgs& a, cudaStream_t s) {
  constexpr int of_expert = kWarps * (32 / S::L) * 4;
  const int smem = of_expert * a.E;
  const cudaError_t e = allow_smem(balance_kernel<S>, smem, of_expert * S::n * S::L);
  if (e != cudaSuccess) return e;
  balance_kernel<S><<<a.blocks + a.adders, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}
cudaError_t launch_balance(BalanceArgs a, cudaStream_t s) {
  a.launch = unique_number() << 2;
  a.hold = diag_hold();
#define CASE(S) return launch_sum<MOE_UNWRAP S>(a, s)
  MOE_BALANCE_SHAPE(a.E, CASE);
#undef CASE
}

template <typename S>
cudaError_t launch_backward(const BalanceArgs& a, const float* dloss, const int32_t* counts,
                            const int32_t* tokens, bool onto, float* out, cudaStream_t s) {
  const auto kern = onto ? balance_backward_kernel<typename S::template Backward<true>, true>
                         : balance_backward_kernel<typename S::template Backward<false>, false>;
  kern<<<a.blocks, kThreads, 0, s>>>(a, dloss, counts, tokens, out);
  return cudaGetLastError();
}
cudaError_t launch_balance_backward(const BalanceArgs& a, const float* dloss, const int32_t* counts,
                                    const int32_t* tokens, bool onto, float* out, cudaStream_t s) {
  const int E = a.E;
#define CASE(S) return launch_backward<MOE_UNWRAP S>(a, dloss, counts, tokens, onto, out, s)
  MOE_BALANCE_SHAPE(E, CASE);
#undef CASE
}

}  // namespace moe
