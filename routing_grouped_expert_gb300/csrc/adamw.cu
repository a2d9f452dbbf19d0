// One AdamW step over many tensors.
//
//   g' = grad_scale g;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// p is the fp32 master weight where there is one (the parameter is then its rounding),
// else the parameter itself.  m and v are fp32, or e4m3 in blocks of 256 elements with an
// fp32 scale each: the block's largest magnitude times fl(1 / 448); v is held as its square root,
// which halves the range its exponents have to span.  The step itself uses m and v before
// they are rounded.
//
// Every array is read and written once, which bounds it: 704 M bf16 parameters in 2.76 ms
// with fp32 moments and masters (19.7 GB, 1.05 of the rate of a plain copy) and in 1.10 ms
// with 8-bit moments (7.1 GB, 0.95; the schedulers issue in three quarters of their cycles).
// 150 ragged tensors of 15.3 M parameters: 68 us (0.93) and, gradients in fp32, 52 us (0.82).
//
// Blocks of 2048 elements in launch order: what is in flight then lies close together in
// each array.  A block that went on to further chunks, with its loads ahead in registers or
// in a ring of shared memory, was slower for that reason: fp32 moments 2.76 -> 2.91 and
// 4.24 ms, 8-bit ones 1.42 -> 2.24 and 1.47 at the same point.  The tensors' table is a
// kernel argument, so a call makes no copy and keeps nothing on the device.
#include <cuda_fp8.h>
#include <math.h>

#include <type_traits>

#include "moe_common.cuh"
#include "status.cuh"

namespace moe {
namespace {

using bf16 = __nv_bfloat16;

// Groups of eight elements per thread, all on their way at once, and blocks per SM.  8-bit
// moments, ms, before small roots had a path of their own (two groups now 1.10): 128 threads of one group 1.27, of two 1.13 (8 blocks) 1.16 (6) 1.25 (5), of
// three 1.20; 256 threads of one 1.33; 64 of two 1.15.  fp32 moments: 2.76 to 2.77 in all.
constexpr int kThreads = 128;
constexpr int kTurns = 2;
constexpr int kTurn = kThreads * 8;
constexpr int kChunk = kTurn * kTurns;     // elements per block
constexpr int kB8 = 8, kB32 = 4;     // for 8-bit and fp32 moments

struct Entry {
  void* param;
  const void* grad;
  long long n;
  uint32_t start;    // the tensor's first block of 256 in the state arrays
  float decay;
};
// As many tensors as kernel arguments hold; fewer where they are enough (the arguments
// are copied at each launch).
template <int N>
struct Table {
  int count;
  uint32_t first[N];   // the tensor's first chunk
  Entry entry[N];
};

struct State {
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
};
struct Hyper {
  float lr, b1, omb1, b2, omb2, eps;   // omb: 1 - b, from 64 bits
  float inv1, root;                    // 1 / (1 - b1^t), 1 / sqrt(1 - b2^t)
  float log_b1, log_b2;
  const long long* step;               // where not null: t, and inv1 and root follow from it
  const float* lr_at;                  // where not null: lr
  const float* grad_scale;             // where not null
};

// Eight consecutive values of a type: as they lie in memory, and as four pairs of fp32, on
// which one instruction works at a time.
template <typename T>
struct Eight;
template <>
struct Eight<bf16> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(bf16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ float2 get(int i) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    return __bfloat1622float2(reinterpret_cast<const __nv_bfloat162&>(w[i]));
  }
  __device__ __forceinline__ void set(const float2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<__nv_bfloat162&>(w[i]) = __float22bfloat162_rn(f[i]);
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Eight<float> {
  float4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = reinterpret_cast<const float4*>(p)[0];
    v[1] = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = v[0];
    reinterpret_cast<float4*>(p)[1] = v[1];
  }
  __device__ __forceinline__ float2 get(int i) const {
    return i & 1 ? make_float2(v[i / 2].z, v[i / 2].w) : make_float2(v[i / 2].x, v[i / 2].y);
  }
  __device__ __forceinline__ void set(const float2 (&f)[4]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) v[i] = make_float4(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x, f[2 * i + 1].y);
  }
};
template <>
struct Eight<__nv_fp8_e4m3> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_fp8_e4m3* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void store(__nv_fp8_e4m3* p) const { *reinterpret_cast<uint2*>(p) = v; }
  __device__ __forceinline__ float2 get(int i) const {
    const uint32_t w = (i < 2 ? v.x : v.y) >> (16 * (i & 1));
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)w, __NV_E4M3)));
  }
  __device__ __forceinline__ void set(const float2 (&f)[4]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = __nv_cvt_float2_to_fp8x2(f[i], __NV_SATFINITE, __NV_E4M3);
    v = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
  }
};

__device__ __forceinline__ float one(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float one(const float* p) { return *p; }
__device__ __forceinline__ void put(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// The eight elements from p on, or `left` of them.
template <bool kAll, typename T>
__device__ __forceinline__ void read(Eight<T>& e, const T* p, int left) {
  if constexpr (kAll) {
    e.load(p);
  } else if (left >= 8) {
    e.load(p);
  } else {
    float2 f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      f[j] = make_float2(2 * j < left ? one(p + 2 * j) : 0.f, 2 * j + 1 < left ? one(p + 2 * j + 1) : 0.f);
    e.set(f);
  }
}
template <bool kAll, typename T>
__device__ __forceinline__ void write(T* p, int left, const float2 (&f)[4]) {
  if (kAll || left >= 8) {
    Eight<T> e;
    e.set(f);
    e.store(p);
    return;
  }
  if constexpr (!kAll) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (2 * j < left) put(p + 2 * j, f[j].x);
      if (2 * j + 1 < left) put(p + 2 * j + 1, f[j].y);
    }
  }
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
// A sum of products, each operation rounded to nearest.  Added one by one: the compiler
// fuses a pair's addition with the multiplication before it.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  return make_float2(__fadd_rn(a.x, b.x), __fadd_rn(a.y, b.y));
}

// The square root: a Newton step from the reciprocal root, whose last operation rounds a value
// that is exact to 2^-44.  Of zero and of 2^-101 to 2^128 it is the correctly rounded one (every
// value compared); below, the remainder leaves fp32.
__device__ __forceinline__ float2 root2(float2 v) {
  float2 y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(fmaxf(v.x, 1.17549435e-38f)));
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(fmaxf(v.y, 1.17549435e-38f)));
  const float2 g = __fmul2_rn(v, y), h = __fmul2_rn(y, both(0.5f));
  const float2 rest = __ffma2_rn(__fmul2_rn(g, both(-1.f)), g, v);
  return __ffma2_rn(rest, h, g);
}
constexpr float kSmall = 0x1p-100f;
// The same of any value, small ones by 2^100 times them.
__device__ __forceinline__ float2 root2_small(float2 v) {
  const bool x = v.x < kSmall, y = v.y < kSmall;
  const float2 r = root2(__fmul2_rn(v, make_float2(x ? 0x1p100f : 1.f, y ? 0x1p100f : 1.f)));
  return __fmul2_rn(r, make_float2(x ? 0x1p-50f : 1.f, y ? 0x1p-50f : 1.f));
}
__device__ __forceinline__ float rcp_approx(float x) {   // of normal numbers
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The largest magnitude of the warp's 32 times eight values.
__device__ __forceinline__ float block_max(const float2 (&f)[4]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(m), "f"(f[i].x), "f"(f[i].y));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}
// f / scale with scale = `most` fl(1 / 448), most the block's largest magnitude; returns the
// scale.  Quotients are correctly rounded (Markstein: with the correctly rounded
// reciprocal, one correction of the quotient by its remainder).  Blocks whose scale is
// below the normal range become zero.
__device__ __forceinline__ float to_units(float2 (&f)[4], float most) {
  const float scale = __fmul_rn(most, 1.f / 448.f);
  const bool some = scale >= 1.17549435e-38f;
  const float inv = some ? __frcp_rn(scale) : 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 q = __fmul2_rn(f[i], both(inv));
    const float2 rest = __ffma2_rn(q, both(-scale), f[i]);
    f[i] = __ffma2_rn(rest, both(inv), q);
  }
  return some ? scale : 0.f;
}

constexpr float kLeast = 1.f / 2048.f;   // the smallest e4m3 value is 2^-9

// Eight elements of a thread, as they lie in memory.  P, G: types of the parameters and
// gradients.  k8: 8-bit moments.
//
// What an 8-bit moment is rounded to is a function of the inputs: m, v, the root, the scale
// and the quotient are fp32 with each operation rounded to nearest, none of them fused.
template <typename P, typename G, bool kMaster, bool k8>
struct Group {
  using M = typename std::conditional<k8, __nv_fp8_e4m3, float>::type;
  using W = typename std::conditional<kMaster, float, P>::type;
  const G* grad;
  W* from;
  P* param;
  M *ms, *vs;
  float *m_scale, *v_scale;   // of the warp's block
  Eight<W> rp;
  Eight<G> rg;
  Eight<M> rm, rv;
  float sm, sv;

  // kWhole: all of the block's elements are there; else `left` of these are.  8-bit arrays
  // hold whole blocks.
  template <bool kWhole>
  __device__ __forceinline__ void load(int left) {
    read<kWhole>(rg, grad, left);
    read<k8 || kWhole>(rm, ms, left);
    read<k8 || kWhole>(rv, vs, left);
    read<kWhole>(rp, from, left);
    sm = sv = 1.f;
    if constexpr (k8) {
      sm = *m_scale;
      sv = *v_scale;
    }
  }
  // Their step; returns whether an element was left as it was.
  template <bool kWhole>
  __device__ __forceinline__ bool step(int left, float rate, float keep, float more, float root,
                                       float gs, const Hyper& h);
};

template <typename P, typename G, bool kMaster, bool k8>
template <bool kWhole>
__device__ __forceinline__ bool Group<P, G, kMaster, k8>::step(int left, float rate, float keep,
                                                               float more, float root, float gs,
                                                               const Hyper& h) {
  float2 m[4], v[4], p[4];
  float2 nan = both(0.f);   // turns NaN with the first moment that is not finite
  // the pairs' moments before and after the step
  auto old = [&](int i, float2& m, float2& v) {
    m = rm.get(i);
    v = rv.get(i);
    if constexpr (k8) {
      // A root that is held as zero in a block that is not stands for a quarter of the
      // smallest value, which is rounded to zero again: where the first moment is still
      // there and the gradient is zero (an expert without a token), its step stays bounded.
      m = __fmul2_rn(m, both(sm));
      v = __fmul2_rn(make_float2(fmaxf(v.x, kLeast), fmaxf(v.y, kLeast)), both(sv));
      v = __fmul2_rn(v, v);
    }
  };
  auto moments = [&](int i, float2& m, float2& v) {
    const float2 g = __fmul2_rn(rg.get(i), both(gs));
    old(i, m, v);
    m = add2(__fmul2_rn(m, both(h.b1)), __fmul2_rn(g, both(h.omb1)));
    v = add2(__fmul2_rn(v, both(h.b2)), __fmul2_rn(__fmul2_rn(g, both(h.omb2)), g));
  };
  // of the second moments that are not zero, the smallest, as its bits less one
  uint32_t least = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    moments(i, m[i], v[i]);
    nan = __ffma2_rn(m[i], both(0.f), nan);
    nan = __ffma2_rn(v[i], both(0.f), nan);
    least = min(min(__float_as_uint(v[i].x) - 1u, __float_as_uint(v[i].y) - 1u), least);
  }
  auto next = [&](int i, const float2& r) {
    const float2 d = __ffma2_rn(r, both(root), both(h.eps));
    const float2 s = __fmul2_rn(m[i], make_float2(rcp_approx(d.x), rcp_approx(d.y)));
    const float2 w = rp.get(i);
    p[i] = __ffma2_rn(w, both(keep), __ffma2_rn(w, both(more), __fmul2_rn(s, both(rate))));
  };
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 r = root2(v[i]);
    next(i, r);
    if constexpr (k8) v[i] = r;
  }
  const bool bad = isnan(nan.x + nan.y);
  if (bad || least < __float_as_uint(kSmall) - 1u) {
    // rare: roots of moments below 2^-100 (gradients of 1e-14), and elements whose moments are
    // not finite, which stay as they were.  Read again: kept, the values would cost every block
    // registers.  As a branch of its own, small roots took 1.24 ms of 704 M parameters with 8-bit
    // moments, here 1.11.
    asm volatile("" ::: "memory");
    load<kWhole>(left);
    auto stay = [&](float& p, float& m, float& v, float op, float om, float ov) {
      if (fabsf(m) < INFINITY && fabsf(v) < INFINITY) return;
      p = op;
      m = om;
      v = ov;
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 om, ov;
      old(i, om, ov);
      moments(i, m[i], v[i]);
      next(i, root2_small(v[i]));
      const float2 op = rp.get(i);
      stay(p[i].x, m[i].x, v[i].x, op.x, om.x, ov.x);
      stay(p[i].y, m[i].y, v[i].y, op.y, om.y, ov.y);
      if constexpr (k8) v[i] = root2_small(v[i]);
    }
  }
  if constexpr (kMaster) write<kWhole>(from, left, p);
  write<kWhole>(param, left, p);
  if constexpr (k8) {
    // v: its roots.  Places past the tensor's end hold zeros and stay so.
    sm = to_units(m, block_max(m));
    sv = to_units(v, block_max(v));
    if ((threadIdx.x & 31) == 0) {
      *m_scale = sm;
      *v_scale = sv;
    }
  }
  write<k8 || kWhole>(ms, left, m);
  write<k8 || kWhole>(vs, left, v);
  return bad;
}

template <typename P, typename G, bool kMaster, bool k8, int N>
__global__ void __launch_bounds__(kThreads, k8 ? kB8 : kB32)
adamw_kernel(const __grid_constant__ Table<N> table, State st, Hyper h, int* status,
             uint64_t launch) {
  status_begin(status, launch);
  int lo = 0, hi = table.count - 1;      // the last tensor whose first chunk is not after this one
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (table.first[mid] <= blockIdx.x) lo = mid;
    else hi = mid - 1;
  }
  const Entry& t = table.entry[lo];
  const size_t chunk = blockIdx.x - table.first[lo];
  const size_t at = chunk * kChunk, state = (size_t)t.start * MOE_ADAMW_BLOCK + at;
  Group<P, G, kMaster, k8> group[kTurns];
#pragma unroll
  for (int u = 0; u < kTurns; ++u) {
    const unsigned i = u * kTurn + threadIdx.x * 8;
    using Gr = Group<P, G, kMaster, k8>;
    group[u].grad = static_cast<const G*>(t.grad) + at + i;
    group[u].param = static_cast<P*>(t.param) + at + i;
    if constexpr (kMaster) group[u].from = st.master + state + i;
    else group[u].from = group[u].param;
    group[u].ms = static_cast<typename Gr::M*>(st.m) + state + i;
    group[u].vs = static_cast<typename Gr::M*>(st.v) + state + i;
    group[u].m_scale = st.m_scale + (state + i) / MOE_ADAMW_BLOCK;
    group[u].v_scale = st.v_scale + (state + i) / MOE_ADAMW_BLOCK;
  }
  const long long rest = t.n - (long long)at;    // of the tensor, from this block on
  const bool whole = rest >= kChunk;
  // everything is on its way before anything is waited for
  if (whole) {
#pragma unroll
    for (int u = 0; u < kTurns; ++u) group[u].template load<true>(8);
  }

  const float lr = h.lr_at != nullptr ? __ldg(h.lr_at) : h.lr;
  float inv1 = h.inv1, root = h.root;
  if (h.step != nullptr) {
    const float s = fmaxf((float)__ldg(h.step), 1.f);
    inv1 = 1.f / -expm1f(s * h.log_b1);
    root = rsqrtf(-expm1f(s * h.log_b2));
  }
  const float rate = -lr * inv1, shrink = -lr * t.decay;
  // 1 - lr decay as a sum, so that p is rounded once: by itself it would be a multiple of 2^-24,
  // and a decay of 2e-8 a step none.  Both parts above zero leave an infinite weight as it is.
  const float keep = __fadd_rd(__fadd_rd(1.f, shrink), -0x1p-24f), more = (1.f - keep) + shrink;
  const float gs = h.grad_scale != nullptr ? __ldg(h.grad_scale) : 1.f;
  // no element takes a step: 8-bit moments would be rounded again by their blocks' largest
  // values, and the scales
  if (!(fabsf(gs) < INFINITY)) {
    if ((threadIdx.x & 31) == 0) status_report(status, launch, MOE_ERR_NONFINITE);
    return;
  }
  bool bad = false;
  if (whole) {
#pragma unroll
    for (int u = 0; u < kTurns; ++u)
      bad |= group[u].template step<true>(8, rate, keep, more, root, gs, h);
  } else {
#pragma unroll 1
    for (int u = 0; u < kTurns; ++u) {
      const int left = (int)rest - u * kTurn - (int)threadIdx.x * 8;
      // an 8-bit block is worked on by a whole warp
      if (k8 ? left + (int)(threadIdx.x & 31) * 8 <= 0 : left <= 0) break;
      Group<P, G, kMaster, k8> part = group[0];
      part.grad += u * kTurn;
      part.param += u * kTurn;
      part.from += u * kTurn;
      part.ms += u * kTurn;
      part.vs += u * kTurn;
      part.m_scale += u * (kTurn / MOE_ADAMW_BLOCK);
      part.v_scale += u * (kTurn / MOE_ADAMW_BLOCK);
      part.template load<false>(left);
      bad |= part.template step<false>(left, rate, keep, more, root, gs, h);
    }
  }
  if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0)
    status_report(status, launch, MOE_ERR_NONFINITE);
}

template <typename P, typename G, bool kMaster, bool k8, int N>
cudaError_t launch_n(const AdamwArgs& a, const Hyper& h, const State& st, int* status,
                     cudaStream_t s) {
  uint64_t launch = 0;
  cudaError_t e = begin_status(status, s, &launch);
  if (e != cudaSuccess) return e;
  Table<N> table;
  table.count = 0;
  unsigned long long chunks = 0;
  auto flush = [&]() {
    adamw_kernel<P, G, kMaster, k8, N><<<(unsigned)chunks, kThreads, 0, s>>>(table, st, h, status,
                                                                             launch);
    launch = 0;   // the launches after the first leave the status word alone
    table.count = 0;
    chunks = 0;
    return cudaGetLastError();
  };
  for (int i = 0; i < a.count; ++i) {
    const moe_adamw_tensor& t = a.tensors[i];
    if (t.n == 0) continue;
    const unsigned long long need = ((unsigned long long)t.n + kChunk - 1) / kChunk;
    if (table.count == N || chunks + need > 0x7fffffffull) {
      e = flush();
      if (e != cudaSuccess) return e;
    }
    table.first[table.count] = (uint32_t)chunks;
    table.entry[table.count++] =
        Entry{t.param, a.grads[i], (long long)t.n, (uint32_t)(t.start / MOE_ADAMW_BLOCK),
              (float)(a.config->weight_decay * t.decay)};
    chunks += need;
  }
  if (chunks > 0) return flush();
  // nothing to do since the last launch; without one the status is still to be cleared
  return launch != 0 ? cudaMemsetAsync(status, 0, 2 * sizeof(int), s) : cudaSuccess;
}

template <typename P, typename G, bool kMaster, bool k8>
cudaError_t launch_t(const AdamwArgs& a, const Hyper& h, const State& st, int* status,
                     cudaStream_t s) {
  if (a.count <= 16) return launch_n<P, G, kMaster, k8, 16>(a, h, st, status, s);
  return launch_n<P, G, kMaster, k8, 256>(a, h, st, status, s);
}

}  // namespace

cudaError_t launch_adamw(const AdamwArgs& a, int* status, cudaStream_t s) {
  const moe_adamw_config& c = *a.config;
  Hyper h{};
  h.lr = (float)c.lr;
  h.b1 = (float)c.beta1;
  h.omb1 = (float)(1.0 - c.beta1);
  h.b2 = (float)c.beta2;
  h.omb2 = (float)(1.0 - c.beta2);
  h.eps = (float)c.eps;
  h.log_b1 = (float)log(c.beta1);
  h.log_b2 = (float)log(c.beta2);
  h.step = reinterpret_cast<const long long*>(a.step_at);
  h.lr_at = a.lr_at;
  h.grad_scale = a.grad_scale;
  const double t = (double)a.step;
  h.inv1 = (float)(1.0 / (1.0 - pow(c.beta1, t)));
  h.root = (float)(1.0 / sqrt(1.0 - pow(c.beta2, t)));
  const State st{a.master, a.exp_avg, a.exp_avg_sq, a.exp_avg_scale, a.exp_avg_sq_scale};
  const bool k8 = c.state_bits == 8, pf = a.param_type == MOE_F32, gf = a.grad_type == MOE_F32;
#define GO(P, G, master)                                                  \
  return k8 ? launch_t<P, G, master, true>(a, h, st, status, s)           \
            : launch_t<P, G, master, false>(a, h, st, status, s)
  if (pf) {
    if (gf) GO(float, float, false);
    GO(float, bf16, false);
  }
  if (a.master != nullptr) {
    if (gf) GO(bf16, float, true);
    GO(bf16, bf16, true);
  }
  if (gf) GO(bf16, float, false);
  GO(bf16, bf16, false);
#undef GO
}

}  // namespace moe
