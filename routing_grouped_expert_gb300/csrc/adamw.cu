// One AdamW step over many tensors.
//
//   g' = grad_scale g;  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr decay) - lr / (1 - b1^t) m / (sqrt(v / (1 - b2^t)) + eps)
//
// p is the fp32 master weight where there is one (the parameter is then its rounding),
// else the parameter itself.  m and v are fp32, or e4m3 in blocks of 256 elements with an
// fp32 scale each: the block's largest magnitude over 448; v is held as its square root,
// which halves the range its exponents have to span.  The step itself uses m and v before
// they are rounded.
//
// Bound by memory: every array is read and written once.  The tensors' table is a kernel
// argument, so a call makes no copy and keeps nothing on the device.
#include <cuda_fp8.h>
#include <math.h>

#include "moe_common.cuh"
#include "status.cuh"

namespace moe {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kThreads = 256;
constexpr int kPerThread = 2;                          // groups of eight elements
constexpr int kChunk = kThreads * 8 * kPerThread;      // elements per block

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

__device__ __forceinline__ void load8(const bf16* p, float (&f)[8]) {
  const uint4 v = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* q = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(q[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0];
  const float4 b = reinterpret_cast<const float4*>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_fp8_e4m3* p, float (&f)[8]) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = i < 2 ? v.x : v.y;
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * (i & 1))), __NV_E4M3);
    const float2 t = __half22float2(__half2(h));
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void store8(bf16* p, const float (&f)[8]) {
  uint4 v;
  __nv_bfloat162* q = reinterpret_cast<__nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) q[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(p) = v;
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ void store8(__nv_fp8_e4m3* p, const float (&f)[8]) {
  uint2 v = make_uint2(0u, 0u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w = __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i], f[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    if (i < 2) v.x |= w << (16 * (i & 1));
    else v.y |= w << (16 * (i & 1));
  }
  *reinterpret_cast<uint2*>(p) = v;
}
__device__ __forceinline__ float get(const bf16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ float get(const float* p) { return *p; }
__device__ __forceinline__ void put(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }

// `left` of the eight elements from p on: all of them by wide accesses.
template <typename T>
__device__ __forceinline__ void read8(const T* p, long long left, float (&f)[8]) {
  if (left >= 8) {
    load8(p, f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = j < left ? get(p + j) : 0.f;
  }
}
template <typename T>
__device__ __forceinline__ void write8(T* p, long long left, const float (&f)[8]) {
  if (left >= 8) {
    store8(p, f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (j < left) put(p + j, f[j]);
  }
}

__device__ __forceinline__ float sqrt_approx(float x) {   // 1 ulp
  float r;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The largest of eight values of each lane of the warp (none negative).
__device__ __forceinline__ float block_max(const float (&f)[8]) {
  float m = fabsf(f[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
}
// Scales f so that its largest magnitude, `most` over the block, is 448, and returns what
// a unit of the result stands for.  Magnitudes that cannot be told from zero become zero.
__device__ __forceinline__ float to_units(float (&f)[8], float most) {
  const float scale = most / 448.f;
  const bool some = scale >= 1.17549435e-38f;
  const float inv = some ? 1.f / scale : 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] *= inv;
  return some ? scale : 0.f;
}

// P, G: types of the parameters and gradients.  k8: 8-bit moments.
template <typename P, typename G, bool kMaster, bool k8, int N>
__global__ void __launch_bounds__(kThreads)
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
  P* param = static_cast<P*>(t.param);
  const G* grad = static_cast<const G*>(t.grad);
  const size_t base = (size_t)t.start * MOE_ADAMW_BLOCK;
  const float lr = h.lr_at != nullptr ? __ldg(h.lr_at) : h.lr;
  float inv1 = h.inv1, root = h.root;
  if (h.step != nullptr) {
    const float s = (float)__ldg(h.step);
    inv1 = 1.f / -expm1f(s * h.log_b1);
    root = rsqrtf(-expm1f(s * h.log_b2));
  }
  const float rate = lr * inv1;
  const float gs = h.grad_scale != nullptr ? __ldg(h.grad_scale) : 1.f;
  const float keep = 1.f - lr * t.decay;
  bool bad = false;
#pragma unroll
  for (int u = 0; u < kPerThread; ++u) {
    const long long at = (long long)(blockIdx.x - table.first[lo]) * kChunk +
                         (u * kThreads + threadIdx.x) * 8;
    const long long left = t.n - at;
    if (k8 ? at - (threadIdx.x & 31) * 8 >= t.n : left <= 0) continue;   // k8: whole warps
    float p[8], g[8], m[8], v[8];
    float ms = 0.f, vs = 0.f;
    const size_t i = base + at, q = i / MOE_ADAMW_BLOCK;
    read8(grad + at, left, g);
    if constexpr (kMaster) read8(st.master + i, left, p);
    else read8(param + at, left, p);
    if constexpr (k8) {
      // the state arrays hold whole blocks
      load8(static_cast<const __nv_fp8_e4m3*>(st.m) + i, m);
      load8(static_cast<const __nv_fp8_e4m3*>(st.v) + i, v);
      ms = st.m_scale[q];
      vs = st.v_scale[q];
    } else {
      read8(static_cast<const float*>(st.m) + i, left, m);
      read8(static_cast<const float*>(st.v) + i, left, v);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (k8) {
        m[j] *= ms;
        v[j] *= vs;
        v[j] *= v[j];
      }
      const float x = g[j] * gs;
      const float nm = fmaf(h.b1, m[j], h.omb1 * x), nv = fmaf(h.b2, v[j], h.omb2 * x * x);
      const bool fine = fabsf(nm) < INFINITY && nv < INFINITY;
      const float r = sqrt_approx(nv);
      const float np = fmaf(p[j], keep, -rate * __fdividef(nm, fmaf(r, root, h.eps)));
      bad |= !fine;
      if (fine) {
        p[j] = np;
        m[j] = nm;
        v[j] = nv;
      }
      if (k8) v[j] = fine ? r : sqrt_approx(v[j]);
    }
    if constexpr (kMaster) write8(st.master + i, left, p);
    write8(param + at, left, p);
    if constexpr (k8) {
      // places past the tensor's end hold zeros and stay so
      ms = to_units(m, block_max(m));
      vs = to_units(v, block_max(v));
      store8(static_cast<__nv_fp8_e4m3*>(st.m) + i, m);
      store8(static_cast<__nv_fp8_e4m3*>(st.v) + i, v);
      if ((threadIdx.x & 31) == 0) {
        st.m_scale[q] = ms;
        st.v_scale[q] = vs;
      }
    } else {
      write8(static_cast<float*>(st.m) + i, left, m);
      write8(static_cast<float*>(st.v) + i, left, v);
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
