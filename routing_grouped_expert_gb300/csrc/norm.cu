// Layer norm of a residual sum, and its backward.
//
//   h = x + residual (rounded to the tensors' type and stored; h = x without one)
//   mean = sum h / H,  rstd = 1 / sqrt(sum (h - mean)^2 / H + eps)
//   y = (h - mean) rstd w + b
//
//   xhat = (h - mean) rstd,  a = sum(w dy) / H,  c = sum(w dy xhat) / H
//   dx = rstd (w dy - a - xhat c) + dh     (dh: the gradient that reaches h past the norm)
//   dw = sum_t dy xhat,  db = sum_t dy
//
// A row is held in registers between its statistics and its output, so memory is
// read once; the variance is taken around the mean (a second pass over the
// registers), not as a difference of two large sums.  Sums are fp32 in a fixed order.
#include <math.h>

#include "moe_common.cuh"

namespace moe {
namespace {

using bf16 = __nv_bfloat16;

// Eight consecutive values: one 16-byte access of bf16, two of fp32.
__device__ __forceinline__ void load8(const bf16* p, float (&f)[8]) {
  const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
  const __nv_bfloat162* q = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __bfloat1622float2(q[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
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
__device__ __forceinline__ float to_f32(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
  else return v;
}
template <typename T>
__device__ __forceinline__ float round_to(float v) { return to_f32(from_f32<T>(v)); }

// Group i of eight of this thread's values of a row of H, for a team of `team` threads
// of which this is number `me`.  kVec: eight consecutive ones (H a multiple of 8);
// otherwise every team-th one.  Places outside the row are 0 / not stored.
template <bool kVec, typename T>
__device__ __forceinline__ void get8(const T* row, int i, int me, int team, int H, float (&f)[8]) {
  if constexpr (kVec) {
    const int at = (i * team + me) * 8;
    if (at < H) {
      load8(row + at, f);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = 0.f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = (i * 8 + j) * team + me;
      f[j] = at < H ? to_f32(row[at]) : 0.f;
    }
  }
}
template <bool kVec, typename T>
__device__ __forceinline__ void put8(T* row, int i, int me, int team, int H, const float (&f)[8]) {
  if constexpr (kVec) {
    const int at = (i * team + me) * 8;
    if (at < H) store8(row + at, f);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int at = (i * 8 + j) * team + me;
      if (at < H) row[at] = from_f32<T>(f[j]);
    }
  }
}
template <bool kVec>
__device__ __forceinline__ bool inside(int i, int j, int me, int team, int H) {
  return kVec ? (i * team + me) * 8 < H : (i * 8 + j) * team + me < H;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
// Sums over a block of n values at once; `part` is n * 32 floats, free to be
// rewritten once all threads have passed another barrier.
template <int n>
__device__ __forceinline__ void block_sum(float (&v)[n], float* part) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int i = 0; i < n; ++i) {
    v[i] = warp_sum(v[i]);
    if (lane == 0) part[32 * i + warp] = v[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < n; ++i) v[i] = warp_sum(lane < warps ? part[32 * i + lane] : 0.f);
}

// kWarp: a row per warp; otherwise a row per block.  n: groups of eight per thread.
template <typename T, typename W, int n, bool kVec, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 128 : 1024)
norm_kernel(const T* __restrict__ x, const T* __restrict__ residual, const W* __restrict__ weight,
            const W* __restrict__ bias, float eps, int rows, int H, T* __restrict__ y,
            T* __restrict__ h, float2* __restrict__ stats) {
  __shared__ float part[2][32];
  const int team = kWarp ? 32 : blockDim.x;
  const int me = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int row = kWarp ? blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5) : blockIdx.x;
  if (kWarp && row >= rows) return;
  const size_t at = (size_t)row * H;
  float v[n][8];
  float sum[1] = {0.f};
#pragma unroll
  for (int i = 0; i < n; ++i) get8<kVec>(x + at, i, me, team, H, v[i]);
  if (residual != nullptr) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float r[8];
      get8<kVec>(residual + at, i, me, team, H, r);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[i][j] = round_to<T>(v[i][j] + r[j]);
      put8<kVec>(h + at, i, me, team, H, v[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < n; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[0] += v[i][j];
  if constexpr (kWarp) sum[0] = warp_sum(sum[0]);
  else block_sum<1>(sum, part[0]);
  const float mean = sum[0] / H;
  float sq[1] = {0.f};
#pragma unroll
  for (int i = 0; i < n; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] -= mean;
      if (inside<kVec>(i, j, me, team, H)) sq[0] = fmaf(v[i][j], v[i][j], sq[0]);
    }
  if constexpr (kWarp) sq[0] = warp_sum(sq[0]);
  else block_sum<1>(sq, part[1]);
  const float rstd = rsqrtf(sq[0] / H + eps);
  if (me == 0 && stats != nullptr) stats[row] = make_float2(mean, rstd);
#pragma unroll
  for (int i = 0; i < n; ++i) {
    float w[8], b[8];
    get8<kVec>(weight, i, me, team, H, w);
    if (bias != nullptr) {
      get8<kVec>(bias, i, me, team, H, b);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = 0.f;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) v[i][j] = fmaf(v[i][j] * rstd, w[j], b[j]);
    put8<kVec>(y + at, i, me, team, H, v[i]);
  }
}

// dx, and this block's share of dw and db in part [gridDim.x][2][H].  A block takes
// every gridDim.x-th row (a warp every so-many-th with kWarp) and keeps its threads'
// columns of dw and db in registers.
template <typename T, typename W, int n, bool kVec, bool kWarp>
__global__ void __launch_bounds__(kWarp ? 128 : n == 1 ? 1024 : 512)
norm_backward_kernel(const T* __restrict__ dy, const T* __restrict__ h,
                     const float2* __restrict__ stats, const W* __restrict__ weight,
                     const T* __restrict__ dh, int rows, int H, T* __restrict__ dx,
                     float* __restrict__ part) {
  extern __shared__ float sums[];   // kWarp: [warps][2][H]; else [2][64]
  const int team = kWarp ? 32 : blockDim.x;
  const int me = kWarp ? threadIdx.x & 31 : threadIdx.x;
  const int warp = threadIdx.x >> 5;
  const int per = kWarp ? blockDim.x >> 5 : 1;
  float dw[n][8], db[n][8];
#pragma unroll
  for (int i = 0; i < n; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = db[i][j] = 0.f;
  int turn = 0;
  for (long long row = (long long)blockIdx.x * per + (kWarp ? warp : 0); row < rows;
       row += (long long)gridDim.x * per) {
    const size_t at = (size_t)row * H;
    const float2 st = __ldg(stats + row);
    float g[n][8], z[n][8];
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < n; ++i) {
      get8<kVec>(dy + at, i, me, team, H, g[i]);
      get8<kVec>(h + at, i, me, team, H, z[i]);
    }
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float w[8];
      get8<kVec>(weight, i, me, team, H, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        z[i][j] = (z[i][j] - st.x) * st.y;
        if (!inside<kVec>(i, j, me, team, H)) z[i][j] = 0.f;
        dw[i][j] = fmaf(g[i][j], z[i][j], dw[i][j]);
        db[i][j] += g[i][j];
        g[i][j] *= w[j];
        s[0] += g[i][j];
        s[1] = fmaf(g[i][j], z[i][j], s[1]);
      }
    }
    if constexpr (kWarp) {
      s[0] = warp_sum(s[0]);
      s[1] = warp_sum(s[1]);
    } else {
      block_sum<2>(s, sums + 64 * turn);   // the other half is read no more: one barrier ago
      turn ^= 1;
    }
    const float a = s[0] / H, c = s[1] / H;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float r[8];
      if (dh != nullptr) {
        get8<kVec>(dh + at, i, me, team, H, r);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) r[j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) r[j] = fmaf(st.y, g[i][j] - a - z[i][j] * c, r[j]);
      put8<kVec>(dx + at, i, me, team, H, r);
    }
  }
  float* mine = part + (size_t)blockIdx.x * 2 * H;
  if constexpr (kWarp) {
    float* to = sums + (size_t)warp * 2 * H;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      put8<kVec>(to, i, me, team, H, dw[i]);
      put8<kVec>(to + H, i, me, team, H, db[i]);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * H; e += blockDim.x) {
      float v = 0.f;
      for (int u = 0; u < per; ++u) v += sums[(size_t)u * 2 * H + e];
      mine[e] = v;
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      put8<kVec>(mine, i, me, team, H, dw[i]);
      put8<kVec>(mine + H, i, me, team, H, db[i]);
    }
  }
}

// dw, db = the sums of the blocks' shares, in block order within each of eight warps.
template <typename W>
__global__ void __launch_bounds__(256)
norm_weight_kernel(const float* __restrict__ part, int blocks, int H, W* __restrict__ dw,
                   W* __restrict__ db) {
  __shared__ float sums[8][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  W* out = blockIdx.y == 0 ? dw : db;
  const float* from = part + (size_t)blockIdx.y * H + e;
  float v = 0.f;
  if (e < H)
    for (int b = warp; b < blocks; b += 8) v += from[(size_t)b * 2 * H];
  sums[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && e < H) {
#pragma unroll
    for (int u = 1; u < 8; ++u) v += sums[u][lane];
    out[e] = from_f32<W>(v);
  }
}

int team_of(int H, int n) {   // threads that hold a row with n groups of eight each
  const int t = (H + 8 * n - 1) / (8 * n);
  return (t + 31) / 32 * 32;
}

template <typename T, typename W, bool kVec>
cudaError_t forward_t(const void* x, const void* residual, const void* weight, const void* bias,
                      float eps, int rows, int H, void* y, void* h, float* stats, cudaStream_t s) {
  const T* xt = static_cast<const T*>(x);
  const T* rt = static_cast<const T*>(residual);
  const W* wt = static_cast<const W*>(weight);
  const W* bt = static_cast<const W*>(bias);
  T* yt = static_cast<T*>(y);
  T* ht = static_cast<T*>(h);
  float2* st = reinterpret_cast<float2*>(stats);
#define MOE_NORM_WARP(n)                                                       \
  norm_kernel<T, W, n, kVec, true><<<(rows - 1) / 4 + 1, 128, 0, s>>>(xt, rt, wt, bt, eps, rows, H, \
                                                                yt, ht, st)
#define MOE_NORM_BLOCK(n)                                                      \
  norm_kernel<T, W, n, kVec, false><<<rows, team_of(H, n), 0, s>>>(xt, rt, wt, bt, eps, rows, H, \
                                                                   yt, ht, st)
  if (H <= 256) MOE_NORM_WARP(1);
  else if (H <= 512) MOE_NORM_WARP(2);
  else if (H <= 1024) MOE_NORM_WARP(4);
  else if (H <= 8192) MOE_NORM_BLOCK(1);
  else MOE_NORM_BLOCK(2);
#undef MOE_NORM_WARP
#undef MOE_NORM_BLOCK
  return cudaGetLastError();
}

template <typename T, typename W, bool kVec>
cudaError_t backward_t(const void* dy, const void* h, const float* stats, const void* weight,
                       const void* dh, int rows, int H, void* dx, void* dw, void* db, int blocks,
                       float* part, cudaStream_t s) {
  const T* gt = static_cast<const T*>(dy);
  const T* ht = static_cast<const T*>(h);
  const T* rt = static_cast<const T*>(dh);
  const W* wt = static_cast<const W*>(weight);
  const float2* st = reinterpret_cast<const float2*>(stats);
  T* xt = static_cast<T*>(dx);
#define MOE_NORM_WARP(n)                                                                           \
  norm_backward_kernel<T, W, n, kVec, true><<<blocks, 128, (size_t)4 * 2 * H * 4, s>>>(gt, ht, st, \
                                                                  wt, rt, rows, H, xt, part)
#define MOE_NORM_BLOCK(n)                                                                          \
  norm_backward_kernel<T, W, n, kVec, false><<<blocks, team_of(H, n), 128 * 4, s>>>(gt, ht, st, wt, \
                                                                  rt, rows, H, xt, part)
  if (rows > 0) {
    if (H <= 256) MOE_NORM_WARP(1);
    else if (H <= 512) MOE_NORM_WARP(2);
    else if (H <= 1024) MOE_NORM_WARP(4);
    else if (H <= 8192) MOE_NORM_BLOCK(1);
    else MOE_NORM_BLOCK(4);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
#undef MOE_NORM_WARP
#undef MOE_NORM_BLOCK
  norm_weight_kernel<W><<<dim3((H + 31) / 32, db != nullptr ? 2 : 1), 256, 0, s>>>(
      part, rows > 0 ? blocks : 0, H, static_cast<W*>(dw), static_cast<W*>(db));
  return cudaGetLastError();
}

}  // namespace

int norm_backward_blocks(int rows, int H) {
  const int most = kSms * (H <= 1024 ? 4 : 1);
  const long long units = H <= 1024 ? ((long long)rows + 3) / 4 : rows;
  return (int)(units < most ? units : most);
}

#define MOE_NORM_TYPES(f, ...)                                                            \
  do {                                                                                    \
    const bool vec = H % 8 == 0;                                                          \
    if (type == MOE_F32)                                                                  \
      return vec ? f<float, float, true>(__VA_ARGS__) : f<float, float, false>(__VA_ARGS__); \
    if (weight_type == MOE_F32)                                                           \
      return vec ? f<bf16, float, true>(__VA_ARGS__) : f<bf16, float, false>(__VA_ARGS__); \
    return vec ? f<bf16, bf16, true>(__VA_ARGS__) : f<bf16, bf16, false>(__VA_ARGS__);    \
  } while (0)

cudaError_t launch_norm(const void* x, const void* residual, const void* weight, const void* bias,
                        float eps, int rows, int H, int type, int weight_type, void* y, void* h,
                        float* stats, cudaStream_t s) {
  MOE_NORM_TYPES(forward_t, x, residual, weight, bias, eps, rows, H, y, h, stats, s);
}

cudaError_t launch_norm_backward(const void* dy, const void* h, const float* stats,
                                 const void* weight, const void* dh, int rows, int H, int type,
                                 int weight_type, void* dx, void* dw, void* db, float* part,
                                 cudaStream_t s) {
  const int blocks = norm_backward_blocks(rows, H);
  MOE_NORM_TYPES(backward_t, dy, h, stats, weight, dh, rows, H, dx, dw, db, blocks, part, s);
}

}  // namespace moe
