// Layer norm of a residual sum:
//
//   h = x + residual (rounded to the tensors' type and stored; h = x without one)
//   mean = sum h / H,  rstd = 1 / sqrt(sum (h - mean)^2 / H + eps)
//   y = (h - mean) rstd w + b
//
// A row is held in registers between its statistics and its output, so memory is read once;
// the variance is taken around the mean (a second pass over the registers), not as a
// difference of two large sums.  Sums are fp32 in a fixed order.
//
// Bound by memory: 8192 x 7168 bf16 with a residual in 70.8 us (470 MB, 0.98 of the rate of a
// plain copy; DRAM read 235 MB), 12000 x 4096 in 58.8 (0.98), 40001 x 512 in 26.2 (0.92),
// without a residual 46 (0.75: half the bytes in flight).  fp32: 8192 x 4096 81.7 us (0.97),
// 4096 x 7168 76.0 (0.91), without a residual 44.5 (0.78), 2000 x 16384 107 (0.72: its groups do
// not fit the registers).  Rows of 7170 102 us (0.68): their weights are cut out of the pieces
// around them, and a row's ends taken one by one.
#include "norm.cuh"

namespace moe {
namespace {

// A row's mean and sum of squares around it, from its warps', so that one barrier is
// enough.  A warp of c values takes the sums r of d and q of d^2 of the distances d to its
// own mean u, as rounded (r is what the rounding left):
//   mean = sum (c u + r) / H,  squares = sum q + 2 (u - mean) r + c (u - mean)^2
struct Moments {
  float4 of[32];
};
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int off = L / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
__device__ __forceinline__ float2 join_moments(int H, float count, float u, float2 s, Moments& sh) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) sh.of[warp] = make_float4(count, u, s.x, s.y);
  __syncthreads();
  const float4 m = lane < warps ? sh.of[lane] : make_float4(0.f, 0.f, 0.f, 0.f);
  const float mean = warp_sum(fmaf(m.x, m.y, m.z)) / H;
  const float d = m.y - mean;
  return make_float2(mean, warp_sum(fmaf(d, fmaf(m.x, d, 2.f * m.z), m.w)));
}

// L = 0: a row per block.  Otherwise a row per L lanes of a warp.  n: groups of eight per
// thread.  A row stays in registers as it lies in memory.
template <typename T, typename W, int n, bool kVec, bool kResidual, int L, int kTeam, int kPer>
__global__ void __launch_bounds__(kTeam, kPer)
norm_kernel(const T* x, const T* residual, const W* __restrict__ weight,
            const W* __restrict__ bias, float eps, int rows, int H, T* y, T* h,
            float2* __restrict__ stats) {
  constexpr bool kBlock = L == 0;
  constexpr int kLanes = kBlock ? 32 : L;
  __shared__ Moments sh;
  Team t{(int)threadIdx.x, (int)blockDim.x, H, 0};
  long long row = blockIdx.x;
  bool there = true;
  if constexpr (!kBlock) {
    t.me &= L - 1;
    t.team = L;
    row = row * (kTeam / L) + threadIdx.x / L;
    // a row that is not there: read and computed as the last one, not stored
    there = row < rows;
    if (!there) row = rows - 1;
  }
  if (!kVec) t.cut = cut_of<T>(row, H);
  const size_t at = (size_t)row * H;
  Eight<T> v[n];
#pragma unroll
  for (int i = 0; i < n; ++i) get<false, kVec>(v[i], x + at, i, t);
  if constexpr (kResidual) {
    Eight<T> r[n];
#pragma unroll
    for (int i = 0; i < n; ++i) get<false, kVec>(r[i], residual + at, i, t);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float a[8], b[8];
      v[i].get(a);
      r[i].get(b);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] += b[j];
      v[i].set(a);
      if (there) put<kVec>(h + at, i, t, v[i]);
    }
  }
  float sum = 0.f;
  int mine = 0;
#pragma unroll
  for (int i = 0; i < n; ++i) {
    float a[8];
    v[i].get(a);
#pragma unroll
    for (int j = 0; j < 8; ++j) sum += a[j];
    if (kBlock) mine += __popc(inside<kVec>(i, t));
  }
  const int count = kBlock ? __reduce_add_sync(0xffffffffu, mine) : H;
  const float u = count > 0 ? lanes_sum<kLanes>(sum) / count : 0.f;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < n; ++i) {
    float a[8];
    v[i].get(a);
    const uint32_t in = inside<kVec>(i, t);
    if (in == 0xffu) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = a[j] - u;
        s.x += d;
        s.y = fmaf(d, d, s.y);
      }
    } else if constexpr (!kVec) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float d = in >> j & 1u ? a[j] - u : 0.f;
        s.x += d;
        s.y = fmaf(d, d, s.y);
      }
    }
  }
  s.x = lanes_sum<kLanes>(s.x);
  s.y = lanes_sum<kLanes>(s.y);
  if constexpr (kBlock) s = join_moments(H, count, u, s, sh);
  else s = make_float2(u + s.x / H, fmaf(-s.x / H, s.x, s.y));
  // rounding may leave a constant row a little below zero
  const float mean = s.x, rstd = rsqrtf((s.y < 0.f ? 0.f : s.y / H) + eps);
  if (t.me == 0 && there && stats != nullptr) stats[row] = make_float2(mean, rstd);
#pragma unroll
  for (int i = 0; i < n; ++i) {
    float a[8], w[8], b[8];
    Eight<W> e;
    get_column<kVec>(e, weight, i, t);
    e.get(w);
    if (bias != nullptr) {
      get_column<kVec>(e, bias, i, t);
      e.get(b);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) b[j] = 0.f;
    }
    v[i].get(a);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] = fmaf((a[j] - mean) * rstd, w[j], b[j]);
    v[i].set(a);
    if (there) put<kVec>(y + at, i, t, v[i]);
  }
}

constexpr int kFewRows = kSms;   // up to here a row has as many threads as it can use: one row 2.6 us
template <typename T, typename W, bool kVec, bool kResidual>
cudaError_t forward_r(const T* x, const T* residual, const W* weight, const W* bias, float eps,
                      int rows, int H, T* y, T* h, float2* stats, cudaStream_t s) {
#define MOE_NORM_WARP(n, L)                                                                       \
  norm_kernel<T, W, n, kVec, kResidual, L, 128, 6><<<(rows - 1) / (128 / L) + 1, 128, 0, s>>>(    \
      x, residual, weight, bias, eps, rows, H, y, h, stats)
#define MOE_NORM_BLOCK(n, team, per)                                                              \
  norm_kernel<T, W, n, kVec, kResidual, 0, team, per><<<rows, team_of(H, n), 0, s>>>(             \
      x, residual, weight, bias, eps, rows, H, y, h, stats)
  // Few threads with several groups each, which are on their way at once, and few rows: all
  // of an SM's threads on one, for the shortest time.  us, threads x groups: 8192 x 7168 with a
  // residual 896 x 1 158, 448 x 2 83, 224 x 4 71; without 224 x 4 47, 128 x 8 49; 20000 x
  // 2048 without 256 x 1 43, 64 x 4 32; 200000 x 128 16 x 1 38, 8 x 2 32.
  const int groups = groups_of(H);
  if (groups <= 16) MOE_NORM_WARP(2, 8);
  else if (groups <= 32) MOE_NORM_WARP(2, 16);
  else if (groups <= 64) MOE_NORM_WARP(2, 32);
  else if (groups <= 128) MOE_NORM_WARP(4, 32);
  else if (groups <= 1024 && rows <= kFewRows) MOE_NORM_BLOCK(1, 1024, 1);
  else if (groups <= 256 && kResidual) MOE_NORM_BLOCK(1, 256, 6);
  else if (groups <= 256) MOE_NORM_BLOCK(4, 64, 16);
  else if (groups <= 512 && kResidual) MOE_NORM_BLOCK(2, 256, 6);
  else if (groups <= 512) MOE_NORM_BLOCK(4, 128, 8);
  else if (groups <= 1024) MOE_NORM_BLOCK(4, 256, kResidual ? 4 : 5);
  else MOE_NORM_BLOCK(5, 512, 2);
#undef MOE_NORM_WARP
#undef MOE_NORM_BLOCK
  return cudaGetLastError();
}
template <typename T, typename W, bool kVec>
cudaError_t forward_t(const void* x, const void* residual, const void* weight, const void* bias,
                      float eps, int rows, int H, void* y, void* h, float* stats, cudaStream_t s) {
  const auto f = residual != nullptr ? forward_r<T, W, kVec, true> : forward_r<T, W, kVec, false>;
  return f(static_cast<const T*>(x), static_cast<const T*>(residual), static_cast<const W*>(weight),
           static_cast<const W*>(bias), eps, rows, H, static_cast<T*>(y), static_cast<T*>(h),
           reinterpret_cast<float2*>(stats), s);
}

}  // namespace

cudaError_t launch_norm(const void* x, const void* residual, const void* weight, const void* bias,
                        float eps, int rows, int H, int type, int weight_type, void* y, void* h,
                        float* stats, cudaStream_t s) {
  MOE_NORM_TYPES(forward_t, x, residual, weight, bias, eps, rows, H, y, h, stats, s);
}

}  // namespace moe
