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
#include "ptx.cuh"

namespace moe {
namespace {

using bf16 = __nv_bfloat16;

// Eight values as they lie in memory: one 16-byte access of bf16, two of fp32.
template <typename T>
struct Eight;
template <>
struct Eight<bf16> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ void load_shared(const bf16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(bf16* p) const { *reinterpret_cast<uint4*>(p) = v; }
  __device__ __forceinline__ float2 pair(int i) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = pair(i);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reinterpret_cast<__nv_bfloat162&>(w[i]) = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void zero() { v = make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct Eight<float> {
  float4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = __ldg(reinterpret_cast<const float4*>(p));
    v[1] = __ldg(reinterpret_cast<const float4*>(p) + 1);
  }
  __device__ __forceinline__ void load_shared(const float* p) {
    v[0] = reinterpret_cast<const float4*>(p)[0];
    v[1] = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = v[0];
    reinterpret_cast<float4*>(p)[1] = v[1];
  }
  __device__ __forceinline__ float2 pair(int i) const {
    return i & 1 ? make_float2(v[i / 2].z, v[i / 2].w) : make_float2(v[i / 2].x, v[i / 2].y);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = v[0].x; f[1] = v[0].y; f[2] = v[0].z; f[3] = v[0].w;
    f[4] = v[1].x; f[5] = v[1].y; f[6] = v[1].z; f[7] = v[1].w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    v[0] = make_float4(f[0], f[1], f[2], f[3]);
    v[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
  __device__ __forceinline__ void zero() { v[0] = v[1] = make_float4(0.f, 0.f, 0.f, 0.f); }
};
__device__ __forceinline__ float to_f32(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(float v) { return v; }
template <typename T>
__device__ __forceinline__ T from_f32(float v) {
  if constexpr (sizeof(T) == 2) return __float2bfloat16_rn(v);
  else return v;
}
template <typename T>
__device__ __forceinline__ float round_to(float v) { return to_f32(from_f32<T>(v)); }

// A thread's group i of eight values of a row of H, for a team of `team` threads of which
// this is number `me`.  Groups start on 16-byte boundaries: where rows do not (kVec false:
// H no multiple of 8), the row's first `cut` values back to the boundary before it are
// missing from group 0, and its last group ends early.  Only those two take values one by
// one.  Places outside the row are 0 / not stored.
template <typename T>
__device__ __forceinline__ int cut_of(long long row, int H) {
  return (int)((unsigned long long)row * H % (16 / sizeof(T)));
}
struct Team {
  int me, team, H, cut;
};
template <bool kVec>
__device__ __forceinline__ int column(const Team& t, int i) {
  return (i * t.team + t.me) * 8 - (kVec ? 0 : t.cut);
}
template <bool kVec>
__device__ __forceinline__ bool whole(const Team& t, int c) {
  return kVec ? c < t.H : c >= 0 && c + 8 <= t.H;
}
template <bool kShared = false, bool kVec, typename T>
__device__ __forceinline__ void get(Eight<T>& e, const T* row, int i, const Team& t) {
  const int c = column<kVec>(t, i);
  if (whole<kVec>(t, c)) {
    if constexpr (kShared) e.load_shared(row + c);
    else e.load(row + c);
  } else {
    e.zero();
    if constexpr (!kVec) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = c + j >= 0 && c + j < t.H ? to_f32(row[c + j]) : 0.f;
      e.set(f);
    }
  }
}
template <bool kVec, typename T>
__device__ __forceinline__ void put(T* row, int i, const Team& t, const Eight<T>& e) {
  const int c = column<kVec>(t, i);
  if (whole<kVec>(t, c)) {
    e.store(row + c);
  } else if constexpr (!kVec) {
    float f[8];
    e.get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j >= 0 && c + j < t.H) row[c + j] = from_f32<T>(f[j]);
  }
}
// The columns' own values, whose place in memory has nothing to do with the rows'.
template <bool kVec, typename W>
__device__ __forceinline__ void get_column(Eight<W>& e, const W* w, int i, const Team& t) {
  if constexpr (kVec) {
    get<false, kVec>(e, w, i, t);
  } else {
    const int c = column<kVec>(t, i);
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = c + j >= 0 && c + j < t.H ? to_f32(w[c + j]) : 0.f;
    e.set(f);
  }
}
template <bool kVec>
__device__ __forceinline__ void put_column(float* w, int i, const Team& t, const float (&f)[8]) {
  const int c = column<kVec>(t, i);
  if constexpr (kVec) {
    Eight<float> e;
    e.set(f);
    put<kVec>(w, i, t, e);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c + j >= 0 && c + j < t.H) w[c + j] = f[j];
  }
}
template <bool kVec>
__device__ __forceinline__ bool inside(int i, int j, const Team& t) {
  const int c = column<kVec>(t, i) + (kVec ? 0 : j);
  return c >= 0 && c < t.H;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
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
norm_kernel(const T* __restrict__ x, const T* __restrict__ residual, const W* __restrict__ weight,
            const W* __restrict__ bias, float eps, int rows, int H, T* __restrict__ y,
            T* __restrict__ h, float2* __restrict__ stats) {
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
    for (int j = 0; j < 8; ++j) {
      sum += a[j];
      mine += kBlock && inside<kVec>(i, j, t);
    }
  }
  const int count = kBlock ? __reduce_add_sync(0xffffffffu, mine) : H;
  const float u = count > 0 ? lanes_sum<kLanes>(sum) / count : 0.f;
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i < n; ++i) {
    float a[8];
    v[i].get(a);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float d = inside<kVec>(i, j, t) ? a[j] - u : 0.f;
      s.x += d;
      s.y = fmaf(d, d, s.y);
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

// Sums of two values over a block: the warps' halves each reduce one of them.  `part`: 32
// pairs, free to be rewritten once all threads have passed another barrier.
__device__ __forceinline__ float2 warp_sum2(float2 v) {
  const int lane = threadIdx.x & 31;
  const float give = lane < 16 ? v.y : v.x, keep = lane < 16 ? v.x : v.y;
  float s = keep + __shfl_xor_sync(0xffffffffu, give, 16);
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  return make_float2(__shfl_sync(0xffffffffu, s, 0), __shfl_sync(0xffffffffu, s, 16));
}
template <int kTeam>
__device__ __forceinline__ float2 block_sum2(float2 v, float2* part) {
  v = warp_sum2(v);
  if constexpr (kTeam == 32) {
    __syncwarp();
    return v;
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  if (lane == 0) part[warp] = v;
  __syncthreads();
  return warp_sum2(lane < warps ? part[lane] : make_float2(0.f, 0.f));
}

// The backward: a row per block, which takes every gridDim.x-th row and keeps its threads'
// columns of dw and db in registers, then writes them as its share to part [gridDim.x][2][H].
// gridDim.x is a multiple of 8 or each block has one row, so that all of a block's rows
// begin at the same place between 16-byte boundaries.  Works on pairs, with d = h - mean:
//   dw += (dy rstd) d,  db += dy,  u = w dy,  a = sum u,  c = sum u d
//   dx = dh - rstd a / H + rstd u - (rstd^3 c / H) d
// The thread's part of a row, from `get_row(tensor, i, group)`, and dx.
template <typename T, typename W, int n, bool kVec, int kTeam>
struct Backward {
  Team t;
  Eight<W> w[n];
  float2 dw[n][4], db[n][4];
  float2 u[n][4], d[n][4];
  Eight<T> r[n];
  __device__ __forceinline__ void begin(const W* weight) {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      get_column<kVec>(w[i], weight, i, t);
#pragma unroll
      for (int j = 0; j < 4; ++j) dw[i][j] = db[i][j] = make_float2(0.f, 0.f);
    }
  }
  template <bool kShared>
  __device__ __forceinline__ float2 take(const T* dy, const T* h, const T* dh, float2 st) {
    float2 sa = make_float2(0.f, 0.f), sc = sa;
    // places past the row hold dy = 0, which is a factor of all that is summed
#pragma unroll
    for (int i = 0; i < n; ++i) {
      Eight<T> g, x;
      get<kShared, kVec>(g, dy, i, t);
      get<kShared, kVec>(x, h, i, t);
      if (dh != nullptr) get<kShared, kVec>(r[i], dh, i, t);
      else r[i].zero();
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 y = g.pair(j);
        d[i][j] = __fadd2_rn(x.pair(j), make_float2(-st.x, -st.x));
        db[i][j] = __fadd2_rn(db[i][j], y);
        dw[i][j] = __ffma2_rn(__fmul2_rn(y, make_float2(st.y, st.y)), d[i][j], dw[i][j]);
        u[i][j] = __fmul2_rn(y, w[i].pair(j));
        sa = __fadd2_rn(sa, u[i][j]);
        sc = __ffma2_rn(u[i][j], d[i][j], sc);
      }
    }
    return make_float2(sa.x + sa.y, sc.x + sc.y);
  }
  __device__ __forceinline__ void give(T* dx, float2 s, float2 st) const {
    const float a = -st.y * (s.x / t.H), c = -st.y * st.y * st.y * (s.y / t.H);
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 x = __ffma2_rn(u[i][j], make_float2(st.y, st.y), make_float2(a, a));
        x = __ffma2_rn(d[i][j], make_float2(c, c), x);
        x = __fadd2_rn(x, r[i].pair(j));
        v[2 * j] = x.x;
        v[2 * j + 1] = x.y;
      }
      Eight<T> e;
      e.set(v);
      put<kVec>(dx, i, t, e);
    }
  }
  __device__ __forceinline__ void end(float* mine) const {
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = dw[i][j].x;
        v[2 * j + 1] = dw[i][j].y;
      }
      put_column<kVec>(mine, i, t, v);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = db[i][j].x;
        v[2 * j + 1] = db[i][j].y;
      }
      put_column<kVec>(mine + t.H, i, t, v);
    }
  }
};

// Rows too wide for a ring of two: read where they lie.
template <typename T, typename W, int n, bool kVec, int kTeam>
__global__ void __launch_bounds__(kTeam, 1)
norm_backward_kernel(const T* __restrict__ dy, const T* __restrict__ h,
                     const float2* __restrict__ stats, const W* __restrict__ weight,
                     const T* __restrict__ dh, int rows, int H, T* __restrict__ dx,
                     float* __restrict__ part, int* __restrict__ flags) {
  pdl_trigger();
  __shared__ float2 sums[2][32];
  Backward<T, W, n, kVec, kTeam> b;
  b.t = Team{(int)threadIdx.x, (int)blockDim.x, H, kVec ? 0 : cut_of<T>(blockIdx.x, H)};
  b.begin(weight);
  int turn = 0;
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const size_t at = (size_t)row * H;
    const float2 st = __ldg(stats + row);
    float2 s = b.template take<false>(dy + at, h + at, dh != nullptr ? dh + at : nullptr, st);
    s = block_sum2<kTeam>(s, sums[turn]);   // the other half is read no more: one barrier ago
    turn ^= 1;
    b.give(dx + at, s, st);
  }
  if (threadIdx.x == 0) flags[blockIdx.x] = 0;
  b.end(part + (size_t)blockIdx.x * 2 * H);
}

// A row of each of up to three tensors, on its way into or in a block's shared memory.  Rows
// come by bulk copies of whole 16-byte pieces: where rows do not start on one, a copy takes
// the pieces that its row touches, and the last few values of a tensor that does not end on
// one are copied one by one.
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr int kMaxStages = 8;
template <typename T>
struct RowRing {
  char* buf;        // [stages][3][pitch]
  uint64_t* full;   // [stages]
  int H, stages, pitch, tensors;
  long long rows;

  static __host__ __device__ int pitch_of(int H) { return (H * (int)sizeof(T) + 31) / 16 * 16; }
  __device__ __forceinline__ T* at(int stage, int tensor) const {
    return reinterpret_cast<T*>(buf + (size_t)(stage * tensors + tensor) * pitch);
  }
  // One thread's work.  cut: values from the 16-byte boundary before a row to its start.
  __device__ __forceinline__ void fetch(int stage, long long row, int cut,
                                        const T* const (&from)[3]) const {
    const size_t first = (size_t)row * H - cut;   // in values, as all that follows
    constexpr int kPiece = 16 / sizeof(T);
    int count = (cut + H + kPiece - 1) / kPiece * kPiece;
    const size_t all = (size_t)rows * H;
    if (first + count > all) {   // the last row, where the tensor ends within a piece
      count -= kPiece;
      for (int i = 0; i < tensors; ++i)
        for (size_t p = max(first + count, (size_t)row * H); p < all; ++p)
          at(stage, i)[p - first] = from[i][p];
    }
    const uint32_t bytes = count * sizeof(T);
    ptx::mbar_arrive_expect_tx(&full[stage], bytes * tensors);
    if (bytes > 0)
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (i < tensors) ptx::bulk_load(at(stage, i), from[i] + first, bytes, &full[stage]);
  }
  // A row's values in shared memory: a pointer to its first.
  __device__ __forceinline__ const T* row(int stage, int tensor, int cut) const {
    return at(stage, tensor) + cut;
  }
};
// Rows fetched ahead by bulk copies.  flags [gridDim.x]: whether a copy did not come.
template <typename T, typename W, int n, bool kVec, int kTeam, int kPer>
__global__ void __launch_bounds__(kTeam, kPer)
norm_backward_ring_kernel(const T* __restrict__ dy, const T* __restrict__ h,
                          const float2* __restrict__ stats, const W* __restrict__ weight,
                          const T* __restrict__ dh, int rows, int H, int stages,
                          T* __restrict__ dx, float* __restrict__ part, int* __restrict__ flags) {
  pdl_trigger();   // the next kernel waits for this one's end all the same
  extern __shared__ __align__(16) char smem[];
  __shared__ uint64_t full[kMaxStages];
  __shared__ float2 sums[2][32];
  __shared__ int dead[2];
  const int me = threadIdx.x;
  const RowRing<T> ring{smem, full, H, stages, RowRing<T>::pitch_of(H), dh != nullptr ? 3 : 2, rows};
  const T* const from[3] = {dy, h, dh};
  if (me == 0) {
    dead[0] = dead[1] = 0;
    for (int s = 0; s < stages; ++s) ptx::mbar_init(&full[s], 1);
    ptx::fence_mbar_init();
  }
  __syncthreads();
  long long ahead = blockIdx.x;   // the next row to be fetched
  const int cut = kVec ? 0 : cut_of<T>(blockIdx.x, H);   // of all of the block's rows
  if (me == 0)
    for (int s = 0; s < stages && ahead < rows; ++s, ahead += gridDim.x)
      ring.fetch(s, ahead, cut, from);
  Backward<T, W, n, kVec, kTeam> b;
  b.t = Team{me, (int)blockDim.x, H, cut};
  b.begin(weight);
  float2 next = __ldg(stats + blockIdx.x);
  int turn = 0, stage = 0;
  uint32_t phase = 0;
  for (long long row = blockIdx.x; row < rows; row += gridDim.x) {
    const float2 st = next;
    if (row + gridDim.x < rows) next = __ldg(stats + row + gridDim.x);
    if (!ptx::mbar_wait(&full[stage], phase, nullptr, kWaitLimitNs)) dead[turn] = 1;
    float2 s = b.template take<true>(ring.row(stage, 0, cut), ring.row(stage, 1, cut),
                                     dh != nullptr ? ring.row(stage, 2, cut) : nullptr, st);
    s = block_sum2<kTeam>(s, sums[turn]);   // the other half is read no more: one barrier ago
    if (dead[turn]) break;
    turn ^= 1;
    // all threads have taken their values of this row
    if (me == 0 && ahead < rows) {
      ring.fetch(stage, ahead, cut, from);
      ahead += gridDim.x;
    }
    b.give(dx + (size_t)row * H, s, st);
    if (++stage == stages) {
      stage = 0;
      phase ^= 1u;
    }
  }
  if (me == 0) {
    const bool late = dead[0] | dead[1];
    flags[blockIdx.x] = late;
    // what is still on its way has to arrive before the block's memory is another's
    if (late)
      for (int s = 0; s < stages; ++s) ptx::mbar_wait(&full[s], phase ^ (s < stage), nullptr, kWaitLimitNs);
  }
  b.end(part + (size_t)blockIdx.x * 2 * H);
}

// dw, db = the sums of the blocks' shares, in block order within each of 32 warps; the
// status from the blocks' flags.
template <typename W>
__global__ void __launch_bounds__(1024)
norm_weight_kernel(const float* __restrict__ part, int blocks, int H, W* __restrict__ dw,
                   W* __restrict__ db, const int* __restrict__ flags, int* __restrict__ status) {
  __shared__ float sums[32][33];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + lane;
  W* out = blockIdx.y == 0 ? dw : db;
  const float* from = part + (size_t)blockIdx.y * H + e;
  float v = 0.f;
  if (e < H) {
#pragma unroll 8
    for (int b = warp; b < blocks; b += 32) v += from[(size_t)b * 2 * H];
  }
  sums[warp][lane] = v;
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    int bad = 0;
    for (int b = threadIdx.x; b < blocks; b += 1024) bad |= flags[b];
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
      status[0] = bad ? MOE_ERR_TIMEOUT : 0;
      status[1] = 0;
    }
  } else {
    __syncthreads();
  }
  v = warp_sum(sums[lane][warp]);   // warp w: column w, lane l: warp l's sum
  const int c = blockIdx.x * 32 + warp;
  if (lane == 0 && c < H) out[c] = from_f32<W>(v);
}

// Shared memory of a ring where `per` blocks share an SM.
constexpr int ring_bytes(int per) { return 227 * 1024 / per - 2048; }
constexpr int kFewRows = kSms;
// Groups of eight that a row takes; one that may begin within a group, up to one more.
int groups_of(int H) { return (H + 7 + (H % 8 != 0 ? 7 : 0)) / 8; }
int team_of(int H, int n) {   // threads that hold a row with n groups each
  const int t = (groups_of(H) + n - 1) / n;
  return (t + 31) / 32 * 32;
}

template <typename T, typename W, bool kVec, bool kResidual>
cudaError_t forward_r(const T* x, const T* residual, const W* weight, const W* bias, float eps,
                      int rows, int H, T* y, T* h, float2* stats, cudaStream_t s) {
#define MOE_NORM_WARP(n, L)                                                                       \
  norm_kernel<T, W, n, kVec, kResidual, L, 128, 6><<<(rows - 1) / (128 / L) + 1, 128, 0, s>>>(    \
      x, residual, weight, bias, eps, rows, H, y, h, stats)
#define MOE_NORM_BLOCK(n, team, per)                                                              \
  norm_kernel<T, W, n, kVec, kResidual, 0, team, per><<<rows, team_of(H, n), 0, s>>>(             \
      x, residual, weight, bias, eps, rows, H, y, h, stats)
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

// A backward's launch shape, by the groups of eight that a row takes: few threads with
// many groups each keep a row's loads and sums in flight at once.
struct Shape {
  int n, per;   // groups per thread, blocks per SM
};
constexpr Shape kShapes[] = {{1, 16}, {2, 12}, {2, 6}, {4, 4}, {4, 2}, {4, 1}, {8, 1}};
int shape_of(int H) {
  const int groups = groups_of(H);
  return groups <= 32 ? 0 : groups <= 64 ? 1 : groups <= 128 ? 2 : groups <= 256 ? 3
         : groups <= 512 ? 4 : groups <= 1024 ? 5 : 6;
}

template <typename T, typename W, bool kVec>
cudaError_t backward_t(const void* dy, const void* h, const float* stats, const void* weight,
                       const void* dh, int rows, int H, void* dx, void* dw, void* db, int blocks,
                       float* part, int* flags, int* status, cudaStream_t s) {
  const T* gt = static_cast<const T*>(dy);
  const T* ht = static_cast<const T*>(h);
  const T* rt = static_cast<const T*>(dh);
  const W* wt = static_cast<const W*>(weight);
  const float2* st = reinterpret_cast<const float2*>(stats);
  T* xt = static_cast<T*>(dx);
  const int stage = RowRing<T>::pitch_of(H) * (rt != nullptr ? 3 : 2);
  constexpr int kWide = kVec ? 256 : 288;   // a row that begins within a group takes one more
#define MOE_NORM_RING(i, team)                                                                    \
  do {                                                                                            \
    constexpr Shape f = kShapes[i];                                                               \
    const auto kern = norm_backward_ring_kernel<T, W, f.n, kVec, team, f.per>;                    \
    int stages = ring_bytes(f.per) / stage;                                                       \
    stages = stages < kMaxStages ? stages : kMaxStages;                                           \
    const cudaError_t e = allow_smem(kern, stages * stage);                                       \
    if (e != cudaSuccess) return e;                                                               \
    kern<<<blocks, team_of(H, f.n), stages * stage, s>>>(gt, ht, st, wt, rt, rows, H, stages, xt, part, \
                                                         flags);                                  \
  } while (0)
  if (rows > 0) {
    switch (shape_of(H)) {
      case 0: MOE_NORM_RING(0, 32); break;
      case 1: MOE_NORM_RING(1, 32); break;
      case 2: MOE_NORM_RING(2, 64); break;
      case 3: MOE_NORM_RING(3, 64); break;
      case 4: MOE_NORM_RING(4, 128); break;
      case 5: MOE_NORM_RING(5, 256); break;
      default:
        // a ring holds two rows at least: fp32 rows of more than 9,500 or 14,000 values do not fit
        if (2 * stage <= ring_bytes(kShapes[6].per)) {
          MOE_NORM_RING(6, kWide);
        } else {
          norm_backward_kernel<T, W, kShapes[6].n, kVec, kWide>
              <<<blocks, team_of(H, kShapes[6].n), 0, s>>>(gt, ht, st, wt, rt, rows, H, xt, part, flags);
        }
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
#undef MOE_NORM_RING
  return launch_k(norm_weight_kernel<W>, dim3((H + 31) / 32, db != nullptr ? 2 : 1), dim3(1024), 0, s,
                  true, static_cast<const float*>(part), rows > 0 ? blocks : 0, H,
                  static_cast<W*>(dw), static_cast<W*>(db), static_cast<const int*>(flags), status);
}

}  // namespace

// Blocks of the backward: as many as the SMs take at once, fewer where that leaves a block
// less than four rows, for every block has a share of dw and db to write.  A multiple of
// 8, or one for each row.
int norm_backward_blocks(int rows, int H) {
  const long long most = (long long)kSms * kShapes[shape_of(H)].per;
  long long want = ((long long)rows + 31) / 32 * 8;
  want = want < kSms ? kSms : want;
  want = want < most ? want : most;
  return (int)(rows < want ? rows : want);
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
                                 int weight_type, void* dx, void* dw, void* db, void* ws,
                                 cudaStream_t s) {
  const int blocks = norm_backward_blocks(rows, H);
  int* status = static_cast<int*>(ws);
  int* flags = status + 64;
  float* part = ws_ptr<float>(ws, kNormHeader);
  MOE_NORM_TYPES(backward_t, dy, h, stats, weight, dh, rows, H, dx, dw, db, blocks, part, flags,
                 status, s);
}

}  // namespace moe
