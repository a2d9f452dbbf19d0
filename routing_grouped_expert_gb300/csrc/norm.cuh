// What layer norm's forward (norm.cu) and backward (norm_backward.cu) share: how a row is
// held, and the types that they are made for.
#pragma once

#include "moe_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

using bf16 = __nv_bfloat16;

// Eight values as they lie in memory: one 16-byte access of bf16, two of fp32.  load_column:
// of memory that no kernel here writes; rows may be those that the same kernel writes (h in the
// place of x, dx in that of dy).
template <typename T>
struct Eight;
template <>
struct Eight<bf16> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void load_column(const bf16* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
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
  // keeps value j where bit j is set
  __device__ __forceinline__ void keep(uint32_t bits) {
    auto word = [&](int i) {
      return (bits >> (2 * i) & 1u ? 0xffffu : 0u) | (bits >> (2 * i + 1) & 1u ? 0xffff0000u : 0u);
    };
    v = make_uint4(v.x & word(0), v.y & word(1), v.z & word(2), v.w & word(3));
  }
};
template <>
struct Eight<float> {
  float4 v[2];
  __device__ __forceinline__ void load(const float* p) {
    v[0] = reinterpret_cast<const float4*>(p)[0];
    v[1] = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void load_column(const float* p) {
    v[0] = __ldg(reinterpret_cast<const float4*>(p));
    v[1] = __ldg(reinterpret_cast<const float4*>(p) + 1);
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
  __device__ __forceinline__ void keep(uint32_t bits) {
    float f[8];
    get(f);
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = bits >> j & 1u ? f[j] : 0.f;
    set(f);
  }
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
// Which of group i's eight places are in the row, as bits.
template <bool kVec>
__device__ __forceinline__ uint32_t inside(int i, const Team& t) {
  const int c = column<kVec>(t, i);
  if (whole<kVec>(t, c)) return 0xffu;
  if (kVec || c >= t.H) return 0u;
  return (c < 0 ? 0xffu << -c : 0xffu) & (c + 8 > t.H ? 0xffu >> (c + 8 - t.H) : 0xffu);
}
// kShared: the row is a copy in shared memory, with room for its first and last groups'
// missing values.
template <bool kShared = false, bool kVec, typename T>
__device__ __forceinline__ void get(Eight<T>& e, const T* row, int i, const Team& t) {
  const int c = column<kVec>(t, i);
  if constexpr (kShared) {
    if (c < t.H) e.load(row + c);
    else e.zero();
    if (!kVec && c < t.H && !whole<kVec>(t, c)) e.keep(inside<kVec>(i, t));
  } else if (whole<kVec>(t, c)) {
    e.load(row + c);
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
// Of the words from a 16-byte boundary on (x), those that begin `skip` words later, for any
// skip below 4: a choice between two places for each of its bits.
template <int have, int want>
__device__ __forceinline__ void skip_words(uint32_t (&x)[have], int skip) {
#pragma unroll
  for (int i = 0; i < want + 1 && i + 2 < have; ++i) x[i] = skip & 2 ? x[i + 2] : x[i];
#pragma unroll
  for (int i = 0; i < want && i + 1 < have; ++i) x[i] = skip & 1 ? x[i + 1] : x[i];
}
// The columns' own values, whose place in memory has nothing to do with the rows'.  Where
// eight of them do not start on a 16-byte boundary they are cut out of the pieces around them:
// one by one, a warp's take four passes through L1 each.
template <bool kVec, typename W>
__device__ __forceinline__ void get_column(Eight<W>& e, const W* w, int i, const Team& t) {
  const int c = column<kVec>(t, i);
  if constexpr (kVec) {
    if (c < t.H) e.load_column(w + c);
    else e.zero();
  } else {
    constexpr int kPiece = 16 / sizeof(W);
    const int s = c & (kPiece - 1);
    // the pieces lie within the array, or are those of its end
    if (c >= 0 && c - s + 8 + kPiece <= t.H) {
      const uint4* from = reinterpret_cast<const uint4*>(w + (c - s));
      if constexpr (sizeof(W) == 2) {
        const uint4 a = __ldg(from), b = __ldg(from + 1);
        uint32_t x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
        skip_words<8, 5>(x, s >> 1);
        uint32_t y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = s & 1 ? __funnelshift_r(x[j], x[j + 1], 16) : x[j];
        e.v = make_uint4(y[0], y[1], y[2], y[3]);
      } else {
        const uint4 a = __ldg(from), b = __ldg(from + 1), d = __ldg(from + 2);
        uint32_t x[12] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, d.x, d.y, d.z, d.w};
        skip_words<12, 8>(x, s);
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(x[j]);
        e.set(f);
      }
    } else {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = c + j >= 0 && c + j < t.H ? to_f32(w[c + j]) : 0.f;
      e.set(f);
    }
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
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  return v;
}
// Groups of eight that a row takes; one that may begin within a group, up to one more.
int groups_of(int H) { return (H + 7 + (H % 8 != 0 ? 7 : 0)) / 8; }
int team_of(int H, int n) {   // threads that hold a row with n groups each
  const int t = (groups_of(H) + n - 1) / n;
  return (t + 31) / 32 * 32;
}

}  // namespace

#define MOE_NORM_TYPES(f, ...)                                                            \
  do {                                                                                    \
    const bool vec = H % 8 == 0;                                                          \
    if (type == MOE_F32)                                                                  \
      return vec ? f<float, float, true>(__VA_ARGS__) : f<float, float, false>(__VA_ARGS__); \
    if (weight_type == MOE_F32)                                                           \
      return vec ? f<bf16, float, true>(__VA_ARGS__) : f<bf16, float, false>(__VA_ARGS__); \
    return vec ? f<bf16, bf16, true>(__VA_ARGS__) : f<bf16, bf16, false>(__VA_ARGS__);    \
  } while (0)

}  // namespace moe
