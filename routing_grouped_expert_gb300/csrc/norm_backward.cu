// The gradients of layer norm (norm.cu):
//
//   xhat = (h - mean) rstd,  a = sum(w dy) / H,  c = sum(w dy xhat) / H
//   dx = rstd (w dy - a - xhat c) + dh     (dh: the gradient that reaches h past the norm)
//   dw = sum_t dy xhat,  db = sum_t dy
//
// One pass over dy, h and dh: each block adds the dw and db of its rows in registers, and a
// second launch adds the blocks' shares.  Sums are fp32 in a fixed order.
//
// Bound by memory: 8192 x 7168 bf16 with dh in 77.1 us (470 MB, 0.90 of the rate of a plain
// copy), of which the second launch is about 5; 12000 x 4096 64.5 (0.90), 20000 x 2048 55
// (0.88), 40001 x 512 35 (0.70: a row per warp, its latency), 200000 x 128 76 (0.40: the same),
// rows of 7170 101 (0.69: the fetching thread's work and the rows' ends), 4000 x 16384 144 to 147
// (0.54: eight groups of a thread do not fit its registers).  fp32: 4096 x 7168 74.7 us (0.93),
// without dh 61.3 (0.84), 8192 x 4096 89 (0.89), 2000 x 16384 157 (0.49).  Few rows: 1 in 5.4 us, 128 of 7168 in 8.9, mostly the
// two launches and their first loads.
#include "norm.cuh"

namespace moe {
namespace {

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
//   dx = dh + rstd (u - a / H - (rstd^2 c / H) d)
// rstd^2 c / H is formed from the right, where it is rstd times a mean of u xhat: rstd^2 by itself
// may leave fp32 with a small eps, in rows of padding say, in which c is 0.
// The thread's part of a row, and of dx.
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
    const float a = -(s.x / t.H), c = -st.y * (st.y * (s.y / t.H));
#pragma unroll
    for (int i = 0; i < n; ++i) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 x = __fadd2_rn(u[i][j], make_float2(a, a));
        x = __ffma2_rn(d[i][j], make_float2(c, c), x);
        x = __ffma2_rn(x, make_float2(st.y, st.y), r[i].pair(j));
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
norm_backward_kernel(const T* dy, const T* h, const float2* __restrict__ stats,
                     const W* __restrict__ weight, const T* dh, int rows, int H, T* dx,
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
constexpr int kMaxStages = 8;
template <typename T>
struct RowRing {
  char* buf;        // [stages][3][pitch]
  uint64_t* full;   // [stages]
  int H, stages, pitch, tensors;
  long long rows;

  // a row and its first and last groups' missing values
  static __host__ __device__ int pitch_of(int H) { return (H * (int)sizeof(T) + 15 + 8 * (int)sizeof(T) + 15) / 16 * 16; }
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
norm_backward_ring_kernel(const T* dy, const T* h, const float2* __restrict__ stats,
                          const W* __restrict__ weight, const T* dh, int rows, int H, int stages,
                          T* dx, float* __restrict__ part, int* __restrict__ flags, Hold hold) {
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
  if (me == 0 && blockIdx.x == 0) ptx::hold_up(hold.at);
  if (me == 0)
    for (int s = 0; s < stages && ahead < rows; ++s, ahead += gridDim.x)
      ring.fetch(s, ahead, cut, from);
  Backward<T, W, n, kVec, kTeam> b;
  b.t = Team{me, (int)blockDim.x, H, cut};
  b.begin(weight);
  float2 next = __ldg(stats + blockIdx.x);
  int turn = 0, stage = 0;
  uint32_t phase = 0;
  long long at = blockIdx.x;   // the row that is worked on
  for (; at < rows; at += gridDim.x) {
    const long long row = at;
    const float2 st = next;
    if (row + gridDim.x < rows) next = __ldg(stats + row + gridDim.x);
    if (!ptx::mbar_wait(&full[stage], phase, nullptr, hold.limit)) dead[turn] = 1;
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
    // what is still on its way has to arrive before the block's memory is another's: the rows
    // from the one that was waited for to the last that was asked for, a place further each
    if (late)
      for (; at < ahead; at += gridDim.x) {
        ptx::mbar_wait(&full[stage], phase, nullptr, hold.limit);
        if (++stage == stages) {
          stage = 0;
          phase ^= 1u;
        }
      }
  }
  b.end(part + (size_t)blockIdx.x * 2 * H);
}

// dw, db = the sums of the blocks' shares, in block order within each of kWarps warps; the
// status from the blocks' flags.  A lane takes V columns; all of a warp's loads are in
// flight at once, eight at a time.
template <typename W, int V, int kWarps>
__global__ void __launch_bounds__(32 * kWarps)
norm_weight_kernel(const float* __restrict__ part, int blocks, int H, W* __restrict__ dw,
                   W* __restrict__ db, const int* __restrict__ flags, int* __restrict__ status) {
  __shared__ float sums[kWarps][32 * V + 1];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 * V + V * lane;
  W* out = blockIdx.y == 0 ? dw : db;
  float v[V];
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = 0.f;
  if (c < H) {   // V > 1: H is a multiple of it
    const float* from = part + (size_t)blockIdx.y * H + c;
#pragma unroll 8
    for (int b = warp; b < blocks; b += kWarps) {
      if constexpr (V == 4) {
        const float4 x = *reinterpret_cast<const float4*>(from + (size_t)b * 2 * H);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
      } else {
        v[0] += from[(size_t)b * 2 * H];
      }
    }
  }
#pragma unroll
  for (int j = 0; j < V; ++j) sums[warp][V * lane + j] = v[j];
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    int bad = 0;
    for (int b = threadIdx.x; b < blocks; b += 32 * kWarps) bad |= flags[b];
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) {
      status[0] = bad ? MOE_ERR_TIMEOUT : 0;
      status[1] = 0;
    }
  } else {
    __syncthreads();
  }
  for (int i = threadIdx.x; i < 32 * V; i += 32 * kWarps) {
    const int at = blockIdx.x * 32 * V + i;
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w][i];
    if (at < H) out[at] = from_f32<W>(s);
  }
}

// Shared memory of a ring where `per` blocks share an SM.
constexpr int ring_bytes(int per) { return 227 * 1024 / per - 2048; }
// A backward's launch shape, by the groups of eight that a row takes: few threads with
// many groups each keep a row's loads and sums in flight at once, and two sums over 7 warps
// take less than over 28.  8192 x 7168, threads x groups, us: 896 x 1 97, 448 x 2 94, 224 x 4
// 77; 12000 x 4096, blocks per SM: 512 x 1 by two 75, 128 x 4 by two 65, by one 73; 20000 x
// 2048: 256 x 1 by three 57, 128 x 2 by three 55, 64 x 4 by four 54.
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
    const cudaError_t e = allow_smem(kern, stages * stage, ring_bytes(f.per));                    \
    if (e != cudaSuccess) return e;                                                               \
    kern<<<blocks, team_of(H, f.n), stages * stage, s>>>(gt, ht, st, wt, rt, rows, H, stages, xt, part, \
                                                         flags, diag_hold());                                  \
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
  // few shares: four columns a lane, all of a warp's loads in flight (128 rows of 7168: 9.0
  // against 9.6 us); many: as many warps as a block has (20000 of 2048: 55.5 against 59.4)
  const bool wide = H % 4 == 0 && H >= 1024 && blocks <= kSms;
  const int columns = wide ? 128 : 32;
  return launch_k(wide ? norm_weight_kernel<W, 4, 16> : norm_weight_kernel<W, 1, 32>,
                  dim3((H + columns - 1) / columns, db != nullptr ? 2 : 1), dim3(wide ? 512 : 1024), 0, s,
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
