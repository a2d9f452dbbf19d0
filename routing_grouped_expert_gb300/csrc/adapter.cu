// Low-rank adapters of many requests at once beside a shared projection:
//   y[t] = x[t] W + z[t] B_a,   z[t] = scale_a * (x[t] A_a^T),   a = adapter_idx[t]
// with W [H, N], A [n, R, H], B [n, R, N]; a token with adapter -1 has no z.
//
// A token block (kNB consecutive tokens) meets a few adapters, its entries (in
// ascending order).  The block's low-rank activations are kept expanded: row t
// of Z holds R columns per entry, zero but for the token's own one.  Then
//   shrink: Z = mask(x [A_a0; A_a1; ..]^T)   one product, masked in its epilogue
//   expand: y = [x | Z] [W; B_a0; B_a1; ..]  the K loop of x W runs on over Z
// so the adapters' part is more K stages of the projection's own tiles: no rows
// are gathered or scattered, and a block of one request pays for one adapter.  A
// block pays for every adapter it meets: few in any order cost little, many in random
// order cost more than the projection (4096 x 4096 x 4096, rank 16: 90 us with one
// adapter, 116 with 16 in random order, 304 with 256; rank 64: 986 with 256, 200 when
// their tokens stand together).  dx = dy W^T + dz A is the same
// pair of products with the roles of A and B exchanged and W read K-major.
//   weight gradients: dA_a = dZ_a^T x, dB_a = Z_a^T dy over the blocks that meet a.
//
// All products run on the 5th-generation tensor cores (weights: the M operand,
// tokens: the N operand), bf16 in, fp32 accumulation in TMEM.  z is rounded to
// bf16 once, as an MMA operand; y, dx, dA and dB are rounded once on output.
#include <cuda.h>

#include <atomic>

#include "moe_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kM = 128;             // output features (or rank rows) per tile
constexpr int kK = 64;              // K per stage: one 128-byte swizzle atom
constexpr int kABytes = kM * kK * 2;
constexpr int kThreads = 224;       // producer, MMA, guard and four epilogue warps
constexpr int kMaxEntries = 256;    // adapters a token block can meet
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr int kSmemMax = 232448;    // dynamic shared memory per CTA (227 KB)
constexpr int kMaxStages = 9;
// Stages of `bytes` that fit beside `other` bytes.
__host__ __device__ constexpr int ring_stages(int bytes, int other) {
  return (kSmemMax - 1024 - other) / bytes < kMaxStages ? (kSmemMax - 1024 - other) / bytes
                                                        : kMaxStages;
}
// A stage of 128 weight rows and nb token rows.
__host__ __device__ constexpr int stage_bytes_of(int nb) { return kABytes + nb * kK * 2; }

// What the shrink kernel leaves about one token block for the kernels after it.
struct BlockPlan {
  int n_ent;                       // adapters the block meets
  int bad;                         // an adapter index was out of range
  int pad[2];                      // `list` 16-byte aligned
  uint32_t bits[32];               // the same adapters as bits
  uint16_t list[kMaxEntries];      // ascending
};
static_assert(sizeof(BlockPlan) <= kAdapterPlanBytes, "plan pitch");

__device__ __forceinline__ const BlockPlan* plan_of(const void* plan, int tt) {
  return reinterpret_cast<const BlockPlan*>(static_cast<const char*>(plan) +
                                            (size_t)tt * kAdapterPlanBytes);
}

// The hand-over of what shrink wrote to a kernel that starts before expand ends: a
// thread of expand, once its own griddepcontrol.wait has made shrink's results
// visible to it, publishes the call's number with release order; the kernel after
// it reads nothing of shrink's before it has read that number with acquire order
// (starting early makes no writes visible).  The word is in the workspace, beside
// the status.
__device__ __forceinline__ uint64_t* hand_over_word(int* status) {
  return reinterpret_cast<uint64_t*>(status + 4);
}
__device__ __forceinline__ void hand_over(int* status, uint64_t call) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(hand_over_word(status)), "l"(call)
               : "memory");
}
// Bounded: expand publishes before it lets the next kernel start, unless it gave up.
__device__ __forceinline__ bool take_over(int* status, uint64_t call) {
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    uint64_t v;
    asm volatile("ld.acquire.gpu.global.u64 %0, [%1];"
                 : "=l"(v)
                 : "l"(hand_over_word(status))
                 : "memory");
    if (v == call) return true;
    if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
}

__device__ __forceinline__ void fence_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
// The sum over kS CTAs of the cluster, in rank order from `first`, of the float4
// at `addr` of their shared memory; all loads in flight at once.
template <int kS>
__device__ __forceinline__ float4 cluster_sum(uint32_t addr, int first = 0) {
  float4 p[kS];
#pragma unroll
  for (int r = 0; r < kS; ++r) p[r] = ld_cluster_f4(mapa_shared(addr, (uint32_t)(first + r)));
#pragma unroll
  for (int r = 1; r < kS; ++r) {
    p[0].x += p[r].x;
    p[0].y += p[r].y;
    p[0].z += p[r].z;
    p[0].w += p[r].w;
  }
  return p[0];
}

__device__ __forceinline__ uint2 pack4(float4 v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  uint2 r;
  r.x = *reinterpret_cast<const uint32_t*>(&lo);
  r.y = *reinterpret_cast<const uint32_t*>(&hi);
  return r;
}

// The role loops run warp-uniform: every lane waits and counts, one lane issues.
// TMA and MMA instructions take their operands from uniform registers, so in
// code that a single lane runs alone each operand is first moved there (a
// producer of two boxes took 500 cycles a stage that way, an MMA warp 430).
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(p));
  return p != 0;
}
// kCluster: the barrier counts arrivals of the pair's other CTA too, whose writes
// are to be seen.
template <bool kCluster>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (kCluster)
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  return ok != 0;
}
template <bool kCluster>
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t i = 1;; ++i) {
    if (try_wait<kCluster>(bar, parity)) return true;
    if ((i & 15) == 0 && (*abort_flag || globaltimer_ns() - t0 > kWaitLimitNs)) return false;
  }
}
// Wait for the phase with `parity` of the barrier at shared address `bar`;
// bounded as ptx::mbar_wait.
template <bool kCluster = false>
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, const volatile int* abort_flag) {
  return try_wait<kCluster>(bar, parity) ? true : wait_slow<kCluster>(bar, parity, abort_flag);
}
// The role loops' instructions on shared addresses (no generic pointers to
// convert at every stage).
__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
               : "memory");
}
// kPair: `bar` may be a barrier of the pair's other CTA (a cluster address).
template <bool kPair = false>
__device__ __forceinline__ void load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                        int y, uint64_t policy) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "l"(policy)
        : "memory");
}
template <bool kPair = false>
__device__ __forceinline__ void load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                        int y, int z, uint64_t policy) {
  if constexpr (kPair)
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "l"(policy)
        : "memory");
}
__device__ __forceinline__ void load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                        int y, int z, int w, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w), "l"(policy)
      : "memory");
}
// Arrive once on `bar`'s place in both CTAs of a pair when the pair's tcgen05
// operations that this thread issued so far have completed.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
      " [%0], %1;" ::"r"(bar),
      "h"((uint16_t)0x3)
      : "memory");
}
// A 128-byte-swizzled operand descriptor from its two words (see
// ptx::sdesc_sw128): the first word moves with the address >> 4.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) {
  return ((uint64_t)hi << 32) | lo;
}
__device__ __forceinline__ uint32_t desc_lo(uint32_t addr, uint32_t lbo) {
  // in a cluster the address carries the CTA's rank above its 18 offset bits
  return ((addr & 0x3ffffu) >> 4) | ((lbo >> 4) << 16);
}
constexpr uint32_t desc_hi(uint32_t sbo) { return (sbo >> 4) | (1u << 14) | (2u << 29); }

// 32 TMEM lanes x 32 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_32x32b_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]),
        "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]),
        "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// This warp's 32 features of the tokens below n, from TMEM to a [token][128] tile.
__device__ __forceinline__ void stage_tile(float* st, uint32_t tb, int n) {
  for (int c0 = 0; c0 < n; c0 += 32) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(tb + c0, v);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (c0 + c < n) st[(c0 + c) * kM] = __uint_as_float(v[c]);
  }
}

// One role's place in a ring of n stages and their barriers.
struct Place {
  int n;
  int stage = 0;
  uint32_t phase = 0;
  int count = 0;   // stages passed
  __device__ __forceinline__ explicit Place(int n_) : n(n_) {}
  __device__ __forceinline__ void next() {
    ++count;
    if (++stage == n) {
      stage = 0;
      phase ^= 1u;
    }
  }
};
// No TMA write may land after the CTA exits (or before its ring is reused by
// ordinary stores): the last loads have arrived.
__device__ __forceinline__ void drain_loads(uint64_t* full, int stages, int from, int issued) {
  for (int i = issued - from > stages ? issued - stages : from; i < issued; ++i)
    mbar_wait(&full[i % stages], (uint32_t)((i / stages) & 1), nullptr, kWaitLimitNs);
}

// ---------------------------------------------------------------- shrink
// Z[t, e R + r] = scale_a * <x[t], A_a[r]> at the token's own entry e, 0 elsewhere,
// in units of 128 rank rows of a token block.  Bound by reading x and the rank
// rows once, so K is split: the kC CTAs of a cluster work on kC / s units at a
// time, s CTAs each taking a share of a unit's K, s chosen per block by how
// many units it turns out to have.  The partial tiles meet in shared memory,
// where only the R values that a token keeps are read.
//
// A block of several units whose entries have few tokens each (at most 64 per
// unit) gathers a unit's own tokens instead of multiplying every token of the
// block by every rank row: two warps copy the rows' 128 bytes of each stage
// by 16-byte asynchronous copies into the swizzled operand.  (TMA
// tile::gather4 took about 16 ns a row: 777 tokens of 24 adapters of rank 64
// spent 31 us on the gathers.)
//
// The gradient's two products, x A^T and dy B^T, are one launch: blockIdx.z says
// which.  While both fit the SMs they run side by side, otherwise one after the other.
//
// Measured: 4096 tokens x 6144, 16 adapters of rank 16, 128 CTAs: 20 us; 8192
// tokens, 7168 + 2048 columns, 8 adapters of rank 16: 43 us for the gradient's
// two products, whose K loops read x at 6.7 TB/s; 777 x 7168, 24 adapters of
// rank 64 (gathered rows): 18 us, bound by the latency of the copies.  About 6 us
// before the first MMA and 4 to 6 us after the last are part of each.
struct ShrinkMaps {
  CUtensorMap p[2];  // the adapters' rank rows [n, R, K], boxes of 64 K x rb rows
  CUtensorMap v[2];  // token rows [T, K], boxes of 64 K x nb rows
};
struct ShrinkArgs {
  int T, nb, n, R, rb, zc;   // nb: tokens per block; rb: rank rows per box, a power
                             // of two that divides R
  int K[2];
  const __nv_bfloat16* rows[2];   // the token rows
  const char* next;         // the adapters' matrices [n][next_bytes] of the expand launch, or null
  long long next_bytes;
  const int32_t* adapter_idx;
  const float* scale;
  __nv_bfloat16* z[2];      // [T, zc]
  void* plan;
  uint32_t* masks;          // [n_tt][256][8]: the tokens of every entry, as bits; or null
  int* status;
};
constexpr int kGatherRows = 64;   // most tokens of a unit that gathers
constexpr int kRowWarps = 2;      // warps 2 and 3 copy them
constexpr int kRowPieces = kGatherRows * 8 / (32 * kRowWarps);   // 16-byte pieces per thread
constexpr int kShrinkOther = 5120;   // ShrinkShared
template <int kNB>
struct ShrinkCfg {
  static constexpr bool kGather = kNB > kGatherRows;
  static constexpr int kTmemCols = kNB < 32 ? 32 : kNB;
  static constexpr int kSmemBytes = kSmemMax;
  static constexpr int kRing = kSmemBytes - 1024 - kShrinkOther;
  static_assert(kNB * kM * 4 <= kRing, "the partial fp32 tile is staged in the ring");
};
struct ShrinkShared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full, drain;
  uint32_t tmem_base;
  int abort, bad, n_ent, most;
  unsigned bits[32];
  uint16_t list[kMaxEntries];
  int count[kMaxEntries];       // tokens of each entry
  int idx[256];                 // adapter of each token of the block, -1 for none
  uint16_t ent[256];            // its entry
  uint16_t tok[kGatherRows];    // the tokens of a gathering unit
  uint16_t pos[256];            // a token's place among them
  int n_tok;
};
static_assert(sizeof(ShrinkShared) <= kShrinkOther, "shared block");

__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// Arrive on `bar` (a counted arrival) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The adapters that token block tt meets, by the whole CTA.
template <bool kCount>
__device__ __forceinline__ void build_list(ShrinkShared* sh, const ShrinkArgs& a, int row0,
                                           int rows) {
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < 32) sh->bits[tid] = 0u;
  if (tid == 32) sh->bad = sh->most = 0;
  if (kCount)
    for (int i = tid; i < kMaxEntries; i += kThreads) sh->count[i] = 0;
  __syncthreads();
  for (int i = tid; i < rows; i += kThreads) {
    int e = __ldg(a.adapter_idx + row0 + i);
    if (e < 0 || e >= a.n) {
      if (e != -1) sh->bad = 1;
      e = -1;
    } else {
      atomicOr(&sh->bits[e >> 5], 1u << (e & 31));
    }
    sh->idx[i] = e;
  }
  __syncthreads();
  if (tid < 32) {
    const int c = __popc(sh->bits[lane]);
    int incl = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += u;
    }
    int at = incl - c;
    for (unsigned w = sh->bits[lane]; w; w &= w - 1)
      sh->list[at++] = (uint16_t)(lane * 32 + __ffs(w) - 1);
    if (lane == 31) sh->n_ent = incl;
  }
  if (kCount) {
    for (int i = tid; i < rows; i += kThreads) {
      const int e = sh->idx[i];
      int at = kMaxEntries;
      if (e >= 0) {
        at = __popc(sh->bits[e >> 5] & ((1u << (e & 31)) - 1u));
        for (int w = 0; w < (e >> 5); ++w) at += __popc(sh->bits[w]);
        atomicAdd(&sh->count[at], 1);
      }
      sh->ent[i] = (uint16_t)at;
    }
  }
  __syncthreads();
}
// ... and the plan of it, for the kernels that follow (one CTA of the block;
// `scratch`: 8 KB that nothing uses yet).
__device__ __forceinline__ void write_plan(ShrinkShared* sh, const ShrinkArgs& a, int tt, int rows,
                                           uint32_t* scratch) {
  const int tid = threadIdx.x;
  BlockPlan* p = const_cast<BlockPlan*>(plan_of(a.plan, tt));
  if (tid < 32) p->bits[tid] = sh->bits[tid];
  if (tid == 32) {
    p->n_ent = sh->n_ent;
    p->bad = sh->bad;
  }
  for (int i = tid; i < sh->n_ent; i += kThreads) p->list[i] = sh->list[i];
  if (a.masks == nullptr) return;
  const int n = sh->n_ent * 8;
  for (int i = tid; i < n; i += kThreads) scratch[i] = 0u;
  __syncthreads();
  for (int i = tid; i < rows; i += kThreads) {
    const int e = sh->idx[i];
    if (e < 0) continue;
    int at = __popc(sh->bits[e >> 5] & ((1u << (e & 31)) - 1u));
    for (int w = 0; w < (e >> 5); ++w) at += __popc(sh->bits[w]);
    atomicOr(&scratch[at * 8 + (i >> 5)], 1u << (i & 31));
  }
  __syncthreads();
  for (int i = tid; i < n; i += kThreads) a.masks[(size_t)tt * kMaxEntries * 8 + i] = scratch[i];
  fence_async_smem();   // the scratch is ring space: TMA loads follow
  __syncthreads();
}

// This CTA's tokens of a finished unit: Z rows of 128 columns, a warp per token.
template <int kS>
__device__ __forceinline__ void store_unit(const ShrinkShared* sh, const ShrinkArgs& a,
                                           __nv_bfloat16* z, const uint8_t* smem, int row0, int rows, int u,
                                           int q_end, bool gather, int first, int r) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this lane's four rank rows belong to one entry (R is a multiple of 8)
  const int ad = 4 * lane < q_end ? (int)sh->list[(u * kM + 4 * lane) / a.R] : -2;
  const float f = ad >= 0 ? __ldg(a.scale + ad) : 0.f;
  const uint32_t mine = smem_u32(smem) + (uint32_t)lane * 16;
#pragma unroll 4
  for (int t = r * (kThreads / 32) + warp; t < rows; t += kS * (kThreads / 32)) {
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (sh->idx[t] == ad) {
      const int j = gather ? (int)sh->pos[t] : t;
      s = cluster_sum<kS>(mine + (uint32_t)j * (kM * 4), first);
      s = make_float4(s.x * f, s.y * f, s.z * f, s.w * f);
    }
    *reinterpret_cast<uint2*>(z + (size_t)(row0 + t) * a.zc + u * kM + 4 * lane) = pack4(s);
  }
}

template <int kNB, int kC>
__global__ void __launch_bounds__(kThreads, 1)
adapter_shrink_kernel(const __grid_constant__ ShrinkMaps maps, const ShrinkArgs a) {
  using C = ShrinkCfg<kNB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  ShrinkShared* sh = reinterpret_cast<ShrinkShared*>(smem + C::kRing);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = kC > 1 ? (int)cluster_ctarank() : 0;
  const int tt = (int)blockIdx.x / kC;
  const int row0 = tt * a.nb, rows = min(a.nb, a.T - row0);
  const int job = (int)blockIdx.z;   // 0 or 1; no indexing of the parameters with it
  const int K = job ? a.K[1] : a.K[0], nk = K / kK;
  const CUtensorMap* map_p = job ? &maps.p[1] : &maps.p[0];
  const CUtensorMap* map_v = job ? &maps.v[1] : &maps.v[0];
  __nv_bfloat16* z = job ? a.z[1] : a.z[0];

  pdl_trigger();
  // the call's status starts clean: this is its first kernel, and nothing is
  // reported before a later kernel of the call or a wait of a second
  if (job == 0 && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x < 2) a.status[threadIdx.x] = 0;
  build_list<C::kGather>(sh, a, row0, rows);
  if (job == 0 && rank == 0 && blockIdx.y == 0)
    write_plan(sh, a, tt, rows, reinterpret_cast<uint32_t*>(smem));
  const int q_all = sh->n_ent * a.R;
  const int units = (q_all + kM - 1) / kM;
  if (a.next != nullptr && warp == 3 && blockIdx.z + 1 == gridDim.z) {
    // the expand launch's adapter rows start on their way into L2
    const int parts = (int)gridDim.y * kC;
    const long long step = 16384, per = (a.next_bytes + step - 1) / step;
    for (long long i = (long long)(blockIdx.y * kC + rank) * 32 + lane; i < per * sh->n_ent;
         i += parts * 32) {
      const int e = (int)(i / per);
      const long long off = (i - e * per) * step;
      const long long left = a.next_bytes - off;
      prefetch_l2(a.next + sh->list[e] * a.next_bytes + off, (uint32_t)(left < step ? left : step));
    }
  }
  // s CTAs per unit: as many as leave a group of CTAs for every unit
  int s = kC;
  while (s > 1 && units * s > (int)gridDim.y * kC) s >>= 1;
  const int groups = kC / s, sub = rank / s, r = rank - sub * s;
  const int u_step = (int)gridDim.y * groups, u_first = (int)blockIdx.y * groups;
  if (u_first >= units) return;   // the same for the whole cluster
  const int kb0 = nk * r / s, kb1 = nk * (r + 1) / s;
  bool gather = false;
  if constexpr (C::kGather) {
    if (units > 1) {
      // the largest number of tokens that one unit's entries have
      for (int u = threadIdx.x; u < units; u += kThreads) {
        int c = 0;
        for (int e = u * kM / a.R; e < sh->n_ent && e * a.R < (u + 1) * kM; ++e) c += sh->count[e];
        atomicMax(&sh->most, c);
      }
      __syncthreads();
      gather = sh->most <= kGatherRows;
    }
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&sh->full[i], gather ? 1 + 32 * kRowWarps : 1);   // TMA, and the threads that copy rows
      mbar_init(&sh->empty[i], 1);
    }
    mbar_init(&sh->acc_full, 1);
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  volatile int* abort_flag = &sh->abort;
  const uint32_t full0 = smem_u32(sh->full), empty0 = smem_u32(sh->empty);
  const int stage_bytes = stage_bytes_of(gather ? kGatherRows : a.nb);
  const int stages = ring_stages(stage_bytes, kShrinkOther);
  Place at(stages);
  uint32_t parity = 0;
  for (int u0 = u_first; u0 < units; u0 += u_step) {
    const int u = u0 + sub;
    const bool have = u < units;   // the groups of a cluster go through the loop together
    const int q_end = min(kM, q_all - u * kM);
    if (C::kGather && gather) {
      if (have && warp == 2) {
        const int e0 = u * kM / a.R, e1 = (u * kM + q_end - 1) / a.R;
        int n = 0;
        for (int t0 = 0; t0 < rows; t0 += 32) {
          const int t = t0 + lane, e = t < rows ? (int)sh->ent[t] : kMaxEntries;
          const bool in = e >= e0 && e <= e1;
          const unsigned m = __ballot_sync(0xffffffffu, in);
          if (in) {
            const int j = n + __popc(m & ((1u << lane) - 1u));
            sh->tok[j] = (uint16_t)t;
            sh->pos[t] = (uint16_t)j;
          }
          n += __popc(m);
        }
        if (lane == 0) sh->n_tok = n;
      }
      __syncthreads();
    }
    const int n_tok = gather && have ? sh->n_tok : rows;   // rows of the partial tile
    const int n_mma = gather ? (n_tok + 15) & ~15 : a.nb;
    // Warps 0, 4, 5 and 6 load the boxes of rank rows (box i: the i-th of them),
    // warp 0 the token rows too; rank rows past the last entry keep what the
    // stage held: their products are not read.
    const int loader = warp == 0 ? 0 : warp >= 4 ? warp - 3 : -1;
    if (have && loader >= 0) {
      const uint64_t pol_p = policy_evict_normal(), pol_v = policy_evict_last();
      const bool leader = elect_lane();
      const int from = at.count;
      const uint32_t sbase = smem_u32(smem);
      const uint32_t bytes = (uint32_t)((q_end + (gather ? 0 : a.nb)) * kK * 2);
      // this warp's boxes: at most 16 of 8 rows over four warps
      int row[4], ad[4];
      bool box[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int q = (loader + 4 * i) * a.rb, e = (u * kM + q) / a.R;
        box[i] = q < q_end;
        row[i] = u * kM + q - e * a.R;
        ad[i] = box[i] ? (int)sh->list[e] : 0;
      }
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = wait_bar(empty0 + at.stage * 8, at.phase ^ 1u, abort_flag);
        if (!ok) break;
        const uint32_t fb = full0 + at.stage * 8, st = sbase + at.stage * stage_bytes;
        if (loader == 0 && leader) {
          expect_tx(fb, bytes);
          if (!gather) load_2d(st + kABytes, map_v, fb, kb * kK, row0, pol_v);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (box[i] && leader)
            load_3d(st + (loader + 4 * i) * a.rb * (kK * 2), map_p, fb, kb * kK, row[i], ad[i],
                    pol_p);
        at.next();
      }
      if (leader && !ok) {
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailProducer);
        *abort_flag = 1;
      }
      if (loader == 0 && leader) drain_loads(sh->full, stages, from, at.count);
      __syncwarp();
    } else if (have && warp == 1) {
      const uint32_t sbase = smem_u32(smem);
      const uint32_t idesc = idesc_bf16(kM, n_mma, false, false);
      const bool leader = elect_lane();
      bool ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = wait_bar(full0 + at.stage * 8, at.phase, abort_flag);
        if (!ok) break;
        // copied rows: ordinary writes that the MMA reads through the async
        // proxy.  The fence is taken here, by a thread without copies in flight:
        // in the copying threads it waits for all of theirs
        if (gather) fence_async_smem();
        tc_fence_after();
        // K-major operands: 8-row groups 1 KB apart, 16 K = 32 bytes
        const uint32_t la = desc_lo(sbase + (uint32_t)(at.stage * stage_bytes), 16);
        const uint32_t lb = la + (kABytes >> 4);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < kK / 16; ++kk)
            mma_bf16_ss(tmem, desc_of(la + 2 * kk, desc_hi(1024)), desc_of(lb + 2 * kk, desc_hi(1024)),
                        idesc, (kb > kb0 || kk) ? 1u : 0u);
          commit(empty0 + at.stage * 8);
        }
        at.next();
      }
      if (leader) {
        if (!ok) {
          set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailMma);
          *abort_flag = 1;
        }
        mma_commit(&sh->acc_full);
        mma_commit(&sh->drain);
        if (!mbar_wait(&sh->drain, parity, nullptr, kWaitLimitNs))
          set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailDrain);
      }
      __syncwarp();
    }
    if (C::kGather && gather && have && warp >= 2 && warp < 2 + kRowWarps) {
      // this thread's 16-byte pieces: piece c of row j, at the swizzled place
      const int n_piece = n_mma * 8;
      const __nv_bfloat16* src[kRowPieces];
      uint32_t dst[kRowPieces];
#pragma unroll
      for (int i = 0; i < kRowPieces; ++i) {
        const int piece = (int)threadIdx.x - 64 + i * (32 * kRowWarps), j = piece >> 3, c = piece & 7;
        dst[i] = piece < n_piece ? (uint32_t)(kABytes + j * 128 + ((c ^ (j & 7)) << 4)) : 0u;
        // rows up to a multiple of 16 repeat the last token
        src[i] = (job ? a.rows[1] : a.rows[0]) + (size_t)(row0 + (int)sh->tok[min(j, n_tok - 1)]) * K +
                 c * 8;
      }
      const uint32_t sbase = smem_u32(smem);
      // every thread arrives when its copies land (64 arrivals a stage; 160, of
      // five warps, took 0.24 us by themselves, and waiting for the copies of
      // an earlier stage before announcing it keeps slots of the ring idle)
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!wait_bar(empty0 + at.stage * 8, at.phase ^ 1u, abort_flag)) break;
#pragma unroll
        for (int i = 0; i < kRowPieces; ++i)
          if (dst[i]) cp_async16(sbase + at.stage * stage_bytes + dst[i], src[i] + (size_t)kb * kK);
        cp_async_arrive(&sh->full[at.stage]);
        at.next();
      }
      asm volatile("cp.async.wait_all;" ::: "memory");   // none is in flight when the CTA leaves
    } else if (have && (warp == 2 || warp == 3)) {
      for (int kb = kb0; kb < kb1; ++kb) at.next();
    }
    const int q = warp & 3;   // TMEM lanes 32 q ..
    if (have && warp >= 3) {
      const bool got = mbar_wait(&sh->acc_full, parity, abort_flag, kWaitLimitNs);
      tc_fence_after();
      if (__all_sync(0xffffffffu, got) && q * 32 < q_end) {
        stage_tile(reinterpret_cast<float*>(smem) + q * 32 + lane, tmem + ((uint32_t)(q * 32) << 16),
                   n_tok);
      }
      tc_fence_before();
    }
    // every partial tile of the cluster is in shared memory
    __syncwarp();
    if constexpr (kC > 1) cluster_sync(); else __syncthreads();
    if (have && !*abort_flag) {
      const int first = sub * s;
      if (kC == 1 || s == 1)
        store_unit<1>(sh, a, z, smem, row0, rows, u, q_end, gather, first, r);
      else if (kC == 2 || s == 2)
        store_unit<2>(sh, a, z, smem, row0, rows, u, q_end, gather, first, r);
      else if (kC == 3)
        store_unit<3>(sh, a, z, smem, row0, rows, u, q_end, gather, first, r);
      else if (kC == 4 || s == 4)
        store_unit<4>(sh, a, z, smem, row0, rows, u, q_end, gather, first, r);
      else
        store_unit<8>(sh, a, z, smem, row0, rows, u, q_end, gather, first, r);
    }
    // no CTA loads the next unit (by TMA, over a tile that ordinary stores
    // wrote), or leaves, while another reads its tile; after a wait that ran out
    // the CTAs still go through their units together
    fence_async_smem();
    __syncwarp();
    if constexpr (kC > 1) cluster_sync(); else __syncthreads();
    tc_fence_after();
    if (have) parity ^= 1u;
  }
  if (warp == 1) tmem_dealloc(tmem, C::kTmemCols);
}

// ---------------------------------------------------------------- expand
// out = v W + Z P, tiles of 128 output features x one token block.
struct ExpandMaps {
  CUtensorMap w;     // the projection's weights
  CUtensorMap v;     // token rows [T, K], boxes of 64 K x nb rows (pairs: nb / 2)
  CUtensorMap p;     // the adapters' matrices [n, R, M], boxes of rb rows x 128 features
  CUtensorMap z;     // Z [T, zc], boxes of 64 columns x nb rows (pairs: nb / 2)
};
struct ExpandArgs {
  int T, nb, K, M, n, R, rb, n_tt;   // nb: tokens per block, a multiple of 16
  __nv_bfloat16* out;       // [T, M]
  const void* plan;
  int* status;
  uint64_t call;            // the call's number where a kernel follows that starts early, or 0
};

// The weight operand of one stage and its `nb` token rows from row0 on.
template <bool kKMajor, bool kPair = false>
__device__ __forceinline__ void load_base(uint32_t st, uint32_t fb, const ExpandMaps& maps, int kb,
                                          int mt, int row0, uint64_t pol_w, uint64_t pol_v) {
  if constexpr (kKMajor)
    load_2d<kPair>(st, &maps.w, fb, kb * kK, mt * kM, pol_w);
  else
    load_3d<kPair>(st, &maps.w, fb, 0, kb * kK, mt * 2, pol_w);
  load_2d<kPair>(st + kABytes, &maps.v, fb, kb * kK, row0, pol_v);
}
// A block's entry list, copied to shared memory by the warp that uses it.
__device__ __forceinline__ void store_list(uint16_t* list, const uint4& v, int lane) {
  __syncwarp();
  reinterpret_cast<uint4*>(list)[lane] = v;
  __syncwarp();
}
__device__ __forceinline__ uint4 load_list(const BlockPlan* plan, int lane) {
  return reinterpret_cast<const uint4*>(plan->list)[lane];
}
// Stage j of the adapters' part, by the whole producer warp: 64 rank rows of
// the block's entries, in boxes of rb rows, each [2 feature atoms][rb rows][128
// bytes].
__device__ __forceinline__ void load_ext(uint32_t st, uint32_t fb, const ExpandMaps& maps,
                                         const ExpandArgs& a, const uint16_t* list, int q_all, int j,
                                         int mt, int nb, int row0, uint64_t pol_w, uint64_t pol_v,
                                         bool leader) {
  if (leader) {
    expect_tx(fb, (uint32_t)(kABytes + nb * kK * 2));
    load_2d(st + kABytes, &maps.z, fb, j * kK, row0, pol_v);
  }
  int e = j * kK / a.R, row = j * kK - e * a.R;
  for (int q = 0; q < kK; q += a.rb) {
    // past the last entry: an adapter that does not exist, read as zeros
    const int ad = j * kK + q < q_all ? (int)list[e] : a.n;
    if (leader) load_4d(st + q * (kM * 2), &maps.p, fb, 0, row, mt * 2, ad, pol_w);
    row += a.rb;
    if (row == a.R) {
      row = 0;
      ++e;
    }
  }
}
// One MMA of a CTA, or of a pair.
template <bool kPair>
__device__ __forceinline__ void mma_of(uint32_t tmem, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  if constexpr (kPair)
    mma_bf16_ss_pair(tmem, a, b, idesc, accumulate);
  else
    mma_bf16_ss(tmem, a, b, idesc, accumulate);
}
// The four MMAs of a stage at shared address a0 (one lane).
template <bool kKMajor, bool kPair = false>
__device__ __forceinline__ void mma_base(uint32_t tmem, uint32_t a0, uint32_t idesc, uint32_t first) {
  // MN-major weights: 64-feature atoms 8 KB apart, 16 K rows = 2 KB; K-major
  // operands: 8-row groups 1 KB apart, 16 K = 32 bytes
  const uint32_t la = kKMajor ? desc_lo(a0, 16) : desc_lo(a0, 8192);
  const uint32_t lb = desc_lo(a0 + kABytes, 16);
#pragma unroll
  for (int kk = 0; kk < kK / 16; ++kk)
    mma_of<kPair>(tmem, desc_of(la + (kKMajor ? 2 : 128) * kk, desc_hi(1024)),
                  desc_of(lb + 2 * kk, desc_hi(1024)), idesc, kk ? 1u : first);
}
// The same of an adapters' stage: MN-major boxes of rb rank rows.
template <bool kPair = false>
__device__ __forceinline__ void mma_ext(uint32_t tmem, uint32_t a0, uint32_t idesc, int rb) {
  const uint32_t lb = desc_lo(a0 + kABytes, 16);
  const uint32_t lbo = (uint32_t)rb * 128, hi = desc_hi(rb == 8 ? 2048u : 1024u);
#pragma unroll
  for (int kk = 0; kk < kK / 16; ++kk) {
    const uint32_t q = 16u * kk, in = q & (uint32_t)(rb - 1);   // rb: a power of two
    const uint32_t la = desc_lo(a0 + (q - in) * 256 + in * 128, lbo);
    mma_of<kPair>(tmem, desc_of(la, hi), desc_of(lb + 2 * kk, desc_hi(1024)), idesc, 1u);
  }
}
// A guard's pass over the 64 x 128 adapter weights of a stage: every
// token of the block is multiplied by every entry's rank rows, its own z or
// zero, so an infinity or NaN there would reach the other requests' tokens as
// 0 * inf.  It counts as zero instead and is reported.
// Slice `part` of `parts` of the stage.
__device__ __forceinline__ bool clear_nonfinite(uint8_t* st, int lane, int part, int parts) {
  // x * 0 + acc stays 0 for finite x and turns NaN for the others: two
  // elements per instruction (one warp checks a stage in 0.2 us; comparing the
  // exponents of every element took 1.75 us, longer than the stage's MMAs)
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
  __nv_bfloat162 acc[4] = {zero, zero, zero, zero};
#pragma unroll 8
  for (int i = part * 32 + lane; i < kABytes / 16; i += 32 * parts) {
    const uint4 v = reinterpret_cast<const uint4*>(st)[i];
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[c] = __hfma2(p[c], zero, acc[c]);
  }
  const __nv_bfloat162 any = __hadd2(__hadd2(acc[0], acc[1]), __hadd2(acc[2], acc[3]));
  const bool found = __hisnan(any.x) || __hisnan(any.y);
  if (!__any_sync(0xffffffffu, found)) return false;
  for (int i = part * 32 + lane; i < kABytes / 16; i += 32 * parts) {
    uint16_t* e = reinterpret_cast<uint16_t*>(st) + 8 * i;
    for (int c = 0; c < 8; ++c)
      if ((e[c] & 0x7f80u) == 0x7f80u) e[c] = 0;
  }
  fence_async_smem();   // the MMA reads what was written here
  return true;
}

// Few tiles: a cluster of kS CTAs per tile, each taking a share of the K
// stages; the partial tiles meet in shared memory and are added in rank order.
// Bound by reading W while there are few tokens (128 x 6144 x 16384, 128 tiles
// unsplit: 42 us for the whole call, 5.4 TB/s of its 230 MB, 0.80 of a copy's
// rate; shrink runs on the SMs that are left), and by the length of a tile's K
// loop otherwise (777 x 7168 x 2048 and 24 stages of adapters, 64 tiles split in
// two: 26 us of the call's 44 after shrink; the tensor pipe is busy 42% of it).
constexpr int kSplitOther = 1024;    // SplitShared
constexpr int kGuards = 5;           // all warps but the producer and the MMA warp
template <int kNB>
struct SplitCfg {
  static constexpr int kTmemCols = kNB < 32 ? 32 : kNB;
  static constexpr int kSmemBytes = kSmemMax;
  static constexpr int kRing = kSmemBytes - 1024 - kSplitOther;
  static_assert(kNB * kM * 4 <= kRing, "the partial fp32 tile is staged in the ring");
};
// Ring slots are handed out in the order of all stages (empty[slot]); arrivals
// are counted apart for the projection's stages (full) and the adapters'
// (loaded, then ready once the guard has passed them), each in its own order,
// since the guard follows the adapters' stages only.
struct SplitShared {
  uint64_t full[kMaxStages], empty[kMaxStages], loaded[kMaxStages], ready[kMaxStages];
  alignas(16) uint16_t list[kMaxEntries];
  uint64_t acc_full, drain;
  uint32_t tmem_base;
  int abort;
};

static_assert(sizeof(SplitShared) <= kSplitOther, "shared block");

template <int kNB, bool kKMajor, int kS>
__global__ void __launch_bounds__(kThreads, 1)
adapter_expand_split_kernel(const __grid_constant__ ExpandMaps maps, const ExpandArgs a) {
  using C = SplitCfg<kNB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  SplitShared* sh = reinterpret_cast<SplitShared*>(smem + C::kRing);
  const int stage_bytes = stage_bytes_of(a.nb), stages = ring_stages(stage_bytes, kSplitOther);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int rank = kS > 1 ? (int)cluster_ctarank() : 0;
  const int tile = (int)blockIdx.x / kS;
  const int tt = tile % a.n_tt, mt = tile / a.n_tt;
  const int row0 = tt * a.nb, rows = min(a.nb, a.T - row0);
  const int nk = a.K / kK;
  const int kb0 = nk * rank / kS, kb1 = nk * (rank + 1) / kS;
  const BlockPlan* plan = plan_of(a.plan, tt);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
      mbar_init(&sh->loaded[s], 1);
      mbar_init(&sh->ready[s], kGuards);
    }
    mbar_init(&sh->acc_full, 1);
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  volatile int* abort_flag = &sh->abort;
  const uint32_t full0 = smem_u32(sh->full), empty0 = smem_u32(sh->empty);
  const uint32_t ready0 = smem_u32(sh->ready), loaded0 = smem_u32(sh->loaded);
  const uint32_t sbase = smem_u32(smem);

  if (warp == 0) {
    // a weight tile read by one block is streamed past L2
    const uint64_t pol_w = a.n_tt == 1 ? policy_evict_first() : policy_evict_normal();
    const uint64_t pol_v = policy_evict_last();
    const bool leader = elect_lane();
    Place at(stages), base(stages), ext(stages);
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!(ok = wait_bar(empty0 + at.stage * 8, at.phase ^ 1u, abort_flag))) break;
      if (leader) {
        expect_tx(full0 + base.stage * 8, (uint32_t)stage_bytes);
        load_base<kKMajor>(sbase + at.stage * stage_bytes, full0 + base.stage * 8, maps, kb, mt, row0,
                           pol_w, pol_v);
      }
      at.next();
      base.next();
    }
    __syncwarp();
    pdl_wait();             // the plan and Z are complete
    if (a.call != 0 && blockIdx.x == 0 && leader) hand_over(a.status, a.call);
    pdl_trigger();
    fence_async_global();
    const int q_all = plan->n_ent * a.R;
    store_list(sh->list, load_list(plan, lane), lane);
    const int ne = (q_all + kK - 1) / kK;
    ok = __all_sync(0xffffffffu, ok);
    for (int j = ne * rank / kS; ok && j < ne * (rank + 1) / kS; ++j) {
      ok = wait_bar(empty0 + at.stage * 8, at.phase ^ 1u, abort_flag);
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      load_ext(sbase + at.stage * stage_bytes, loaded0 + ext.stage * 8, maps, a, sh->list, q_all, j,
               mt, a.nb, row0, pol_w, pol_v, leader);
      at.next();
      ext.next();
    }
    if (leader) {
      if (!ok) {
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailProducer);
        *abort_flag = 1;
      }
      if (mt == 0 && rank == 0 && plan->bad) set_status(a.status, MOE_ERR_INVALID_ARG);
      drain_loads(sh->full, stages, 0, base.count);
      drain_loads(sh->loaded, stages, 0, ext.count);
    }
  } else if (warp == 1) {
    const uint32_t id_base = idesc_bf16(kM, a.nb, /*a_mn=*/!kKMajor, false);
    const uint32_t id_ext = idesc_bf16(kM, a.nb, /*a_mn=*/true, false);
    const bool leader = elect_lane();
    Place at(stages), base(stages), ext(stages);
    bool ok = true;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!(ok = wait_bar(full0 + base.stage * 8, base.phase, abort_flag))) break;
      tc_fence_after();
      if (leader) {
        mma_base<kKMajor>(tmem, sbase + (uint32_t)(at.stage * stage_bytes), id_base,
                          kb > kb0 ? 1u : 0u);
        commit(empty0 + at.stage * 8);
      }
      at.next();
      base.next();
    }
    __syncwarp();
    pdl_wait();
    const int ne = (plan->n_ent * a.R + kK - 1) / kK;
    for (int j = ne * rank / kS; ok && j < ne * (rank + 1) / kS; ++j) {
      if (!(ok = wait_bar(ready0 + ext.stage * 8, ext.phase, abort_flag))) break;
      tc_fence_after();
      if (leader) {
        mma_ext(tmem, sbase + (uint32_t)(at.stage * stage_bytes), id_ext, a.rb);
        commit(empty0 + at.stage * 8);
      }
      at.next();
      ext.next();
    }
    if (leader) {
      if (!ok) {
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailMma);
        *abort_flag = 1;
      }
      mma_commit(&sh->acc_full);
      mma_commit(&sh->drain);
      if (!mbar_wait(&sh->drain, 0, nullptr, kWaitLimitNs))
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailDrain);
    }
  } else {   // the guards, warps 2 .. 6
    Place at(stages), ext(stages);
    for (int kb = kb0; kb < kb1; ++kb) at.next();
    pdl_wait();
    const int ne = (plan->n_ent * a.R + kK - 1) / kK;
    bool found = false;
    for (int j = ne * rank / kS; j < ne * (rank + 1) / kS; ++j) {
      const bool got = mbar_wait(&sh->loaded[ext.stage], ext.phase, abort_flag, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, got)) break;
      found |= clear_nonfinite(smem + at.stage * stage_bytes, lane, warp - 2, kGuards);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->ready[ext.stage]);
      at.next();
      ext.next();
    }
    if (found) set_status(a.status, MOE_ERR_NONFINITE);
  }
  if (warp >= 3) {
    const bool got = mbar_wait(&sh->acc_full, 0, abort_flag, kWaitLimitNs);
    tc_fence_after();
    if (__all_sync(0xffffffffu, got)) {
      // TMEM lane = feature, column = token
      const int q = warp & 3;
      stage_tile(reinterpret_cast<float*>(smem) + q * 32 + lane, tmem + ((uint32_t)(q * 32) << 16),
                 rows);
    }
    tc_fence_before();
  }
  __syncwarp();
  if constexpr (kS > 1) cluster_sync(); else __syncthreads();
  if (!*abort_flag) {
    const uint32_t mine = smem_u32(smem) + (uint32_t)lane * 16;
    constexpr int kStep = kS * (kThreads / 32);
#pragma unroll 4
    for (int t = rank * (kThreads / 32) + warp; t < rows; t += kStep) {
      float4 s;
      if constexpr (kS == 1)
        s = *reinterpret_cast<const float4*>(smem + t * (kM * 4) + lane * 16);
      else
        s = cluster_sum<kS>(mine + (uint32_t)t * (kM * 4));
      *reinterpret_cast<uint2*>(a.out + (size_t)(row0 + t) * a.M + mt * kM + 4 * lane) = pack4(s);
    }
  }
  __syncwarp();
  // no CTA leaves while another reads its shared memory
  if constexpr (kS > 1) cluster_sync(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Many tiles: persistent CTAs, two accumulators of 256 tokens in TMEM, so the
// epilogue of one tile runs under the main loop of the next.  Two CTAs of a
// cluster take neighbouring feature tiles of the same token block as one tile of
// 256 features (.cta_group::2): each stages its own weights and half of the
// block's rows, 32 KB a stage instead of 48 KB, in a ring of six stages instead of
// four.  Rank 0 issues the MMAs: its `full` counts both CTAs' loads, its `ready`
// both guards, its acc_empty both epilogues; each CTA's own `loaded` counts what
// its guard has to pass, and `empty` and acc_full are announced to both.
// Bound by the tensor cores: 4096 x 6144 x 10752 in 287 us by itself, 1.89 PFLOP/s
// (0.97 of cuBLAS's burst rate, tensor pipe 88%), about 300 in calls one after the
// other, under the power limit; the gradient's 8192 x 2048 x 7168 in 138 us, 1.74
// PFLOP/s (79%).  With each CTA staging the whole block's rows for an MMA of its own,
// sent to both, the two calls took 338 and 211 us; they take 320 and 207.
struct FullCfg {
  static constexpr int kNB = 256;
  static constexpr int kStgBytes = 16 * 32 * 2;            // 16 tokens x 32 features per warp
  static constexpr int kOther = 1024 + 4 * kStgBytes;      // FullShared, staging
  static constexpr int kSmemBytes = kSmemMax;
  static constexpr int kRing = kSmemBytes - 1024 - kOther;
};
struct FullShared {
  uint64_t full[kMaxStages], empty[kMaxStages], loaded[kMaxStages], ready[kMaxStages];   // as in SplitShared
  alignas(16) uint16_t list[kMaxEntries];
  uint64_t acc_full[2], acc_empty[2], drain;
  uint32_t tmem_base;
  int abort;
  uint32_t issued;   // rank 0: the projection's stages that rank 1 has loaded
};

static_assert(sizeof(FullShared) <= 1024, "shared block");

template <bool kKMajor>
__global__ void __launch_bounds__(kThreads, 1)
adapter_expand_kernel(const __grid_constant__ ExpandMaps maps, const ExpandArgs a) {
  // maps.v and maps.z: boxes of half a block's rows (a.nb: a multiple of 32, as the
  // pair's MMAs need)
  using C = FullCfg;
  constexpr int kNB = C::kNB;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  FullShared* sh = reinterpret_cast<FullShared*>(smem + C::kRing);
  const int half = a.nb / 2;   // a multiple of 16
  const int stage_bytes = stage_bytes_of(half), stages = ring_stages(stage_bytes, C::kOther);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int nk = a.K / kK;
  const int rank = (int)cluster_ctarank();
  const int n_mp = (a.M / kM + 1) / 2;      // pairs of feature tiles (the last may be half empty)
  const int total = a.n_tt * n_mp;
  const int first = (int)blockIdx.x >> 1, step = (int)gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
      mbar_init(&sh->loaded[s], 1);
      mbar_init(&sh->ready[s], 2);    // both CTAs' guards
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sh->acc_full[b], 1);
      mbar_init(&sh->acc_empty[b], 8);   // both CTAs' epilogue warps
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&sh->tmem_base, 2 * kNB);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();   // both CTAs' barriers are set before either signals the other's
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  volatile int* abort_flag = &sh->abort;
  int issued0 = -1;   // rank 0's producer: the projection's stages it has loaded
  // arrive on rank 0's barrier
  auto arrive_rank0 = [=](uint64_t* bar) {
    if (rank == 0) mbar_arrive(bar);
    else mbar_arrive_cluster(mapa_shared(smem_u32(bar), 0));
  };
  // a role that gives up stops the roles of both CTAs
  auto raise_abort = [=]() {
    *abort_flag = 1;
    st_cluster_u32(mapa_shared(smem_u32(&sh->abort), (uint32_t)(rank ^ 1)), 1u);
  };

  const uint32_t full0 = smem_u32(sh->full), empty0 = smem_u32(sh->empty);
  const uint32_t ready0 = smem_u32(sh->ready), loaded0 = smem_u32(sh->loaded);
  const uint32_t sbase = smem_u32(smem);

  if (warp == 0) {
    const uint64_t pol_w = policy_evict_normal(), pol_v = policy_evict_last();
    const bool leader = elect_lane();
    const uint32_t counted0 = mapa_shared(full0, 0);   // rank 0's barriers
    Place at(stages), base(stages), ext(stages);
    bool ok = true;
    for (int tile = first; ok && tile < total; tile += step) {
      // row0: of this CTA's half of the block
      const int tt = tile % a.n_tt, mt = 2 * (tile / a.n_tt) + rank, row0 = tt * a.nb + rank * half;
      const BlockPlan* plan = plan_of(a.plan, tt);
      // from the second tile on the plan is known to be complete: its words
      // are on their way while the projection's stages are loaded
      const bool later = tile != first;
      int n_ent = later ? plan->n_ent : 0;
      uint4 list = later ? load_list(plan, lane) : make_uint4(0, 0, 0, 0);
      for (int kb = 0; kb < nk; ++kb) {
        if (!(ok = wait_bar(empty0 + at.stage * 8, at.phase ^ 1u, abort_flag))) break;
        if (leader) {
          if (rank == 0) expect_tx(full0 + base.stage * 8, 2u * (uint32_t)stage_bytes);
          load_base<kKMajor, true>(sbase + at.stage * stage_bytes, counted0 + base.stage * 8, maps, kb,
                                   mt, row0, pol_w, pol_v);
        }
        at.next();
        base.next();
      }
      __syncwarp();
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (!later) {
        pdl_wait();             // the plan and Z are complete
        if (a.call != 0 && blockIdx.x == 0 && leader) hand_over(a.status, a.call);
        pdl_trigger();
        fence_async_global();
        n_ent = plan->n_ent;
        list = load_list(plan, lane);
      }
      const int q_all = n_ent * a.R;
      store_list(sh->list, list, lane);
      for (int j = 0; j * kK < q_all; ++j) {
        ok = wait_bar(empty0 + at.stage * 8, at.phase ^ 1u, abort_flag);
        if (!(ok = __all_sync(0xffffffffu, ok))) break;
        load_ext(sbase + at.stage * stage_bytes, loaded0 + ext.stage * 8, maps, a, sh->list, q_all, j,
                 mt, half, row0, pol_w, pol_v, leader);
        at.next();
        ext.next();
      }
      if (leader && mt == 0 && plan->bad) set_status(a.status, MOE_ERR_INVALID_ARG);
    }
    pdl_wait();
    if (leader) {
      if (!ok) {
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailProducer);
        raise_abort();
      }
      if (rank == 0) {
        issued0 = base.count;
        if (ok) drain_loads(sh->full, stages, 0, base.count);   // both CTAs' loads
      } else {
        st_cluster_u32(mapa_shared(smem_u32(&sh->issued), 0), (uint32_t)base.count);
      }
      drain_loads(sh->loaded, stages, 0, ext.count);
    }
  } else if (warp == 1 && rank == 0) {
    const uint32_t id_base = idesc_bf16(2 * kM, a.nb, /*a_mn=*/!kKMajor, false);
    const uint32_t id_ext = idesc_bf16(2 * kM, a.nb, /*a_mn=*/true, false);
    const bool leader = elect_lane();
    const uint32_t acc_full0 = smem_u32(sh->acc_full), acc_empty0 = smem_u32(sh->acc_empty);
    Place at(stages), base(stages), ext(stages);
    Place buf(2);
    bool ok = true;
    for (int tile = first; ok && tile < total; tile += step) {
      if (!(ok = wait_bar<true>(acc_empty0 + buf.stage * 8, buf.phase ^ 1u, abort_flag))) break;
      tc_fence_after();
      const uint32_t d = tmem + (uint32_t)(buf.stage * kNB);
      const BlockPlan* plan = plan_of(a.plan, tile % a.n_tt);
      const bool later = tile != first;
      int n_ent = later ? plan->n_ent : 0;   // early, as the producer's
      for (int kb = 0; kb < nk; ++kb) {
        if (!(ok = wait_bar<true>(full0 + base.stage * 8, base.phase, abort_flag))) break;
        tc_fence_after();
        if (leader) {
          mma_base<kKMajor, true>(d, sbase + (uint32_t)(at.stage * stage_bytes), id_base, kb ? 1u : 0u);
          commit_pair(empty0 + at.stage * 8);
        }
        at.next();
        base.next();
      }
      __syncwarp();
      if (!later) {
        pdl_wait();
        n_ent = plan->n_ent;
      }
      const int q_all = n_ent * a.R;
      for (int j = 0; ok && j * kK < q_all; ++j) {
        if (!(ok = wait_bar<true>(ready0 + ext.stage * 8, ext.phase, abort_flag))) break;
        tc_fence_after();
        if (leader) {
          mma_ext<true>(d, sbase + (uint32_t)(at.stage * stage_bytes), id_ext, a.rb);
          commit_pair(empty0 + at.stage * 8);
        }
        at.next();
        ext.next();
      }
      if (!(ok = __all_sync(0xffffffffu, ok))) break;
      if (leader) commit_pair(acc_full0 + buf.stage * 8);
      buf.next();
    }
    if (leader) {
      if (!ok) {
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailMma);
        raise_abort();
      }
      commit_pair(smem_u32(&sh->drain));
      if (!mbar_wait(&sh->drain, 0, nullptr, kWaitLimitNs))
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailDrain);
    }
  } else if (warp == 2) {
    Place at(stages), ext(stages);
    bool ok = true, found = false;
    for (int tile = first; ok && tile < total; tile += step) {
      for (int kb = 0; kb < nk; ++kb) at.next();
      pdl_wait();
      const int q_all = plan_of(a.plan, tile % a.n_tt)->n_ent * a.R;
      for (int j = 0; j * kK < q_all; ++j) {
        const bool got = mbar_wait(&sh->loaded[ext.stage], ext.phase, abort_flag, kWaitLimitNs);
        if (!(ok = __all_sync(0xffffffffu, got))) break;
        found |= clear_nonfinite(smem + at.stage * stage_bytes, lane, 0, 1);
        __syncwarp();
        if (lane == 0) arrive_rank0(&sh->ready[ext.stage]);
        at.next();
        ext.next();
      }
    }
    if (found) set_status(a.status, MOE_ERR_NONFINITE);
  } else if (warp >= 3) {
    const int q = warp & 3;
    __nv_bfloat16* stg =
        reinterpret_cast<__nv_bfloat16*>(smem + C::kRing + 1024 + (warp - 3) * C::kStgBytes);
    Place buf(2);
    pdl_wait();   // the limit of the first wait does not run while shrink does
    for (int tile = first; tile < total; tile += step) {
      const int tt = tile % a.n_tt, mt = 2 * (tile / a.n_tt) + rank;
      const int row0 = tt * a.nb, rows = min(a.nb, a.T - row0);
      const bool got = mbar_wait(&sh->acc_full[buf.stage], buf.phase, abort_flag, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, got)) break;
      tc_fence_after();
      const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16) + (uint32_t)(buf.stage * kNB);
      const bool real = mt * kM < a.M;   // not the second tile of a half-empty pair
      __nv_bfloat16* o = a.out + (size_t)row0 * a.M + mt * kM + q * 32;
      for (int c0 = 0; real && c0 < rows; c0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tb + c0, v);
        tmem_ld_wait();
        // 16 tokens x 32 features, then rows of 64 bytes by four lanes each
#pragma unroll
        for (int c = 0; c < 16; ++c)
          stg[c * 32 + lane] = __float2bfloat16_rn(__uint_as_float(v[c]));
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = 8 * h + (lane >> 2);
          const uint4 w = *reinterpret_cast<const uint4*>(stg + r * 32 + (lane & 3) * 8);
          if (c0 + r < rows)
            *reinterpret_cast<uint4*>(o + (size_t)(c0 + r) * a.M + (lane & 3) * 8) = w;
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_rank0(&sh->acc_empty[buf.stage]);
      buf.next();
    }
    // rank 1's last announcements have arrived: `drain` is the last of them
    if (rank == 1 && warp == 3 && lane == 0 && !mbar_wait(&sh->drain, 0, nullptr, kWaitLimitNs))
      set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailDrain);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();   // neither CTA leaves while the other may still write to it
  if (*abort_flag) {
    // a wait ran out: the loads on rank 0's `full` that no drain has waited for,
    // rank 1's beyond rank 0's among them, which nothing has announced
    if (rank == 0 && issued0 >= 0) {
      const int issued1 = (int)sh->issued;
      for (int i = issued0; i < issued1; ++i) expect_tx(full0 + (i % stages) * 8, (uint32_t)stage_bytes);
      drain_loads(sh->full, stages, 0, issued0 > issued1 ? issued0 : issued1);
    }
    __syncwarp();
    cluster_sync();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * kNB);
  }
}

// ------------------------------------------------------- weight gradients
// G[a][r][d] = sum over the tokens t of adapter a of Z[t, entry(a) R + r] V[t, d]:
// one cluster of kS CTAs per (adapter, 128 columns of V), K = the tokens of every
// 64-token group that holds one of adapter a, ascending, the groups dealt to the
// CTAs in turn; their tiles meet in shared memory and are added in rank order.
// Both gradients in one launch:
// dA from (x, dZ), then dB from (dy, Z).  Bound by reading x and dy once more:
// 8192 tokens, 7168 + 2048 columns, 8 adapters in 42 us by itself, 3.6 TB/s (the
// 576 CTAs are a round and a quarter of three per SM, of unequal lengths).  Adapters in
// random order share most 64-token groups, and each reads those it shares: 4096 x
// 4096 x 4096, 256 adapters of rank 16, 1.41 ms for the gradient call, 0.36 where
// their tokens stand together.
// It may start while the expand launch before it still runs, since nothing that
// expand writes is read: expand hands shrink's results over (see take_over), and
// this kernel does not end before expand.  In a captured launch, whose number would
// be the same in every replay, it waits for the end of expand before it reads (4 to 5
// us of a gradient call).
struct WgradMaps {
  CUtensorMap v[2];   // [T, D] as (64 features, tokens, D / 64)
  CUtensorMap z[2];   // [T, zc], boxes of 64 columns x 64 tokens
};
struct WgradArgs {
  int T, n, R, nb, n_tt;       // nb: tokens per block of the plan
  int D[2];
  const void* plan;
  const uint32_t* masks;       // [n_tt][256][8]: the tokens of every entry, as bits
  __nv_bfloat16* out[2];       // [n, R, D]
  int* status;
  uint64_t call;               // the number that expand hands shrink's results over with, or 0
};
// kCols: 64-column boxes of Z per stage (ranks up to 64, or up to 128).
template <int kCols>
struct WgradCfg {
  static constexpr int kStageBytes = kABytes + kCols * 64 * kK * 2;
  static constexpr int kStages = 3;      // three CTAs per SM at kCols = 1
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kSmemBytes = kRing + 1024 + 1024;
  static constexpr int kTmemCols = 64 * kCols;
};
static_assert(WgradCfg<1>::kRing >= 64 * kM * 4 && WgradCfg<2>::kRing >= 128 * kM * 4,
              "a CTA's fp32 tile is staged in the ring");
struct WgradShared {
  uint64_t full[4], empty[4], ready[4];
  uint64_t acc_full, drain;
  uint32_t tmem_base;
  int abort;
  volatile int stages;         // K stages in all, once the producer has issued them
  volatile uint32_t mask[4][2];   // the adapter's own tokens among the 64 of each stage
  volatile int rows[4];           // rows of the stage that belong to its block
};

template <int kCols, int kS>
__global__ void __launch_bounds__(kThreads, 1)
adapter_wgrad_kernel(const __grid_constant__ WgradMaps maps, const WgradArgs a) {
  using C = WgradCfg<kCols>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  WgradShared* sh = reinterpret_cast<WgradShared*>(smem + C::kRing);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int units0 = a.n * (a.D[0] / kM);
  const int rank = kS > 1 ? (int)cluster_ctarank() : 0;
  const int which = (int)blockIdx.x / kS < units0 ? 0 : 1;
  const int unit = (int)blockIdx.x / kS - (which ? units0 : 0);
  const int D = a.D[which], n_dt = D / kM;
  const int ad = unit / n_dt, d0 = (unit - ad * n_dt) * kM;
  const int N = (a.R + 15) & ~15;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
      mbar_init(&sh->ready[s], 1);
    }
    mbar_init(&sh->acc_full, 1);
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    sh->stages = -1;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem_base, C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem_base;
  volatile int* abort_flag = &sh->abort;
  if (a.call == 0) pdl_wait();
  if (warp == 0) {
    const uint64_t pol = policy_evict_normal();
    const bool leader = elect_lane();
    bool ok = a.call == 0 || take_over(a.status, a.call);
    ok = __all_sync(0xffffffffu, ok);
    fence_async_global();   // Z and dZ were written by ordinary stores
    const uint32_t empty0 = smem_u32(sh->empty), full0 = smem_u32(sh->full);
    const uint32_t sbase = smem_u32(smem);
    Place at(C::kStages);
    int group = 0;   // of the adapter's
    for (int tb = 0; ok && tb < a.n_tt; tb += 32) {
      // lane: block tb + lane, ad's entry in it and its tokens there
      int e = 0;
      uint4 m0 = make_uint4(0, 0, 0, 0), m1 = m0;
      if (tb + lane < a.n_tt) {
        const BlockPlan* p = plan_of(a.plan, tb + lane);
        const unsigned w = __ldcg(&p->bits[ad >> 5]);
        if ((w >> (ad & 31)) & 1u) {
          e = __popc(w & ((1u << (ad & 31)) - 1u));
          for (int i = 0; i < (ad >> 5); ++i) e += __popc(__ldcg(&p->bits[i]));
          const uint4* m =
              reinterpret_cast<const uint4*>(a.masks + ((size_t)(tb + lane) * kMaxEntries + e) * 8);
          m0 = __ldcg(m);
          m1 = __ldcg(m + 1);
        }
      }
      const uint32_t lo[4] = {m0.x, m0.z, m1.x, m1.z}, hi[4] = {m0.y, m0.w, m1.y, m1.w};
      const bool any = (m0.x | m0.y | m0.z | m0.w | m1.x | m1.y | m1.z | m1.w) != 0u;
      for (unsigned have = __ballot_sync(0xffffffffu, any); ok && have; have &= have - 1) {
        const int src = __ffs(have) - 1;
        const int eb = __shfl_sync(0xffffffffu, e, src);
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const uint32_t ml = __shfl_sync(0xffffffffu, lo[g], src);
          const uint32_t mh = __shfl_sync(0xffffffffu, hi[g], src);
          if (!ok || (ml | mh) == 0u) continue;   // no token of ad in this group
          if (kS > 1 && (group++ & (kS - 1)) != rank) continue;
          const int t0 = (tb + src) * a.nb + g * kK;
          ok = wait_bar(empty0 + at.stage * 8, at.phase ^ 1u, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          if (ok && leader) {
            const uint32_t st = sbase + at.stage * C::kStageBytes, fb = full0 + at.stage * 8;
            sh->mask[at.stage][0] = ml;
            sh->mask[at.stage][1] = mh;
            sh->rows[at.stage] = min(64, a.nb - g * kK);
            expect_tx(fb, C::kStageBytes);
            load_3d(st, &maps.v[which], fb, 0, t0, d0 >> 6, pol);
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              load_2d(st + kABytes + c * 64 * kK * 2, &maps.z[which], fb, eb * a.R + 64 * c, t0, pol);
          }
          if (ok) at.next();
        }
      }
    }
    if (lane == 0) {
      int from = 0;
      if (ok) ok = mbar_wait(&sh->empty[at.stage], at.phase ^ 1u, abort_flag, kWaitLimitNs);
      if (ok) {
        // the end of the list travels as one more stage without data; the
        // load that used this slot before has been read
        sh->stages = at.count;
        mbar_arrive(&sh->full[at.stage]);
        if (at.count >= C::kStages) from = at.count - C::kStages + 1;
      } else {
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailProducer);
        *abort_flag = 1;
      }
      drain_loads(sh->full, C::kStages, from, at.count);
    }
  } else if (warp == 1) {
    const uint32_t sbase = smem_u32(smem), ready0 = smem_u32(sh->ready);
    const uint32_t idesc = idesc_bf16(kM, N, true, true);
    const bool leader = elect_lane();
    Place at(C::kStages);
    bool ok = true;
    while (true) {
      if (!(ok = wait_bar(ready0 + at.stage * 8, at.phase, abort_flag))) break;
      if (sh->stages == at.count) break;
      tc_fence_after();
      const uint32_t a0 = sbase + (uint32_t)(at.stage * C::kStageBytes);
      const uint32_t la = desc_lo(a0, 8192), lb = desc_lo(a0 + kABytes, 8192);
      if (leader) {
#pragma unroll
        for (int kk = 0; kk < kK / 16; ++kk)
          mma_bf16_ss(tmem, desc_of(la + 128 * kk, desc_hi(1024)), desc_of(lb + 128 * kk, desc_hi(1024)),
                      idesc, (at.count || kk) ? 1u : 0u);
        mma_commit(&sh->empty[at.stage]);
      }
      at.next();
    }
    if (leader) {
      if (!ok) {
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailMma);
        *abort_flag = 1;
      }
      mma_commit(&sh->acc_full);
      mma_commit(&sh->drain);
      if (!mbar_wait(&sh->drain, 0, nullptr, kWaitLimitNs))
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailDrain);
    }
  } else if (warp == 2) {
    // Rows of V of other requests' tokens meet a zero of Z, which does not
    // stop an infinity or NaN in them: they are cleared.
    Place at(C::kStages);
    while (true) {
      const bool got = mbar_wait(&sh->full[at.stage], at.phase, abort_flag, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, got)) break;
      if (sh->stages == at.count) {
        if (lane == 0) mbar_arrive(&sh->ready[at.stage]);
        break;
      }
      uint8_t* st = smem + at.stage * C::kStageBytes;
      // rows past the block are another block's: what Z holds there, in this
      // entry's columns, is not defined
      for (int i = sh->rows[at.stage] * 8 + lane; i < 64 * 8; i += 32)
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          reinterpret_cast<uint4*>(st + kABytes + c * 64 * kK * 2)[i] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // two rows at a time: row r is 128 bytes in each of the two feature
        // atoms, a half warp's 16 vectors
        for (unsigned m = ~sh->mask[at.stage][h]; m;) {
          const int r0 = __ffs(m) - 1;
          m &= m - 1;
          const int r1 = m ? __ffs(m) - 1 : r0;
          m &= m - 1;
          const int r = 32 * h + (lane < 16 ? r0 : r1), v = lane & 15;
          *reinterpret_cast<uint4*>(st + (v >> 3) * 8192 + r * 128 + (v & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->ready[at.stage]);
      at.next();
    }
  } else {   // warps 3 to 6, TMEM lanes 32 (warp % 4) ..
    const bool got = mbar_wait(&sh->acc_full, 0, abort_flag, kWaitLimitNs);
    if (__all_sync(0xffffffffu, got) && !*abort_flag) {
      tc_fence_after();
      const bool none = sh->stages == 0;   // no token: a zero gradient
      const int q = warp & 3;
      __nv_bfloat16* o = a.out[which] + (size_t)ad * a.R * D + d0 + q * 32 + lane;
      float* st = reinterpret_cast<float*>(smem) + q * 32 + lane;   // the ring: every load was read
      for (int c0 = 0; c0 < a.R; c0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tmem + ((uint32_t)(q * 32) << 16) + c0, v);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          const float f = none ? 0.f : __uint_as_float(v[c]);
          if constexpr (kS > 1) {
            if (c0 + c < a.R) st[(c0 + c) * kM] = f;
          } else {
            if (c0 + c < a.R) o[(size_t)(c0 + c) * D] = __float2bfloat16_rn(f);
          }
        }
      }
    }
    tc_fence_before();
  }
  if constexpr (kS > 1) {
    __syncwarp();
    cluster_sync();
    if (!*abort_flag) {
      const uint32_t tile = smem_u32(smem);
      __nv_bfloat16* o = a.out[which] + (size_t)ad * a.R * D + d0;
      for (int i = rank * kThreads + (int)threadIdx.x; i < a.R * (kM / 4); i += kS * kThreads)
        *reinterpret_cast<uint2*>(o + (size_t)(i >> 5) * D + (i & 31) * 4) =
            pack4(cluster_sum<kS>(tile + (uint32_t)i * 16));
    }
    __syncwarp();
    cluster_sync();   // no CTA leaves while another reads its tile
  }
  __syncwarp();
  __syncthreads();
  pdl_wait();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// ------------------------------------------------------------------ host
using u64 = unsigned long long;

int rank_box(int R) {
  int rb = 8;
  while (rb < 64 && R % (2 * rb) == 0) rb *= 2;
  return rb;
}

// [rows, cols] bf16, boxes of 64 columns x box_rows rows.
bool map_rows(CUtensorMap* m, const void* p, int rows, int cols, int box_rows) {
  const u64 dims[2] = {(u64)cols, (u64)rows}, st[1] = {(u64)cols * 2};
  const unsigned box[2] = {64, (unsigned)box_rows};
  return make_tensor_map_bf16(m, p, 2, dims, st, box);
}
// [rows, cols] bf16 as (64 columns, rows, cols / 64): boxes of 64 rows x 128 columns.
bool map_atoms(CUtensorMap* m, const void* p, int rows, int cols) {
  const u64 dims[3] = {64, (u64)rows, (u64)cols / 64}, st[2] = {(u64)cols * 2, 128};
  const unsigned box[3] = {64, 64, 2};
  return make_tensor_map_bf16(m, p, 3, dims, st, box);
}
// [n, R, cols] bf16, boxes of 64 columns x rb rows of one adapter.
bool map_rank_rows(CUtensorMap* m, const void* p, int n, int R, int cols, int rb) {
  const u64 dims[3] = {(u64)cols, (u64)R, (u64)n}, st[2] = {(u64)cols * 2, (u64)R * cols * 2};
  const unsigned box[3] = {64, (unsigned)rb, 1};
  return make_tensor_map_bf16(m, p, 3, dims, st, box);
}
// The same as (64 columns, R, cols / 64, n): boxes of rb rows x 128 columns.
bool map_rank_atoms(CUtensorMap* m, const void* p, int n, int R, int cols, int rb) {
  const u64 dims[4] = {64, (u64)R, (u64)cols / 64, (u64)n};
  const u64 st[3] = {(u64)cols * 2, 128, (u64)R * cols * 2};
  const unsigned box[4] = {64, (unsigned)rb, 2, 1};
  return make_tensor_map_bf16(m, p, 4, dims, st, box);
}

// How an expand launch runs: persistent pairs of CTAs over `blocks` token blocks
// of nb tokens (split 0), or a tile per cluster of `split` CTAs.
struct ExpandPlan {
  int blocks, nb, split;
};
constexpr int kMoreBlocks = 7;   // token blocks tried beyond the fewest
// Tokens per block for a number of blocks: equal blocks, whole MMA columns (16,
// for a pair of CTAs 32).
int block_rows(int T, int blocks, int step = 16) {
  return ((T + blocks - 1) / blocks + step - 1) / step * step;
}
// The cheapest of both by a cost in microseconds: a K stage of 64 takes 0.3 us
// at 256 tokens (measured alone; its MMAs 0.27), in proportion to the tokens
// down to 0.15 us, a CTA's set-up, first loads and epilogue 6 us, which the
// persistent CTAs pay once, and joining s partial tiles of 256 tokens 6 + 3 log2 s
// us.  More blocks are more work for shrink, whose K stages (shrink_k in all) take
// 0.25 us per unit (777 x 7168 x 2048, 24 adapters of rank 64: 70 us in pairs, 44 in
// four blocks of clusters of two).  Over 379 calls (1 to 8192 tokens, H and N from 512
// to 16384, both directions) every form was timed: the choice is 1.9% slower than the
// best on average, at most 33% (1024 x 4096 x 1024, 16 adapters in random order: 29.8 us
// in pairs, 22.5 in clusters of two); without the join's cost and the limit on clusters
// of eight it would be 8% and 85% (1024 x 2048 x 1024: 21.2 us in clusters of four, 13.9
// in pairs; 128 x 7168 x 2048: 27.0 us in clusters of eight, 18.4 in clusters of four).
ExpandPlan plan_expand(int T, int K, int M, int n, int R, int shrink_k) {
  // sizes are asked for on hosts without a device too: there the count is 1
  const int nk = K / kK, sms = device_sm_count() > 1 ? device_sm_count() : 2;
  auto stage = [](int nb) { return nb > 128 ? 0.3 * nb / 256 : 0.15; };
  const int least = (T + 255) / 256;
  auto shrink = [&](int blocks, int nb) {
    const int units = ((n < nb ? n : nb) * R + kM - 1) / kM;
    return 0.25 * blocks * units * (shrink_k / kK) / sms;
  };
  ExpandPlan best{least, block_rows(T, least), 1};
  double cost = 1e30;
  for (int s = 1; s <= 8 && (s == 1 || nk / s >= 4); s *= 2) {
    const long long ctas = (long long)least * (M / kM) * s;
    // clusters of eight do not tile the GPU's processing clusters, and shrink's
    // take some of their places: above three quarters of the SMs the last of
    // them start when shrink ends
    const int room = s == 8 ? sms * 3 / 4 : sms;
    const double join = s == 1 ? 0.0 : best.nb / 256.0 * (s == 2 ? 9 : s == 4 ? 12 : 15);
    const double c = (double)((ctas + room - 1) / room) * (nk * stage(best.nb) / s + 6.0 + join) +
                     shrink(least, best.nb);
    if (c < cost) {
      cost = c;
      best.split = s;
    }
  }
  const int pairs = sms / 2;
  for (int blocks = least; blocks <= least + kMoreBlocks; ++blocks) {
    const int nb = block_rows(T, blocks, 32);
    if (nb <= 128) break;
    const long long tiles = (long long)blocks * ((M / kM + 1) / 2);
    const double c = (double)((tiles + pairs - 1) / pairs) * nk * stage(nb) + 6.0 + shrink(blocks, nb);
    if (c < cost) {
      cost = c;
      best = ExpandPlan{blocks, nb, 0};
    }
  }
  return best;
}

// Launches kKern as clusters of `cluster` CTAs.  Its shared-memory limit is raised
// once per device (half a microsecond a call otherwise), and again should a
// launch find it back at its default, as after a device reset.
template <auto kKern, typename... Args>
cudaError_t launch_cluster(dim3 grid, int cluster, int smem, bool pdl, cudaStream_t s,
                           Args&&... args) {
  static std::atomic<uint64_t> raised{0};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  const uint64_t bit = 1ull << (dev & 63);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  if (pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  if (raised.load(std::memory_order_relaxed) & bit) {
    err = cudaLaunchKernelEx(&cfg, kKern, args...);
    if (err != cudaErrorInvalidValue) return err;
    (void)cudaGetLastError();
  }
  err = cudaFuncSetAttribute(kKern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (err != cudaSuccess) return err;
  raised.fetch_or(bit, std::memory_order_relaxed);
  return cudaLaunchKernelEx(&cfg, kKern, args...);
}

template <int kNB>
cudaError_t launch_shrink_nb(int cluster, int gy, int jobs, const ShrinkMaps& m,
                             const ShrinkArgs& a, int n_tt, cudaStream_t s) {
  const dim3 grid(n_tt * cluster, gy, jobs);
  constexpr int smem = ShrinkCfg<kNB>::kSmemBytes;
  switch (cluster) {
    case 1: return launch_cluster<adapter_shrink_kernel<kNB, 1>>(grid, 1, smem, false, s, m, a);
    case 2: return launch_cluster<adapter_shrink_kernel<kNB, 2>>(grid, 2, smem, false, s, m, a);
    case 3: return launch_cluster<adapter_shrink_kernel<kNB, 3>>(grid, 3, smem, false, s, m, a);
    case 4: return launch_cluster<adapter_shrink_kernel<kNB, 4>>(grid, 4, smem, false, s, m, a);
    default: return launch_cluster<adapter_shrink_kernel<kNB, 8>>(grid, 8, smem, false, s, m, a);
  }
}

// One product: Z [T, zc] of the rows v [T, K] and the adapters' matrices P [n, R, K].
struct ShrinkJob {
  const __nv_bfloat16 *v, *P;
  int K;
  __nv_bfloat16* z;
};
// One or two of them, the first launch of a call.  `next` [n, R, next_cols]: the
// adapters' matrices that the expand launch reads; `v_map`: the map of the last
// job's rows, which is the expand launch's too if its boxes are equal.
cudaError_t launch_shrink(const AdapterSizes& z, int jobs, const ShrinkJob* job, const float* scale,
                          const int32_t* adapter_idx, void* plan, uint32_t* masks, int* status,
                          const __nv_bfloat16* next, int next_cols, CUtensorMap* v_map,
                          cudaStream_t s) {
  ShrinkMaps m;
  ShrinkArgs a{};
  const int rb = rank_box(z.R);
  int least = job[0].K;
  for (int i = 0; i < jobs; ++i) {
    if (!map_rank_rows(&m.p[i], job[i].P, z.n, z.R, job[i].K, rb) ||
        !map_rows(&m.v[i], job[i].v, z.T, job[i].K, z.nb))
      return cudaErrorInvalidValue;
    a.K[i] = job[i].K;
    a.rows[i] = job[i].v;
    a.z[i] = job[i].z;
    if (job[i].K < least) least = job[i].K;
  }
  *v_map = m.v[jobs - 1];
  // few blocks: the expand's tiles meet their adapters' rows cold, after the
  // projection's weights; with many blocks most of those reads hit L2 anyway
  const bool ahead = z.n_tt <= 4;
  a.T = z.T;
  a.nb = z.nb;
  a.n = z.n;
  a.R = z.R;
  a.rb = rb;
  a.zc = z.zc;
  a.next = ahead ? reinterpret_cast<const char*>(next) : nullptr;
  a.next_bytes = (long long)z.R * next_cols * 2;
  a.adapter_idx = adapter_idx;
  a.scale = scale;
  a.plan = plan;
  a.masks = masks;
  a.status = status;
  // as many clusters per block as the SMs take in one round and the block can
  // have units for; the CTAs share them out once they know its adapters
  int sms = device_sm_count();
  // One block beside an expand launch of fewer CTAs than SMs (a decode batch):
  // shrink keeps to the SMs that are left, since the expand's weights stream
  // meanwhile and a tile that waited for shrink's SMs came out last (8 of 128
  // tiles, 18 us late).
  if (z.n_tt == 1 && z.ctas < sms && sms - z.ctas >= 8) sms -= (int)z.ctas;
  // clusters of eight do not tile the GPU's processing clusters: more than
  // three quarters of the SMs' worth of them run in two rounds (16 blocks of
  // 4096 tokens: 30 us against 18)
  int cluster = 8;
  while (cluster > 1 && (z.n_tt * cluster > (cluster == 8 ? sms * 3 / 4 : sms) ||
                         least / kK / cluster < 4))
    cluster /= 2;
  // s of the kernel for as many units as a block can have
  auto share = [&](int c) {
    const int per = sms / (jobs * z.n_tt * c) * c;
    int n = c;
    while (n > 1 && z.zc / kM * n > per) n >>= 1;
    return n;
  };
  // three CTAs per unit where a power of two leaves a third of the SMs idle
  if (cluster > 3 && share(cluster) == 2 && share(3) == 3) cluster = 3;
  const int most = (z.zc / kM * 8 + cluster - 1) / cluster;   // up to eight CTAs per unit
  int gy = sms / (jobs * z.n_tt * cluster);
  gy = gy < 1 ? 1 : gy > most ? most : gy;
  if (z.nb <= 32) return launch_shrink_nb<32>(cluster, gy, jobs, m, a, z.n_tt, s);
  if (z.nb <= 64) return launch_shrink_nb<64>(cluster, gy, jobs, m, a, z.n_tt, s);
  if (z.nb <= 128) return launch_shrink_nb<128>(cluster, gy, jobs, m, a, z.n_tt, s);
  return launch_shrink_nb<256>(cluster, gy, jobs, m, a, z.n_tt, s);
}

template <int kNB, bool kKMajor>
cudaError_t launch_split_nb(int split, const ExpandMaps& m, const ExpandArgs& a, cudaStream_t s) {
  const dim3 grid((unsigned)(a.n_tt * (a.M / kM) * split));
  constexpr int smem = SplitCfg<kNB>::kSmemBytes;
  switch (split) {
    case 1:
      return launch_cluster<adapter_expand_split_kernel<kNB, kKMajor, 1>>(grid, 1, smem, true, s, m,
                            a);
    case 2:
      return launch_cluster<adapter_expand_split_kernel<kNB, kKMajor, 2>>(grid, 2, smem, true, s, m,
                            a);
    case 4:
      return launch_cluster<adapter_expand_split_kernel<kNB, kKMajor, 4>>(grid, 4, smem, true, s, m,
                            a);
    default:
      return launch_cluster<adapter_expand_split_kernel<kNB, kKMajor, 8>>(grid, 8, smem, true, s, m,
                            a);
  }
}

template <bool kKMajor>
cudaError_t launch_expand_t(int split, const ExpandMaps& m, const ExpandArgs& a, cudaStream_t s) {
  if (split == 0)
    return launch_cluster<adapter_expand_kernel<kKMajor>>(dim3(device_sm_count() / 2 * 2), 2,
                          FullCfg::kSmemBytes, true, s, m, a);
  if (a.nb <= 32) return launch_split_nb<32, kKMajor>(split, m, a, s);
  if (a.nb <= 64) return launch_split_nb<64, kKMajor>(split, m, a, s);
  if (a.nb <= 128) return launch_split_nb<128, kKMajor>(split, m, a, s);
  return launch_split_nb<256, kKMajor>(split, m, a, s);
}

// out [T, M] = v [T, K] W + Z P, with P [n, R, M]; W [K, M] or (k_major) [M, K].
cudaError_t launch_expand(const AdapterSizes& z, const CUtensorMap& v_map,
                          const __nv_bfloat16* v, const __nv_bfloat16* W,
                          bool k_major, const __nv_bfloat16* Z, const __nv_bfloat16* P, int K,
                          int M, const void* plan, __nv_bfloat16* out, int* status, uint64_t call,
                          cudaStream_t s) {
  ExpandMaps m;
  const int rb = rank_box(z.R);
  const int box = z.split == 0 ? z.nb / 2 : z.nb;
  if (!(k_major ? map_rows(&m.w, W, M, K, kM) : map_atoms(&m.w, W, K, M)) ||
      (box != z.nb && !map_rows(&m.v, v, z.T, K, box)) || !map_rank_atoms(&m.p, P, z.n, z.R, M, rb) ||
      !map_rows(&m.z, Z, z.T, z.zc, box))
    return cudaErrorInvalidValue;
  if (box == z.nb) m.v = v_map;
  const ExpandArgs a{z.T, z.nb, K, M, z.n, z.R, rb, z.n_tt, out, plan, status, call};
  return k_major ? launch_expand_t<true>(z.split, m, a, s)
                 : launch_expand_t<false>(z.split, m, a, s);
}

template <int kCols>
cudaError_t launch_wgrad(const AdapterSizes& z, const WgradMaps& m, const WgradArgs& a,
                         cudaStream_t s) {
  // Few units (one adapter trained alone: 72 of them with H 7168, N 2048) are
  // split until there are about two CTAs per SM, with 8 stages or more each.
  // 8192 tokens, one adapter, the whole gradient call: 228 us unsplit, 206, 200
  // and 212 us with 2, 4 and 8; two adapters 206, 202, 207 and 218 us; at eight a split
  // only adds (200 us, 207 with 2).  1000 tokens x 2048 x 1024, one adapter, replayed
  // from a graph: 31.5, 27.3, 26.1 and 25.5 us.
  const int units = z.n * ((z.H + z.N) / kM);
  const int groups = (z.T + kK - 1) / kK / z.n;   // of an adapter, on average
  int split = 1;
  while (split < 8 && units * split <= device_sm_count() && groups / split >= 16) split *= 2;
  const dim3 grid((unsigned)(units * split));
  constexpr int smem = WgradCfg<kCols>::kSmemBytes;
  switch (split) {
    case 1: return launch_cluster<adapter_wgrad_kernel<kCols, 1>>(grid, 1, smem, true, s, m, a);
    case 2: return launch_cluster<adapter_wgrad_kernel<kCols, 2>>(grid, 2, smem, true, s, m, a);
    case 4: return launch_cluster<adapter_wgrad_kernel<kCols, 4>>(grid, 4, smem, true, s, m, a);
    default: return launch_cluster<adapter_wgrad_kernel<kCols, 8>>(grid, 8, smem, true, s, m, a);
  }
}

}  // namespace

AdapterSizes adapter_sizes(int T, int H, int N, int n, int R, bool backward) {
  AdapterSizes z{};
  z.T = T;
  z.H = H;
  z.N = N;
  z.n = n;
  z.R = R;
  const ExpandPlan e = T > 0 ? (backward ? plan_expand(T, N, H, n, R, H + N)
                                       : plan_expand(T, H, N, n, R, H))
                             : ExpandPlan{0, 16, 1};
  z.nb = e.nb;
  z.n_tt = (T + e.nb - 1) / e.nb;
  z.split = e.split;
  // CTAs of the expand launch, of which one block's shrink keeps clear
  z.ctas = e.split ? (long long)z.n_tt * ((backward ? H : N) / kM) * e.split : device_sm_count();
  auto columns = [&](int nb) {
    const int entries = n < nb ? n : nb;
    return (int)align_up((size_t)entries * R, kM);
  };
  z.zc = columns(z.nb);
  // The layout has room for every launch shape that plan_expand may choose for T
  // tokens, and so for fewer tokens too: a caller sizes its workspace once, for its
  // largest batch.
  const size_t most_blocks = (size_t)(T + 255) / 256 + kMoreBlocks;
  const size_t z_bytes = (size_t)T * columns(T < 256 ? (T + 31) & ~31 : 256) * 2;
  size_t o = 1024;   // the status word
  z.plan = o;
  o += most_blocks * kAdapterPlanBytes;
  z.z = o;
  o = align_up(o + z_bytes, 1024);
  if (backward) {
    z.dz = o;
    o = align_up(o + z_bytes, 1024);
    z.masks = o;
    o = align_up(o + most_blocks * kMaxEntries * 8 * 4, 1024);
  }
  z.total = o;
  return z;
}

cudaError_t launch_adapter_project(const AdapterSizes& z, const __nv_bfloat16* x,
                                   const __nv_bfloat16* W, const __nv_bfloat16* A,
                                   const __nv_bfloat16* B, const float* scale,
                                   const int32_t* adapter_idx, __nv_bfloat16* y, void* ws,
                                   cudaStream_t s) {
  int* status = static_cast<int*>(ws);
  void* plan = ws_ptr<void>(ws, z.plan);
  __nv_bfloat16* Z = ws_ptr<__nv_bfloat16>(ws, z.z);
  const ShrinkJob job{x, A, z.H, Z};
  CUtensorMap v_map;
  const cudaError_t err =
      launch_shrink(z, 1, &job, scale, adapter_idx, plan, nullptr, status, B, z.N, &v_map, s);
  if (err != cudaSuccess) return err;
  return launch_expand(z, v_map, x, W, false, Z, B, z.H, z.N, plan, y, status, 0, s);
}

cudaError_t launch_adapter_backward(const AdapterSizes& z, const __nv_bfloat16* dy,
                                    const __nv_bfloat16* x, const __nv_bfloat16* W,
                                    const __nv_bfloat16* A, const __nv_bfloat16* B,
                                    const float* scale, const int32_t* adapter_idx,
                                    __nv_bfloat16* dx, __nv_bfloat16* dA, __nv_bfloat16* dB,
                                    void* ws, cudaStream_t s) {
  int* status = static_cast<int*>(ws);
  void* plan = ws_ptr<void>(ws, z.plan);
  __nv_bfloat16* Z = ws_ptr<__nv_bfloat16>(ws, z.z);
  __nv_bfloat16* dZ = ws_ptr<__nv_bfloat16>(ws, z.dz);
  uint32_t* masks = ws_ptr<uint32_t>(ws, z.masks);
  const ShrinkJob job[2] = {{x, A, z.H, Z}, {dy, B, z.N, dZ}};
  CUtensorMap v_map;
  uint64_t call = 0;
  cudaError_t err = launch_number(s, &call);
  if (err == cudaSuccess)
    err = launch_shrink(z, 2, job, scale, adapter_idx, plan, masks, status, A, z.H, &v_map, s);
  if (err == cudaSuccess)
    err = launch_expand(z, v_map, dy, W, true, dZ, A, z.N, z.H, plan, dx, status, call, s);
  if (err != cudaSuccess) return err;
  WgradMaps m;
  if (!map_atoms(&m.v[0], x, z.T, z.H) || !map_rows(&m.z[0], dZ, z.T, z.zc, 64) ||
      !map_atoms(&m.v[1], dy, z.T, z.N) || !map_rows(&m.z[1], Z, z.T, z.zc, 64))
    return cudaErrorInvalidValue;
  const WgradArgs a{z.T, z.n, z.R, z.nb, z.n_tt, {z.H, z.N}, plan, masks, {dA, dB}, status, call};
  return z.R > 64 ? launch_wgrad<2>(z, m, a, s) : launch_wgrad<1>(z, m, a, s);
}

}  // namespace moe
