// Low-rank adapters of many requests at once beside a shared projection:
//   y[t] = x[t] W + z[t] B_a,   z[t] = scale_a * (x[t] A_a^T),   a = adapter_idx[t]
// with W [H, N], A [n, R, H], B [n, R, N]; a token with adapter -1 has no z.
//
// A token block (kNB consecutive tokens) meets a few adapters, its entries (in
// ascending order).  The block's low-rank activations are kept expanded: row t
// of Z holds R columns per entry, zero but for the token's own one.  Then
//   shrink: Z = mask(x [A_a0; A_a1; ..]^T)   one product, masked in its epilogue
//   expand: y = [x | Z] [W; B_a0; B_a1; ..]  the K loop of x W runs on over Z
// so the adapters' part is a few more K stages of the projection's own tiles,
// whatever the order of the tokens: no rows are gathered or scattered, and a
// block of one request pays for one adapter.  dx = dy W^T + dz A is the same
// pair of products with the roles of A and B exchanged and W read K-major.
//   weight gradients: dA_a = dZ_a^T x, dB_a = Z_a^T dy over the blocks that meet a.
//
// All products run on the 5th-generation tensor cores (weights: the M operand,
// tokens: the N operand), bf16 in, fp32 accumulation in TMEM.  z is rounded to
// bf16 once, as an MMA operand; y, dx, dA and dB are rounded once on output.
#include <cuda.h>

#include "moe_common.cuh"
#include "ptx.cuh"

namespace moe {
namespace {

using namespace ptx;

constexpr int kM = 128;             // output features (or rank rows) per tile
constexpr int kK = 64;              // K per stage: one 128-byte swizzle atom
constexpr int kABytes = kM * kK * 2;
constexpr int kThreads = 192;       // producer, MMA and four epilogue warps
constexpr int kEpiThreads = 128;
constexpr int kMaxEntries = 256;    // adapters a token block can meet
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr int kSmemRing = 196608;

template <int kNB>
struct Cfg {
  static constexpr int kBBytes = kNB * kK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = kSmemRing / kStageBytes < 8 ? kSmemRing / kStageBytes : 8;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kTmemCols = kNB < 32 ? 32 : kNB;
  static constexpr int kSmemBytes = kRing + 1024 /* alignment */ + 4096 /* Shared */;
  static_assert(kNB * kM * 4 <= kRing, "the split's fp32 tile is staged in the ring");
};

struct Shared {
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t acc_full;
  uint64_t list_ready;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  int n_ent;
  unsigned bits[32];
  uint16_t list[kMaxEntries];   // the block's adapters, ascending
  int idx[256];                 // adapter of each token of the block, -1 for none
};
static_assert(sizeof(Shared) <= 4096, "shared block");

struct Maps {
  CUtensorMap w;     // expand: the projection's weights; shrink: the adapters' rank rows
  CUtensorMap x;     // token rows [T, K]
  CUtensorMap ext;   // expand: the adapters' other matrix
  CUtensorMap z;     // expand: Z
};

struct Args {
  int T, K, n, R, rb;       // rb: rank rows per TMA box, a power of two that divides R
  int n_tt, split;          // token blocks; CTAs of a cluster that share a tile's K
  const int32_t* adapter_idx;
  const float* scale;
  __nv_bfloat16* out;       // expand: y [T, ld]; shrink: Z [T, ld]
  int ld;
  int32_t* plan;            // shrink: [n_tt][kPlanInts], the blocks' adapters as bits
  int* status;
};
constexpr int kPlanInts = 32;

__device__ __forceinline__ void fence_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
__device__ __forceinline__ void epi_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// The adapters that token block tt meets (the four epilogue warps).
__device__ __forceinline__ void build_list(Shared* sh, const Args& a, int row0, int rows,
                                           bool report) {
  const int tid = threadIdx.x - 64, lane = threadIdx.x & 31;
  if (tid < 32) sh->bits[tid] = 0u;
  epi_sync();
  bool bad = false;
  for (int i = tid; i < rows; i += kEpiThreads) {
    int e = __ldg(a.adapter_idx + row0 + i);
    if (e < 0 || e >= a.n) {
      bad |= e != -1;
      e = -1;
    } else {
      atomicOr(&sh->bits[e >> 5], 1u << (e & 31));
    }
    sh->idx[i] = e;
  }
  if (bad && report) set_status(a.status, MOE_ERR_INVALID_ARG);
  epi_sync();
  if (tid < 32) {
    unsigned w = sh->bits[lane];
    const int c = __popc(w);
    int incl = c;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, off);
      if (lane >= off) incl += u;
    }
    int at = incl - c;
    for (; w; w &= w - 1) sh->list[at++] = (uint16_t)(lane * 32 + __ffs(w) - 1);
    if (lane == 31) sh->n_ent = incl;
  }
  epi_sync();
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ uint2 pack4(float4 v) {
  const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
  uint2 r;
  r.x = *reinterpret_cast<const uint32_t*>(&lo);
  r.y = *reinterpret_cast<const uint32_t*>(&hi);
  return r;
}

// One tile (128 output features x kNB tokens) per cluster of `split` CTAs, each
// taking a contiguous share of the K stages; the partial tiles meet in
// shared memory and are added in rank order.
template <int kNB, bool kShrink, bool kKMajor>
__global__ void __launch_bounds__(kThreads, 1)
adapter_gemm_kernel(const __grid_constant__ Maps maps, const Args a) {
  using C = Cfg<kNB>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  Shared* sh = reinterpret_cast<Shared*>(smem + C::kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.split;
  const int rank = S > 1 ? (int)cluster_ctarank() : 0;
  const int tile = (int)blockIdx.x / S;
  const int tt = tile % a.n_tt, mt = tile / a.n_tt;
  const int row0 = tt * kNB;
  const int rows = min(kNB, a.T - row0);
  const int nk = a.K / kK;
  const int kb0 = (int)((long long)nk * rank / S), kb1 = (int)((long long)nk * (rank + 1) / S);

  if (kShrink) pdl_trigger();
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
    }
    mbar_init(&sh->acc_full, 1);
    mbar_init(&sh->list_ready, 1);
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

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol_w = a.n_tt == 1 ? policy_evict_first() : policy_evict_normal();
      const uint64_t pol_x = policy_evict_last();
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      bool ok = true;
      auto next = [&]() {
        ++issued;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      };
      if (kShrink) ok = mbar_wait(&sh->list_ready, 0, abort_flag, kWaitLimitNs);
      for (int kb = kb0; ok && kb < kb1; ++kb) {
        if (!(ok = mbar_wait(&sh->empty[stage], phase ^ 1u, abort_flag, kWaitLimitNs))) break;
        uint8_t* sA = smem + stage * C::kStageBytes;
        uint64_t* fb = &sh->full[stage];
        const int k0 = kb * kK;
        if constexpr (kShrink) {
          // the rank rows of this tile's entries; rows past the last entry keep
          // what the stage held (their products are dropped by the epilogue)
          const int q_end = min(kM, sh->n_ent * a.R - mt * kM);
          if (q_end <= 0) break;
          mbar_arrive_expect_tx(fb, (uint32_t)(q_end * kK * 2 + C::kBBytes));
          for (int q = 0; q < q_end; q += a.rb) {
            const int qq = mt * kM + q, e = qq / a.R;
            tma_load_3d(sA + q * (kK * 2), &maps.w, fb, k0, qq - e * a.R, sh->list[e], pol_w);
          }
        } else {
          mbar_arrive_expect_tx(fb, C::kStageBytes);
          if constexpr (kKMajor)
            tma_load_2d(sA, &maps.w, fb, k0, mt * kM, pol_w);
          else
            tma_load_3d(sA, &maps.w, fb, 0, k0, mt * 2, pol_w);
        }
        tma_load_2d(sA + kABytes, &maps.x, fb, k0, row0, pol_x);
        next();
      }
      if constexpr (!kShrink) {
        // K goes on over Z and the entries' rank rows
        if (ok) ok = mbar_wait(&sh->list_ready, 0, abort_flag, kWaitLimitNs);
        pdl_wait();             // Z is complete
        fence_async_global();
        const int q_all = ok ? sh->n_ent * a.R : 0;
        const int ne = (q_all + kK - 1) / kK;
        const int j0 = ne * rank / S, j1 = ne * (rank + 1) / S;
        for (int j = j0; ok && j < j1; ++j) {
          if (!(ok = mbar_wait(&sh->empty[stage], phase ^ 1u, abort_flag, kWaitLimitNs))) break;
          uint8_t* sA = smem + stage * C::kStageBytes;
          uint64_t* fb = &sh->full[stage];
          mbar_arrive_expect_tx(fb, C::kStageBytes);
          for (int q = 0; q < kK; q += a.rb) {
            const int qq = j * kK + q;
            const int e = qq / a.R;
            // past the last entry: an adapter that does not exist, read as zeros
            const int ad = qq < q_all ? (int)sh->list[e] : a.n;
            tma_load_4d(sA + q * (kM * 2), &maps.ext, fb, 0, qq - e * a.R, mt * 2, ad, pol_w);
          }
          tma_load_2d(sA + kABytes, &maps.z, fb, j * kK, row0, pol_x);
          next();
        }
      }
      if (!ok) {
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailProducer);
        *abort_flag = 1;
      }
      // no TMA write may land after the CTA exits: wait for the last loads
      for (int i = issued > C::kStages ? issued - C::kStages : 0; i < issued; ++i)
        mbar_wait(&sh->full[i % C::kStages], (uint32_t)((i / C::kStages) & 1), nullptr,
                  kWaitLimitNs);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t sbase = smem_u32(smem);
      int stage = 0;
      uint32_t phase = 0, acc = 0;
      bool ok = true;
      constexpr uint32_t kIdesc = idesc_bf16(kM, kNB, /*a_mn=*/!kShrink && !kKMajor, false);
      constexpr uint32_t kIdescExt = idesc_bf16(kM, kNB, /*a_mn=*/true, false);
      int kend = kb1;
      if (kShrink) {
        ok = mbar_wait(&sh->list_ready, 0, abort_flag, kWaitLimitNs);
        if (sh->n_ent * a.R <= mt * kM) kend = kb0;   // no such tile
      }
      auto advance = [&]() {
        mma_commit(&sh->empty[stage]);
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      };
      for (int kb = kb0; ok && kb < kend; ++kb) {
        if (!(ok = mbar_wait(&sh->full[stage], phase, abort_flag, kWaitLimitNs))) break;
        tc_fence_after();
        const uint32_t a0 = sbase + (uint32_t)(stage * C::kStageBytes), b0 = a0 + kABytes;
#pragma unroll
        for (int kk = 0; kk < kK / 16; ++kk) {
          // MN-major weights: 64-feature atoms 8 KB apart, 16 K rows = 2 KB;
          // K-major operands: 8-row groups 1 KB apart, 16 K = 32 bytes
          const uint64_t da = (kShrink || kKMajor) ? sdesc_sw128(a0 + kk * 32, 16, 1024)
                                                   : sdesc_sw128(a0 + kk * 2048, 8192, 1024);
          mma_bf16_ss(tmem, da, sdesc_sw128(b0 + kk * 32, 16, 1024), kIdesc, acc);
          acc = 1u;
        }
        advance();
      }
      if constexpr (!kShrink) {
        if (ok) ok = mbar_wait(&sh->list_ready, 0, abort_flag, kWaitLimitNs);
        const int ne = ok ? (sh->n_ent * a.R + kK - 1) / kK : 0;
        const int j0 = ne * rank / S, j1 = ne * (rank + 1) / S;
        // boxes of rb rank rows, each [2 feature atoms][rb rows][128 bytes]
        const uint32_t lbo = (uint32_t)a.rb * 128, sbo = a.rb == 8 ? 2048u : 1024u;
        for (int j = j0; ok && j < j1; ++j) {
          if (!(ok = mbar_wait(&sh->full[stage], phase, abort_flag, kWaitLimitNs))) break;
          tc_fence_after();
          const uint32_t a0 = sbase + (uint32_t)(stage * C::kStageBytes), b0 = a0 + kABytes;
#pragma unroll
          for (int kk = 0; kk < kK / 16; ++kk) {
            const uint32_t q = 16u * kk, box = q / a.rb;
            const uint32_t at = a0 + box * (uint32_t)a.rb * 256 + (q - box * a.rb) * 128;
            mma_bf16_ss(tmem, sdesc_sw128(at, lbo, sbo), sdesc_sw128(b0 + kk * 32, 16, 1024),
                        kIdescExt, acc);
            acc = 1u;
          }
          advance();
        }
      }
      if (!ok) {
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailMma);
        *abort_flag = 1;
      }
      mma_commit(&sh->acc_full);
      mma_commit(&sh->drain);
      if (!mbar_wait(&sh->drain, 0, nullptr, kWaitLimitNs))
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailDrain);
    }
  } else {
    build_list(sh, a, row0, rows, mt == 0 && rank == 0);
    if (threadIdx.x == 64) mbar_arrive(&sh->list_ready);
    if (kShrink && mt == 0 && rank == 0 && warp == 2)
      a.plan[(size_t)tt * kPlanInts + lane] = (int)sh->bits[lane];
  }
  bool have = true;
  if (warp >= 2) {
    // a shrink tile past the block's entries has nothing to store
    if (kShrink) have = sh->n_ent * a.R > mt * kM;
    const bool got = mbar_wait(&sh->acc_full, 0, abort_flag, kWaitLimitNs);
    if (!__all_sync(0xffffffffu, got)) have = false;
    tc_fence_after();
    if (have) {
      // TMEM lane = feature, column = token
      const int q = warp & 3;
      const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16);
      const int f = q * 32 + lane;
      for (int c0 = 0; c0 < rows; c0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tb + c0, v);
        tmem_ld_wait();
        float* st = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int c = 0; c < 16; ++c) st[(c0 + c) * kM + f] = __uint_as_float(v[c]);
      }
    }
    tc_fence_before();
  }
  // every partial tile of the cluster is in shared memory
  __syncwarp();
  if (S > 1) cluster_sync(); else __syncthreads();
  if (warp >= 2 && have && !*abort_flag) {
    const int w = warp - 2;
    const uint32_t mine = smem_u32(smem);
    for (int t = rank * 4 + w; t < rows; t += 4 * S) {
      const uint32_t at = mine + (uint32_t)(t * kM * 4 + lane * 16);
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      if (S == 1) {
        s = *reinterpret_cast<const float4*>(smem + t * kM * 4 + lane * 16);
      } else {
        for (int r = 0; r < S; ++r) {
          const float4 p = ld_cluster_f4(mapa_shared(at, (uint32_t)r));
          s.x += p.x;
          s.y += p.y;
          s.z += p.z;
          s.w += p.w;
        }
      }
      if constexpr (kShrink) {
        const int e = (mt * kM + 4 * lane) / a.R;   // the entry of these four rank rows
        const int own = sh->idx[t];
        if (own >= 0 && e < sh->n_ent && sh->list[e] == own) {
          const float f = __ldg(a.scale + own);
          s = make_float4(s.x * f, s.y * f, s.z * f, s.w * f);
        } else {
          s = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
      *reinterpret_cast<uint2*>(a.out + (size_t)(row0 + t) * a.ld + mt * kM + 4 * lane) = pack4(s);
    }
  }
  __syncwarp();
  tc_fence_before();
  // no CTA leaves while another reads its shared memory
  if (S > 1) cluster_sync(); else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// dG[a][r][d] = sum over the tokens t of adapter a of Z[t, entry(a) R + r] V[t, d]:
// one CTA per (adapter, 128 features of V), K = the tokens of every 64-token
// group that holds one of adapter a, in ascending order.
struct WgradMaps {
  CUtensorMap v;   // [T, D] as (64 features, tokens, D / 64)
  CUtensorMap z;   // [T, zc], boxes of 64 columns x 64 tokens
};
struct WgradArgs {
  int T, D, n, R, nb, n_tt;    // nb: tokens per block of the plan
  const int32_t* adapter_idx;
  const int32_t* plan;
  __nv_bfloat16* out;          // [n, R, D]
  int* status;
};
struct WgradCfg {
  static constexpr int kBBytes = 2 * 64 * kK * 2;   // up to 128 rank columns
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 6;
  static constexpr int kRing = kStages * kStageBytes;
  static constexpr int kSmemBytes = kRing + 1024 + 1024;
  static constexpr int kTmemCols = 128;
};
struct WgradShared {
  uint64_t full[WgradCfg::kStages];
  uint64_t empty[WgradCfg::kStages];
  uint64_t acc_full;
  uint64_t drain;
  uint32_t tmem_base;
  int abort;
  volatile int stages;   // K stages in all, written by the producer before its last arrival
};

__global__ void __launch_bounds__(kThreads, 1)
adapter_wgrad_kernel(const __grid_constant__ WgradMaps maps, const WgradArgs a) {
  using C = WgradCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  WgradShared* sh = reinterpret_cast<WgradShared*>(smem + C::kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n_dt = a.D / kM;
  const int ad = (int)blockIdx.x / n_dt, d0 = ((int)blockIdx.x % n_dt) * kM;
  const int n_cols = a.R > 64 ? 2 : 1;                   // 64-column boxes of Z
  const int N = (a.R + 15) & ~15;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], 1);
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
  if (warp == 0) {
    const uint64_t pol = policy_evict_normal();
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int tt = 0; ok && tt < a.n_tt; ++tt) {
      // the block's entries below `ad`, and whether ad is one
      const unsigned w = (unsigned)__ldg(a.plan + (size_t)tt * kPlanInts + lane);
      const unsigned mine = __shfl_sync(0xffffffffu, w, ad >> 5);
      if (!((mine >> (ad & 31)) & 1u)) continue;
      const unsigned below = lane < (ad >> 5) ? w : lane == (ad >> 5) ? w & ((1u << (ad & 31)) - 1u)
                                                                      : 0u;
      const int e = (int)__reduce_add_sync(0xffffffffu, (unsigned)__popc(below));
      const int t_end = min(a.T, (tt + 1) * a.nb);
      for (int t0 = tt * a.nb; ok && t0 < t_end; t0 += kK) {
        const int ta = t0 + lane, tb = ta + 32;
        const bool any = (ta < t_end && __ldg(a.adapter_idx + ta) == ad) ||
                         (tb < t_end && __ldg(a.adapter_idx + tb) == ad);
        if (!__any_sync(0xffffffffu, any)) continue;
        int got = 1;
        if (lane == 0) {
          got = mbar_wait(&sh->empty[stage], phase ^ 1u, abort_flag, kWaitLimitNs);
          if (got) {
            uint8_t* sA = smem + stage * C::kStageBytes;
            uint64_t* fb = &sh->full[stage];
            mbar_arrive_expect_tx(fb, (uint32_t)(kABytes + n_cols * 64 * kK * 2));
            tma_load_3d(sA, &maps.v, fb, 0, t0, d0 >> 6, pol);
            for (int c = 0; c < n_cols; ++c)
              tma_load_2d(sA + kABytes + c * 64 * kK * 2, &maps.z, fb, e * a.R + 64 * c, t0, pol);
          }
        }
        ok = __shfl_sync(0xffffffffu, got, 0) != 0;
        if (!ok) break;
        ++issued;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (lane == 0) {
      int last = issued > C::kStages ? issued - C::kStages : 0;   // first load not known to be read
      if (ok) ok = mbar_wait(&sh->empty[stage], phase ^ 1u, abort_flag, kWaitLimitNs);
      if (ok) {
        // the end of the list travels as one more stage without data; the
        // load that used this slot before has been read
        sh->stages = issued;
        mbar_arrive(&sh->full[stage]);
        if (issued >= C::kStages) last = issued - C::kStages + 1;
      } else {
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailProducer);
        *abort_flag = 1;
      }
      for (int i = last; i < issued; ++i)
        mbar_wait(&sh->full[i % C::kStages], (uint32_t)((i / C::kStages) & 1), nullptr,
                  kWaitLimitNs);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t sbase = smem_u32(smem);
      const uint32_t idesc = idesc_bf16(kM, N, true, true);
      int stage = 0, done = 0;
      uint32_t phase = 0;
      bool ok = true;
      while (true) {
        if (!(ok = mbar_wait(&sh->full[stage], phase, abort_flag, kWaitLimitNs))) break;
        if (sh->stages == done) break;
        tc_fence_after();
        const uint32_t a0 = sbase + (uint32_t)(stage * C::kStageBytes), b0 = a0 + kABytes;
#pragma unroll
        for (int kk = 0; kk < kK / 16; ++kk)
          mma_bf16_ss(tmem, sdesc_sw128(a0 + kk * 2048, 8192, 1024),
                      sdesc_sw128(b0 + kk * 2048, 8192, 1024), idesc, (done || kk) ? 1u : 0u);
        mma_commit(&sh->empty[stage]);
        ++done;
        if (++stage == C::kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) {
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailMma);
        *abort_flag = 1;
      }
      mma_commit(&sh->acc_full);
      mma_commit(&sh->drain);
      if (!mbar_wait(&sh->drain, 0, nullptr, kWaitLimitNs))
        set_status(a.status, MOE_ERR_TIMEOUT, kWaitDetailDrain);
    }
  } else {
    const bool got = mbar_wait(&sh->acc_full, 0, abort_flag, kWaitLimitNs);
    if (__all_sync(0xffffffffu, got) && !*abort_flag) {
      tc_fence_after();
      const bool none = sh->stages == 0;   // no token: a zero gradient
      const int q = warp & 3;
      const uint32_t tb = tmem + ((uint32_t)(q * 32) << 16);
      __nv_bfloat16* o = a.out + (size_t)ad * a.R * a.D + d0 + q * 32 + lane;
      for (int c0 = 0; c0 < a.R; c0 += 16) {
        uint32_t v[16];
        tmem_ld_32x32b_x16(tb + c0, v);
        tmem_ld_wait();
#pragma unroll
        for (int c = 0; c < 16; ++c)
          if (c0 + c < a.R)
            o[(size_t)(c0 + c) * a.D] =
                none ? __float2bfloat16_rn(0.f) : __float2bfloat16_rn(__uint_as_float(v[c]));
      }
    }
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
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

// CTAs per tile: the split of K (1, 2, 4 or 8 ways) that needs the fewest
// rounds of the SMs per share of the work, at least four stages each.
int split_of(long long tiles, int nk) {
  int best = 1;
  double cost = 1e30;
  for (int s = 1; s <= 8 && (s == 1 || nk / s >= 4); s *= 2) {
    const long long rounds = (tiles * s + device_sm_count() - 1) / device_sm_count();
    const double c = (double)rounds / s + 0.02 * s;   // joining more parts costs more
    if (c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

template <int kNB, bool kShrink, bool kKMajor>
cudaError_t launch_gemm(const Maps& maps, const Args& args, long long tiles, bool pdl,
                        cudaStream_t s) {
  using C = Cfg<kNB>;
  auto kern = adapter_gemm_kernel<kNB, kShrink, kKMajor>;
  cudaError_t err =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * args.split));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (args.split > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = args.split;
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
  return cudaLaunchKernelEx(&cfg, kern, maps, args);
}

template <bool kShrink, bool kKMajor>
cudaError_t launch_gemm_nb(int nb, const Maps& maps, const Args& args, long long tiles, bool pdl,
                           cudaStream_t s) {
  switch (nb) {
    case 32: return launch_gemm<32, kShrink, kKMajor>(maps, args, tiles, pdl, s);
    case 64: return launch_gemm<64, kShrink, kKMajor>(maps, args, tiles, pdl, s);
    case 128: return launch_gemm<128, kShrink, kKMajor>(maps, args, tiles, pdl, s);
    default: return launch_gemm<256, kShrink, kKMajor>(maps, args, tiles, pdl, s);
  }
}

// Z of the rows v [T, D] and the adapters' matrices P [n, R, D].
cudaError_t launch_shrink(const AdapterSizes& z, const __nv_bfloat16* v, const __nv_bfloat16* P,
                          int D, const float* scale, const int32_t* adapter_idx, int32_t* plan,
                          __nv_bfloat16* Z, int* status, cudaStream_t s) {
  const int nb = z.nb, rb = rank_box(z.R);
  Maps m;
  if (!map_rank_rows(&m.w, P, z.n, z.R, D, rb) || !map_rows(&m.x, v, z.T, D, nb))
    return cudaErrorInvalidValue;
  m.ext = m.z = m.x;
  Args a{z.T, D, z.n, z.R, rb, z.n_tt, 1, adapter_idx, scale, Z, z.zc, plan, status};
  const long long tiles = (long long)z.n_tt * (z.zc / kM);
  a.split = split_of(z.n_tt, D / kK);
  return launch_gemm_nb<true, true>(nb, m, a, tiles, false, s);
}

// out [T, M] = v [T, K] W + Z P, with P [n, R, M]; W [K, M] or (k_major) [M, K].
cudaError_t launch_expand(const AdapterSizes& z, const __nv_bfloat16* v, const __nv_bfloat16* W,
                          bool k_major, const __nv_bfloat16* Z, const __nv_bfloat16* P, int K,
                          int M, const int32_t* adapter_idx, __nv_bfloat16* out, int* status,
                          cudaStream_t s) {
  const int nb = z.nb, rb = rank_box(z.R);
  Maps m;
  if (!(k_major ? map_rows(&m.w, W, M, K, kM) : map_atoms(&m.w, W, K, M)) ||
      !map_rows(&m.x, v, z.T, K, nb) || !map_rank_atoms(&m.ext, P, z.n, z.R, M, rb) ||
      !map_rows(&m.z, Z, z.T, z.zc, nb))
    return cudaErrorInvalidValue;
  Args a{z.T, K, z.n, z.R, rb, z.n_tt, 1, adapter_idx, nullptr, out, M, nullptr, status};
  const long long tiles = (long long)z.n_tt * (M / kM);
  a.split = split_of(tiles, K / kK);
  return k_major ? launch_gemm_nb<false, true>(nb, m, a, tiles, true, s)
                 : launch_gemm_nb<false, false>(nb, m, a, tiles, true, s);
}

// G [n, R, D] = the adapters' sums of Z^T v.
cudaError_t launch_wgrad(const AdapterSizes& z, const __nv_bfloat16* v, const __nv_bfloat16* Z,
                         int D, const int32_t* adapter_idx, const int32_t* plan, __nv_bfloat16* G,
                         int* status, cudaStream_t s) {
  WgradMaps m;
  if (!map_atoms(&m.v, v, z.T, D) || !map_rows(&m.z, Z, z.T, z.zc, 64))
    return cudaErrorInvalidValue;
  const WgradArgs a{z.T, D, z.n, z.R, z.nb, z.n_tt, adapter_idx, plan, G, status};
  cudaError_t err = cudaFuncSetAttribute(
      adapter_wgrad_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, WgradCfg::kSmemBytes);
  if (err != cudaSuccess) return err;
  return launch_k(adapter_wgrad_kernel, dim3((unsigned)(z.n * (D / kM))), dim3(kThreads),
                  WgradCfg::kSmemBytes, s, false, m, a);
}

}  // namespace

AdapterSizes adapter_sizes(int T, int H, int N, int n, int R) {
  AdapterSizes z{};
  z.T = T;
  z.H = H;
  z.N = N;
  z.n = n;
  z.R = R;
  z.nb = T <= 32 ? 32 : T <= 64 ? 64 : T <= 128 ? 128 : 256;
  z.n_tt = (T + z.nb - 1) / z.nb;
  const int entries = n < z.nb ? n : z.nb;
  z.zc = (int)align_up((size_t)entries * R, kM);
  size_t o = 256;   // the status word
  z.plan = o;
  o = align_up(o + (size_t)z.n_tt * kPlanInts * 4, 1024);
  z.z = o;
  o = align_up(o + (size_t)T * z.zc * 2, 1024);
  z.total = o;
  z.dz = o;
  z.total_backward = align_up(o + (size_t)T * z.zc * 2, 1024);
  return z;
}

cudaError_t launch_adapter_project(const AdapterSizes& z, const __nv_bfloat16* x,
                                   const __nv_bfloat16* W, const __nv_bfloat16* A,
                                   const __nv_bfloat16* B, const float* scale,
                                   const int32_t* adapter_idx, __nv_bfloat16* y, void* ws,
                                   cudaStream_t s) {
  int* status = static_cast<int*>(ws);
  __nv_bfloat16* Z = ws_ptr<__nv_bfloat16>(ws, z.z);
  cudaError_t err = launch_shrink(z, x, A, z.H, scale, adapter_idx, ws_ptr<int32_t>(ws, z.plan), Z,
                                  status, s);
  if (err != cudaSuccess) return err;
  return launch_expand(z, x, W, false, Z, B, z.H, z.N, adapter_idx, y, status, s);
}

cudaError_t launch_adapter_backward(const AdapterSizes& z, const __nv_bfloat16* dy,
                                    const __nv_bfloat16* x, const __nv_bfloat16* W,
                                    const __nv_bfloat16* A, const __nv_bfloat16* B,
                                    const float* scale, const int32_t* adapter_idx,
                                    __nv_bfloat16* dx, __nv_bfloat16* dA, __nv_bfloat16* dB,
                                    void* ws, cudaStream_t s) {
  int* status = static_cast<int*>(ws);
  int32_t* plan = ws_ptr<int32_t>(ws, z.plan);
  __nv_bfloat16* Z = ws_ptr<__nv_bfloat16>(ws, z.z);
  __nv_bfloat16* dZ = ws_ptr<__nv_bfloat16>(ws, z.dz);
  cudaError_t err = launch_shrink(z, x, A, z.H, scale, adapter_idx, plan, Z, status, s);
  if (err == cudaSuccess)
    err = launch_shrink(z, dy, B, z.N, scale, adapter_idx, plan, dZ, status, s);
  if (err == cudaSuccess)
    err = launch_expand(z, dy, W, true, dZ, A, z.N, z.H, adapter_idx, dx, status, s);
  if (err == cudaSuccess) err = launch_wgrad(z, x, dZ, z.H, adapter_idx, plan, dA, status, s);
  if (err == cudaSuccess) err = launch_wgrad(z, dy, Z, z.N, adapter_idx, plan, dB, status, s);
  return err;
}

}  // namespace moe
