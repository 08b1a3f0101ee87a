// attention_backward.cuh -- backward pass of full-sequence attention per head
// on tcgen05 tensor cores (sm_100a), recomputing the probabilities from the
// row log-sum-exp of the forward pass.
//
// Per (batch, head), for queries i and keys k below N:
//   P_ik = exp(scale q_i.k_k - lse_i)        delta_i = sum_c dO_ic O_ic
//   dV_k = sum_i P_ik dO_i                   dP_ik   = dO_i . v_k
//   dS_ik = P_ik (dP_ik - delta_i)
//   dQ_i = scale sum_k dS_ik k_k             dK_k    = scale sum_i dS_ik q_i
// Five products of N x N x D per head, so the tensor core is the floor.
//
// Three kernels: one computes delta and puts the statistics in the form the
// tiles want; the main one makes a single pass over the N x N scores; the
// last one rounds dQ, which the main kernel leaves in fp32.
//
// Main kernel: a CTA owns 128 keys of one head and walks the 128-query tiles
// in order.  K, V stay in shared memory, dK and dV in tensor memory; scores
// are computed transposed (keys in the lanes), so that P^T and dS^T, rounded
// to bf16 for the tensor core as the forward pass rounds P, are the A operands
// of dV += P^T dO and dK += dS^T Q straight from tensor memory.  Only dQ needs
// dS the other way round: it goes through shared memory, one 32 KB tile.
// Roles (16 warps):
//   warps 0-7   elementwise: warpgroup h takes queries 64h .. 64h+63 of a tile,
//               one thread per key
//   warps 8-11  dQ tiles from tensor memory to global fp32 accumulators
//   warp 12     TMA producer
//   warp 13     TMEM allocator and the single MMA-issuing thread
// Tensor memory (512 columns): R0 = 0..127 holds S^T, then P^T; R1 = 128..255
// holds dP^T, then dS^T, then dQ; dV at 256, dK at 256 + D.  Per query tile j
// the MMA thread issues
//   dP_j,  dV += P_j^T dO_j,  S_{j+1},  dK += dS_j^T Q_j,  dQ_j
// so that the elementwise work on dS_j runs beside dV and S_{j+1}, and the
// exponentials of S_{j+1} beside dK, dQ and the dQ tile's way out of R1.
//
// dQ_i sums over all keys, i.e. over CTAs.  The key tiles of a head add into
// the fp32 accumulators in key order, each tile passing a per-(query tile,
// 32 rows) turn counter on to the next: results repeat bit for bit and depend
// neither on timing nor on P.  A CTA takes its key tile from a ticket, so the
// tile before it is always held by a CTA that already runs and no wait can
// close a cycle; consecutive key tiles of a head run about one query tile
// apart.  Up to kMaxPartial key tiles, where that stagger would be felt, each
// key tile writes a partial dQ of its own and the last kernel adds them in
// the same order (so both give the same bits).
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <type_traits>

#include "attention.cuh"
#include "projection.cuh"
#include "sm100.cuh"

namespace sp {

struct AttnBwdParams {
  int32_t N, Np, H, B;   // true tokens, token slots, heads, batch
  int32_t hsplit;        // heads per tensor-map "batch" slot (Hl or H)
  int32_t T;             // tiles of 128 tokens
  int32_t BH;            // B * H
  int32_t head_group;    // heads whose key tiles run at the same time
  int32_t partial;       // every key tile has its own dQ buffer
  int32_t nl_split;      // as in AttnParams
  float scale, scale_log2e;
  const uint8_t *q, *k, *v, *o, *dout;
  const float *lse;      // [B][H][Np]
  __nv_bfloat16 *dq, *dk, *dv;
  int64_t row_el, batch_el, rank_el;  // strides of tokens, slots, rank slabs
  // workspace
  float *dq_acc;         // [BH][T][key tiles or 1][4 x 32 rows][D / 32][8][32 rows] float4
  float *ndelta;         // [BH][128 T]: -delta, 0 past N
  float *nlse2;          // [BH][128 T]: -lse * log2(e), -inf past N
  uint32_t *turn;        // [BH][T][4]: key tiles that added their part
  uint32_t *ticket;      // [2]: next work item, abort
  int32_t *status;
};

// Element offset of token `t` of head bh's row in q, k, v, o and their gradients.
__device__ __forceinline__ int64_t bwd_row(const AttnBwdParams &p, int bh, int t, int D) {
  const int b = bh / p.H, hg = bh - b * p.H;
  const int hs = hg / p.hsplit, head = hg - hs * p.hsplit;
  int64_t off;
  if (p.nl_split) {
    const int rk = t / p.nl_split;
    off = rk * p.rank_el + b * p.batch_el + (t - rk * p.nl_split) * p.row_el;
  } else {
    off = (static_cast<int64_t>(hs) * p.B + b) * p.batch_el + t * p.row_el;
  }
  return off + static_cast<int64_t>(head) * D;
}

// One block per (query tile, head): delta in fp32 from 16-byte loads, D / 8
// lanes a row, and the turn counters' zeros.
template <int D>
__global__ void __launch_bounds__(256) attention_delta_kernel(const __grid_constant__ AttnBwdParams p) {
  constexpr int kLanes = D / 8, kRows = 256 / kLanes;
  const int qt = blockIdx.x % p.T, bh = blockIdx.x / p.T;
  if (threadIdx.x < 4) p.turn[blockIdx.x * 4ll + threadIdx.x] = 0u;
  if (blockIdx.x == 0 && threadIdx.x < 2) p.ticket[threadIdx.x] = 0u;
  const int c = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  uint4 vo[128 / kRows], vd[128 / kRows];
#pragma unroll
  for (int i = 0; i < 128 / kRows; ++i) {
    const int t = qt * 128 + r0 + i * kRows;
    vo[i] = vd[i] = make_uint4(0u, 0u, 0u, 0u);
    if (t < p.N) {
      const int64_t off = bwd_row(p, bh, t, D) * 2 + c * 16;
      vo[i] = ld_global_nc_v4(p.o + off);
      vd[i] = ld_global_nc_v4(p.dout + off);
    }
  }
#pragma unroll
  for (int i = 0; i < 128 / kRows; ++i) {
    const uint32_t a[4] = {vo[i].x, vo[i].y, vo[i].z, vo[i].w};
    const uint32_t b[4] = {vd[i].x, vd[i].y, vd[i].z, vd[i].w};
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      s = fmaf(__uint_as_float(a[e] << 16), __uint_as_float(b[e] << 16), s);
      s = fmaf(__uint_as_float(a[e] & 0xffff0000u), __uint_as_float(b[e] & 0xffff0000u), s);
    }
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const int t = qt * 128 + r0 + i * kRows;
    if (c == 0) {
      const int64_t w = static_cast<int64_t>(bh) * p.T * 128 + t;
      p.ndelta[w] = -s;
      // rows without a key (lse = -inf) get no gradient: probability 2^-inf
      const float l = t < p.N ? p.lse[static_cast<int64_t>(bh) * p.Np + t] : -INFINITY;
      p.nlse2[w] = l == -INFINITY ? -INFINITY : -l * 1.4426950408889634f;
    }
  }
}

template <int D>
struct AttnBwdCfg {
  static constexpr int kHalves = D / 64;              // 128-byte column blocks per row
  static constexpr int kBlockBytes = 128 * 128;
  static constexpr int kTileBytes = kHalves * kBlockBytes;
  static constexpr int kOffK = 0;
  static constexpr int kOffV = kTileBytes;
  static constexpr int kOffQ = 2 * kTileBytes;        // two stages
  static constexpr int kOffDO = 4 * kTileBytes;       // one stage
  static constexpr int kOffDS = 5 * kTileBytes;       // [2 query halves][128 keys][128 bytes]
  // dQ on its way out: [4 warps][2 buffers][32 rows x 32 columns] fp32
  static constexpr int kChunkBytes = 32 * 32 * 4;
  static constexpr int kOffOut = kOffDS + 2 * kBlockBytes;
  static constexpr int kOffStat = kOffOut + 8 * kChunkBytes;  // [2 stages][nlse2, ndelta][128]
  static constexpr int kOffBar = kOffStat + 2 * 2 * 512;
  static constexpr int kNumBar = 20;
  static constexpr int kOffMisc = kOffBar + kNumBar * 8;  // TMEM base, abort flag, work item
  static constexpr int kSmemBytes = kOffMisc + 16;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  static constexpr int kThreads = 512;
  static constexpr uint32_t kColR1 = 128;
  static constexpr uint32_t kColDV = 256;
  static constexpr uint32_t kColDK = 256 + D;
  static constexpr uint32_t kTmemCols = 512;
};

// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ uint32_t ld_acquire_gpu_u32(const uint32_t *p) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void st_release_gpu_u32(uint32_t *p, uint32_t v) {
  asm volatile("st.release.gpu.global.u32 [%0], %1;" ::"l"(p), "r"(v) : "memory");
}
// Bulk copies shared -> global in this thread's groups (16-byte aligned,
// multiples of 16 bytes): a plain store, or fp32 adds performed in L2.
__device__ __forceinline__ void bulk_store(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;"
               ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_add_f32(void *dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.reduce.async.bulk.global.shared::cta.bulk_group.add.f32 [%0], [%1], %2;"
               ::"l"(dst), "r"(src), "r"(bytes)
               : "memory");
}
// Waits until at most kPending of this thread's bulk groups are incomplete.
template <int kPending>
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group %0;" ::"n"(kPending) : "memory");
}

// Matrix products of bf16 operands whose descriptors differ from one another
// only in the low word: high word = stride 1,024 bytes, version 1, 128-byte
// swizzle (make_sdesc_sw128).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);

__device__ __forceinline__ void umma_ss_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void umma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
      ::"r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "n"(kDescHi)
      : "memory");
}

// Untiled bulk copy global -> shared (16-byte aligned, multiple of 16 bytes).
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

template <int D>
__global__ void __launch_bounds__(512, 1)
attention_backward_kernel(const __grid_constant__ CUtensorMap tmQ,
                          const __grid_constant__ CUtensorMap tmK,
                          const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ CUtensorMap tmDO,
                          const __grid_constant__ AttnBwdParams p) {
  using C = AttnBwdCfg<D>;
  // The swizzled tiles want 1,024-byte alignment, which the dynamic shared
  // memory of a kernel without static shared memory has; there is no room
  // to round up, so it is checked.
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = p.T;

  const uint32_t bar_k = sbase + C::kOffBar, bar_v = bar_k + 8;
  const uint32_t bar_q_full = bar_k + 16, bar_q_empty = bar_k + 32;
  const uint32_t bar_do_full = bar_k + 48, bar_dv = bar_k + 56;
  const uint32_t bar_s = bar_k + 80;
  const uint32_t bar_p = bar_k + 88;    // [2]
  const uint32_t bar_dp = bar_k + 104;
  const uint32_t bar_ds = bar_k + 112;  // [2]
  const uint32_t bar_dq = bar_k + 128, bar_dq_free = bar_k + 136;
  const uint32_t bar_acc = bar_k + 144, bar_drain = bar_k + 152;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);
  volatile int *work_slot = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 8);

  if ((sbase & 1023u) != 0) {  // uniform
    if (threadIdx.x == 0) atomicExch(p.status, kStatusTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    *work_slot = static_cast<int>(atomicAdd(p.ticket, 1u));
    mbar_init(bar_k, 1);
    mbar_init(bar_v, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_q_full + 8 * s, 1);
      mbar_init(bar_q_empty + 8 * s, 1);
      mbar_init(bar_p + 8 * s, 128);
      mbar_init(bar_ds + 8 * s, 128);
    }
    mbar_init(bar_do_full, 1);
    mbar_init(bar_dv, 1);
    mbar_init(bar_s, 1);
    mbar_init(bar_dp, 1);
    mbar_init(bar_dq, 1);
    mbar_init(bar_dq_free, 128);
    mbar_init(bar_acc, 1);
    mbar_init(bar_drain, 2);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 13) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // Work item -> (head, key tile): the heads of a group take turns, so a
  // group's Q, dO and dQ stay in L2 while its key tiles run.
  const int work = *work_slot;
  const int gsize = p.head_group * T;
  const int g = work / gsize, gr = work - g * gsize;
  const int gh = min(p.head_group, p.BH - g * p.head_group);
  const int n = gr / gh;
  const int bh = g * p.head_group + (gr - n * gh);
  const int b = bh / p.H, hg = bh - b * p.H;
  const int k0 = n * 128;

  bool ok = true;
  int issued = 0;  // loads of query tiles issued: Q_0, dO_0, Q_1, ...
  bool kv_issued = false;
  bool leader = false;   // the lanes of warps 13 and 14 that issue MMAs
  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;");
    if (warp == 12) {
      // -------------------------------------------------------------- producer
      const int hs = hg / p.hsplit;
      const int map_head = hg - hs * p.hsplit, map_batch = hs * p.B + b;
      const uint64_t pol_kv = policy_evict_first(), pol_q = policy_evict_last();
      const int nl = p.nl_split;
      if (lane == 0) {
        prefetch_tmap(&tmQ);
        prefetch_tmap(&tmK);
        prefetch_tmap(&tmV);
        prefetch_tmap(&tmDO);
      }
      // Rank-major layout: a tile that crosses a shard boundary, or holds
      // padding slots of the last shard, is copied row by row.
      auto tma_ok = [&](int t0) {
        if (nl == 0) return true;
        const int r0 = t0 / nl;
        return t0 - r0 * nl + 128 <= nl && t0 + 128 <= p.N;
      };
      // The swizzled layout of copy_rows, inlined: the call's registers would
      // not be held to this warpgroup's share.
      auto copy_tile = [&](const uint8_t *base, uint32_t dst, int t0) {
        constexpr int kChunks = D / 8;
#pragma unroll 2
        for (int idx = lane; idx < 128 * kChunks; idx += 32) {
          const int r = idx / kChunks, cc = idx % kChunks;
          uint4 val = make_uint4(0u, 0u, 0u, 0u);
          if (t0 + r < p.N) val = ld_global_nc_v4(base + bwd_row(p, bh, t0 + r, D) * 2 + cc * 16);
          st_shared_v4(dst + (cc >> 3) * C::kBlockBytes + r * 128 + (((cc & 7) ^ (r & 7)) << 4), val);
        }
        fence_proxy_async_smem();
      };
      // Loads one tile (and, with stat, the tile's statistics) on barrier bar.
      auto load = [&](const CUtensorMap *m, const uint8_t *base, uint32_t dst, uint32_t bar, int t0,
                      uint64_t pol, bool stat, uint32_t stat_dst) {
        const bool tma = tma_ok(t0);
        if (!tma) copy_tile(base, dst, t0);
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, (tma ? C::kTileBytes : 0) + (stat ? 1024u : 0u));
          if (tma) {
            for (int h = 0; h < C::kHalves; ++h) {
              if (nl == 0) {
                tma_load_4d(dst + h * C::kBlockBytes, m, bar, h * 64, map_head, t0, map_batch, pol);
              } else {
                const int r0 = t0 / nl;
                tma_load_5d(dst + h * C::kBlockBytes, m, bar, h * 64, map_head, t0 - r0 * nl, b, r0,
                            pol);
              }
            }
          }
          if (stat) {
            const int64_t w = static_cast<int64_t>(bh) * T * 128 + t0;
            bulk_load(stat_dst, p.nlse2 + w, 512, bar);
            bulk_load(stat_dst + 512, p.ndelta + w, 512, bar);
          }
        }
        __syncwarp();
      };
      load(&tmK, p.k, sbase + C::kOffK, bar_k, k0, pol_kv, false, 0);
      for (int j = 0; j < T && ok; ++j) {
        const int s = j & 1;
        const uint32_t free_par = ((j >> 1) & 1) ^ 1;
        bool got = mbar_wait(bar_q_empty + 8 * s, free_par, abort_flag, kWaitLimitNs);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        load(&tmQ, p.q, sbase + C::kOffQ + s * C::kTileBytes, bar_q_full + 8 * s, j * 128, pol_q,
             true, sbase + C::kOffStat + s * 1024);
        issued = 2 * j + 1;
        if (j == 0) {
          load(&tmV, p.v, sbase + C::kOffV, bar_v, k0, pol_kv, false, 0);
          kv_issued = true;
        }
        // dV and dP of the tile before have both read the stage
        got = j == 0 || (mbar_wait(bar_dv, s ^ 1, abort_flag, kWaitLimitNs) &&
                         mbar_wait(bar_dp, s ^ 1, abort_flag, kWaitLimitNs));
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        load(&tmDO, p.dout, sbase + C::kOffDO, bar_do_full, j * 128, pol_q, false, 0);
        issued = 2 * j + 2;
      }
    } else if (warp < 15) {
      // -------------------------------------------------------------- MMA issue
      // Warp 13 issues the products that feed the elementwise warps, warp 14
      // those that they feed.  The whole warp runs the loop and one elected
      // lane issues, and every address is a constant or warp-uniform (the
      // kernel holds all of tensor memory, so its base is 0), so that
      // descriptors stay in uniform registers.
      constexpr uint32_t idesc_kk = make_idesc_bf16(128, 128, 0, 0);  // S^T, dP^T
      constexpr uint32_t idesc_acc = make_idesc_bf16(128, D, 0, 1);   // dV, dK
      constexpr uint32_t idesc_dq = make_idesc_bf16(128, D, 1, 1);    // dQ
      // Low descriptor words: start address / 16 and the leading offset.
      constexpr uint32_t kLboK = 1u << 16;                               // K-major: unused
      constexpr uint32_t kLboMn = static_cast<uint32_t>(C::kBlockBytes >> 4) << 16;
      constexpr uint32_t R0 = 0, R1 = C::kColR1;
      constexpr uint32_t kStage = C::kTileBytes >> 4;
      const uint32_t s16 = sbase >> 4;
      const uint32_t aK = s16 + (C::kOffK >> 4), aV = s16 + (C::kOffV >> 4);
      const uint32_t aQ = s16 + (C::kOffQ >> 4), aDO = s16 + (C::kOffDO >> 4);
      const uint32_t aDS = s16 + (C::kOffDS >> 4);
      leader = elect_one();
      auto wait = [&](uint32_t bar, uint32_t parity) {
        const bool got = mbar_wait(bar, parity, abort_flag, kWaitLimitNs);
        tc_fence_after();
        return __all_sync(0xffffffffu, got) != 0;
      };
      ok = tmem == 0;
      if (warp == 13) {
        // [128 x 128] = A B^T over D, both operands K-major
        auto issue_kk = [&](uint32_t d, uint32_t a, uint32_t bb) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (((kk >> 2) * C::kBlockBytes + (kk & 3) * 32) >> 4) | kLboK;
            umma_ss_lo(d, a + off, bb + off, idesc_kk, kk > 0 ? 1u : 0u);
          }
        };
        ok = ok && wait(bar_k, 0);
        for (int j = 0; j < T && ok; ++j) {
          const int s = j & 1;
          // R0 is free when dV has used the tile's probabilities
          ok = wait(bar_q_full + 8 * s, (j >> 1) & 1) && (j == 0 || wait(bar_dv, s ^ 1));
          if (!ok) break;
          if (leader) {
            issue_kk(R0, aK, aQ + s * kStage);
            umma_commit(bar_s);
          }
          // R1 is free when the tile's dQ has left it
          ok = (j > 0 || wait(bar_v, 0)) && wait(bar_do_full, s) &&
               (j == 0 || wait(bar_dq_free, s ^ 1));
          if (!ok) break;
          if (leader) {
            issue_kk(R1, aV, aDO);
            umma_commit(bar_dp);
          }
        }
      } else {
        // acc += X[:, 64h .. 64h+63] B[64h .. 64h+63, :], X in tensor memory
        auto issue_acc = [&](uint32_t d, uint32_t x, uint32_t bb, int h, uint32_t more) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_ts_lo(d, x + 64 * h + 8 * k, bb + ((((4 * h + k) * 16 * 128) >> 4) | kLboMn),
                       idesc_acc, (h == 0 && k == 0) ? more : 1u);
        };
        for (int j = 0; j < T && ok; ++j) {
          const int s = j & 1;
          const uint32_t par = s, more = j > 0 ? 1u : 0u;
          ok = wait(bar_do_full, par) && wait(bar_p, par);
          if (!ok) break;
          if (leader) issue_acc(C::kColDV, R0, aDO, 0, more);
          ok = wait(bar_p + 8, par);
          if (!ok) break;
          if (leader) {
            issue_acc(C::kColDV, R0, aDO, 1, 1u);
            umma_commit(bar_dv);
          }
          ok = wait(bar_ds, par);
          if (!ok) break;
          if (leader) issue_acc(C::kColDK, R1, aQ + s * kStage, 0, more);
          ok = wait(bar_ds + 8, par);
          if (!ok) break;
          if (leader) {
            issue_acc(C::kColDK, R1, aQ + s * kStage, 1, 1u);
            umma_commit(bar_q_empty + 8 * s);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) {
              const uint32_t off = ((kk * 16 * 128) >> 4) | kLboMn;
              umma_ss_lo(R1, aDS + off, aK + off, idesc_dq, kk > 0 ? 1u : 0u);
            }
            umma_commit(bar_dq);
          }
        }
        if (ok && leader) umma_commit(bar_acc);
      }
      __syncwarp();
    }
  } else if (warp >= 8) {
    // ---------------------------------------------------------------- dQ tiles
    asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    const int wq = warp & 3;
    const uint32_t tR1 = tmem + (static_cast<uint32_t>(wq * 32) << 16) + C::kColR1;
    const int parts = p.partial ? T : 1;
    constexpr int kChunks = D / 32;
    // this warp's 32 rows of the head's accumulators, query tile 0
    uint8_t *acc = reinterpret_cast<uint8_t *>(p.dq_acc) +
                   ((static_cast<int64_t>(bh) * T * parts + (p.partial ? n : 0)) * 4 + wq) *
                       (kChunks * C::kChunkBytes);
    const int64_t acc_tile = static_cast<int64_t>(parts) * 4 * kChunks * C::kChunkBytes;
    uint32_t *turn = p.turn + static_cast<int64_t>(bh) * T * 4 + wq;
    const bool add = !p.partial && n > 0, pass = !p.partial && n + 1 < T;
    const uint32_t buf = sbase + C::kOffOut + wq * 2 * C::kChunkBytes;
    // Tile j's adds are complete: pass its turn on.
    auto release = [&](int j) {
      fence_proxy_async_global();
      st_release_gpu_u32(turn + 4 * j, static_cast<uint32_t>(n + 1));
    };
    for (int j = 0; j < T; ++j) {
      // asked for before the tile is there, so that the answer's way is hidden
      uint32_t seen = add && lane == 0 ? ld_acquire_gpu_u32(turn + 4 * j) : 0u;
      const bool got = mbar_wait(bar_dq, j & 1, abort_flag, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t r[D];
#pragma unroll
      for (int c = 0; c < D; c += 32) tmem_ld32(tR1 + c, r + c);
      tmem_wait_ld();
      tc_fence_before();
      mbar_arrive(bar_dq_free);
      bool mine = true;
      if (add && lane == 0) {
        if (seen < static_cast<uint32_t>(n)) {
          const uint64_t t0 = globaltimer_ns();
          while (ld_acquire_gpu_u32(turn + 4 * j) < static_cast<uint32_t>(n)) {
            if (*abort_flag || globaltimer_ns() - t0 > kWaitLimitNs ||
                ld_acquire_gpu_u32(p.ticket + 1) != 0u) {
              mine = false;
              break;
            }
          }
        }
        fence_proxy_async_global();
      }
      if (!__all_sync(0xffffffffu, mine)) {
        ok = false;
        break;
      }
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
        const uint32_t dst = buf + (c & 1) * C::kChunkBytes;
        if (lane == 0) bulk_wait_read<1>();  // the buffer's last copy has been read
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          st_shared_v4(dst + i * 512 + lane * 16,
                       make_uint4(r[32 * c + 4 * i], r[32 * c + 4 * i + 1], r[32 * c + 4 * i + 2],
                                  r[32 * c + 4 * i + 3]));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          uint8_t *g_dst = acc + j * acc_tile + c * C::kChunkBytes;
          if (add) bulk_add_f32(g_dst, dst, C::kChunkBytes);
          else bulk_store(g_dst, dst, C::kChunkBytes);
          bulk_commit();
          if (c == 1 && pass && j > 0) {
            bulk_wait<2>();  // all but this tile's two chunks
            release(j - 1);
          }
        }
      }
    }
    if (lane == 0) {
      bulk_wait_all();  // (no copy outlives the CTA's shared memory either)
      if (ok && pass) release(T - 1);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- elementwise
    asm volatile("setmaxnreg.inc.sync.aligned.u32 144;");
    const int h = warp >> 2;             // query half of a tile
    const int wq = warp & 3;
    const int row = wq * 32 + lane;      // key within the tile
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tR0 = tmem + lane_bits + 64 * h;
    const uint32_t tR1 = tmem + lane_bits + C::kColR1 + 64 * h;
    const bool valid = k0 + row < p.N;
    const uint64_t k_sl2 = f2_pack(p.scale_log2e, p.scale_log2e);
    const uint64_t zero2 = f2_pack(0.f, 0.f);
    const uint32_t ds_row = sbase + C::kOffDS + h * C::kBlockBytes + row * 128;
    for (int j = 0; j < T; ++j) {
      const int s = j & 1;
      bool got = mbar_wait(bar_s, j & 1, abort_flag, kWaitLimitNs) &&
                 mbar_wait(bar_q_full + 8 * s, (j >> 1) & 1, abort_flag, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const ulonglong2 *nlse = reinterpret_cast<const ulonglong2 *>(smem + C::kOffStat + s * 1024) + 16 * h;
      const ulonglong2 *ndelta = nlse + 32;
      uint32_t pr[64];  // the tile row's scores, then its probabilities
      tmem_ld32(tR0, pr);
      tmem_ld32(tR0 + 32, pr + 32);
      tmem_wait_ld();
      if (!valid) {  // keys past N: probability 0 whatever lse is
#pragma unroll
        for (int i = 0; i < 64; ++i) pr[i] = 0xFF800000u;
      }
      uint32_t pk[32];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const ulonglong2 nl = nlse[i];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = 4 * i + 2 * e;
          const uint64_t x = f2_fma(f2_pack_bits(pr[c], pr[c + 1]), k_sl2, e ? nl.y : nl.x);
          float p0, p1;
          f2_unpack(x, p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          pr[c] = __float_as_uint(p0);
          pr[c + 1] = __float_as_uint(p1);
          pk[2 * i + e] = pack_bf16x2(p0, p1);
        }
      }
      tmem_st32(tR0, pk);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar_p + 8 * h);

      got = mbar_wait(bar_dp, j & 1, abort_flag, kWaitLimitNs);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc_fence_after();
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t dp[32];
        tmem_ld32(tR1 + 32 * hh, dp);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const ulonglong2 nd = ndelta[8 * hh + i];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int c = 4 * i + 2 * e;
            const uint64_t x = f2_add(f2_pack_bits(dp[c], dp[c + 1]), e ? nd.y : nd.x);
            const uint64_t y =
                f2_fma(f2_pack_bits(pr[32 * hh + c], pr[32 * hh + c + 1]), x, zero2);
            float d0, d1;
            f2_unpack(y, d0, d1);
            pk[16 * hh + 2 * i + e] = pack_bf16x2(d0, d1);
          }
        }
#pragma unroll
        for (int c = 0; c < 4; ++c)
          st_shared_v4(ds_row + (((4 * hh + c) ^ (row & 7)) << 4),
                       make_uint4(pk[16 * hh + 4 * c], pk[16 * hh + 4 * c + 1],
                                  pk[16 * hh + 4 * c + 2], pk[16 * hh + 4 * c + 3]));
      }
      tmem_st32(tR1, pk);
      fence_proxy_async_smem();
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar_ds + 8 * h);
    }
    // epilogue: warpgroup 0 stores dV, warpgroup 1 stores dK, a row per thread
    if (ok) ok = mbar_wait(bar_acc, 0, abort_flag, kWaitLimitNs);
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      const uint32_t tA = tmem + lane_bits + (h == 0 ? C::kColDV : C::kColDK);
      const float f = h == 0 ? 1.0f : p.scale;
      __nv_bfloat16 *dst = (h == 0 ? p.dv : p.dk) + bwd_row(p, bh, k0 + row, D);
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(tA + c, o);
        tmem_wait_ld();
        if (valid) {
          uint4 *d4 = reinterpret_cast<uint4 *>(dst + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * e]) * f,
                                 __uint_as_float(o[8 * i + 2 * e + 1]) * f);
            d4[i] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    } else {
      ok = false;
    }
  }

  // ------------------------------------------------------------------ teardown
  if (!ok) {
    *abort_flag = 1;
    atomicExch(p.ticket + 1, 1u);
    atomicExch(p.status, kStatusTimeout);
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // asynchronous work lands before shared and tensor memory are released
    if (warp == 12 && lane == 0) {
      mbar_wait_drain(bar_k, 0, kWaitLimitNs);
      if (kv_issued) mbar_wait_drain(bar_v, 0, kWaitLimitNs);
      const int nq = (issued + 1) >> 1, ndo = issued >> 1;  // loads issued
      for (int j = max(nq - 2, 0); j < nq; ++j)
        mbar_wait_drain(bar_q_full + 8 * (j & 1), (j >> 1) & 1, kWaitLimitNs);
      if (ndo > 0) mbar_wait_drain(bar_do_full, (ndo - 1) & 1, kWaitLimitNs);
    }
    if (leader) {
      umma_commit(bar_drain);
      mbar_wait_drain(bar_drain, 0, kWaitLimitNs);
    }
    __syncthreads();
  }
  if (warp == 13) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// One block per (query tile, head): dQ = scale * the accumulators, rounded
// once.  A thread takes 16 columns of a row: every load of a warp is 512
// contiguous bytes, every row piece stored is a whole 32-byte sector.  Past
// the tiles' blocks, one block per (head, padding token) zeroes that token's
// row of all three gradients.
template <int D>
__global__ void __launch_bounds__(256) attention_dq_kernel(const __grid_constant__ AttnBwdParams p) {
  const int64_t tiles = static_cast<int64_t>(p.BH) * p.T;
  if (blockIdx.x >= tiles) {
    const int pad = p.Np - p.N;
    const int i = static_cast<int>(blockIdx.x - tiles);
    const int bh = i / pad;
    const int64_t off = bwd_row(p, bh, p.N + (i - bh * pad), D);
    if (threadIdx.x < 3 * D / 8) {
      const int which = threadIdx.x / (D / 8), c = threadIdx.x % (D / 8);
      __nv_bfloat16 *base = which == 0 ? p.dq : which == 1 ? p.dk : p.dv;
      reinterpret_cast<uint4 *>(base + off)[c] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const int qt = static_cast<int>(blockIdx.x % p.T), bh = static_cast<int>(blockIdx.x / p.T);
  const int parts = p.partial ? p.T : 1;
  const float4 *src = reinterpret_cast<const float4 *>(p.dq_acc) +
                      static_cast<int64_t>(blockIdx.x) * parts * (D / 4) * 128;
  const int row = threadIdx.x & 127, t = qt * 128 + row;
  if (t >= p.N) return;
  src += (row >> 5) * (D / 4) * 32 + (row & 31);
  uint4 *dst = reinterpret_cast<uint4 *>(p.dq + bwd_row(p, bh, t, D));
#pragma unroll
  for (int c = threadIdx.x >> 7; c < D / 16; c += 2) {
    float4 a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = src[(4 * c + i) * 32];
    for (int k = 1; k < parts; ++k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float4 v = src[static_cast<int64_t>(k) * (D / 4) * 128 + (4 * c + i) * 32];
        a[i].x += v.x, a[i].y += v.y, a[i].z += v.z, a[i].w += v.w;
      }
    }
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[2 * i] = pack_bf16x2(a[i].x * p.scale, a[i].y * p.scale);
      w[2 * i + 1] = pack_bf16x2(a[i].z * p.scale, a[i].w * p.scale);
    }
    dst[2 * c] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[2 * c + 1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

}  // namespace sp
