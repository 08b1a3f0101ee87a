// attention_backward.cuh -- backward pass of full-sequence attention per head
// on tcgen05 tensor cores (sm_100a), recomputing the probabilities from the
// row log-sum-exp of the forward pass.
//
// Per (batch, head), for queries i and keys k below N:
//   P_ik = exp(scale q_i.k_k - lse_i)        delta_i = sum_c dO_ic O_ic
//   dV_k = sum_i P_ik dO_i                   dP_ik   = dO_i . v_k
//   dS_ik = P_ik (dP_ik - delta_i)
//   dQ_i = scale sum_k dS_ik k_k             dK_k    = scale sum_i dS_ik q_i
// Five products of N x N x D per head.  dK and dV sum over queries, dQ over
// keys: one of the two has to leave its CTA.  A single pass that adds 128 x 128
// fp32 tiles of dQ to global memory in key order (which repeats bit for bit)
// moves 64 KB out of every SM per tile; it took 18.5 ms at 480p (12 heads,
// 32,760 tokens) and 1.52 ms at 4,096 tokens x 40 heads.  Here scores and dP are
// computed twice instead, seven products, and every sum stays in tensor memory:
// 17.9 and 1.00 ms.  Results repeat bit for bit and depend neither on timing nor
// on P.
// What bounds it: at 480p the 1,000 W power cap (1.5 GHz of 1.97; seven products
// at 1.28 PFLOP/s, cuBLAS holds 1.38 there).  A 128 x 128 tile takes 2,700 cycles
// in a dK/dV CTA (its four products 2,048) and 2,050 in a dQ CTA (1,536); a
// polynomial for part of the exponentials brought that to 2,450 and 1,970, and
// the time, at the cap, not at all (D = 64 has one, see below).  Short problems
// are bound by a CTA's chain.
//
// One launch holds both kinds of CTA:
//   dK, dV: 128 keys; walks the 128-query tiles.  Scores are computed
//           transposed (keys in the lanes), so that P^T and dS^T, rounded to
//           bf16 for the tensor core as the forward pass rounds P, are the A
//           operands of dV += P^T dO and dK += dS^T Q from tensor memory.
//   dQ:     two tiles of 128 queries, which take turns at each 128-key tile
//           (one K, V load serves both), or one tile (the launcher has the
//           rule); dS is the A operand of dQ += dS K.
// Roles (12 warps):
//   warps 0-7   elementwise: warpgroup h takes columns 64h .. 64h+63 of a tile,
//               one thread per row (key, or query for dQ)
//   warps 8, 10 TMA producers, one per operand pair
//   warp 9      TMEM allocator and the single MMA-issuing warp
// Tensor memory (512 columns): R0 = 0..127 scores, then P^T (dK, dV only), and with
// D = 64 a second tile of them at 384; R1 = 128..255 dP, then dS; two accumulators
// from 256.  MMAs of one thread run
// in order, so nothing waits for an operand's last reader.  The MMA warp issues
//   dK, dV:  dV_j, S_{j+1}, dK_j, dP_{j+1}
//   dQ:      S_{i+1}, dQ_i, dP_{i+1}
// so that exponentials run beside dK and dP, and dS beside dV and S.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>

#include "attention.cuh"
#include "permute.cuh"
#include "sm100.cuh"

namespace sp {

struct AttnBwdParams {
  int32_t N, Np, H, B;   // true tokens, token slots, heads, batch
  int32_t hsplit;        // heads per tensor-map "batch" slot (Hl or H)
  int32_t T;             // tiles of 128 tokens
  int32_t BH;            // B * H
  int32_t dq_tiles;      // query tiles of a dQ CTA: 1 or 2
  int32_t nl_split;      // as in AttnParams
  FastDiv div_nl;
  float scale, scale_log2e;
  const uint8_t *q, *k, *v, *o, *dout;
  const float *lse;      // [B][H][Np]
  __nv_bfloat16 *dq, *dk, *dv;
  int64_t row_el, batch_el, rank_el;  // strides of tokens, slots, rank slabs
  float *stat;           // workspace, [BH][T][2][128]: -lse * log2(e), -delta
  int32_t *status;
};

// Tensor maps of Q, K, V and dO with boxes of 128 rows and, for rank-major
// shards, of 32 and of 8.
struct AttnBwdMaps {
  CUtensorMap tile[4], quad[4], group[4];
};

// Element offset of token `t` of head bh's row in q, k, v, o and their gradients.
__device__ __forceinline__ int64_t bwd_row(const AttnBwdParams &p, int bh, int t, int D) {
  const int b = bh / p.H, hg = bh - b * p.H;
  const int hs = hg / p.hsplit, head = hg - hs * p.hsplit;
  int64_t off;
  if (p.nl_split) {
    const int rk = fdiv(t, p.div_nl);
    off = rk * p.rank_el + b * p.batch_el + (t - rk * p.nl_split) * p.row_el;
  } else {
    off = (static_cast<int64_t>(hs) * p.B + b) * p.batch_el + t * p.row_el;
  }
  return off + static_cast<int64_t>(head) * D;
}

// One block per (query tile, head): delta in fp32 from 16-byte loads, D / 8
// lanes a row.  Past the tiles' blocks, one block per (head, padding token)
// zeroes that token's row of all three gradients.
template <int D>
__global__ void __launch_bounds__(256) attention_delta_kernel(const __grid_constant__ AttnBwdParams p) {
  constexpr int kLanes = D / 8, kRows = 256 / kLanes;
  // the main kernel's blocks may begin to fetch their tiles beside this one
  asm volatile("griddepcontrol.launch_dependents;");
  const int64_t tiles = static_cast<int64_t>(p.BH) * p.T;
  if (blockIdx.x >= tiles) {
    const int pad = p.Np - p.N;
    const int i = static_cast<int>(blockIdx.x - tiles);
    const int bh = i / pad;
    const int64_t off = bwd_row(p, bh, p.N + (i - bh * pad), D);
    if (threadIdx.x < 3 * kLanes) {
      const int which = threadIdx.x / kLanes, c = threadIdx.x % kLanes;
      __nv_bfloat16 *base = which == 0 ? p.dq : which == 1 ? p.dk : p.dv;
      reinterpret_cast<uint4 *>(base + off)[c] = make_uint4(0u, 0u, 0u, 0u);
    }
    return;
  }
  const int qt = blockIdx.x % p.T, bh = blockIdx.x / p.T;
  const int c = threadIdx.x % kLanes, r0 = threadIdx.x / kLanes;
  uint4 vo[128 / kRows], vd[128 / kRows];
  float lse[128 / kRows];
#pragma unroll
  for (int i = 0; i < 128 / kRows; ++i) {
    const int t = qt * 128 + r0 + i * kRows;
    vo[i] = vd[i] = make_uint4(0u, 0u, 0u, 0u);
    // rows past N: probability 2^-inf
    lse[i] = -INFINITY;
    if (t < p.N) {
      if (c == 0) lse[i] = __ldg(p.lse + static_cast<int64_t>(bh) * p.Np + t);
      const int64_t off = bwd_row(p, bh, t, D) * 2 + c * 16;
      vo[i] = ld_global_nc_v4(p.o + off);
      vd[i] = ld_global_nc_v4(p.dout + off);
    }
  }
  float *stat = p.stat + static_cast<int64_t>(blockIdx.x) * 256;
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
    const int r = r0 + i * kRows;
    if (c == 0) {
      // (rows without a key, lse = -inf, too)
      stat[r] = lse[i] == -INFINITY ? -INFINITY : -lse[i] * 1.4426950408889634f;
      stat[128 + r] = -s;
    }
  }
}

template <int D>
struct AttnBwdCfg {
  static constexpr int kHalves = D / 64;              // 128-byte column blocks per row
  static constexpr int kBlockBytes = 128 * 128;
  static constexpr int kTileBytes = kHalves * kBlockBytes;
  // Seven tiles.  dK, dV: K, V, three stages of Q, two of dO.
  // dQ: Q and dO of both query tiles, two stages of K, one of V.
  static constexpr int kOffOwn = 0;
  static constexpr int kOffX = 2 * kTileBytes;        // dK, dV: Q stages
  static constexpr int kOffY = 5 * kTileBytes;        // dK, dV: dO stages
  static constexpr int kOffK2 = 4 * kTileBytes;       // dQ: K stages
  static constexpr int kOffV1 = 6 * kTileBytes;       // dQ: V
  static constexpr int kOffStat = 7 * kTileBytes;     // dK, dV: [2 stages][2][128] fp32
  static constexpr int kOffBar = kOffStat + 2 * 1024;
  static constexpr int kNumBar = 30;
  static constexpr int kOffMisc = kOffBar + kNumBar * 8;  // TMEM base, abort flag
  static constexpr int kSmemBytes = kOffMisc + 16;
  static_assert(kSmemBytes <= 227 * 1024, "shared memory per CTA");
  static constexpr int kThreads = 384;
  static constexpr uint32_t kColR1 = 128;
  static constexpr uint32_t kColA0 = 256;             // dV, or dQ of tile 0
  static constexpr uint32_t kColA1 = 256 + D;         // dK, or dQ of tile 1
  static constexpr uint32_t kTmemCols = 512;
  // With D = 64 tensor memory holds a second tile of scores, so that S_{j+1}
  // need not wait for the tile before it: 32,760 tokens x 12 heads 12.3 instead of
  // 12.9 ms, 1,024 x 4 heads 17.6 instead of 18.8 us.
  static constexpr int kScores = D == 64 ? 2 : 1;
  static constexpr uint32_t kColS1 = 384;
};

// Blocks: every head's pairs of query tiles first, since they run longest, then
// every head's key tiles (2,048 tokens x 12 heads 78 us; head by head 92.5,
// and the same within 1 % from 4,096 tokens on).  The CTAs that run together
// belong to one or two heads, whose Q, K, V and dO stay in L2.
template <int D>
__global__ void __launch_bounds__(384, 1)
attention_backward_kernel(const __grid_constant__ AttnBwdMaps maps,
                          const __grid_constant__ AttnBwdParams p) {
  using C = AttnBwdCfg<D>;
  // The swizzled tiles want 1,024-byte alignment, which the dynamic shared
  // memory of a kernel without static shared memory has; there is no room
  // to round up, so it is checked.
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t sbase = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int T = p.T;

  const uint32_t bar_own = sbase + C::kOffBar;      // [4]: K, V; or Q0, dO0, Q1, dO1
  const uint32_t bar_x_full = bar_own + 32;         // [3]: Q (K)
  const uint32_t bar_x_empty = bar_own + 56;        // [3]
  const uint32_t bar_y_full = bar_own + 80;         // [2]: dO (V)
  const uint32_t bar_y_empty = bar_own + 96;        // [2]
  const uint32_t bar_stat = bar_own + 112;          // [2]
  const uint32_t bar_s = bar_own + 128;             // [score tiles]
  const uint32_t bar_s_free = bar_own + 144;        // dQ, one score tile
  const uint32_t bar_p = bar_own + 152;             // [score tiles][2]
  const uint32_t bar_dp = bar_own + 184;
  const uint32_t bar_ds = bar_own + 192;            // [2]
  const uint32_t bar_acc = bar_own + 208, bar_drain = bar_own + 216;
  const uint32_t bar_stat_empty = bar_own + 224;    // [2]
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + C::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::kOffMisc + 4);

  if ((sbase & 1023u) != 0) {  // uniform
    if (threadIdx.x == 0) atomicExch(p.status, kStatusTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < 4; ++s) mbar_init(bar_own + 8 * s, 1);
    for (int s = 0; s < 3; ++s) {
      mbar_init(bar_x_full + 8 * s, 1);
      mbar_init(bar_x_empty + 8 * s, 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar_y_full + 8 * s, 1);
      mbar_init(bar_y_empty + 8 * s, 1);
      mbar_init(bar_stat + 8 * s, 1);
      mbar_init(bar_stat_empty + 8 * s, 1);
      mbar_init(bar_s + 8 * s, 1);
      mbar_init(bar_p + 8 * s, 128);
      mbar_init(bar_p + 16 + 8 * s, 128);
      mbar_init(bar_ds + 8 * s, 128);
    }
    mbar_init(bar_s_free, 256);
    mbar_init(bar_dp, 1);
    mbar_init(bar_acc, 1);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), C::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int T2 = (T + p.dq_tiles - 1) / p.dq_tiles;
  const int n_dq = p.BH * T2, blk = blockIdx.x;
  const bool is_dq = blk < n_dq;
  const int i_kind = is_dq ? blk : blk - n_dq, per = is_dq ? T2 : T;
  const int bh = i_kind / per;
  const int t0 = (i_kind - bh * per) * (is_dq ? p.dq_tiles * 128 : 128);  // first own token
  const int nt = is_dq && p.dq_tiles == 2 && t0 + 128 < p.N ? 2 : 1;
  const int b = bh / p.H, hg = bh - b * p.H;

  // Item i's score tile: its column, index and the parity of its barriers (one
  // for both tiles could be two phases ahead of a waiting warp).
  auto s_col = [](int i) { return C::kScores == 2 && (i & 1) ? C::kColS1 : 0u; };
  auto s_idx = [](int i) { return C::kScores == 2 ? static_cast<uint32_t>(i & 1) : 0u; };
  auto s_par = [](int i) { return static_cast<uint32_t>(C::kScores == 2 ? i >> 1 : i) & 1u; };

  bool ok = true;
  bool leader = false;   // the lane of warp 9 that issues MMAs
  // loads issued by a producer warp: own tiles, tiles of its ring, statistics
  int n_own = 0, n_ring = 0, n_stat = 0;
  const int stages = (is_dq ? 1 : 2) + (warp == 8 ? 1 : 0);  // of its ring
  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8 || warp == 10) {
      // -------------------------------------------------------------- producers
      // Warp 8: K, the Q ring and the statistics; for dQ the Q tiles and the
      // K ring.  Warp 10: V and the dO ring; for dQ the dO tiles and V.
      const int hs = hg / p.hsplit;
      const int map_head = hg - hs * p.hsplit, map_batch = hs * p.B + b;
      const uint64_t pol_own = policy_evict_first(), pol_ring = policy_evict_last();
      const int nl = p.nl_split;
      if (lane < 4) prefetch_tmap(&maps.tile[lane]);
      // Rank-major layout: a tile that crosses a shard boundary, or holds
      // padding slots of the last shard, is loaded in pieces.
      auto rank_of = [&](int n) { return static_cast<int>(fdiv(n, p.div_nl)); };
      auto tma_ok = [&](int tok) {
        if (nl == 0) return true;
        const int r0 = rank_of(tok);
        return tok - r0 * nl + 128 <= nl && tok + 128 <= p.N;
      };
      // Lane g has group g, eight rows, 1,024 bytes of each column block as the
      // TMA swizzles it.  Four groups, or one, that lie within a shard or past N
      // (zeros, from a box past the shard) are one more TMA load a column block;
      // the few others are copied row by row, 16-byte chunk cc of row r to chunk
      // cc ^ (r mod 8).  2,050 tokens in 8 shards, 2 x 8 heads: 123 us (in one
      // shard 112); all rows copied 160; groups by TMA but not fours 140; single
      // rows by TMA too 150.  Shards of 6 tokens (all rows copied): 58 us where a
      // copy that steps through the rows took 49.
      auto load_pieces = [&](int which, const uint8_t *base, uint32_t dst, uint32_t bar, int tok,
                             uint64_t pol) {
        auto whole = [&](int n, int rows) {
          return nl >= rows && (n >= p.N || (n - rank_of(n) * nl + rows <= nl && n + rows <= p.N));
        };
        const int n0 = tok + 8 * lane;
        const bool quad = lane < 16 && whole(tok + 32 * (lane >> 2), 32);
        const bool tma = quad || (lane < 16 && whole(n0, 8));
        const uint32_t by_tma = __ballot_sync(0xffffffffu, tma);
        if (lane == 0) mbar_expect_tx(bar, __popc(by_tma) * 1024 * C::kHalves);
        __syncwarp();
        if (quad ? (lane & 3) == 0 : tma) {
          const CUtensorMap *m = quad ? &maps.quad[which] : &maps.group[which];
          const int rk = n0 >= p.N ? 0 : rank_of(n0), loc = n0 >= p.N ? nl : n0 - rk * nl;
          for (int h = 0; h < C::kHalves; ++h)
            tma_load_5d(dst + h * C::kBlockBytes + lane * 1024, m, bar, h * 64, map_head, loc, b, rk,
                        pol);
        }
        __syncwarp();
        constexpr int kChunks = D / 8;
        const int cc = lane % kChunks;
        const uint32_t col = dst + (cc >> 3) * C::kBlockBytes;
        for (uint32_t rest = ~by_tma & 0xffffu; rest != 0; rest &= rest - 1) {
          const int g8 = 8 * (__ffs(rest) - 1);
#pragma unroll
          for (int i = lane / kChunks; i < 8; i += 32 / kChunks) {
            const int n = tok + g8 + i, rk = rank_of(n);
            const bool in = n < p.N;
            const uint8_t *src = base + cc * 16 +
                                 2 * (rk * p.rank_el + b * p.batch_el + (n - rk * nl) * p.row_el +
                                      static_cast<int64_t>(map_head) * D);
            cp_async16(col + (g8 + i) * 128 + (((cc & 7) ^ i) << 4), in ? src : base, in ? 16 : 0);
          }
        }
        cp_async_wait();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      auto load = [&](int which, const uint8_t *base, uint32_t dst, uint32_t bar, int tok,
                      uint64_t pol) {
        if (!tma_ok(tok)) {
          load_pieces(which, base, dst, bar, tok, pol);
        } else if (lane == 0) {
          const CUtensorMap *m = &maps.tile[which];
          mbar_arrive_expect_tx(bar, C::kTileBytes);
          for (int h = 0; h < C::kHalves; ++h) {
            if (nl == 0) {
              tma_load_4d(dst + h * C::kBlockBytes, m, bar, h * 64, map_head, tok, map_batch, pol);
            } else {
              const int r0 = rank_of(tok);
              tma_load_5d(dst + h * C::kBlockBytes, m, bar, h * 64, map_head, tok - r0 * nl, b, r0,
                          pol);
            }
          }
        }
        __syncwarp();
      };
      auto wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, kWaitLimitNs)) != 0;
      };
      const bool first = warp == 8;
      // 0 .. 3: Q, K, V, dO
      const int mO = first ? (is_dq ? 0 : 1) : (is_dq ? 3 : 2);    // own
      const int mR = first ? (is_dq ? 1 : 0) : (is_dq ? 2 : 3);    // ring
      const uint8_t *gO = first ? (is_dq ? p.q : p.k) : (is_dq ? p.dout : p.v);
      const uint8_t *gR = first ? (is_dq ? p.k : p.q) : (is_dq ? p.v : p.dout);
      const uint32_t ring = sbase + (first ? (is_dq ? C::kOffK2 : C::kOffX)
                                           : (is_dq ? C::kOffV1 : C::kOffY));
      const uint32_t own = first ? 0 : 1;
      const uint32_t bar_full = first ? bar_x_full : bar_y_full;
      const uint32_t bar_empty = first ? bar_x_empty : bar_y_empty;
      int rs = 0, rp = 1;  // ring stage, parity of its empty barrier
      load(mO, gO, sbase + own * C::kTileBytes, bar_own + 8 * own, t0, pol_own);
      n_own = 1;
      for (int j = 0; j < T && ok; ++j) {
        ok = wait(bar_empty + 8 * rs, rp);
        if (!ok) break;
        load(mR, gR, ring + rs * C::kTileBytes, bar_full + 8 * rs, j * 128, pol_ring);
        ++n_ring;
        if (++rs == stages) rs = 0, rp ^= 1;
        if (!is_dq && first) {
          const int s = j & 1;
          ok = wait(bar_stat_empty + 8 * s, ((j >> 1) & 1) ^ 1);
          if (!ok) break;
          if (lane == 0) {
            // (written by the kernel in front of this one)
            if (j == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
            mbar_arrive_expect_tx(bar_stat + 8 * s, 1024);
            bulk_load(sbase + C::kOffStat + s * 1024,
                      p.stat + (static_cast<int64_t>(bh) * T + j) * 256, 1024, bar_stat + 8 * s);
          }
          __syncwarp();
          ++n_stat;
        }
        if (j == 0 && nt == 2) {
          load(mO, gO, sbase + (2 + own) * C::kTileBytes, bar_own + 8 * (2 + own), t0 + 128, pol_own);
          n_own = 2;
        }
      }
    } else if (warp == 9) {
      // -------------------------------------------------------------- MMA issue
      // The whole warp runs the loops and one elected lane issues, and every
      // address is a constant or warp-uniform (the kernel holds all of tensor
      // memory, so its base is 0), so that descriptors stay in uniform
      // registers.
      constexpr uint32_t idesc_kk = make_idesc_bf16(128, 128, 0, 0);  // S, dP
      constexpr uint32_t idesc_acc = make_idesc_bf16(128, D, 0, 1);   // dV, dK, dQ
      // Low descriptor words: start address / 16 and the leading offset.
      constexpr uint32_t kLboK = 1u << 16;                               // K-major: unused
      constexpr uint32_t kLboMn = static_cast<uint32_t>(C::kBlockBytes >> 4) << 16;
      constexpr uint32_t R1 = C::kColR1;
      constexpr uint32_t kStage = C::kTileBytes >> 4;
      const uint32_t s16 = sbase >> 4;
      leader = elect_one();
      auto wait = [&](uint32_t bar, uint32_t parity) {
        const bool got = mbar_wait(bar, parity, abort_flag, kWaitLimitNs);
        tc_fence_after();
        return __all_sync(0xffffffffu, got) != 0;
      };
      // [128 x 128] = A B^T over D, both operands K-major
      auto issue_kk = [&](uint32_t d, uint32_t a, uint32_t bb) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (((kk >> 2) * C::kBlockBytes + (kk & 3) * 32) >> 4) | kLboK;
          umma_ss_lo(d, a + off, bb + off, idesc_kk, kk > 0 ? 1u : 0u);
        }
      };
      // acc += X[:, 64h .. 64h+63] B[64h .. 64h+63, :], X in tensor memory
      auto issue_acc = [&](uint32_t d, uint32_t x, uint32_t bb, int h, uint32_t more) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
          umma_ts_lo(d, x + 64 * h + 8 * k, bb + ((((4 * h + k) * 16 * 128) >> 4) | kLboMn),
                     idesc_acc, (h == 0 && k == 0) ? more : 1u);
      };
      ok = tmem == 0;
      const uint32_t aOwn = s16;
      const uint32_t aX = s16 + ((is_dq ? C::kOffK2 : C::kOffX) >> 4);
      const uint32_t aY = s16 + ((is_dq ? C::kOffV1 : C::kOffY) >> 4);
      if (!is_dq) {
        ok = ok && wait(bar_own, 0) && wait(bar_x_full, 0);
        if (ok) {
          if (leader) {
            issue_kk(s_col(0), aOwn, aX);
            umma_commit(bar_s + 8 * s_idx(0));
          }
          ok = wait(bar_own + 8, 0) && wait(bar_y_full, 0);
        }
        if (ok && leader) {
          issue_kk(R1, aOwn + kStage, aY);
          umma_commit(bar_dp);
        }
        int xs = 0, xp = 0;  // Q stage of tile j, its parity
        for (int j = 0; j < T && ok; ++j) {
          const uint32_t par = j & 1, more = j > 0 ? 1u : 0u;
          const int ys = j & 1;
          const bool next = j + 1 < T;
          int xn = xs + 1, xnp = xp;
          if (xn == 3) xn = 0, xnp ^= 1;
          // Q_{j+1} first: a wait costs 100 to 200 cycles even when its barrier
          // stands, and between dV and S it would idle the tensor core (1.5 %;
          // dO_{j+1} likewise before dK: nothing gained)
          ok = !next || wait(bar_x_full + 8 * xn, xnp);
          if (!ok) break;
          const auto next_scores = [&] {
            if (next && leader) {
              issue_kk(s_col(j + 1), aOwn, aX + xn * kStage);
              umma_commit(bar_s + 8 * s_idx(j + 1));
            }
          };
          if (C::kScores == 2) next_scores();
          ok = wait(bar_p + 16 * s_idx(j), s_par(j));
          if (!ok) break;
          if (leader) issue_acc(C::kColA0, s_col(j), aY + ys * kStage, 0, more);
          ok = wait(bar_p + 16 * s_idx(j) + 8, s_par(j));
          if (!ok) break;
          if (leader) {
            issue_acc(C::kColA0, s_col(j), aY + ys * kStage, 1, 1u);
            umma_commit(bar_y_empty + 8 * ys);
          }
          if (C::kScores == 1) next_scores();
          ok = wait(bar_ds, par);
          if (!ok) break;
          if (leader) issue_acc(C::kColA1, R1, aX + xs * kStage, 0, more);
          ok = wait(bar_ds + 8, par);
          if (!ok) break;
          if (leader) {
            issue_acc(C::kColA1, R1, aX + xs * kStage, 1, 1u);
            umma_commit(bar_x_empty + 8 * xs);
            mbar_arrive(bar_stat_empty + 8 * ys);  // dS stands: its statistics were read
          }
          if (next) {
            ok = wait(bar_y_full + 8 * (ys ^ 1), ((j + 1) >> 1) & 1);
            if (!ok) break;
            if (leader) {
              issue_kk(R1, aOwn + kStage, aY + (ys ^ 1) * kStage);
              umma_commit(bar_dp);
            }
          }
          xs = xn, xp = xnp;
        }
      } else {
        // item i: key tile j = i / nt, query tile t = i % nt
        ok = ok && wait(bar_own, 0) && wait(bar_x_full, 0);
        if (ok) {
          if (leader) {
            issue_kk(s_col(0), aOwn, aX);
            umma_commit(bar_s + 8 * s_idx(0));
          }
          ok = wait(bar_own + 8, 0) && wait(bar_y_full, 0);
        }
        if (ok && leader) {
          issue_kk(R1, aOwn + kStage, aY);
          umma_commit(bar_dp);
          if (nt == 1) umma_commit(bar_y_empty);
        }
        if (ok && nt == 2) ok = wait(bar_own + 16, 0) && wait(bar_own + 24, 0);
        int j = 0, t = 0;
        for (int i = 0; j < T && ok; ++i) {
          const uint32_t par = i & 1;
          int jn = j, tn = t + 1;
          if (tn == nt) tn = 0, ++jn;
          const bool next = jn < T;
          const int xs = j & 1, xn = jn & 1;
          if (next) {
            // (of two score tiles, the other one's item is done: its dS was used)
            ok = (tn != 0 || wait(bar_x_full + 8 * xn, (jn >> 1) & 1)) &&
                 (C::kScores == 2 || wait(bar_s_free, par));
            if (!ok) break;
            if (leader) {
              issue_kk(s_col(i + 1), aOwn + 2 * tn * kStage, aX + xn * kStage);
              umma_commit(bar_s + 8 * s_idx(i + 1));
            }
          }
          const uint32_t acc = t ? C::kColA1 : C::kColA0, more = j > 0 ? 1u : 0u;
          ok = wait(bar_ds, par);
          if (!ok) break;
          if (leader) issue_acc(acc, R1, aX + xs * kStage, 0, more);
          ok = wait(bar_ds + 8, par);
          if (!ok) break;
          if (leader) {
            issue_acc(acc, R1, aX + xs * kStage, 1, 1u);
            if (t == nt - 1) umma_commit(bar_x_empty + 8 * xs);
          }
          if (next) {
            if (tn == 0) ok = wait(bar_y_full, jn & 1);
            if (!ok) break;
            if (leader) {
              issue_kk(R1, aOwn + (2 * tn + 1) * kStage, aY);
              umma_commit(bar_dp);
              if (tn == nt - 1) umma_commit(bar_y_empty);
            }
          }
          j = jn, t = tn;
        }
      }
      if (ok && leader) umma_commit(bar_acc);
      __syncwarp();
    }
  } else {
    // ---------------------------------------------------------------- elementwise
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int h = warp >> 2;             // column half of a tile
    const int wq = warp & 3;
    const int row = wq * 32 + lane;      // row within the tile
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t tS = tmem + lane_bits + 64 * h;
    const uint32_t tR1 = tmem + lane_bits + C::kColR1 + 64 * h;
    const uint64_t k_sl2 = f2_pack(p.scale_log2e, p.scale_log2e);
    auto wait = [&](uint32_t bar, uint32_t parity) {
      const bool got = mbar_wait(bar, parity, abort_flag, kWaitLimitNs);
      return __all_sync(0xffffffffu, got) != 0;
    };
    // pr = 2^(pr * scale * log2(e) + bias pair), 32 columns.  With D = 64 the
    // products take half as long and the special-function unit bounds a tile,
    // so four of sixteen pairs go to the FMA pipe (32,760 tokens x 12 heads: 12.25
    // instead of 12.55 ms, 1,024 x 4 heads 17.8 instead of 19.2 us; six the same,
    // eight 12.8 ms; the factor 2^n that keeps NaN, in the place of an addition to
    // the exponent, 12.4).  With D = 128 it cost 1 to 2 % at the power cap.
    constexpr int kPolyPairs = D == 64 ? 4 : 0;
    auto exps = [&](uint32_t *pr, auto bias) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const uint64_t x = f2_fma(f2_pack_bits(pr[2 * i], pr[2 * i + 1]), k_sl2, bias(i));
        if ((i * kPolyPairs) % 16 < kPolyPairs) {
          ex2_poly(x, pr[2 * i], pr[2 * i + 1]);
        } else {
          float p0, p1;
          f2_unpack(x, p0, p1);
          pr[2 * i] = __float_as_uint(ex2(p0));
          pr[2 * i + 1] = __float_as_uint(ex2(p1));
        }
      }
    };
    auto pack16 = [](const uint32_t *v, uint32_t *w) {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        w[i] = pack_bf16x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
    };
    // dS = P (dP - delta) of 32 columns, rounded
    auto dscores = [&](const uint32_t *pr, const uint32_t *dp, uint32_t *w, auto ndelta) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float d0, d1;
        f2_unpack(f2_mul(f2_add(f2_pack_bits(dp[2 * i], dp[2 * i + 1]), ndelta(i)),
                         f2_pack_bits(pr[2 * i], pr[2 * i + 1])),
                  d0, d1);
        w[i] = pack_bf16x2(d0, d1);
      }
    };
    if (!is_dq) {
      for (int j = 0; j < T; ++j) {
        const int s = j & 1;
        ok = wait(bar_stat + 8 * s, (j >> 1) & 1) && wait(bar_s + 8 * s_idx(j), s_par(j));
        if (!ok) break;
        tc_fence_after();
        const ulonglong2 *nlse =
            reinterpret_cast<const ulonglong2 *>(smem + C::kOffStat + s * 1024) + 16 * h;
        const ulonglong2 *ndelta = nlse + 32;
        const uint32_t tR0 = tS + s_col(j);
        uint32_t pr[64], pk[32], dp[64];
        tmem_ld32(tR0, pr);
        tmem_ld32(tR0 + 32, pr + 32);
        tmem_wait_ld();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          exps(pr + 32 * hh, [&](int i) {
            const ulonglong2 v = nlse[8 * hh + (i >> 1)];
            return i & 1 ? v.y : v.x;
          });
          pack16(pr + 32 * hh, pk + 16 * hh);
        }
        tmem_st32(tR0, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar_p + 16 * s_idx(j) + 8 * h);

        ok = wait(bar_dp, s);
        if (!ok) break;
        tc_fence_after();
        tmem_ld32(tR1, dp);
        tmem_ld32(tR1 + 32, dp + 32);
        tmem_wait_ld();
#pragma unroll
        for (int hh = 0; hh < 2; ++hh)
          dscores(pr + 32 * hh, dp + 32 * hh, pk + 16 * hh, [&](int i) {
            const ulonglong2 v = ndelta[8 * hh + (i >> 1)];
            return i & 1 ? v.y : v.x;
          });
        tmem_st32(tR1, pk);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar_ds + 8 * h);
      }
    } else {
      // this thread's rows' statistics, both query tiles
      float nlse[2], ndelta[2];
      asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float *stat =
            p.stat + (static_cast<int64_t>(bh) * T + t0 / 128 + (t < nt ? t : 0)) * 256 + row;
        nlse[t] = stat[0];
        ndelta[t] = stat[128];
      }
      int i = 0;  // item
      for (int j = 0; j < T && ok; ++j) {
        const int lim = p.N - j * 128 - 64 * h;  // keys of this half that exist
        for (int t = 0; t < nt; ++t, ++i) {
          const uint32_t par = i & 1;
          ok = wait(bar_s + 8 * s_idx(i), s_par(i));
          if (!ok) break;
          tc_fence_after();
          const float nl = t ? nlse[1] : nlse[0], nd = t ? ndelta[1] : ndelta[0];
          const uint64_t nl2 = f2_pack(nl, nl), nd2 = f2_pack(nd, nd);
          const uint32_t tR0 = tS + s_col(i);
          uint32_t pr[64], pk[32], dp[64];
          tmem_ld32(tR0, pr);
          tmem_ld32(tR0 + 32, pr + 32);
          tmem_wait_ld();
          if (C::kScores == 1) {
            tc_fence_before();
            mbar_arrive(bar_s_free);
          }
          if (lim < 64) {  // keys past N: probability 0 whatever lse is
#pragma unroll
            for (int k = 0; k < 64; ++k)
              if (k >= lim) pr[k] = 0xFF800000u;
          }
          exps(pr, [&](int) { return nl2; });
          exps(pr + 32, [&](int) { return nl2; });
          ok = wait(bar_dp, par);
          if (!ok) break;
          tc_fence_after();
          tmem_ld32(tR1, dp);
          tmem_ld32(tR1 + 32, dp + 32);
          tmem_wait_ld();
          dscores(pr, dp, pk, [&](int) { return nd2; });
          dscores(pr + 32, dp + 32, pk + 16, [&](int) { return nd2; });
          tmem_st32(tR1, pk);
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(bar_ds + 8 * h);
        }
      }
    }
    // epilogue: warpgroup h stores accumulator h (dV and dK, or dQ of query
    // tile h).  A thread has a row; through shared memory (the own tiles, which
    // the last MMA has read; chunks swizzled as there) a warp's stores cover
    // whole rows instead of 16 bytes of each of 32 (4,096 tokens x 40 heads 996
    // instead of 1,046 us, 1,024 x 18 heads 48 instead of 53).
    if (ok) ok = wait(bar_acc, 0);
    if (ok && (!is_dq || h < nt)) {
      tc_fence_after();
      const int tok = is_dq ? t0 + 128 * h + row : t0 + row;
      const float f = !is_dq && h == 0 ? 1.0f : p.scale;
      __nv_bfloat16 *base = is_dq ? p.dq : h == 0 ? p.dv : p.dk;
      const uint64_t dst =
          tok < p.N ? reinterpret_cast<uint64_t>(base + bwd_row(p, bh, tok, D)) : 0;
      const uint32_t tA = tmem + lane_bits + (h == 0 ? C::kColA0 : C::kColA1);
      const uint32_t stage = sbase + C::kOffOwn + warp * (64 * D);
#pragma unroll
      for (int c = 0; c < D; c += 32) {
        uint32_t o[32];
        tmem_ld32(tA + c, o);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = pack_bf16x2(__uint_as_float(o[8 * i + 2 * e]) * f,
                               __uint_as_float(o[8 * i + 2 * e + 1]) * f);
          st_shared_v4(stage + lane * 2 * D + (((c / 8 + i) ^ (lane & 7)) << 4),
                       make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
      __syncwarp();
      constexpr int kChunks = D / 8;
      const int cc = lane % kChunks;
#pragma unroll
      for (int r0 = 0; r0 < 32; r0 += 32 / kChunks) {
        const int r = r0 + lane / kChunks;
        const uint64_t d = __shfl_sync(0xffffffffu, dst, r);
        if (d != 0)
          reinterpret_cast<uint4 *>(d)[cc] = ld_shared_v4(stage + r * 2 * D + ((cc ^ (r & 7)) << 4));
      }
    }
  }

  // ------------------------------------------------------------------ teardown
  if (!ok) {
    *abort_flag = 1;
    atomicExch(p.status, kStatusTimeout);
  }
  tc_fence_before();
  __syncthreads();
  if (*abort_flag) {
    // asynchronous work lands before shared and tensor memory are released:
    // of every stage the last load issued into it
    if ((warp == 8 || warp == 10) && lane == 0) {
      const uint32_t own = warp == 8 ? 0 : 1, bar_full = warp == 8 ? bar_x_full : bar_y_full;
      for (int i = 0; i < n_own; ++i)
        mbar_wait_drain(bar_own + 8 * (2 * i + own), 0, kWaitLimitNs);
      for (int i = max(n_ring - stages, 0); i < n_ring; ++i)
        mbar_wait_drain(bar_full + 8 * (i % stages), (i / stages) & 1, kWaitLimitNs);
      for (int i = max(n_stat - 2, 0); i < n_stat; ++i)
        mbar_wait_drain(bar_stat + 8 * (i & 1), (i >> 1) & 1, kWaitLimitNs);
    }
    if (leader) {
      umma_commit(bar_drain);
      mbar_wait_drain(bar_drain, 0, kWaitLimitNs);
    }
    __syncthreads();
  }
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace sp
