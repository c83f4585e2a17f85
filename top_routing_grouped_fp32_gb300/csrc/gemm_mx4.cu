// gemm_mx4.cu -- the experts' products on 4-bit microscaled operands.
//
// For every dispatched row r of expert e, with A the row's e2m1 elements times
// its scales and W the weights held the same way (mx.cuh):
//   gate/up : g = A . W_gate^T, u = A . W_up^T in one accumulator tile, then
//             h = silu(g) u, rounded to e2m1 blocks in the epilogue (a lane
//             holds a row's 32 features of a block, so neither the largest
//             value nor the scale leaves the lane) and stored as the operand
//             of the down product with its scales in product order;
//   down    : out = h . W_down^T, stored in dispatch order or, times the
//             routing weight of its slot, as FP32 at that token slot.
// tcgen05.mma kind::mxf4 takes both operands packed (64 values deep a step) and
// multiplies by the scales itself; sums are FP32 in TMEM.  Elements times
// scales have at most four significant bits, so products are exact.
//
// The kernel is the segmented, persistent one of the 16-bit products (tiles
// visited expert by expert, a TMA warp, an MMA thread, four epilogue warps,
// two accumulators, bounded waits), with these differences:
//   * a 128-byte swizzled row holds 256 values, so a ring stage is 256 deep;
//   * scales travel with their stage: one kilobyte for 128 rows, copied from
//     shared memory to TMEM (tcgen05.cp, 32 lanes by 16 bytes, replicated to
//     the four lane quarters) by the thread that issues the MMAs, in order
//     with them.  Two sets of scale columns are used in turn;
//   * N = 192 on CTA pairs: two accumulators of 256 columns would leave no
//     TMEM for the scales, and accumulators that share columns would stop the
//     MMAs at every tile's end until the epilogue has read the shared part.
//     192 columns are three blocks of 32 gate features with their up features;
//   * gate and up rows alternate by 32 (gate, up, gate, up ...), so that a
//     tile's columns hold both values of the same features in blocks.  Weight
//     scales are laid out once in that order, 128 rows a piece: a tile that
//     begins in the middle of a piece addresses its scales two columns on.
// Single CTAs with N = 64 serve batches that hold few rows an expert: they are
// bound by reading weights, and many small tiles spread over the SMs.
#include <algorithm>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "tcgen05.cuh"

namespace moe {

struct Mx4Weights {
  CUtensorMap gate32, up32;    // boxes of 32 rows by 256 values
  CUtensorMap down96, down64;  // boxes of 96 and 64 rows
  CUtensorMap sgu2, sgu1;      // scale pairs of two pieces, of one
  CUtensorMap sd2, sd1;
  int64_t E, I, H;
};

namespace mx4 {

using namespace tc;

constexpr int BM = 128;
constexpr uint32_t ROW_BYTES = 128;              // 256 values of a row
constexpr uint32_t A_BYTES = BM * ROW_BYTES;     // 16 KiB
constexpr uint32_t SF_BYTES = 1024;              // scales of 128 rows by 256 values
constexpr int THREADS = 192;
constexpr uint32_t TMEM_COLS = 512;
constexpr int MAX_E = 1024;

template <int PAIR, int BN>
struct Cfg {
  static constexpr int B_ROWS = BN / PAIR;
  static constexpr uint32_t B_BYTES = B_ROWS * ROW_BYTES;
  static constexpr int SFB_PIECES = BN > 128 ? 2 : 1;
  static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES + SF_BYTES * (1 + SFB_PIECES);
  static constexpr int STAGES = (int)(222208 / STAGE_BYTES);
  static constexpr int TILE_M = BM * PAIR;
  // TMEM columns: two accumulators, then two sets of scales (A: 2 x 4, B: 2 x 8)
  static constexpr uint32_t SF_COL = 2 * BN;
  static constexpr uint32_t SF_SET = 32;
  static_assert(SF_COL + 2 * SF_SET <= TMEM_COLS, "TMEM");
  static_assert(STAGE_BYTES % 1024 == 0, "stages keep the swizzle's alignment");
};

struct Params {
  const uint32_t* offsets;
  int E;
  int nb;         // n-tiles per m-tile
  int panel;
  int steps;      // 256-deep steps
  int gate_up;
  int b_pieces;   // 128-row scale pieces per expert and step
  int64_t n_out;  // I (gate/up) or H (down)
  int h_steps;    // depth steps of h (gate/up)
  uint8_t* hq;
  uint8_t* hs;
  void* out;
  const uint32_t* perm;
  const void* weights;
  int wdt;
  int thin_a;
  uint32_t* status;
};

// D (+)= A . B^T, 64 values deep, scales in TMEM
template <int PAIR>
__device__ __forceinline__ void umma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                         uint32_t sfb, uint32_t accumulate) {
  if constexpr (PAIR == 2) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  }
}
// 32 lanes by 16 bytes of shared memory to four TMEM columns, in every lane quarter
template <int PAIR>
__device__ __forceinline__ void copy_scales(uint32_t taddr, uint64_t desc) {
  if constexpr (PAIR == 2)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc) : "memory");
}
// 512 contiguous bytes without swizzle: groups of 8 rows of 16 bytes, 128 bytes apart
__device__ __forceinline__ uint64_t scale_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(128 >> 4) << 32) | ((uint64_t)1 << 46);
}
// e2m1 A and B, both K-major, exponent scales, FP32 accumulator; the scale ids
// (which pair of a column's four bytes a step uses) are added per step
__host__ __device__ constexpr uint32_t make_idesc(int M, int N) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}

struct Tile {
  int e, nb;
  int64_t m0;
  uint32_t piece;  // scale piece of the tile's first row
  bool thin;
};

__device__ __forceinline__ Tile decode_tile(uint32_t tile, const Params& p, const uint32_t* s_pref,
                                            const uint32_t* s_piece, const uint32_t* s_off, int tile_m) {
  const uint32_t q = tile / (uint32_t)p.nb;
  int lo = 0, hi = p.E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_pref[mid] <= q) lo = mid; else hi = mid;
  }
  const uint32_t mte = s_pref[lo + 1] - s_pref[lo];
  const uint32_t L = tile - s_pref[lo] * (uint32_t)p.nb;
  const uint32_t w = (uint32_t)p.panel;
  const uint32_t pid = L / (mte * w);
  const uint32_t rem = L - pid * mte * w;
  const uint32_t width = min(w, (uint32_t)p.nb - pid * w);
  const uint32_t mt = rem / width;
  Tile t;
  t.e = lo;
  t.nb = (int)(pid * w + rem % width);
  t.m0 = (int64_t)s_off[lo] + (int64_t)mt * tile_m;
  t.piece = tile_m == 256 ? 2 * (s_pref[lo] + mt) : 2 * s_piece[lo] + mt;
  t.thin = p.thin_a && (int64_t)s_off[lo + 1] - t.m0 <= 32;
  return t;
}

template <typename T, int PAIR, int BN>
__global__ void __launch_bounds__(THREADS, 1)
gemm_mx4_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapA32,
                const __grid_constant__ CUtensorMap mapB0, const __grid_constant__ CUtensorMap mapB1,
                const __grid_constant__ CUtensorMap mapSA, const __grid_constant__ CUtensorMap mapSB, const Params p) {
  using C = Cfg<PAIR, BN>;
  constexpr int STAGES = C::STAGES;
  constexpr bool kCluster = PAIR == 2;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t ring = (raw_s + 1023u) & ~1023u;
  uint8_t* ring_ptr = smem_raw + (ring - raw_s);
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring_ptr + STAGES * C::STAGE_BYTES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  uint32_t* s_off = reinterpret_cast<uint32_t*>(ring_ptr + STAGES * C::STAGE_BYTES + 256);
  uint32_t* s_pref = s_off + (p.E + 1);
  uint32_t* s_piece = s_pref + (p.E + 1);  // PAIR == 1 only: a pair's tile is two pieces

  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int E = p.E;
  const uint32_t rank = kCluster ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  const uint32_t cluster_id = blockIdx.x / PAIR, num_clusters = gridDim.x / PAIR;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4 * PAIR);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    prefetch_map(&mapA);
    if (p.thin_a) prefetch_map(&mapA32);
    prefetch_map(&mapB0);
    prefetch_map(&mapB1);
    prefetch_map(&mapSA);
    prefetch_map(&mapSB);
  }
  if (warp == 1) tmem_alloc<PAIR>(smem_u32(tmem_slot), TMEM_COLS);
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i <= E; i += THREADS) s_off[i] = p.offsets[i];
  __syncthreads();
  if (warp == 2 || (warp == 3 && PAIR == 1)) {
    // warp 2: tiles of experts < e; warp 3: 256-row units of scales of experts < e
    const uint32_t unit = warp == 2 ? (uint32_t)C::TILE_M : 256u;
    uint32_t* dst = warp == 2 ? s_pref : s_piece;
    const int per = (E + 31) / 32;
    uint32_t loc = 0;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < E) loc += (s_off[e + 1] - s_off[e] + unit - 1) / unit;
    }
    uint32_t incl = loc;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    uint32_t run = incl - loc;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < E) {
        dst[e] = run;
        run += (s_off[e + 1] - s_off[e] + unit - 1) / unit;
      }
    }
    if (lane == 31) dst[E] = incl;
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kCluster) cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t total_tiles = s_pref[E] * (uint32_t)p.nb;
  auto tile_at = [&](uint32_t tile) { return decode_tile(tile, p, s_pref, s_piece, s_off, C::TILE_M); };
  const uint32_t full0_leader = kCluster ? mapa(full_bar(0), 0) : full_bar(0);
  const uint32_t tempty0_leader = kCluster ? mapa(tempty_bar(0), 0) : tempty_bar(0);

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t last_fill[STAGES];
      bool filled[STAGES];
      for (int s = 0; s < STAGES; ++s) filled[s] = false, last_fill[s] = 0;
      bool ok = true;
      for (uint32_t tile = cluster_id; ok && tile < total_tiles; tile += num_clusters) {
        const Tile t = tile_at(tile);
        const int a_row = (int)(t.m0 + (int64_t)rank * BM);
        const CUtensorMap* ma = t.thin ? &mapA32 : &mapA;
        const uint32_t stage_tx = (t.thin ? C::STAGE_BYTES - (A_BYTES - A_BYTES / 4) : C::STAGE_BYTES) * PAIR;
        const int n0 = t.nb * BN;
        const int sa_row = (int)((t.piece + rank) * (uint32_t)p.steps);
        const int sb_row = t.e * p.steps * p.b_pieces + (n0 >> 7);
        for (int kb = 0; kb < p.steps; ++kb) {
          if (!mbar_wait<kCluster>(empty_bar(stage), phase ^ 1u, abort_flag, p.status)) {
            ok = false;
            break;
          }
          const uint32_t sa = ring + stage * C::STAGE_BYTES;
          const uint32_t sb = sa + A_BYTES, sf = sb + C::B_BYTES;
          const uint32_t fb = full0_leader + 8u * stage;
          const int kx = kb * (int)ROW_BYTES;
          if (leader) mbar_expect_tx(full_bar(stage), stage_tx);
          tma_load_2d<PAIR>(sa, ma, kx, a_row, fb);
          if (p.gate_up) {
#pragma unroll
            for (int q = 0; q < C::B_ROWS / 32; ++q) {
              const int grp = (n0 >> 5) + (int)rank * (C::B_ROWS / 32) + q;  // gate, up, gate, up ...
              tma_load_3d<PAIR>(sb + q * 32 * ROW_BYTES, (grp & 1) ? &mapB1 : &mapB0, kx, (grp >> 1) * 32, t.e, fb);
            }
          } else {
            tma_load_3d<PAIR>(sb, &mapB0, kx, n0 + (int)rank * C::B_ROWS, t.e, fb);
          }
          tma_load_2d<PAIR>(sf, &mapSA, 0, sa_row + kb, fb);
          tma_load_2d<PAIR>(sf + SF_BYTES, &mapSB, 0, sb_row + kb * p.b_pieces, fb);
          filled[stage] = true;
          last_fill[stage] = phase;
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (!ok && leader) {  // aborting: let the copies in flight land before exit
        for (int s = 0; s < STAGES; ++s) {
          if (!filled[s]) continue;
          const uint64_t t0 = global_timer();
          while (!mbar_test<kCluster>(full_bar(s), last_fill[s]) && global_timer() - t0 < kWaitLimitNs) {
          }
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader CTA)
    if (lane == 0 && leader) {
      constexpr uint32_t idesc = make_idesc(C::TILE_M, BN);
      const uint64_t hi = sw128_desc(0), sf_hi = scale_desc(0);
      int stage = 0;
      uint32_t phase = 0, acc = 0, acc_phase = 0, set = 0;
      bool ok = true;
      for (uint32_t tile = cluster_id; ok && tile < total_tiles; tile += num_clusters) {
        const Tile t = tile_at(tile);
        const uint32_t shift = (uint32_t)((t.nb * BN) & 127) >> 5;  // columns into the first scale piece
        if (!mbar_wait<kCluster>(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p.status)) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = 0; kb < p.steps; ++kb) {
          if (!mbar_wait<kCluster>(full_bar(stage), phase, abort_flag, p.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = ring + stage * C::STAGE_BYTES;
          const uint32_t sb = sa + A_BYTES, sf = sb + C::B_BYTES;
          const uint32_t ta = tmem_base + C::SF_COL + set * C::SF_SET, tb = ta + 8;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            copy_scales<PAIR>(ta + half * 4, sf_hi | ((sf + half * 512) & 0x3FFFFu) >> 4);
#pragma unroll
            for (int q = 0; q < C::SFB_PIECES; ++q)
              copy_scales<PAIR>(tb + half * 8 + q * 4, sf_hi | ((sf + SF_BYTES * (1 + q) + half * 512) & 0x3FFFFu) >> 4);
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t id = idesc | (uint32_t)(k & 1) * ((2u << 29) | (2u << 4));
            umma_mx4<PAIR>(d_tmem, hi | ((sa + k * 32) & 0x3FFFFu) >> 4, hi | ((sb + k * 32) & 0x3FFFFu) >> 4, id,
                           ta + (k >> 1) * 4, tb + (k >> 1) * 8 + shift, (kb | k) != 0 ? 1u : 0u);
          }
          set ^= 1u;
          umma_commit<PAIR>(empty_bar(stage));
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        umma_commit<PAIR>(tfull_bar(acc));
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
      umma_commit_local<PAIR>(drain_bar);
      const uint64_t t0 = global_timer();
      while (!mbar_test<false>(drain_bar, 0) && global_timer() - t0 < kWaitLimitNs) {
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;
    uint32_t acc = 0, acc_phase = 0;
    for (uint32_t tile = cluster_id; tile < total_tiles; tile += num_clusters) {
      const Tile t = tile_at(tile);
      const int row = quarter * 32 + lane;
      const int64_t grow = t.m0 + (int64_t)rank * BM + row;
      const bool row_ok = grow < (int64_t)s_off[t.e + 1];
      int64_t slot = grow;
      float wscale = 1.f;
      if (p.perm != nullptr && row_ok) {
        const uint32_t s = __ldg(p.perm + grow);
        slot = s;
        wscale = load_dyn(p.weights, p.wdt, s);
      }
      int ok = 1;
      if (lane == 0) ok = mbar_wait<kCluster>(tfull_bar(acc), acc_phase, abort_flag, p.status) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * BN;
      // the warps' 32 rows have rows to store, or nothing is read
      const bool any = __any_sync(0xffffffffu, row_ok);
      if (any && p.gate_up) {
        const int blocks = (int)(p.n_out / 32), b0 = t.nb * (BN / 64);
        uint8_t* hrow = p.hq + grow * (p.n_out / 2);
        uint8_t* srow = p.hs + (int64_t)(t.piece + rank) * p.h_steps * 1024;
#pragma unroll 1
        for (int b = 0; b < BN / 64; ++b) {
          const int blk = b0 + b;
          if (blk >= blocks) break;
          uint32_t g[32], u[32];
          __syncwarp();
          tmem_ld32(taddr + b * 64, g);
          tmem_ld32(taddr + b * 64 + 32, u);
          tmem_wait_ld(g);
          reg_fence(u);
          float h[32];
          uint32_t a = 0;
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float gg = __uint_as_float(g[i]), uu = __uint_as_float(u[i]);
            // a few ulp of FP32: far below an e2m1 step
            h[i] = __fdividef(gg * uu, 1.f + __expf(-gg));
            a = max(a, mx::abs_bits(h[i]));
          }
          const uint32_t sb = mx::scale_byte<MOE_MXFP4>(a);
          const float inv = mx::inverse_scale(sb);
          uint32_t w[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            float q[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = sb == 255u ? 0.f : h[v * 8 + i] * inv;
            w[v] = mx::to_e2m1x8(q);
          }
          if (row_ok) {
            *reinterpret_cast<uint4*>(hrow + blk * 16) = make_uint4(w[0], w[1], w[2], w[3]);
            uint8_t* d = srow + (int64_t)(blk >> 3) * 1024;
            d[mx::pair_byte((uint32_t)row, (uint32_t)blk & 7u)] = (uint8_t)sb;
            if (blk == blocks - 1)  // the row's last pair: finite scales behind its end
              for (int c = (blk & 7) + 1; c < 8; ++c) d[mx::pair_byte((uint32_t)row, (uint32_t)c)] = 0;
          }
        }
      } else if (any) {
        const int64_t c0 = (int64_t)t.nb * BN;
#pragma unroll 1
        for (int c = 0; c < BN; c += 32) {
          if (c0 + c >= p.n_out) break;
          uint32_t o[32];
          __syncwarp();
          tmem_ld32(taddr + c, o);
          tmem_wait_ld(o);
          if (row_ok && p.perm != nullptr) {
            float4* d = reinterpret_cast<float4*>(static_cast<float*>(p.out) + slot * p.n_out + c0 + c);
#pragma unroll
            for (int v = 0; v < 8; ++v)
              d[v] = make_float4(__uint_as_float(o[4 * v]) * wscale, __uint_as_float(o[4 * v + 1]) * wscale,
                                 __uint_as_float(o[4 * v + 2]) * wscale, __uint_as_float(o[4 * v + 3]) * wscale);
          } else if (row_ok) {
            uint4* d = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + slot * p.n_out + c0 + c);
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(o[v * 8 + i]);
              d[v] = pack8<T>(f);
            }
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kCluster) mbar_arrive_cluster(tempty0_leader + 8u * acc);
        else mbar_arrive(tempty_bar(acc));
      }
      acc ^= 1u;
      if (acc == 0) acc_phase ^= 1u;
    }
  }

  __syncthreads();
  if constexpr (kCluster) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<PAIR>(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- host side
// rows x bytes (rows of whole 16-byte vectors), box `box_rows` x 128 bytes, swizzled
bool encode_rows(CUtensorMap* m, const void* base, uint64_t rows, uint64_t bytes, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {bytes, rows};
  cuuint64_t strides[1] = {bytes};
  cuuint32_t box[2] = {ROW_BYTES, box_rows};
  cuuint32_t estr[2] = {1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool encode_weights(CUtensorMap* m, const void* base, uint64_t E, uint64_t rows, uint64_t bytes, uint32_t box_rows) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {bytes, rows, E};
  cuuint64_t strides[2] = {bytes, rows * bytes};
  cuuint32_t box[3] = {ROW_BYTES, box_rows, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// n kilobytes of scales, `box_kb` of them a load
bool encode_scales(CUtensorMap* m, const void* base, uint64_t n, uint32_t box_kb) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {SF_BYTES / 4, n};
  cuuint64_t strides[1] = {SF_BYTES};
  cuuint32_t box[2] = {SF_BYTES / 4, box_kb};
  cuuint32_t estr[2] = {1u, 1u};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int PAIR, int BN>
size_t smem_bytes(int E) {
  return 1024 + (size_t)Cfg<PAIR, BN>::STAGES * Cfg<PAIR, BN>::STAGE_BYTES + 256 +
         4 * (size_t)(PAIR == 2 ? 2 : 3) * (E + 1);
}

// Clusters of PAIR CTAs that can be resident at once (one CTA per SM), asked
// once per device.
template <typename T, int PAIR, int BN>
cudaError_t resident_clusters(int num_sms, int* out) {
  static std::mutex lock;
  static int clusters[64] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  std::lock_guard<std::mutex> g(lock);
  int n = clusters[dev & 63];
  if (n == 0) {
    const size_t smem = smem_bytes<PAIR, BN>(MAX_E);
    err = cudaFuncSetAttribute(gemm_mx4_kernel<T, PAIR, BN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (err != cudaSuccess) return err;
    n = num_sms;
    if (PAIR == 2) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = PAIR;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(PAIR * (num_sms / PAIR));
      cfg.blockDim = dim3(THREADS);
      cfg.dynamicSmemBytes = smem;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      err = cudaOccupancyMaxActiveClusters(&n, gemm_mx4_kernel<T, PAIR, BN>, &cfg);
      if (err != cudaSuccess) return err;
    }
    clusters[dev & 63] = n;
  }
  *out = n;
  return cudaSuccess;
}

template <typename T, int PAIR, int BN>
cudaError_t launch_t(const Mx4Args& a, const Mx4Weights* w, int num_sms, cudaStream_t s) {
  using C = Cfg<PAIR, BN>;
  const int64_t K = a.gate_up ? a.H : a.I;
  CUtensorMap mA, mA32, mSA;
  const uint64_t a_kb = mx4_row_scale_bytes(a.N, a.E, K) / SF_BYTES;
  if (!encode_rows(&mA, a.a, a.N, K / 2, BM) || !encode_rows(&mA32, a.a, a.N, K / 2, 32) ||
      !encode_scales(&mSA, a.a_scales, a_kb, 1))
    return cudaErrorInvalidValue;
  Params p{};
  p.offsets = a.offsets;
  p.E = a.E;
  p.steps = (int)mx::depth_steps(K);
  p.gate_up = a.gate_up;
  p.n_out = a.gate_up ? a.I : a.H;
  const int64_t cols = a.gate_up ? 2 * a.I : a.H;  // columns of the product
  p.nb = (int)((cols + BN - 1) / BN);
  p.b_pieces = (int)(a.gate_up ? mx4_gate_up_pieces(a.I) : mx4_down_pieces(a.H));
  p.h_steps = (int)mx::depth_steps(a.I);
  p.hq = static_cast<uint8_t*>(a.hq);
  p.hs = static_cast<uint8_t*>(a.hs);
  p.out = a.out;
  p.perm = a.perm;
  p.weights = a.weights;
  p.wdt = (int)a.wdt;
  p.thin_a = PAIR == 1;
  p.status = a.status;
  int clusters = 0;
  cudaError_t err = resident_clusters<T, PAIR, BN>(num_sms, &clusters);
  if (err != cudaSuccess) return err;
  if (clusters < 1) return cudaErrorLaunchOutOfResources;
  constexpr int TM = C::TILE_M;
  const int64_t mt_max = (a.N + TM - 1) / TM + std::min<int64_t>(a.E, a.N);
  const int nclu = (int)std::max<int64_t>(1, std::min<int64_t>(clusters, mt_max * p.nb));
  // panel width: about one wave of clusters spread over an expert's expected m-tiles
  const int64_t mt_per_expert = std::max<int64_t>(1, (a.N + (int64_t)TM * a.E - 1) / ((int64_t)TM * a.E));
  p.panel = (int)std::max<int64_t>(1, std::min<int64_t>(p.nb, (nclu + mt_per_expert - 1) / mt_per_expert));
  const CUtensorMap& b0 = a.gate_up ? w->gate32 : PAIR == 2 ? w->down96 : w->down64;
  const CUtensorMap& b1 = a.gate_up ? w->up32 : b0;
  const CUtensorMap& sb = a.gate_up ? (C::SFB_PIECES == 2 ? w->sgu2 : w->sgu1) : (C::SFB_PIECES == 2 ? w->sd2 : w->sd1);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PAIR;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(nclu * PAIR);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem_bytes<PAIR, BN>(a.E);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_mx4_kernel<T, PAIR, BN>, mA, mA32, b0, b1, mSA, sb, p);
}

}  // namespace mx4

int64_t mx4_gate_up_pieces(int64_t I) { return (2 * I + 127) / 128; }
int64_t mx4_down_pieces(int64_t H) { return (H + 127) / 128; }
size_t mx4_gate_up_scale_bytes(int64_t E, int64_t I, int64_t H) {
  return (size_t)(E * mx::depth_steps(H) * mx4_gate_up_pieces(I)) * mx4::SF_BYTES;
}
size_t mx4_down_scale_bytes(int64_t E, int64_t I, int64_t H) {
  return (size_t)(E * mx::depth_steps(I) * mx4_down_pieces(H)) * mx4::SF_BYTES;
}
size_t mx4_row_scale_bytes(int64_t N, int64_t E, int64_t C) {
  // every expert's rows begin an even piece of their own
  return (size_t)(2 * ((N + 255) / 256 + std::min<int64_t>(E, N))) * mx::depth_steps(C) * mx4::SF_BYTES;
}

Mx4Weights* mx4_weights_create(const void* gate, const void* up, const void* down, const void* sgu, const void* sd,
                               int64_t E, int64_t I, int64_t H, const char** err) {
  if (!tc::encode_fn()) {
    *err = "cuTensorMapEncodeTiled is not available from the driver";
    return nullptr;
  }
  Mx4Weights* w = new (std::nothrow) Mx4Weights();
  if (!w) {
    *err = "out of host memory";
    return nullptr;
  }
  w->E = E;
  w->I = I;
  w->H = H;
  const uint64_t ngu = mx4_gate_up_scale_bytes(E, I, H) / mx4::SF_BYTES, nd = mx4_down_scale_bytes(E, I, H) / mx4::SF_BYTES;
  if (!mx4::encode_weights(&w->gate32, gate, E, I, H / 2, 32) || !mx4::encode_weights(&w->up32, up, E, I, H / 2, 32) ||
      !mx4::encode_weights(&w->down96, down, E, H, I / 2, 96) ||
      !mx4::encode_weights(&w->down64, down, E, H, I / 2, 64) || !mx4::encode_scales(&w->sgu2, sgu, ngu, 2) ||
      !mx4::encode_scales(&w->sgu1, sgu, ngu, 1) || !mx4::encode_scales(&w->sd2, sd, nd, 2) ||
      !mx4::encode_scales(&w->sd1, sd, nd, 1)) {
    *err = "cuTensorMapEncodeTiled rejected a 4-bit expert weight tensor";
    delete w;
    return nullptr;
  }
  return w;
}

void mx4_weights_destroy(Mx4Weights* w) { delete w; }

cudaError_t launch_gemm_mx4(const Mx4Args& a, const Mx4Weights* w, int num_sms, cudaStream_t s) {
  // CTA pairs where experts hold at least a full 128-row tile on average
  const bool pair = a.N >= (int64_t)128 * a.E;
  if (a.dt == MOE_BF16)
    return pair ? mx4::launch_t<__nv_bfloat16, 2, 192>(a, w, num_sms, s)
                : mx4::launch_t<__nv_bfloat16, 1, 64>(a, w, num_sms, s);
  return pair ? mx4::launch_t<__half, 2, 192>(a, w, num_sms, s) : mx4::launch_t<__half, 1, 64>(a, w, num_sms, s);
}

}  // namespace moe
