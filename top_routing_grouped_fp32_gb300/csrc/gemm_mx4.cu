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
// visited expert by expert, a TMA warp, an MMA warp, epilogue warps, two
// accumulators, bounded waits), with these differences:
//   * a 128-byte swizzled row holds 256 values, so a ring slot is 256 deep, and
//     its four MMAs take about 400 cycles: what the issuing thread does between
//     them counts.  Slots are therefore filled and freed one by one but handed
//     over in pairs (512 columns, a span): one wait for eight MMAs.  The TMA and
//     the MMA warp run their loops as whole warps and elect a lane to issue, so
//     that operands are known to be uniform;
//   * six more warps bring the scales: two copy them several spans ahead into
//     a ring of their own (cp.async, beside the TMA unit, which is busy); each
//     of the four others reads a span's (16 bytes a lane for 32 rows), writes
//     them to its quarter of the TMEM lanes with tcgen05.st (the MMA reads
//     scales from all four), one set of columns for each slot pair, and arrives
//     on the barrier of the pair's copies.  Copied by the same four, 430 cycles
//     a span, the scales were the kernel's pace (1070 cycles a span; the
//     headline's products 502 -> 479 us with the rows, the wide ones' 544 -> 506).
//     Copying them from shared memory (tcgen05.cp) instead holds up the MMAs:
//     about 50 cycles a copy, six copies a slot (the headline's gate/up without
//     its loads and epilogue: 367 us, 250 us of it MMAs), and loading them by
//     TMA takes a fifth of the loads' time;
//   * eight epilogue warps, four for each accumulator, and nothing released
//     later than it must: an arrival on the peer's barrier that orders memory
//     waits for every store and load in flight (2000 cycles of a tile's 6000);
//   * N = 192 on CTA pairs: two accumulators of 256 columns would leave no
//     TMEM for the scales, and accumulators that share columns would stop the
//     MMAs at every tile's end until the epilogue has read the shared part;
//   * a gate/up tile's columns are its gate features, then the same up
//     features (on CTA pairs the leader stages the gate rows, its peer the up
//     rows), so that a lane holds both values of a feature.
// Where rows are 1025 to 2048 values long (HELD), an n-tile's B stays in shared
// memory for up to four m-tiles, and the ring carries A alone.
// What bounds it: on CTA pairs power (200 us of the headline's gate/up are 1.7 GHz
// of 2.07), the MMAs' step of 64 (two thirds of the nominal 4-bit rate; PTX has one
// of 96 for this architecture, not tried here) and the depth that shared memory
// leaves the ring, three spans.  A span
// takes 1070 to 1100 cycles at prompt batches, 800 of them MMAs; the MMA warp waits
// 500 for copies, and these for free slots, or with HELD 260 for copies and 180 for
// the epilogue (all eight warps on each tile, half its columns each, end that wait,
// but not the time: 441 and 440 us).  N = 256 would move a tenth less, for TMEM see
// above.
// Single CTAs serve batches that hold few rows an expert: they are bound by
// reading weights (32 tokens over 256 experts of 7168 x 2048, top-8: 580 us,
// 6.6 TB/s), and many small tiles spread over the SMs.
#include <algorithm>
#include <new>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "tcgen05.cuh"

namespace moe {

struct Mx4Weights {
  CUtensorMap gate96, up96, down96;  // boxes of 96 rows by 256 values
  CUtensorMap gate64, up64, down128;  // boxes of 64 and 128 rows
  const uint8_t *sg, *su, *sd;       // scales in product order
};

namespace mx4 {

using namespace tc;

constexpr int BM = 128;
constexpr uint32_t ROW_BYTES = 128;              // 256 values of a row
constexpr uint32_t A_BYTES = BM * ROW_BYTES;     // 16 KiB
constexpr int THREADS = 512;  // TMA, MMA, eight epilogue and six scale warps
constexpr uint32_t TMEM_COLS = 512;
constexpr int MAX_E = 1024;

constexpr int HELD_MIN = 3, HELD_SPANS = 4;  // spans of B that HELD keeps

template <int PAIR, int BN, bool HELD>
struct Cfg {
  static constexpr int B_ROWS = BN / PAIR;
  static constexpr uint32_t B_BYTES = B_ROWS * ROW_BYTES;
  static constexpr uint32_t SLOT_BYTES = A_BYTES + (HELD ? 0 : B_BYTES);  // 256 columns
  static constexpr uint32_t HELD_BYTES = HELD ? 2 * HELD_SPANS * B_BYTES : 0;
  static constexpr int TABLES = PAIR == 2 && !HELD ? 2 : 3;
  static constexpr uint32_t SF_BYTES = (4 + BN / 32) * mx::kGroupBytes;  // a span's scales
  // what 227 KiB hold beside the tables of MAX_E experts and the barriers
  static constexpr int ROOM = 232448 - 1024 - 512 - 4 * TABLES * (MAX_E + 1) - (int)HELD_BYTES;
  static constexpr int PAIRS = (ROOM - (HELD ? 4 * (int)SF_BYTES : 0)) / (int)SLOT_BYTES / 2;  // of slots
  // depth of the scales' ring, in what is left
  static constexpr int SF_RING = std::min<int>(8, (ROOM - 2 * PAIRS * (int)SLOT_BYTES) / (int)SF_BYTES);
  static_assert(SF_RING >= 4, "scales are read ahead");
  // A held span is read last a row's spans before it is written again, which the
  // wait for A's slots of PAIRS spans ago then covers.
  static_assert(!HELD || PAIRS <= HELD_MIN, "spans between two uses of a held span's place");
  static constexpr int TILE_M = BM * PAIR;
  static constexpr int GROUPS = BN / 32;  // 32-row groups of B
  // TMEM columns: two accumulators, then a set of a span's scales for each slot
  // pair (A: four words of 4 groups, B: four words of GROUPS groups)
  static constexpr uint32_t SF_COL = 2 * BN;
  static constexpr int SF_WORDS = 16 + 4 * GROUPS;
  static_assert(SF_COL + PAIRS * SF_WORDS <= TMEM_COLS, "TMEM");
  static_assert(SLOT_BYTES % 1024 == 0, "slots keep the swizzle's alignment");
};

struct Params {
  const uint32_t* offsets;
  int E;
  int nb;         // n-tiles per m-tile
  int panel;
  int chunk;      // HELD: m-tiles that share an n-tile's B, at most
  int steps;      // slots of a row: 256 columns each
  int gate_up;
  const uint8_t* sa;   // scales in product order
  const uint8_t* sb0;  // gate, or down
  const uint8_t* sb1;  // up, or down again
  int64_t n_out;  // I (gate/up) or H (down)
  int h_spans;    // spans of a row of h (gate/up)
  uint8_t* hq;
  uint8_t* hs;
  void* out;
  const uint32_t* perm;
  const void* weights;
  int wdt;
  int thin_a;
  int v8_out;  // out is 32-byte aligned
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
// R consecutive words of this warp's 32 TMEM lanes
template <int R>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t* r) {
  static_assert(R == 8 || R == 32, "");
  if constexpr (R == 8) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  } else {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
  }
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
// e2m1 A and B, both K-major, exponent scales, FP32 accumulator; the scale ids
// (which pair of a column's four bytes a step uses) are added per step
__host__ __device__ constexpr uint32_t make_idesc(int M, int N) {
  return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) | ((uint32_t)(M >> 4) << 24);
}

struct Tile {
  int e, nb;
  int64_t m0;
  uint32_t unit;  // 256-row unit of scales, and the tile's first group in it
  uint32_t group;
  int a_rows;  // rows of A to load: 128, or 64 or 32 that hold all there are
  int count;   // HELD: m-tiles in a row, from this one, with one B
};

// By a converged warp: every role asks for a tile at its start, and what that
// takes is time without copies.
__device__ __forceinline__ Tile decode_tile(uint32_t tile, const Params& p, const uint32_t* s_pref,
                                            const uint32_t* s_unit, const uint32_t* s_off, int tile_m) {
  const uint32_t q = small_div(tile, (uint32_t)p.nb);
  const int lo = warp_search(s_pref, p.E, q);
  const uint32_t mte = s_pref[lo + 1] - s_pref[lo];
  const uint32_t L = tile - s_pref[lo] * (uint32_t)p.nb;
  const uint32_t w = (uint32_t)p.panel;
  const uint32_t pid = small_div(L, mte * w);
  const uint32_t rem = L - pid * mte * w;
  const uint32_t width = min(w, (uint32_t)p.nb - pid * w);
  const uint32_t mt = small_div(rem, width);
  Tile t;
  t.e = lo;
  t.nb = (int)(pid * w + rem - mt * width);
  t.m0 = (int64_t)s_off[lo] + (int64_t)mt * tile_m;
  t.unit = tile_m == 256 ? s_pref[lo] + mt : s_unit[lo] + (mt >> 1);
  t.group = tile_m == 256 ? 0u : 4u * (mt & 1u);
  const int64_t left = (int64_t)s_off[lo + 1] - t.m0;
  t.a_rows = !p.thin_a || left > 64 ? BM : left > 32 ? 64 : 32;
  t.count = 1;
  return t;
}
// HELD: an n-tile's neighbours take other n-tiles of the same rows.  s_chunk:
// chunks of m-tiles of experts < e
__device__ __forceinline__ Tile decode_chunk(uint32_t tile, const Params& p, const uint32_t* s_pref,
                                             const uint32_t* s_chunk, const uint32_t* s_off, int tile_m) {
  const uint32_t q = small_div(tile, (uint32_t)p.nb);
  const int lo = warp_search(s_chunk, p.E, q);
  const uint32_t mte = s_pref[lo + 1] - s_pref[lo], chunks = s_chunk[lo + 1] - s_chunk[lo], c = q - s_chunk[lo];
  const uint32_t each = small_div(mte, chunks), more = mte - each * chunks;  // the first `more` have one more
  const uint32_t m0 = c * each + min(c, more);
  Tile t;
  t.e = lo;
  t.nb = (int)(tile - q * (uint32_t)p.nb);
  t.m0 = (int64_t)s_off[lo] + (int64_t)m0 * tile_m;
  t.unit = s_pref[lo] + m0;
  t.group = 0;
  t.a_rows = BM;
  t.count = (int)(each + (c < more ? 1u : 0u));
  return t;
}

template <typename T, int PAIR, int BN, bool HELD>
__global__ void __launch_bounds__(THREADS, 1)
gemm_mx4_kernel(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapA64,
                const __grid_constant__ CUtensorMap mapA32,
                const __grid_constant__ CUtensorMap mapB0, const __grid_constant__ CUtensorMap mapB1, const Params p) {
  using C = Cfg<PAIR, BN, HELD>;
  constexpr int PAIRS = C::PAIRS;
  constexpr bool kCluster = PAIR == 2;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t ring = (raw_s + 1023u) & ~1023u;
  uint8_t* ring_ptr = smem_raw + (ring - raw_s);
  const uint32_t held = ring + 2 * PAIRS * C::SLOT_BYTES;
  uint8_t* sf_ring = ring_ptr + 2 * PAIRS * C::SLOT_BYTES + C::HELD_BYTES;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sf_ring + C::SF_RING * C::SF_BYTES);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 3 * PAIRS + 5 + 2 * C::SF_RING);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  uint32_t* s_off = reinterpret_cast<uint32_t*>(reinterpret_cast<uint8_t*>(bars) + 512);
  uint32_t* s_pref = s_off + (p.E + 1);
  uint32_t* s_unit = s_pref + (p.E + 1);  // PAIR == 1 (a pair's tile is a unit), or HELD's chunks

  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int q) { return bar0 + 8u * q; };               // a pair's copies and scales are there
  auto empty_bar = [&](int q, int h) { return bar0 + 8u * (PAIRS + 2 * q + h); };  // slot h's MMAs are done
  auto tfull_bar = [&](int a) { return bar0 + 8u * (3 * PAIRS + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (3 * PAIRS + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (3 * PAIRS + 4);
  auto sfull_bar = [&](int q) { return bar0 + 8u * (3 * PAIRS + 5 + q); };              // scales copied
  auto sempty_bar = [&](int q) { return bar0 + 8u * (3 * PAIRS + 5 + C::SF_RING + q); };  // and read by four warps

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int E = p.E;
  const uint32_t rank = kCluster ? cluster_rank() : 0u;
  const bool leader = rank == 0;
  const uint32_t cluster_id = blockIdx.x / PAIR, num_clusters = gridDim.x / PAIR;

  if (threadIdx.x == 0) {
    for (int q = 0; q < PAIRS; ++q) {
      mbar_init(full_bar(q), 1 + 4 * PAIR);  // the copies, and one arrival per scale warp
      mbar_init(empty_bar(q, 0), 1);
      mbar_init(empty_bar(q, 1), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4 * PAIR);
    }
    for (int q = 0; q < C::SF_RING; ++q) {
      mbar_init(sfull_bar(q), 64);  // every thread that copies
      mbar_init(sempty_bar(q), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    prefetch_map(&mapA);
    if (p.thin_a) {
      prefetch_map(&mapA64);
      prefetch_map(&mapA32);
    }
    prefetch_map(&mapB0);
    prefetch_map(&mapB1);
  }
  if (warp == 1) tmem_alloc<PAIR>(smem_u32(tmem_slot), TMEM_COLS);
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i <= E; i += THREADS) s_off[i] = p.offsets[i];
  __syncthreads();
  if (warp == 2 || (warp == 3 && C::TABLES == 3)) {
    // warp 2: tiles of experts < e; warp 3: 256-row units of scales, or chunks, of experts < e
    const uint32_t unit = warp == 2 ? (uint32_t)C::TILE_M : HELD ? (uint32_t)(C::TILE_M * p.chunk) : 256u;
    uint32_t* dst = warp == 2 ? s_pref : s_unit;
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
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  // (HELD: "tiles" are chunks of m-tiles)
  const uint32_t total_tiles = __shfl_sync(0xffffffffu, (HELD ? s_unit : s_pref)[E] * (uint32_t)p.nb, 0);
  auto tile_at = [&](uint32_t tile) {
    return HELD ? decode_chunk(tile, p, s_pref, s_unit, s_off, C::TILE_M)
                : decode_tile(tile, p, s_pref, s_unit, s_off, C::TILE_M);
  };
  // the m-tiles of a chunk
  auto count_of = [&](const Tile& t) { return HELD ? __shfl_sync(0xffffffffu, t.count, 0) : 1; };
  const uint32_t full0_leader = kCluster ? mapa(full_bar(0), 0) : full_bar(0);
  const uint32_t tempty0_leader = kCluster ? mapa(tempty_bar(0), 0) : tempty_bar(0);
  const int spans = (p.steps + 1) / 2;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    // The whole warp runs the loop, so that what the copies and the MMAs take
    // is known to be the same in every lane; one elected lane issues.
    int pr = 0;
    uint32_t phase = 0, fills = 0;
    bool ok = true;
    for (uint32_t tile = cluster_id; ok && tile < total_tiles; tile += num_clusters) {
      const Tile t = tile_at(tile);
      const int a_row = __shfl_sync(0xffffffffu, (int)(t.m0 + (int64_t)rank * BM), 0);
      const int te = __shfl_sync(0xffffffffu, t.e, 0);
      const int tnb = __shfl_sync(0xffffffffu, t.nb, 0);
      const int a_rows = __shfl_sync(0xffffffffu, t.a_rows, 0);
      const int count = count_of(t);
      const int n0 = tnb * (p.gate_up ? BN / 2 : BN);  // first feature, or first output column
      const int b_row = PAIR == 2 && !p.gate_up ? n0 + (int)rank * C::B_ROWS : n0;
      int sp = 0, m = 0;
      for (int i = 0; i < spans * count; ++i) {
        const bool two = 2 * sp + 1 < p.steps;
        const uint32_t slot_tx = ((m == 0 ? C::B_BYTES : 0u) + (uint32_t)a_rows * ROW_BYTES) * PAIR;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ok = __all_sync(0xffffffffu, mbar_wait<kCluster>(empty_bar(pr, h), phase ^ 1u, abort_flag, p.status));
          if (!ok) {
            fills += h;  // the pair's first copies are in flight
            break;
          }
          if ((h == 0 || two) && elect_one()) {
            const uint32_t sa = ring + (2 * pr + h) * C::SLOT_BYTES;
            const uint32_t sb = HELD ? held + (2 * sp + h) * C::B_BYTES : sa + A_BYTES;
            const uint32_t fb = full0_leader + 8u * pr;
            const int kx = (2 * sp + h) * (int)ROW_BYTES;
            if (leader && h == 0) mbar_expect_tx(full_bar(pr), two ? 2 * slot_tx : slot_tx);
            if (a_rows == 32) tma_load_2d<PAIR>(sa, &mapA32, kx, a_row, fb);
            else if (a_rows == 64) tma_load_2d<PAIR>(sa, &mapA64, kx, a_row, fb);
            else tma_load_2d<PAIR>(sa, &mapA, kx, a_row + m * C::TILE_M, fb);
            if (HELD && m != 0) {  // B is there
            } else if (PAIR == 2) {  // gate rows and up rows, or the two halves of the down rows
              if (leader) tma_load_3d<PAIR>(sb, &mapB0, kx, b_row, te, fb);
              else tma_load_3d<PAIR>(sb, &mapB1, kx, b_row, te, fb);
            } else {
              tma_load_3d<PAIR>(sb, &mapB0, kx, b_row, te, fb);
              if (p.gate_up) tma_load_3d<PAIR>(sb + C::B_BYTES / 2, &mapB1, kx, b_row, te, fb);
            }
          }
          __syncwarp();
        }
        if (!ok) break;
        ++fills;
        if (++pr == PAIRS) {
          pr = 0;
          phase ^= 1u;
        }
        if (++sp == spans) {
          sp = 0;
          ++m;
        }
      }
    }
    if (!ok && leader && lane == 0) {  // aborting: let the copies in flight land before exit
      for (uint32_t i = fills > PAIRS ? fills - PAIRS : 0; i < fills; ++i) {
        const uint64_t t0 = global_timer();
        while (!mbar_test<kCluster>(full_bar(i % PAIRS), (i / PAIRS) & 1u) && global_timer() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader CTA)
    if (leader) {
      constexpr uint32_t idesc = make_idesc(C::TILE_M, BN);
      const uint64_t hi = sw128_desc(0);
      int pr = 0;
      uint32_t phase = 0, acc = 0, acc_phase = 0;
      bool ok = true;
      int count = HELD && cluster_id < total_tiles ? count_of(tile_at(cluster_id)) : 1;
      for (uint32_t tile = cluster_id; ok && tile < total_tiles;) {
        ok = __all_sync(0xffffffffu, mbar_wait<kCluster>(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p.status));
        if (!ok) break;
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int sp = 0; sp < spans; ++sp) {
          ok = __all_sync(0xffffffffu, mbar_wait<kCluster>(full_bar(pr), phase, abort_flag, p.status));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sf = tmem_base + C::SF_COL + pr * C::SF_WORDS;
            const uint32_t s0 = ring + 2 * pr * C::SLOT_BYTES;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              if (h == 0 || 2 * sp + 1 < p.steps) {
                const uint32_t sa = s0 + h * C::SLOT_BYTES;
                const uint32_t sb = HELD ? held + (2 * sp + h) * C::B_BYTES : sa + A_BYTES;
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // scales: bytes 0-1 or 2-3 of word 2 h + k / 2
                  const uint32_t id = idesc | (uint32_t)(k & 1) * ((2u << 29) | (2u << 4));
                  const int w = 2 * h + (k >> 1);
                  umma_mx4<PAIR>(d_tmem, hi | ((sa + k * 32) & 0x3FFFFu) >> 4, hi | ((sb + k * 32) & 0x3FFFFu) >> 4,
                                 id, sf + w * 4, sf + 16 + w * C::GROUPS, (h | k) != 0 ? 1u : sp != 0);
                }
              }
              umma_commit<PAIR>(empty_bar(pr, h));
            }
            if (sp == spans - 1) umma_commit<PAIR>(tfull_bar(acc));
          }
          __syncwarp();
          if (++pr == PAIRS) {
            pr = 0;
            phase ^= 1u;
          }
        }
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
        if (--count == 0) {
          tile += num_clusters;
          count = HELD && tile < total_tiles ? count_of(tile_at(tile)) : 1;
        }
      }
      if (elect_one()) {
        umma_commit_local<PAIR>(drain_bar);
        const uint64_t t0 = global_timer();
        while (!mbar_test<false>(drain_bar, 0) && global_timer() - t0 < kWaitLimitNs) {
        }
      }
      __syncwarp();
    }
  } else if (warp >= 14) {
    // ------------------------------------------------------------ scales: copies
    constexpr int G = C::GROUPS, MINE = (4 + G) / 2;  // of A's 4 and B's G groups, every other one
    static_assert(G % 2 == 0, "");
    const int wi = warp - 14;
    const uint32_t dst0 = smem_u32(sf_ring) + wi * mx::kGroupBytes + lane * 16;
    const int64_t per = p.n_out / 32;  // groups of an expert
    uint32_t slot = 0, phase = 0;
    bool ok = true;
    for (uint32_t tile = cluster_id; ok && tile < total_tiles; tile += num_clusters) {
      const Tile t = tile_at(tile);
      const int count = count_of(t);
      const uint8_t* pa =
          p.sa + ((int64_t)t.unit * spans * mx::kUnitGroups + t.group + rank * 4 + wi) * mx::kGroupBytes + lane * 16;
      const uint8_t* pb[MINE - 2];
#pragma unroll
      for (int i = 0; i < MINE - 2; ++i) {
        const int j = wi + 2 * i;  // the halves of the columns: gate and up features, or down columns
        const bool second = p.gate_up && j >= G / 2;
        const int64_t g = p.gate_up ? (int64_t)t.nb * (G / 2) + (second ? j - G / 2 : j) : (int64_t)t.nb * G + j;
        pb[i] = g < per ? (second ? p.sb1 : p.sb0) + ((int64_t)t.e * spans * per + g) * mx::kGroupBytes + lane * 16
                        : nullptr;
      }
      int sp = 0;
      for (int i = 0; i < spans * count; ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait<false>(sempty_bar(slot), phase ^ 1u, abort_flag, p.status));
        if (!ok) break;
        const uint32_t dst = dst0 + slot * C::SF_BYTES;
        async_copy16(dst, pa);
        async_copy16(dst + 2 * mx::kGroupBytes, pa + 2 * mx::kGroupBytes);
        pa += mx::kUnitGroups * mx::kGroupBytes;
#pragma unroll
        for (int j = 0; j < MINE - 2; ++j)
          if (pb[j]) async_copy16(dst + (4 + 2 * j) * mx::kGroupBytes, pb[j] + sp * per * mx::kGroupBytes);
        async_copy_arrive(sfull_bar(slot));
        if (++sp == spans) sp = 0;
        if (++slot == C::SF_RING) {
          slot = 0;
          phase ^= 1u;
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp >= 10) {
    // ------------------------------------------------------------ scales: to TMEM
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    constexpr int G = C::GROUPS, W = C::SF_WORDS, RING = C::SF_RING;
    bool ok = true;
    uint32_t pr = 0, phase = 0, slot = 0, sphase = 0;
    for (uint32_t mine = cluster_id; ok && mine < total_tiles; mine += num_clusters) {
      const int all = HELD ? spans * count_of(tile_at(mine)) : spans;
      for (int sp = 0; sp < all; ++sp) {
        ok = __all_sync(0xffffffffu, mbar_wait<false>(sfull_bar(slot), sphase, abort_flag, p.status));
        if (!ok) break;
        uint32_t w[W];
        const uint4* src = reinterpret_cast<const uint4*>(sf_ring + slot * C::SF_BYTES) + lane;
#pragma unroll
        for (int j = 0; j < 4 + G; ++j) {
          const uint4 v = src[j * 32];
          const int at = j < 4 ? j : 12 + j, step = j < 4 ? 4 : G;
          w[at] = v.x;
          w[at + step] = v.y;
          w[at + 2 * step] = v.z;
          w[at + 3 * step] = v.w;
        }
        // the MMAs that read this set last are done
        ok = __all_sync(0xffffffffu, mbar_wait<kCluster>(empty_bar(pr, 1), phase ^ 1u, abort_flag, p.status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t ta = tmem_base + lanes + C::SF_COL + pr * C::SF_WORDS;
        tmem_st<32>(ta, w);
        if constexpr (W > 32) tmem_st<8>(ta + 32, w + 32);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if constexpr (kCluster) mbar_arrive_cluster_relaxed(full0_leader + 8u * pr);
          else mbar_arrive(full_bar(pr));
          mbar_arrive(sempty_bar(slot));  // every lane has used what it read
        }
        if (++pr == PAIRS) {
          pr = 0;
          phase ^= 1u;
        }
        if (++slot == RING) {
          slot = 0;
          sphase ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // four warps for each accumulator: they have the time of two tiles
    const int quarter = warp & 3;
    const uint32_t acc = (uint32_t)(warp - 2) >> 2;
    uint32_t acc_phase = 0;
    int ok = 1, parity = 0;
    for (uint64_t tile = cluster_id + (HELD ? 0 : acc * num_clusters); ok && tile < total_tiles;
         tile += (HELD ? 1 : 2) * num_clusters) {
      Tile t = tile_at((uint32_t)tile);
      const int count = count_of(t);
      // HELD: every other one of the m-tiles that follow one another
      for (int m = 0; m < count; ++m, t.m0 += C::TILE_M, ++t.unit, parity ^= 1) {
        if (HELD && parity != (int)acc) continue;
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
          uint8_t* srow =
              p.hs + ((int64_t)t.unit * p.h_spans * mx::kUnitGroups + t.group + rank * 4 + quarter) * mx::kGroupBytes +
              lane * 16;
#pragma unroll 1
          for (int b = 0; b < BN / 64; ++b) {
            const int blk = b0 + b;
            if (blk >= blocks) break;
            uint32_t g[32], u[32];
            __syncwarp();
            tmem_ld32(taddr + b * 32, g);
            tmem_ld32(taddr + BN / 2 + b * 32, u);
            tmem_wait_ld(g);
            reg_fence(u);
            float2 h[16];
            uint32_t a = 0;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 gg = make_float2(__uint_as_float(g[2 * i]), __uint_as_float(g[2 * i + 1]));
              const float2 uu = make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
              const float2 t = mul2(gg, both(-kLog2e));
              const float2 n = add2(make_float2(exp2_fast(t.x), exp2_fast(t.y)), both(1.f));
              // a few ulp of FP32: far below an e2m1 step.  silu(g) first: g u may
              // leave FP32's range where silu(g) u does not (g far below 0)
              h[i] = mul2(mul2(gg, make_float2(rcp_fast(n.x), rcp_fast(n.y))), uu);
              a = max(a, max(mx::abs_bits(h[i].x), mx::abs_bits(h[i].y)));
            }
            const uint32_t sb = mx::scale_byte<MOE_MXFP4>(a);
            // (a block with a NaN has scale NaN; its elements then do not matter)
            const float2 inv = both(mx::inverse_scale(sb));
            uint32_t w[4];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float q[8];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 y = mul2(h[4 * v + i], inv);
                q[2 * i] = y.x;
                q[2 * i + 1] = y.y;
              }
              w[v] = mx::to_e2m1x8(q);
            }
            if (row_ok) {
              *reinterpret_cast<uint4*>(hrow + blk * 16) = make_uint4(w[0], w[1], w[2], w[3]);
              uint8_t* d = srow + (int64_t)(blk >> 4) * (mx::kUnitGroups * mx::kGroupBytes);
              d[blk & 15] = (uint8_t)sb;
              if (blk == blocks - 1)  // the row's last span: finite scales behind its end
                for (int c = (blk & 15) + 1; c < 16; ++c) d[c] = 0;
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
              uint32_t* d = reinterpret_cast<uint32_t*>(static_cast<T*>(p.out) + slot * p.n_out + c0 + c);
              uint32_t q[16];
#pragma unroll
              for (int v = 0; v < 4; ++v) {
                float f[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(o[v * 8 + i]);
                const uint4 r = pack8<T>(f);
                q[4 * v] = r.x;
                q[4 * v + 1] = r.y;
                q[4 * v + 2] = r.z;
                q[4 * v + 3] = r.w;
              }
              if (p.v8_out) {  // whole 32-byte sectors
                st_v8(d, q);
                st_v8(d + 8, q + 8);
              } else {
#pragma unroll
                for (int v = 0; v < 4; ++v)
                  reinterpret_cast<uint4*>(d)[v] = make_uint4(q[4 * v], q[4 * v + 1], q[4 * v + 2], q[4 * v + 3]);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          // its TMEM reads are done; a release would wait for the tile's stores
          if constexpr (kCluster) mbar_arrive_cluster_relaxed(tempty0_leader + 8u * acc);
          else mbar_arrive(tempty_bar(acc));
        }
        acc_phase ^= 1u;
      }
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
template <int PAIR, int BN, bool HELD>
size_t smem_bytes(int E) {
  using C = Cfg<PAIR, BN, HELD>;
  return 1024 + (size_t)C::PAIRS * 2 * C::SLOT_BYTES + C::HELD_BYTES + (size_t)C::SF_RING * C::SF_BYTES + 512 +
         4 * (size_t)C::TABLES * (E + 1);
}

template <typename T, int PAIR, int BN, bool HELD = false>
cudaError_t launch_t(const Mx4Args& a, const Mx4Weights* w, int num_sms, cudaStream_t s, int chunk = 1) {
  using C = Cfg<PAIR, BN, HELD>;
  const int64_t K = a.gate_up ? a.H : a.I;
  CUtensorMap mA, mA64, mA32;
  if (!encode_rows(&mA, a.a, a.N, K / 2, BM)) return cudaErrorInvalidValue;
  mA64 = mA32 = mA;  // CTA pairs load whole tiles
  if (PAIR == 1 && (!encode_rows(&mA64, a.a, a.N, K / 2, 64) || !encode_rows(&mA32, a.a, a.N, K / 2, 32)))
    return cudaErrorInvalidValue;
  Params p{};
  p.offsets = a.offsets;
  p.E = a.E;
  p.steps = (int)((K + 255) / 256);
  p.gate_up = a.gate_up;
  p.n_out = a.gate_up ? a.I : a.H;
  const int64_t cols = a.gate_up ? 2 * a.I : a.H;  // columns of the product
  p.nb = (int)((cols + BN - 1) / BN);
  p.sa = static_cast<const uint8_t*>(a.a_scales);
  p.sb0 = a.gate_up ? w->sg : w->sd;
  p.sb1 = a.gate_up ? w->su : w->sd;
  p.h_spans = (int)mx::spans(a.I);
  p.hq = static_cast<uint8_t*>(a.hq);
  p.hs = static_cast<uint8_t*>(a.hs);
  p.out = a.out;
  p.v8_out = reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
  p.perm = a.perm;
  p.weights = a.weights;
  p.wdt = (int)a.wdt;
  p.thin_a = PAIR == 1;
  p.chunk = chunk;
  p.status = a.status;
  static PerDevice known;
  int clusters = 0;
  cudaError_t err = resident_clusters<PAIR>(gemm_mx4_kernel<T, PAIR, BN, HELD>, THREADS, smem_bytes<PAIR, BN, HELD>(MAX_E),
                                            num_sms, known, &clusters);
  if (err != cudaSuccess) return err;
  if (clusters < 1) return cudaErrorLaunchOutOfResources;
  constexpr int TM = C::TILE_M;
  const int64_t mt_max = (a.N + TM - 1) / TM + std::min<int64_t>(a.E, a.N);
  const int nclu = (int)std::max<int64_t>(1, std::min<int64_t>(clusters, mt_max * p.nb));
  // panel width: about one wave of clusters spread over an expert's expected m-tiles
  const int64_t mt_per_expert = std::max<int64_t>(1, (a.N + (int64_t)TM * a.E - 1) / ((int64_t)TM * a.E));
  p.panel = (int)std::max<int64_t>(1, std::min<int64_t>(p.nb, (nclu + mt_per_expert - 1) / mt_per_expert));
  const CUtensorMap& b0 = PAIR == 2 ? (a.gate_up ? w->gate96 : w->down96) : (a.gate_up ? w->gate64 : w->down128);
  const CUtensorMap& b1 = !a.gate_up ? b0 : PAIR == 2 ? w->up96 : w->up64;
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
  cfg.dynamicSmemBytes = smem_bytes<PAIR, BN, HELD>(a.E);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, gemm_mx4_kernel<T, PAIR, BN, HELD>, mA, mA64, mA32, b0, b1, p);
}

// m-tiles that share a B held in shared memory, or 1: B is loaded for each.  Held,
// an SM takes in 44 instead of 62 KiB a span, but by larger pieces of work: six
// chunks a CTA pair at least.  2048 x 1408, us of both products and the rows,
// loaded and held: 98304 rows over 64 experts 483 and 446, 32768 over eight 172
// and 157, 8192 over eight 61 and 66 (here not held).  Rows of one or two spans
// lose (65536 of 1024 x 512 over 32 experts: 123 and 129), longer ones than four
// have no room.
int held_chunk(const Mx4Args& a, int num_sms) {
  const int64_t K = a.gate_up ? a.H : a.I, cols = a.gate_up ? 2 * a.I : a.H;
  if (mx::spans(K) < HELD_MIN || mx::spans(K) > HELD_SPANS) return 1;
  const int64_t tiles = (a.N + 255) / 256 * ((cols + 191) / 192) / std::max(1, num_sms / 2);
  const int64_t mean = (a.N + 256 * (int64_t)a.E - 1) / (256 * (int64_t)a.E);  // m-tiles of an expert
  return (int)std::max<int64_t>(1, std::min<int64_t>({tiles / 6, mean, 4}));
}

}  // namespace mx4

size_t mx4_weight_scale_bytes(int64_t rows, int64_t C) {
  return (size_t)(rows / mx::kGroupRows) * mx::spans(C) * mx::kGroupBytes;
}
size_t mx4_row_scale_bytes(int64_t N, int64_t E, int64_t C) {
  // every expert's rows begin a 256-row unit of their own
  return (size_t)(mx::kUnitGroups * ((N + 255) / 256 + std::min<int64_t>(E, N))) * mx::spans(C) * mx::kGroupBytes;
}

Mx4Weights* mx4_weights_create(const void* gate, const void* up, const void* down, const uint8_t* sg,
                               const uint8_t* su, const uint8_t* sd, int64_t E, int64_t I, int64_t H,
                               const char** err) {
  if (!tc::encode_fn()) {
    *err = "cuTensorMapEncodeTiled is not available from the driver";
    return nullptr;
  }
  Mx4Weights* w = new (std::nothrow) Mx4Weights();
  if (!w) {
    *err = "out of host memory";
    return nullptr;
  }
  w->sg = sg;
  w->su = su;
  w->sd = sd;
  using mx4::encode_weights;
  if (!encode_weights(&w->gate96, gate, E, I, H / 2, 96) || !encode_weights(&w->up96, up, E, I, H / 2, 96) ||
      !encode_weights(&w->down96, down, E, H, I / 2, 96) || !encode_weights(&w->gate64, gate, E, I, H / 2, 64) ||
      !encode_weights(&w->up64, up, E, I, H / 2, 64) || !encode_weights(&w->down128, down, E, H, I / 2, 128)) {
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
  const int chunk = pair ? mx4::held_chunk(a, num_sms) : 1;
  if (chunk > 1)
    return a.dt == MOE_BF16 ? mx4::launch_t<__nv_bfloat16, 2, 192, true>(a, w, num_sms, s, chunk)
                            : mx4::launch_t<__half, 2, 192, true>(a, w, num_sms, s, chunk);
  if (a.dt == MOE_BF16)
    return pair ? mx4::launch_t<__nv_bfloat16, 2, 192>(a, w, num_sms, s)
                : mx4::launch_t<__nv_bfloat16, 1, 128>(a, w, num_sms, s);
  return pair ? mx4::launch_t<__half, 2, 192>(a, w, num_sms, s) : mx4::launch_t<__half, 1, 128>(a, w, num_sms, s);
}

}  // namespace moe
