// gemm_tc.cu -- persistent segmented grouped GEMM on Blackwell tensor cores.
//
// Computes the three expert products of SwiGluExperts::forward_dispatched_with_
// strategy in src/moe/experts.rs (ruDNN 0.1.25 source view): for every
// dispatched row r of expert e, A[r,:] . W[e]^T, with
//   gate/up : both products in one accumulator tile, epilogue h = silu(g) * u
//             (silu(z) = z * sigmoid(z), MindSpeed-Ops PR 163, rms_norm_gated
//             notes), stored as the 16-bit operand of the down product;
//   down    : o = h . W_down[e]^T, stored either in dispatch order
//             (moe_experts_forward) or multiplied by the routing weight of
//             its slot and stored at that token slot (fused forward: the
//             weight scale and the un-permute of the user guide's combine,
//             section 6, move into this epilogue).
// The pages' own grouped product is a scalar or "cooperative matrix" loop
// (prior art); this is an sm_103a design:
//
//   * persistent CTAs over a tile list built on the device from offsets[]
//     (segment lengths are never read by the host); a tile is 128*PAIR rows
//     x 256 FP32 accumulator columns of one expert, except that on CTA pairs
//     a segment's last tile holding at most 128 rows runs as a half tile
//     (M = 128 over the pair, 64 rows per CTA), halving its padding;
//   * PAIR = 2 (the default): a cluster of two CTAs on two SMs runs one
//     tcgen05.mma.cta_group::2 of M=256: each CTA stages its own 128 rows of A
//     and one 128-row half of B (for gate/up: 64 gate rows and the same 64 up
//     rows, so that every accumulator lane holds gate and up of the same
//     features; for down: one half of the 256 down rows), so an SM moves
//     32 KiB per 64-deep k-block instead of 48 KiB; the forward products
//     ring three 128-deep stages of 64 KiB (KS = 2), the backward products
//     and long-K down projections six 64-deep ones; PAIR = 1 is the
//     single-CTA form (M=128, both B halves staged locally, 4 stages; a tile
//     of at most 32 rows loads A through a 32-row box);
//   * warp 0: TMA producer (cp.async.bulk.tensor, 128-byte swizzle); its
//     copies complete on the leader CTA's "full" barrier;
//   * warp 1: allocates 512 TMEM columns; in the leader CTA one thread issues
//     the MMAs (kind::f16, FP32 accumulate) and tcgen05.commit frees ring
//     stages and hands finished accumulators to both CTAs' epilogues;
//   * warps 2-5: epilogue; each reads its 32 TMEM lanes (= 32 tile rows) with
//     tcgen05.ld while the MMA fills the other accumulator;
//   * rows past the end of a segment are computed (the A box may run into the
//     next expert's rows or past the buffer, where TMA fills zeros) and never
//     stored, so segments of any length are handled without padding;
//   * tiles are visited expert by expert; inside an expert, column panels of
//     `panel` n-blocks are swept over all its m-tiles so that CTAs running at
//     the same time share weight tiles in L2;
//   * the same kernel runs the five products of the expert backward
//     (ExpertTrainingCache::backward in src/moe/experts.rs): operands may be
//     MN-major in shared memory (weights and row blocks read as stored, no
//     transposes), the weight-gradient products take a per-expert K range
//     over 64-padded rows, and their epilogues store FP32 tiles.
//
// Every wait on an mbarrier is bounded: after ~2 s the CTA records
// MOE_ERR_DEVICE_TIMEOUT in the workspace status word, stops issuing work,
// waits (bounded) for its own copies and MMAs in flight, frees its TMEM and
// returns.
#include <cudaTypedefs.h>

#include <algorithm>
#include <limits>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "parts.h"
#include "tcgen05.cuh"

namespace moe {

// Prebuilt TMA descriptors of one expert-weight set (gate, up [E,I,H]; down [E,H,I]).
struct TcWeights {
  CUtensorMap gate;  // CUtensorMap carries its own 64-byte alignment
  CUtensorMap up;
  CUtensorMap down;
  CUtensorMap gate64;  // 64-row boxes: the interleaved gate/up operand of CTA pairs
  CUtensorMap up64;
  int64_t E, I, H;
};

namespace tc {

constexpr int BM = 128;        // rows per CTA
constexpr int BN = 256;        // FP32 accumulator columns per tile
constexpr int BK = 64;         // 64 16-bit elements = one 128-byte swizzle row
static_assert(BM == parts::kRows && BN == parts::kCols && BK == parts::kDepth, "what parts.h counts in");
constexpr int UMMA_K = 16;
constexpr uint32_t A_BYTES = BM * BK * 2;        // 16 KiB
constexpr uint32_t B_HALF_BYTES = 128 * BK * 2;  // 16 KiB
// TMA warp, MMA warp, and four epilogue warps, or four for each accumulator in
// the checkpointed backward, whose epilogues do more than its products
template <int CK>
constexpr int kEpilogues = CK == 2 ? 2 : 1;
template <int CK>
constexpr int kThreads = 64 + 128 * kEpilogues<CK>;
constexpr uint32_t TMEM_COLS = 2 * BN;
constexpr int MAX_E = 1024;
constexpr float kFltMax = std::numeric_limits<float>::max();

// KS: 64-deep K sub-blocks per ring stage.  KS = 2 (forward CTA-pair GEMMs,
// K-major operands) halves the barrier round trips and commits per MMA: one
// stage holds A sub-blocks 0..KS-1, then B sub-blocks 0..KS-1, each in the
// 128-byte-swizzled layout of one TMA box.
template <int PAIR, int KS = 1>
struct Cfg {
  static constexpr int STAGES = KS == 2 ? 3 : (PAIR == 1 ? 4 : 6);
  static constexpr uint32_t B_BYTES = (PAIR == 1 ? 2u : 1u) * B_HALF_BYTES;  // B staged per CTA per sub-block
  static constexpr uint32_t STAGE_BYTES = KS * (A_BYTES + B_BYTES);
  static constexpr int TILE_M = BM * PAIR;
};

struct Params {
  const uint32_t* offsets;
  int E;
  int nb;             // n-blocks per m-tile
  int panel;          // n-blocks per raster panel
  int k_blocks;       // k-blocks per tile: 64-deep, 128-deep when KS = 2
  int mode;
  int cols_per_tile;  // output columns per tile: 128 (gate/up) or 256 (down)
  int b1_row_off;     // row offset of the second B box inside the n-block
  int64_t n_out;
  void* out;
  const uint32_t* perm;
  const void* weights;
  int wdt;
  uint32_t* status;
  // backward products
  void* out2;          // second output (kSwigluBwd: a; kWgrad: rows >= split)
  const void* da;      // kSwigluBwd: da = dout W_down, 16-bit [rows, n_out]
  const uint32_t* pad; // pad[e] = sum over e' < e of roundup(rows of e', 64)
  // operand forms: A K-major (rows x K) or MN-major (K rows x M columns);
  // B K-major 3-D, MN-major 3-D (experts x K rows x N columns) or MN-major 2-D
  int a_mn;
  int b_form;
  int a_row_pad;       // A rows live in the 64-padded row space (row - offsets[e] + pad[e])
  int kb_split;        // > 0: k-blocks from here on read map B1 and A columns from a_k2 on
  int a_k2;
  // kWgrad: per-expert product over the padded row range [pad[e], pad[e+1])
  int wgrad;
  int mb;              // m-tiles per expert
  // kWgrad with a_tail: A's rows are read where they are, not from a padded
  // copy; a segment's last rows, short of 64, come from a copy of their own
  // (64 rows an expert, zeros behind them; the mapA64 slot)
  int a_tail;
  // parts that K is cut into, each a tile of its own with an FP32 output: of
  // kWgrad [E, k_parts, ...], of kPartial [k_parts, m_total, n_out]; 0 or 1: none
  int k_parts;
  int64_t m_total;     // M of the product
  int64_t split;       // output rows per buffer (M, or I for the [dgate; dup] pair)
  // forward products on CTA pairs: a segment's last m-tile holding at most
  // 128 rows runs as a half tile, an M = 128 tcgen05.mma.cta_group::2 (64 rows
  // per CTA, A loaded through mapA64): half the MMA work of a padded 256-row tile
  int half_tails;
  // gate/up on CTA pairs: B is staged interleaved, each CTA's 128-row half of
  // the N = 256 operand being [64 gate rows | the same 64 up rows] (mapB0 /
  // mapB1 then have 64-row boxes), so that every accumulator lane holds the
  // gate and up values of the same features in both tile forms
  int b_inter;
  int v8_out;  // out rows are 32-byte aligned segments (n_out % 16 == 0, 32-byte base)
  // 8-bit checkpoints of the gate and up products [rows, I] with a scale a
  // 32-column block: written by the gate/up product (CK = kSave), read by the
  // da product (CK = kUse)
  uint8_t* ck_g;
  uint8_t* ck_u;
  uint8_t* ck_gs;
  uint8_t* ck_us;
  // single CTAs (decode-sized batches): a tile of at most 32 rows loads A
  // through a 32-row box (the mapA64 slot); the MMA still runs M = 128, and
  // its other 96 rows multiply whatever the ring stage held before -- rows
  // that are never stored
  int thin_a;
};

// ---------------------------------------------------------------- epilogue stores
// Each lane of an epilogue warp holds one tile row; storing straight from
// registers would make every store instruction touch 32 rows.  Instead a
// warp's 32 rows x WORDS 32-bit words pass through its staging buffer (rows
// padded by 4 words against bank conflicts) and are written back CH = WORDS/4
// lanes per row, so each store instruction covers whole row segments
// (4 rows x 128 bytes for WORDS = 32, 8 rows x 64 bytes for WORDS = 16).
constexpr int STG_STRIDE = 36;                         // words per staged row
constexpr uint32_t STG_BYTES_PER_WARP = 32 * STG_STRIDE * 4;
constexpr uint32_t STG_BYTES = 4 * STG_BYTES_PER_WARP;  // 18 KiB
constexpr uint32_t STG16_BYTES_PER_WARP = 32 * 20 * 4;   // rows of 16 words
template <int CK>
constexpr uint32_t kStgBytes = CK == 2 ? 8 * STG16_BYTES_PER_WARP : STG_BYTES;

__device__ __forceinline__ void put4(uint32_t* w, uint4 q) {
  w[0] = q.x;
  w[1] = q.y;
  w[2] = q.z;
  w[3] = q.w;
}
// 32-bit words of a row segment that lie inside the output (cols_left >= 0)
template <typename V>
__device__ __forceinline__ int valid_words(int64_t cols_left) {
  const int64_t w = cols_left * (int64_t)sizeof(V) / 4;
  return w < 0 ? 0 : (int)(w < 32 ? w : 32);
}
// dst: this lane's row segment (nullptr: the row is not stored); the
// segment's first `valid` words are written (a multiple of 4).
template <int WORDS>
__device__ __forceinline__ void staged_store(uint32_t* stg, const uint32_t* w, uint32_t* dst, int valid,
                                             int lane) {
  constexpr int STRIDE = WORDS + 4;
  constexpr int CH = WORDS / 4;   // 16-byte chunks per row
  constexpr int RPI = 32 / CH;    // rows per store instruction
#pragma unroll
  for (int j = 0; j < CH; ++j)
    *reinterpret_cast<uint4*>(stg + lane * STRIDE + 4 * j) =
        make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
  __syncwarp();
  const int j = lane % CH;
#pragma unroll
  for (int it = 0; it < CH; ++it) {
    const int r = lane / CH + RPI * it;
    const uint4 v = *reinterpret_cast<const uint4*>(stg + r * STRIDE + 4 * j);
    uint32_t* d = reinterpret_cast<uint32_t*>(
        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), r));
    if (d != nullptr && 4 * j < valid) *reinterpret_cast<uint4*>(d + 4 * j) = v;
  }
  __syncwarp();
}

// 32 words of each of the warp's 32 rows as whole lines, 16 rows at a time
// through 16 x 36 words of shared memory: where stores set the pace (weight
// gradients of 128 experts of 2048 x 768 over 16384 rows) 183 and 116 us, with
// staged_store's half lines 222 and 138
__device__ __forceinline__ void staged_lines(uint32_t* stg, const uint32_t* w, uint32_t* dst, int valid, int lane) {
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (lane >> 4 == half)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4*>(stg + (lane & 15) * 36 + 4 * j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    __syncwarp();
    const int j = lane & 7;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int r = (lane >> 3) + 4 * it;
      const uint4 v = *reinterpret_cast<const uint4*>(stg + r * 36 + 4 * j);
      uint32_t* d = reinterpret_cast<uint32_t*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(dst), 16 * half + r));
      if (d != nullptr && 4 * j < valid) *reinterpret_cast<uint4*>(d + 4 * j) = v;
    }
    __syncwarp();
  }
}

// The descriptor of sw128_desc for an MN-major tile: each TMA box holds 64 K rows of 64
// consecutive M (or N) elements, 128 bytes a row, swizzled in 8-row groups
// 1024 bytes apart (stride offset); boxes for the next 64 M/N elements follow
// 8 KiB apart (leading offset).
constexpr uint32_t MN_BOX_BYTES = 64 * BK * 2;  // 8 KiB
__device__ __forceinline__ uint64_t sw128_mn_desc(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4)
         | ((uint64_t)(MN_BOX_BYTES >> 4) << 16)   // leading offset: next 64 M/N elements
         | ((uint64_t)(1024 >> 4) << 32)           // stride offset: next 8 K rows
         | ((uint64_t)1 << 46)
         | ((uint64_t)2 << 61);
}
// A 32-column block of a row in 8 bits: `left` of its columns (a multiple of 8)
// lie inside the row; those behind hold zeros and do not move the scale.
__device__ __forceinline__ void store_mx8(const uint32_t (&r)[32], uint8_t* dst, int64_t left, uint8_t* scale) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) a = max(a, r[i] & 0x7FFFFFFFu);
  const uint32_t sb = mx::scale_byte<MOE_MXFP8>(a);
  const float inv = mx::inverse_scale(sb);
  uint32_t w[8];
#pragma unroll
  for (int v = 0; v < 8; ++v) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = sb == 255u ? 0.f : __uint_as_float(r[4 * v + i]) * inv;
    w[v] = mx::to_e4m3x4(q);
  }
  if (left >= 32 && reinterpret_cast<uintptr_t>(dst) % 16 == 0) {
    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v)
      if (left >= 8 * v + 8) reinterpret_cast<uint2*>(dst)[v] = make_uint2(w[2 * v], w[2 * v + 1]);
  }
  *scale = (uint8_t)sb;
}
// The elements of such a block (zeros past `left`)
__device__ __forceinline__ void load_mx8(const uint8_t* src, int64_t left, uint32_t (&w)[8]) {
  if (left >= 32 && reinterpret_cast<uintptr_t>(src) % 32 == 0) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(src));
  } else {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const uint2 a = left >= 8 * v + 8 ? __ldg(reinterpret_cast<const uint2*>(src) + v) : make_uint2(0u, 0u);
      w[2 * v] = a.x;
      w[2 * v + 1] = a.y;
    }
  }
}

// What a kernel does with the 8-bit checkpoints of the gate and up products
enum Checkpoint { kNone = 0, kSave = 1, kUse = 2 };
enum BForm { kBKmajor3d = 0, kBMNmajor3d = 1, kBMNmajor2d = 2 };
// Instruction descriptor: FP32 accumulator, 16-bit A/B (bf16 or f16), both
// K-major (bits 15/16 set below make A/B MN-major), M = 128*PAIR, N = 256.
__host__ __device__ constexpr uint32_t make_idesc(bool bf16, int M) {
  return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) |
         ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// ---------------------------------------------------------------- tile list
struct Tile {
  int e;
  int nb;
  int64_t m0;  // first row of the (pair) tile
  int kx0;     // first K coordinate (0, or pad[e] for weight gradients)
  int nk;      // k-blocks of this tile
  int kb0;     // its first k-block, where K is cut into parts
  int eo;      // weight gradients: (expert, part of K), where its output lies; else the part of K
  bool half;   // M = 128 pair tile (64 rows per CTA): see Params::half_tails
  bool thin;   // single-CTA tile of at most 32 rows: see Params::thin_a
};

// By a converged warp.
__device__ __forceinline__ Tile decode_tile(uint32_t tile, const Params& p, const uint32_t* s_pref,
                                            const uint32_t* s_off, int tile_m) {
  uint32_t part = 0;
  if (p.k_parts > 1) {  // the tiles of one part of K, then those of the next
    const uint32_t base = s_pref[p.E] * (uint32_t)p.nb;
    part = small_div(tile, base);
    tile -= part * base;
  }
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
  t.kx0 = 0;
  t.kb0 = p.k_parts > 1 ? (int)((uint32_t)p.k_blocks * part / (uint32_t)p.k_parts) : 0;
  t.nk = (p.k_parts > 1 ? (int)((uint32_t)p.k_blocks * (part + 1) / (uint32_t)p.k_parts) : p.k_blocks) - t.kb0;
  t.eo = (int)part;
  t.half = p.half_tails && (int64_t)s_off[lo + 1] - t.m0 <= BM;
  t.thin = p.thin_a && (int64_t)s_off[lo + 1] - t.m0 <= 32;
  return t;
}

// Weight-gradient tiles: expert-major, then m-tile, then n-block; the K range
// is the expert's padded column range of the transposed operands.
__device__ __forceinline__ Tile decode_wgrad(uint32_t tile, const Params& p, const uint32_t* s_pad, int tile_m) {
  const uint32_t per = (uint32_t)(p.mb * p.nb);
  Tile t;
  t.eo = (int)small_div(tile, per);
  t.e = p.k_parts > 1 ? (int)small_div((uint32_t)t.eo, (uint32_t)p.k_parts) : t.eo;
  const uint32_t rem = tile - (uint32_t)t.eo * per;
  const uint32_t m = small_div(rem, (uint32_t)p.nb);
  t.m0 = (int64_t)m * tile_m;
  t.nb = (int)(rem - m * (uint32_t)p.nb);
  const uint32_t k0 = s_pad[t.e], k1 = s_pad[t.e + 1];
  // this part's share of the expert's k-blocks
  const uint32_t nkb = (k1 - k0) / BK, part = (uint32_t)(t.eo - t.e * p.k_parts);
  const uint32_t f0 = p.k_parts > 1 ? small_div(nkb * part, (uint32_t)p.k_parts) : 0u;
  const uint32_t f1 = p.k_parts > 1 ? small_div(nkb * (part + 1), (uint32_t)p.k_parts) : nkb;
  t.kx0 = (int)(k0 + f0 * BK);
  t.kb0 = (int)f0;
  t.nk = (int)(f1 - f0);
  t.half = false;
  t.thin = false;
  return t;
}

// ---------------------------------------------------------------- the kernel
// CK = kSave: the gate/up product also writes its checkpoints.  CK = kUse: the
// da product of the checkpointed backward (kSwigluBwd on da's own accumulators)
// and weight gradients stored in T.
template <typename T, int PAIR, int KS, int CK>
__global__ void __launch_bounds__(kThreads<CK>, 1)
grouped_gemm_tc(const __grid_constant__ CUtensorMap mapA, const __grid_constant__ CUtensorMap mapB0,
                const __grid_constant__ CUtensorMap mapB1, const __grid_constant__ CUtensorMap mapA64,
                const Params p) {
  using C = Cfg<PAIR, KS>;
  constexpr int STAGES = C::STAGES;
  constexpr bool kCluster = PAIR == 2;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t ring = (raw_s + 1023u) & ~1023u;  // 1024-byte aligned for the swizzle
  uint8_t* ring_ptr = smem_raw + (ring - raw_s);
  uint32_t* staging = reinterpret_cast<uint32_t*>(ring_ptr + STAGES * C::STAGE_BYTES);
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring_ptr + STAGES * C::STAGE_BYTES + kStgBytes<CK>);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 5);
  volatile uint32_t* abort_flag = tmem_slot + 1;
  uint32_t* s_off = reinterpret_cast<uint32_t*>(ring_ptr + STAGES * C::STAGE_BYTES + kStgBytes<CK> + 256);
  uint32_t* s_pref = s_off + (p.E + 1);

  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
  auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
  auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int E = p.E;
  const uint32_t rank = kCluster ? cluster_rank() : 0u;  // this CTA's half of the pair tile
  const bool leader = rank == 0;
  const uint32_t cluster_id = blockIdx.x / PAIR, num_clusters = gridDim.x / PAIR;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull_bar(a), 1);
      mbar_init(tempty_bar(a), 4 * PAIR);  // one arrival per epilogue warp of every CTA
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    prefetch_map(&mapA);
    if (p.half_tails || p.thin_a || p.a_tail) prefetch_map(&mapA64);
    prefetch_map(&mapB0);
    prefetch_map(&mapB1);
  }
  if (warp == 1) tmem_alloc<PAIR>(smem_u32(tmem_slot), TMEM_COLS);
  // everything above overlaps the predecessor kernel (programmatic launch);
  // from here on the kernel reads what earlier kernels wrote
  pdl_wait();
  pdl_trigger();
  for (int i = threadIdx.x; i <= E; i += kThreads<CK>) s_off[i] = p.offsets[i];
  __syncthreads();
  if (p.wgrad) {  // s_pref[e] = first padded row of expert e
    for (int i = threadIdx.x; i <= E; i += kThreads<CK>) s_pref[i] = p.pad[i];
  } else if (warp == 2) {  // s_pref[e] = number of (128*PAIR)-row tiles of experts < e
    const int per = (E + 31) / 32;
    uint32_t loc = 0;
    for (int i = 0; i < per; ++i) {
      const int e = lane * per + i;
      if (e < E) loc += (s_off[e + 1] - s_off[e] + C::TILE_M - 1) / C::TILE_M;
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
        s_pref[e] = run;
        run += (s_off[e + 1] - s_off[e] + C::TILE_M - 1) / C::TILE_M;
      }
    }
    if (lane == 31) s_pref[E] = incl;
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kCluster) cluster_sync();  // the peer's barriers exist before any remote use
  tc_fence_after();
  const uint32_t tmem_base = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  const uint32_t total_tiles = __shfl_sync(
      0xffffffffu, p.wgrad ? (uint32_t)E * (uint32_t)(p.mb * p.nb * p.k_parts) : s_pref[E] * (uint32_t)(p.nb * max(p.k_parts, 1)), 0);
  auto tile_at = [&](uint32_t tile) {
    return p.wgrad ? decode_wgrad(tile, p, s_pref, C::TILE_M) : decode_tile(tile, p, s_pref, s_off, C::TILE_M);
  };
  // the leader CTA's barriers, as seen from this CTA
  const uint32_t full0_leader = kCluster ? mapa(full_bar(0), 0) : full_bar(0);
  const uint32_t tempty0_leader = kCluster ? mapa(tempty_bar(0), 0) : tempty_bar(0);

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    // This warp and the next run their loops whole, so that the operands of
    // copies and MMAs are known to be the same in every lane, and elect one
    // lane to issue (issued by a single lane in a branch of its own, four MMAs
    // take as long to issue as to run).
    int stage = 0;
    uint32_t phase = 0, fills = 0;
    bool ok = true;
    for (uint32_t tile = cluster_id; ok && tile < total_tiles; tile += num_clusters) {
      const Tile t = tile_at(tile);
      const int te = __shfl_sync(0xffffffffu, t.e, 0);
      const int tnb = __shfl_sync(0xffffffffu, t.nb, 0);
      const int kx0 = __shfl_sync(0xffffffffu, t.kx0, 0);
      const int nk = __shfl_sync(0xffffffffu, t.nk, 0);
      const bool half = __all_sync(0xffffffffu, t.half), thin = __all_sync(0xffffffffu, t.thin);
      // A's row (K-major) or M column (MN-major) of this CTA's half: 128
      // rows, or 64 for a half tile
      int row = (int)(t.m0 + (int64_t)rank * (half ? BM / 2 : BM));
      if (p.a_row_pad) row += (int)(__ldg(p.pad + t.e) - s_off[t.e]);
      const int a_row = __shfl_sync(0xffffffffu, row, 0);
      const int a_k0 = p.a_tail ? __shfl_sync(0xffffffffu, (int)s_off[t.e] + t.kb0 * BK, 0) : 0;
      // this tile's last k-block is the segment's, and is cut
      const bool a_cut = p.a_tail && __all_sync(0xffffffffu, s_off[t.e] + (uint32_t)(t.kb0 + t.nk) * BK > s_off[t.e + 1]);
      const int b0row = tnb * p.cols_per_tile;
      const int b1row = b0row + p.b1_row_off;
      // interleaved gate/up B (pairs): this CTA's 64 gate rows and the same 64 up rows
      const int birow = b0row + (int)rank * 64;
      const CUtensorMap* ma = (half || thin) ? &mapA64 : &mapA;
      const uint32_t stage_tx = half   ? (C::STAGE_BYTES - KS * A_BYTES / 2) * PAIR
                                : thin ? (C::STAGE_BYTES - KS * (A_BYTES - A_BYTES / 4)) * PAIR
                                       : C::STAGE_BYTES * PAIR;
      // k-blocks of weight gradients count from the tile's first row, others from the row's start
      const int kfirst = p.wgrad ? 0 : __shfl_sync(0xffffffffu, t.kb0, 0);
      for (int kb = kfirst; kb < kfirst + nk; ++kb) {
        ok = __all_sync(0xffffffffu, mbar_wait<kCluster>(empty_bar(stage), phase ^ 1u, abort_flag, p.status));
        if (!ok) break;
        if (elect_one()) {
          const uint32_t sa = ring + stage * C::STAGE_BYTES;
          const uint32_t fb = full0_leader + 8u * stage;
          // K coordinates of this k-block: A's, and B's (row or column)
          const bool second = p.kb_split > 0 && kb >= p.kb_split;  // [dg | du] . [W_gate ; W_up]: up half
          const int kx = second ? p.a_k2 + (kb - p.kb_split) * BK : kx0 + kb * BK * KS;
          const int kb_b = second ? (kb - p.kb_split) * BK : kx0 + kb * BK;
          const CUtensorMap* mb = second ? &mapB1 : &mapB0;
          if (leader) mbar_expect_tx(full_bar(stage), stage_tx);
          if constexpr (KS == 2) {  // K-major A and B only: KS sub-blocks of 64
#pragma unroll
            for (int sub = 0; sub < KS; ++sub) {
              const int kxs = kx + sub * BK;
              const uint32_t sbs = sa + KS * A_BYTES + sub * C::B_BYTES;
              tma_load_2d<PAIR>(sa + sub * A_BYTES, ma, kxs, a_row, fb);
              if constexpr (PAIR == 1) {
                tma_load_3d<PAIR>(sbs, &mapB0, kxs, b0row, te, fb);
                tma_load_3d<PAIR>(sbs + B_HALF_BYTES, &mapB1, kxs, b1row, te, fb);
              } else if (p.b_inter) {
                tma_load_3d<PAIR>(sbs, &mapB0, kxs, birow, te, fb);
                tma_load_3d<PAIR>(sbs + B_HALF_BYTES / 2, &mapB1, kxs, birow, te, fb);
              } else if (leader) {
                tma_load_3d<PAIR>(sbs, &mapB0, kxs, b0row, te, fb);
              } else {
                tma_load_3d<PAIR>(sbs, &mapB1, kxs, b1row, te, fb);
              }
            }
          } else if (p.a_mn) {  // two 64-column boxes of this CTA's 128 M values
            const bool cut = a_cut && kb == nk - 1;
            const CUtensorMap* mk = cut ? &mapA64 : &mapA;
            const int ka = cut ? te * BK : p.a_tail ? a_k0 + kb * BK : kx;
            tma_load_2d<PAIR>(sa, mk, a_row, ka, fb);
            tma_load_2d<PAIR>(sa + MN_BOX_BYTES, mk, a_row + 64, ka, fb);
          } else {
            tma_load_2d<PAIR>(sa, ma, kx, a_row, fb);
          }
          if (KS == 2) {
            // loaded above
          } else if (p.b_form == kBKmajor3d) {
            if constexpr (PAIR == 1) {
              tma_load_3d<PAIR>(sa + A_BYTES, &mapB0, kx, b0row, te, fb);
              tma_load_3d<PAIR>(sa + A_BYTES + B_HALF_BYTES, &mapB1, kx, b1row, te, fb);
            } else if (p.b_inter) {
              tma_load_3d<PAIR>(sa + A_BYTES, &mapB0, kx, birow, te, fb);
              tma_load_3d<PAIR>(sa + A_BYTES + B_HALF_BYTES / 2, &mapB1, kx, birow, te, fb);
            } else if (leader) {
              tma_load_3d<PAIR>(sa + A_BYTES, &mapB0, kx, b0row, te, fb);
            } else {
              tma_load_3d<PAIR>(sa + A_BYTES, &mapB1, kx, b1row, te, fb);
            }
          } else {  // MN-major B: this CTA's N columns in boxes of 64
            const int n0 = tnb * 256 + (PAIR == 2 ? (int)rank * 128 : 0);
#pragma unroll
            for (int j = 0; j < (PAIR == 2 ? 2 : 4); ++j) {
              const uint32_t dst = sa + A_BYTES + j * MN_BOX_BYTES;
              if (p.b_form == kBMNmajor3d) tma_load_3d<PAIR>(dst, mb, n0 + 64 * j, kb_b, te, fb);
              else tma_load_2d<PAIR>(dst, mb, n0 + 64 * j, kb_b, fb);
            }
          }
        }
        __syncwarp();
        ++fills;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    if (!ok && leader && lane == 0) {  // aborting: let the copies in flight land before exit
      for (uint32_t i = fills > STAGES ? fills - STAGES : 0; i < fills; ++i) {
        const uint64_t t0 = global_timer();
        while (!mbar_test<kCluster>(full_bar(i % STAGES), (i / STAGES) & 1u) &&
               global_timer() - t0 < kWaitLimitNs) {
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer (leader CTA)
    if (leader) {
      const uint32_t idesc = make_idesc(sizeof(T) == 2 && !std::is_same<T, __half>::value, C::TILE_M) |
                             ((uint32_t)(p.a_mn != 0) << 15) | ((uint32_t)(p.b_form != kBKmajor3d) << 16);
      // half tile: M = 128 over the pair (the M field is bits 24-28, M >> 4)
      const uint32_t idesc_half = (idesc & ~(0x1Fu << 24)) | ((uint32_t)(C::TILE_M / 2 >> 4) << 24);
      // per 16-deep MMA step: 32 bytes along a K-major row, 16 rows of an MN-major box
      const uint32_t a_step = p.a_mn ? 16u * 128u : UMMA_K * 2u;
      const uint32_t b_step = p.b_form != kBKmajor3d ? 16u * 128u : UMMA_K * 2u;
      // descriptor bits other than the start address
      const uint64_t a_hi = p.a_mn ? sw128_mn_desc(0) : sw128_desc(0);
      const uint64_t b_hi = p.b_form != kBKmajor3d ? sw128_mn_desc(0) : sw128_desc(0);
      int stage = 0;
      uint32_t phase = 0, acc = 0, acc_phase = 0;
      bool ok = true;
      for (uint32_t tile = cluster_id; ok && tile < total_tiles; tile += num_clusters) {
        const Tile tt = tile_at(tile);
        const int nk = __shfl_sync(0xffffffffu, tt.nk, 0);  // 0 for an expert without rows (weight gradients)
        const uint32_t id = __all_sync(0xffffffffu, tt.half) ? idesc_half : idesc;
        ok = __all_sync(0xffffffffu, mbar_wait<kCluster>(tempty_bar(acc), acc_phase ^ 1u, abort_flag, p.status));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + acc * BN;
        for (int kb = 0; kb < nk; ++kb) {
          ok = __all_sync(0xffffffffu, mbar_wait<kCluster>(full_bar(stage), phase, abort_flag, p.status));
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t sa = ring + stage * C::STAGE_BYTES;
            const uint32_t sb = sa + KS * A_BYTES;
#pragma unroll
            for (int q = 0; q < KS * (BK / UMMA_K); ++q) {
              const int sub = q / (BK / UMMA_K), kk = q % (BK / UMMA_K);
              const uint32_t ak = sa + sub * A_BYTES + kk * a_step, bk = sb + sub * C::B_BYTES + kk * b_step;
              umma_f16<PAIR>(d_tmem, a_hi | ((ak & 0x3FFFFu) >> 4), b_hi | ((bk & 0x3FFFFu) >> 4), id,
                             (kb | q) != 0 ? 1u : 0u);
            }
            umma_commit<PAIR>(empty_bar(stage));  // ring stage free (in every CTA) once done
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) umma_commit<PAIR>(tfull_bar(acc));  // accumulator ready for the epilogues
        __syncwarp();
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
      // every MMA this warp issued must be complete before TMEM is freed
      if (elect_one()) {
        umma_commit_local<PAIR>(drain_bar);
        const uint64_t t0 = global_timer();
        while (!mbar_test<false>(drain_bar, 0) && global_timer() - t0 < kWaitLimitNs) {
        }
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ epilogue
    const int quarter = warp & 3;  // this warp may access TMEM lanes 32*quarter .. +31
    uint32_t* stg = CK == kUse ? staging + (warp - 2) * (STG16_BYTES_PER_WARP / 4) : staging + quarter * (STG_BYTES_PER_WARP / 4);
    constexpr int EG = kEpilogues<CK>;  // with two groups of warps, each keeps to its accumulator
    uint32_t acc = EG == 2 ? (uint32_t)(warp - 2) >> 2 : 0u, acc_phase = 0;
    T* out = static_cast<T*>(p.out);
    for (uint64_t tile = cluster_id + acc * num_clusters; tile < total_tiles; tile += EG * num_clusters) {
      const Tile t = tile_at((uint32_t)tile);
      // full tile: lane l of quarter q is row 32q + l of this CTA's 128, all
      // N columns.  Half tile (M = 128 over the pair): the CTA's 64 rows sit
      // in lanes 0-63 with N columns 0-127 and again in lanes 64-127 with N
      // columns 128-255, each in TMEM columns 0-127; quarter q then holds rows
      // 32*(q & 1) + l and the N-column half q >> 1.
      const int row = t.half ? (quarter & 1) * 32 + lane : quarter * 32 + lane;
      const int nhalf = t.half ? quarter >> 1 : 0;
      const int64_t grow = t.m0 + (int64_t)rank * (t.half ? BM / 2 : BM) + row;
      const bool row_ok = p.wgrad ? grow < p.m_total : grow < (int64_t)s_off[t.e + 1];
      // the weighted epilogue's slot and routing weight: loaded before the
      // accumulator wait so that their latency overlaps the MMAs
      int64_t wslot = grow;
      float wscale = 1.f;
      if (p.mode == kDownWeighted && row_ok) {
        const uint32_t s = __ldg(p.perm + grow);
        wslot = s;
        wscale = load_dyn(p.weights, p.wdt, s);
      }
      int ok = 1;
      if (lane == 0) ok = mbar_wait<kCluster>(tfull_bar(acc), acc_phase, abort_flag, p.status) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      const uint32_t taddr = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * BN;
      if constexpr (CK == kUse) {
        if (p.mode == kSwigluBwd) {
          // accumulator da = dout . W_down[e]; g and u of the forward from
          // their 8-bit checkpoints: dg = da u silu'(g), du = da silu(g) and a
          // = silu(g) u in the 16-bit dtype, in the 64-padded row space (its
          // padding rows zero).  da itself stays in FP32 and in TMEM.
          const int64_t I = p.n_out, nblk = (I + 31) / 32;
          const int64_t col0 = (int64_t)t.nb * 256 + (int64_t)nhalf * 128;
          const int64_t local = grow - (int64_t)s_off[t.e];
          const uint32_t pe = __ldg(p.pad + t.e);
          const bool zero_row = !row_ok && local < (int64_t)(__ldg(p.pad + t.e + 1) - pe);
          const bool store = row_ok || zero_row;
          const int64_t prow = (int64_t)pe + local;
          uint32_t* dgp = store ? reinterpret_cast<uint32_t*>(out + prow * 2 * I + col0) : nullptr;
          uint32_t* dup_p = store ? reinterpret_cast<uint32_t*>(out + prow * 2 * I + I + col0) : nullptr;
          uint32_t* ap = store ? reinterpret_cast<uint32_t*>(static_cast<T*>(p.out2) + prow * I + col0) : nullptr;
          const int nch = t.half ? 4 : 8;
          // the next block's elements and scales are asked for before this one is computed
          uint32_t gq[8], uq[8], gb = 0, ub = 0;
          auto load = [&](int ci) {
            const int64_t c = col0 + 32 * ci, left = row_ok ? I - c : 0;
            load_mx8(p.ck_g + grow * I + c, left, gq);
            load_mx8(p.ck_u + grow * I + c, left, uq);
            gb = left > 0 ? (uint32_t)__ldg(p.ck_gs + grow * nblk + c / 32) : 0u;
            ub = left > 0 ? (uint32_t)__ldg(p.ck_us + grow * nblk + c / 32) : 0u;
          };
          load(0);
#pragma unroll 1
          for (int ci = 0; ci < nch; ++ci) {
            if (col0 + 32 * ci >= I) break;
            uint32_t d[32];
            tmem_ld32(taddr + 32 * ci, d);
            float g[32], u[32];
            const float gs = mx::scale_value(gb), us = mx::scale_value(ub);
#pragma unroll
            for (int v = 0; v < 8; ++v) {
              mx::from_e4m3x4(gq[v], g + 4 * v);
              mx::from_e4m3x4(uq[v], u + 4 * v);
            }
            if (ci + 1 < nch) load(ci + 1);
            tmem_wait_ld(d);
            if (!row_ok)  // rows not stored may hold anything; g and u are 0 there
#pragma unroll
              for (int i = 0; i < 32; ++i) d[i] = 0u;
            // two values an instruction: at one, this arithmetic takes longer
            // than the product (631 against 373 us for the headline's da)
            uint32_t wdg[16], wdu[16], wa[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 gg = mul2(make_float2(g[2 * i], g[2 * i + 1]), both(gs));
              const float2 uu = mul2(make_float2(u[2 * i], u[2 * i + 1]), both(us));
              const float2 dv = make_float2(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]));
              const float2 t = mul2(gg, both(-kLog2e));
              const float2 n = add2(make_float2(exp2_fast(t.x), exp2_fast(t.y)), both(1.f));
              const float2 sg = make_float2(rcp_fast(n.x), rcp_fast(n.y));  // 16-bit outputs
              const float2 silu = mul2(gg, sg);
              const float2 slope = fma2(silu, fma2(sg, both(-1.f), both(1.f)), sg);
              // (da u may leave FP32's range where the slope brings it back)
              wdg[i] = pack2<T>(mul2(dv, mul2(uu, slope)));
              wdu[i] = pack2<T>(mul2(dv, silu));
              wa[i] = pack2<T>(mul2(silu, uu));
            }
            const int vw = min(16, valid_words<T>(I - col0 - 32 * ci));
            staged_store<16>(stg, wdg, dgp ? dgp + 16 * ci : nullptr, vw, lane);
            staged_store<16>(stg, wdu, dup_p ? dup_p + 16 * ci : nullptr, vw, lane);
            staged_store<16>(stg, wa, ap ? ap + 16 * ci : nullptr, vw, lane);
          }
        } else if (p.mode == kPartial) {
          // one part of a long K: FP32 sums, joined afterwards
          const int64_t col0 = (int64_t)t.nb * 256 + (int64_t)nhalf * 128;
          float* row = static_cast<float*>(p.out) + ((int64_t)t.eo * p.m_total + grow) * p.n_out + col0;
#pragma unroll 1
          for (int c = 0; c < (t.half ? 128 : 256); c += 32) {
            if (col0 + c >= p.n_out) break;
            uint32_t o[32];
            __syncwarp();
            tmem_ld32(taddr + c, o);
            tmem_wait_ld(o);
            const int vw = valid_words<float>(p.n_out - col0 - c);
            if (row_ok)
#pragma unroll
              for (int v = 0; v < 8; ++v)
                if (4 * v < vw)
                  *reinterpret_cast<uint4*>(row + c + 4 * v) = make_uint4(o[4 * v], o[4 * v + 1], o[4 * v + 2], o[4 * v + 3]);
          }
        } else {
          // kWgrad: rows of a weight-gradient tile, rounded once to T: an FP32
          // gradient would double the stores, which set the pace where experts
          // are many and small (an expert without rows gets zeros)
          const int64_t col0 = (int64_t)t.nb * 256;
          T* rowt = nullptr;
          if (row_ok) {
            if (grow < p.split)
              rowt = out + ((int64_t)t.e * p.split + grow) * p.n_out + col0;
            else
              rowt = static_cast<T*>(p.out2) + ((int64_t)t.e * (p.m_total - p.split) + grow - p.split) * p.n_out + col0;
          }
          uint32_t* rowp = reinterpret_cast<uint32_t*>(rowt);
          // the next 32 columns are read from TMEM while these are packed and stored
          uint32_t ob[2][32], w[32];
          tmem_ld32(taddr, ob[0]);
          tmem_wait_ld(ob[0]);
#pragma unroll
          for (int ci = 0; ci < 8; ++ci) {
            if (ci + 1 < 8) tmem_ld32(taddr + 32 * ci + 32, ob[(ci + 1) & 1]);
            const uint32_t* o = ob[ci & 1];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = t.nk == 0 ? 0.f : __uint_as_float(o[v * 8 + i]);
              put4(w + 16 * (ci & 1) + 4 * v, pack8<T>(f));
            }
            if (ci & 1) {
              const int vw = min(32, valid_words<T>(p.n_out - col0 - 32 * (ci - 1)));
              staged_lines(stg, w, rowp ? rowp + 16 * (ci - 1) : nullptr, vw, lane);
            }
            if (ci + 1 < 8) tmem_wait_ld(ob[(ci + 1) & 1]);
          }
        }
      } else if (p.mode == kGateUpSwiglu) {
        // h = silu(g) * u: stored straight from registers (one 16-byte vector
        // per 8 columns); this epilogue is not store-bound, and measured
        // faster without the staging round trip.  Interleaved B: accumulator
        // columns [128 b, 128 b + 64) hold gate features 64 b .. 64 b + 63 of
        // the tile (64 (b + nhalf) for a half tile) and the next 64 columns
        // the up values of the same features; otherwise gate columns 0-127,
        // up columns 128-255.
        const int fw = p.b_inter ? 64 : 128;       // features per block
        const int nblk = t.half ? 1 : 128 / fw;
        const int64_t col0 = (int64_t)t.nb * 128 + (int64_t)nhalf * 64;
        T* dst = out + grow * p.n_out + col0;
#pragma unroll 1
        for (int i32 = 0; i32 < nblk * fw; i32 += 32) {
          const int b = i32 / fw, c = i32 - b * fw;
          const uint32_t gcol = (uint32_t)(b * 2 * fw + c);
          uint32_t g[32], u[32];
          __syncwarp();
          tmem_ld32(taddr + gcol, g);
          tmem_ld32(taddr + gcol + fw, u);
          tmem_wait_ld(g);
          reg_fence(u);
          if constexpr (CK == kSave) {
            if (row_ok && col0 + i32 < p.n_out) {
              const int64_t c = col0 + i32, at = grow * ((p.n_out + 31) / 32) + c / 32;
              store_mx8(g, p.ck_g + grow * p.n_out + c, p.n_out - c, p.ck_gs + at);
              store_mx8(u, p.ck_u + grow * p.n_out + c, p.n_out - c, p.ck_us + at);
            }
          }
          if (row_ok) {
            uint32_t hw[16];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float f[8], top = 0.f;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const float gg = __uint_as_float(g[v * 8 + i]);
                const float uu = __uint_as_float(u[v * 8 + i]);
                // 16-bit output: the fast divide's ~2 ulp are far below its rounding
                f[i] = __fdividef(gg * uu, 1.f + __expf(-gg));
                top = fmaxf(top, fabsf(gg * uu));
              }
              if (top > kFltMax) {  // g u leaves FP32's range: silu(g) u need not, for g below 0
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  const float gg = __uint_as_float(g[v * 8 + i]);
                  const float uu = __uint_as_float(u[v * 8 + i]);
                  if (fabsf(gg * uu) > kFltMax) f[i] = gg / (1.f + __expf(-gg)) * uu;
                }
              }
              put4(hw + 4 * v, pack8<T>(f));
            }
            if (p.v8_out && col0 + i32 + 32 <= p.n_out) {
              uint32_t* d32 = reinterpret_cast<uint32_t*>(dst + i32);
              st_v8(d32, hw);
              st_v8(d32 + 8, hw + 8);
            } else {
#pragma unroll
              for (int v = 0; v < 4; ++v)
                if (col0 + i32 + v * 8 + 8 <= p.n_out)
                  *reinterpret_cast<uint4*>(dst + i32 + v * 8) =
                      make_uint4(hw[4 * v], hw[4 * v + 1], hw[4 * v + 2], hw[4 * v + 3]);
            }
          }
        }
      } else if (CK == kNone && p.mode == kSwigluBwd) {
        // accumulators g = x . W_gate[e]^T, u = x . W_up[e]^T (recomputed); with
        // da = dout . W_down[e] (16-bit, from the previous product):
        // dg = da * u * silu'(g), du = da * silu(g) and the activation
        // a = silu(g) * u, stored in the 16-bit dtype in the 64-padded row
        // space (row - offsets[e] + pad[e]); the padding rows after an
        // expert's last row are written as zeros (a segment's padding ends
        // inside its last tile, half tiles included).  The gate and up
        // accumulator columns are laid out as in the forward gate/up product.
        const int fw = p.b_inter ? 64 : 128;
        const int64_t col0 = (int64_t)t.nb * 128 + (int64_t)nhalf * 64;  // this warp's first feature
        const int64_t I = p.n_out;
        const int64_t local = grow - (int64_t)s_off[t.e];
        const uint32_t pe = __ldg(p.pad + t.e);
        const bool zero_row = !row_ok && local < (int64_t)(__ldg(p.pad + t.e + 1) - pe);
        const int64_t prow = (int64_t)pe + local;
        const T* dasrc = static_cast<const T*>(p.da) + grow * I + col0;
        const bool store = row_ok || zero_row;
        uint32_t* dgp = store ? reinterpret_cast<uint32_t*>(out + prow * 2 * I + col0) : nullptr;
        uint32_t* dup_p = store ? reinterpret_cast<uint32_t*>(out + prow * 2 * I + I + col0) : nullptr;
        uint32_t* ap = store ? reinterpret_cast<uint32_t*>(static_cast<T*>(p.out2) + prow * I + col0) : nullptr;
        // da of this row (16-bit), 32 columns per chunk; the next chunk's loads
        // are issued before the current chunk is computed so that their latency
        // overlaps the TMEM reads and the arithmetic
        auto load_da = [&](int c, float (&d)[32]) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 q = make_uint4(0u, 0u, 0u, 0u);
            if (row_ok && col0 + c + v * 8 + 8 <= I) q = __ldg(reinterpret_cast<const uint4*>(dasrc + c + v * 8));
            unpack8<T>(q, d + v * 8);
          }
        };
        // NF features of this warp: 128 (full tile) or 64 (half tile)
        auto features = [&](auto nf) {
        constexpr int NF = decltype(nf)::value;
        float dcur[32];
        load_da(0, dcur);
#pragma unroll
        for (int c = 0; c < NF; c += 32) {
          float dnext[32];
          if (c + 32 < NF) load_da(c + 32, dnext);
          const int b = c / fw;
          const uint32_t gcol = (uint32_t)(b * 2 * fw + (c - b * fw));
          uint32_t g[32], u[32], wdg[16], wdu[16], wa[16];
          tmem_ld32(taddr + gcol, g);
          tmem_ld32(taddr + gcol + fw, u);
          tmem_wait_ld(g);
          reg_fence(u);
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            float fdg[8], fdu[8], fa[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              // padding rows (and rows not stored) have da = 0 and store zeros
              const float gg = row_ok ? __uint_as_float(g[v * 8 + i]) : 0.f;
              const float uu = row_ok ? __uint_as_float(u[v * 8 + i]) : 0.f;
              const float dv = dcur[v * 8 + i];
              const float sg = __fdividef(1.f, 1.f + __expf(-gg));  // 16-bit outputs
              const float silu = gg * sg;
              fdg[i] = dv * uu * (sg + silu * (1.f - sg));
              fdu[i] = dv * silu;
              fa[i] = silu * uu;
            }
            put4(wdg + 4 * v, pack8<T>(fdg));
            put4(wdu + 4 * v, pack8<T>(fdu));
            put4(wa + 4 * v, pack8<T>(fa));
          }
          const int vw = valid_words<T>(I - col0 - c);
          staged_store<16>(stg, wdg, dgp ? dgp + c / 2 : nullptr, vw, lane);
          staged_store<16>(stg, wdu, dup_p ? dup_p + c / 2 : nullptr, vw, lane);
          staged_store<16>(stg, wa, ap ? ap + c / 2 : nullptr, vw, lane);
          if (c + 32 < NF) {
#pragma unroll
            for (int i = 0; i < 32; ++i) dcur[i] = dnext[i];
          }
        }
        };
        if (t.half) features(std::integral_constant<int, 64>{});
        else features(std::integral_constant<int, 128>{});
      } else if (CK == kNone && p.mode == kWgrad) {
        // FP32 rows of a weight-gradient tile (rows at or past `split` go to
        // out2; an expert without rows gets zeros).  A half tile's warp holds
        // 128 of the 256 columns.
        const int64_t col0 = (int64_t)t.nb * 256 + (int64_t)nhalf * 128;
        float* rowf = nullptr;
        if (row_ok) {
          if (grow < p.split)
            rowf = static_cast<float*>(p.out) + ((int64_t)t.eo * p.split + grow) * p.n_out + col0;
          else
            rowf = static_cast<float*>(p.out2) +
                   ((int64_t)t.eo * (p.m_total - p.split) + grow - p.split) * p.n_out + col0;
        }
        uint32_t* rowp = reinterpret_cast<uint32_t*>(rowf);
        const bool empty = t.nk == 0;
        if (empty) {
          uint32_t z[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) z[i] = 0u;
#pragma unroll 1
          for (int c = 0; c < 256; c += 32)
            staged_store<32>(stg, z, rowp ? rowp + c : nullptr, valid_words<float>(p.n_out - col0 - c), lane);
        } else {
          // the next 32 columns are read from TMEM while this chunk is stored
          auto chunks = [&](auto nch) {
            constexpr int NCH = decltype(nch)::value;
            uint32_t ob[2][32];
            tmem_ld32(taddr, ob[0]);
            tmem_wait_ld(ob[0]);
#pragma unroll
            for (int ci = 0; ci < NCH; ++ci) {
              const int c = ci * 32;
              if (ci + 1 < NCH) tmem_ld32(taddr + c + 32, ob[(ci + 1) & 1]);
              staged_store<32>(stg, ob[ci & 1], rowp ? rowp + c : nullptr,
                               valid_words<float>(p.n_out - col0 - c), lane);
              if (ci + 1 < NCH) tmem_wait_ld(ob[(ci + 1) & 1]);
            }
          };
          if (t.half) chunks(std::integral_constant<int, 4>{});
          else chunks(std::integral_constant<int, 8>{});
        }
      } else {
        // the next 32 columns are read from TMEM while this chunk is scaled,
        // packed and stored.  A half tile's warp holds 128 of the 256 columns.
        const int64_t col0 = (int64_t)t.nb * 256 + (int64_t)nhalf * 128;
        uint32_t* rowp = row_ok ? reinterpret_cast<uint32_t*>(out + wslot * p.n_out + col0) : nullptr;
        // NCH 32-column chunks: 8 for a full tile, 4 for a half tile (a
        // compile-time count in each form, so the double buffer stays in registers)
        auto chunks = [&](auto nch) {
          constexpr int NCH = decltype(nch)::value;
          uint32_t ob[2][32];
          tmem_ld32(taddr, ob[0]);
          tmem_wait_ld(ob[0]);
#pragma unroll
          for (int ci = 0; ci < NCH; ++ci) {
            const int c = ci * 32;
            if (ci + 1 < NCH) tmem_ld32(taddr + c + 32, ob[(ci + 1) & 1]);
            const uint32_t* o = ob[ci & 1];
            uint32_t w[16];
#pragma unroll
            for (int v = 0; v < 4; ++v) {
              float f[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(o[v * 8 + i]) * wscale;
              put4(w + 4 * v, pack8<T>(f));
            }
            if (p.v8_out && col0 + c + 32 <= p.n_out) {  // warp-uniform: whole 64-byte row segments
              if (rowp) {
                st_v8(rowp + c / 2, w);
                st_v8(rowp + c / 2 + 8, w + 8);
              }
            } else {
              staged_store<16>(stg, w, rowp ? rowp + c / 2 : nullptr, valid_words<T>(p.n_out - col0 - c), lane);
            }
            if (ci + 1 < NCH) tmem_wait_ld(ob[(ci + 1) & 1]);
          }
        };
        if (t.half) chunks(std::integral_constant<int, 4>{});
        else chunks(std::integral_constant<int, 8>{});
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        // its TMEM reads are done; a release would wait for the tile's stores
        if constexpr (kCluster) mbar_arrive_cluster_relaxed(tempty0_leader + 8u * acc);
        else mbar_arrive(tempty_bar(acc));
      }
      if constexpr (EG == 1) acc ^= 1u;
      if (EG == 2 || acc == 0) acc_phase ^= 1u;
    }
  }

  __syncthreads();
  // PAIR == 2: the leader's MMAs write the peer's TMEM and the peer arrives on
  // the leader's barriers, so neither CTA frees TMEM or exits before both are done
  if constexpr (kCluster) cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc<PAIR>(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------- self-test
// Exercises the path every bounded wait of this file takes when it gives up:
// one warp waits on an mbarrier that nothing will complete; after limit_ns
// the wait records MOE_ERR_DEVICE_TIMEOUT in the status word and the kernel
// returns normally, leaving the context usable.
__global__ void bounded_wait_selftest(uint32_t* status, uint64_t limit_ns) {
  __shared__ uint64_t bar;
  __shared__ uint32_t abort_flag;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bar), 1);
    abort_flag = 0u;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  if (threadIdx.x == 0) mbar_wait<false>(smem_u32(&bar), 0, &abort_flag, status, limit_ns);
  __syncthreads();
}

// ---------------------------------------------------------------- host side
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

CUtensorMapDataType tmap_type(moe_dtype dt) {
  return dt == MOE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// rows x cols (cols contiguous), box `box_rows` (128, or 64) rows x 64 columns
bool encode_2d(CUtensorMap* m, const void* base, moe_dtype dt, uint64_t rows, uint64_t cols,
               uint32_t box_rows = 128) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {(cuuint32_t)BK, box_rows};
  cuuint32_t estr[2] = {1u, 1u};
  return fn(m, tmap_type(dt), 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// experts x rows x cols (cols contiguous), box 1 x `box_rows` (128, or 64) x 64
bool encode_3d(CUtensorMap* m, const void* base, moe_dtype dt, uint64_t E, uint64_t rows,
               uint64_t cols, uint32_t box_rows = 128) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {cols, rows, E};
  cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
  cuuint32_t box[3] = {(cuuint32_t)BK, box_rows, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, tmap_type(dt), 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int PAIR, int KS = 1, int CK = kNone>
size_t smem_bytes(int E) {
  return 1024 + (size_t)Cfg<PAIR, KS>::STAGES * Cfg<PAIR, KS>::STAGE_BYTES + kStgBytes<CK> + 256 +
         8 * (size_t)(E + 1);
}

// mA64: A with 64-row boxes, for the half tiles of p.half_tails (else unused)
template <typename T, int PAIR, int KS = 1, int CK = kNone>
cudaError_t launch_t(int64_t N, int E, const CUtensorMap& mA, const CUtensorMap& mB0,
                     const CUtensorMap& mB1, Params p, int num_sms, cudaStream_t s,
                     const CUtensorMap* mA64 = nullptr) {
  if (!mA64 || PAIR != 2) p.half_tails = 0;
  if (!mA64 || PAIR != 1) p.thin_a = 0;
  static PerDevice known;
  int clusters = 0;
  cudaError_t err = resident_clusters<PAIR>(grouped_gemm_tc<T, PAIR, KS, CK>, kThreads<CK>, smem_bytes<PAIR, KS, CK>(MAX_E),
                                            num_sms, known, &clusters);
  if (err != cudaSuccess) return err;
  if (clusters < 1) return cudaErrorLaunchOutOfResources;
  constexpr int TM = Cfg<PAIR>::TILE_M;
  int64_t tiles_max;
  if (p.wgrad) {
    tiles_max = (int64_t)E * p.mb * p.nb * p.k_parts;
  } else {
    const int64_t mt_max = (N + TM - 1) / TM + std::min<int64_t>(E, N);
    tiles_max = mt_max * p.nb * std::max(p.k_parts, 1);
  }
  const int nclu = (int)std::max<int64_t>(1, std::min<int64_t>(clusters, tiles_max));
  // panel width: about one wave of clusters spread over an expert's expected m-tiles
  const int64_t mt_per_expert = std::max<int64_t>(1, (N + (int64_t)TM * E - 1) / ((int64_t)TM * E));
  p.panel = (int)std::max<int64_t>(1, std::min<int64_t>(p.nb, (nclu + mt_per_expert - 1) / mt_per_expert));
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = PAIR;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see pdl_wait
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(nclu * PAIR);
  cfg.blockDim = dim3(kThreads<CK>);
  cfg.dynamicSmemBytes = smem_bytes<PAIR, KS, CK>(E);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, grouped_gemm_tc<T, PAIR, KS, CK>, mA, mB0, mB1, mA64 ? *mA64 : mA, p);
}

template <typename T, int CK = kNone>
cudaError_t launch_any(bool pair, int64_t N, int E, const CUtensorMap& mA, const CUtensorMap& mB0,
                       const CUtensorMap& mB1, const Params& p, int num_sms, cudaStream_t s,
                       const CUtensorMap* mA64 = nullptr) {
  return pair ? launch_t<T, 2, 1, CK>(N, E, mA, mB0, mB1, p, num_sms, s, mA64)
              : launch_t<T, 1, 1, CK>(N, E, mA, mB0, mB1, p, num_sms, s);
}

// ---------------------------------------------------------------- backward
// Scratch of the tensor-core expert backward; every buffer 1024-byte aligned.
// Row buffers marked P live in the 64-padded row space (npad rows).
struct BwdLayout {
  int64_t npad;  // >= pad[E] for any offsets: N + 63 E
  size_t pad, da, dgduP, actP, xP, doutP, total;
};

BwdLayout bwd_layout(int64_t N, int E, int64_t H, int64_t I) {
  BwdLayout L{};
  L.npad = N + 63 * (int64_t)E;
  size_t off = 0;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += (bytes + 1023) & ~(size_t)1023;
    return at;
  };
  L.pad = take((size_t)(E + 1) * 4);
  L.da = take((size_t)N * I * 2);
  L.dgduP = take((size_t)L.npad * 2 * I * 2);
  L.actP = take((size_t)L.npad * I * 2);
  L.xP = take((size_t)L.npad * H * 2);
  L.doutP = take((size_t)L.npad * H * 2);
  L.total = off;
  return L;
}

// rows x cols (cols contiguous), box 64 rows x 64 columns: an MN-major operand
bool encode_2d_mn(CUtensorMap* m, const void* base, moe_dtype dt, uint64_t rows, uint64_t cols) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {cols, rows};
  cuuint64_t strides[1] = {cols * 2};
  cuuint32_t box[2] = {64u, (cuuint32_t)BK};
  cuuint32_t estr[2] = {1u, 1u};
  return fn(m, tmap_type(dt), 2, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// experts x rows x cols (cols contiguous), box 1 x 64 x 64: an MN-major weight operand
bool encode_3d_mn(CUtensorMap* m, const void* base, moe_dtype dt, uint64_t E, uint64_t rows,
                  uint64_t cols) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {cols, rows, E};
  cuuint64_t strides[2] = {cols * 2, rows * cols * 2};
  cuuint32_t box[3] = {64u, (cuuint32_t)BK, 1u};
  cuuint32_t estr[3] = {1u, 1u, 1u};
  return fn(m, tmap_type(dt), 3, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Products of the backward, each one launch of grouped_gemm_tc, every weight
// read in its stored layout (MN-major where the product needs it transposed):
//   1. da     = dout W_down (W_down MN-major), in the 16-bit dtype
//   2. g, u   = x W_gate^T, x W_up^T recomputed; the epilogue forms dg, du
//               and a from them and da, in the padded row space
//   3. dinput = dg W_gate + du W_up (weights MN-major; one accumulator over
//               the gate k-blocks, then the up k-blocks)
//   4. [dgate ; dup] = [dg | du]^T x per expert   (both operands MN-major over
//   5. ddown         = dout^T a per expert         the expert's padded rows)
template <typename T>
cudaError_t backward_t(const ExpertsBwdArgs& a, const TcWeights* w, char* ws, int num_sms, cudaStream_t s) {
  const int64_t N = a.N, H = a.H, I = a.I;
  const int E = a.E;
  const moe_dtype dt = a.dt;
  const BwdLayout L = bwd_layout(N, E, H, I);
  uint32_t* pad = reinterpret_cast<uint32_t*>(ws + L.pad);
  void* da = ws + L.da;
  void* dgduP = ws + L.dgduP;
  void* actP = ws + L.actP;
  void* xP = ws + L.xP;
  void* doutP = ws + L.doutP;
  cudaError_t err;
#define MOE_TC_TRY(x) \
  if ((err = (x)) != cudaSuccess) return err
  CUtensorMap mX, mDo, mDgduP, mWdMN, mWgMN, mWuMN, mDgduMN, mXMN, mDoMN, mActMN;
  CUtensorMap mX64, mDo64, mDgduP64;  // 64-row A boxes: half tiles of products 1-3
  if (!encode_2d(&mX64, a.x_disp, dt, N, H, 64) || !encode_2d(&mDo64, a.dout, dt, N, H, 64) ||
      !encode_2d(&mDgduP64, dgduP, dt, L.npad, 2 * I, 64))
    return cudaErrorInvalidValue;
  if (!encode_2d(&mX, a.x_disp, dt, N, H) || !encode_2d(&mDo, a.dout, dt, N, H) ||
      !encode_2d(&mDgduP, dgduP, dt, L.npad, 2 * I) || !encode_3d_mn(&mWdMN, a.down, dt, E, H, I) ||
      !encode_3d_mn(&mWgMN, a.gate, dt, E, I, H) || !encode_3d_mn(&mWuMN, a.up, dt, E, I, H) ||
      !encode_2d_mn(&mDgduMN, dgduP, dt, L.npad, 2 * I) || !encode_2d_mn(&mXMN, xP, dt, L.npad, H) ||
      !encode_2d_mn(&mDoMN, doutP, dt, L.npad, H) || !encode_2d_mn(&mActMN, actP, dt, L.npad, I))
    return cudaErrorInvalidValue;
  MOE_TC_TRY(launch_pad_offsets(a.offsets, E, pad, s));
  // x and dout into the padded row space on a side stream: they are needed
  // only by products 4 and 5 and co-run with products 1-3 (whose CTAs leave
  // registers and threads free on every SM).  While `s` is being captured
  // into a CUDA graph they run on `s` itself (no per-call stream then).
  cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
  MOE_TC_TRY(cudaStreamIsCapturing(s, &capture));
  if (capture != cudaStreamCaptureStatusNone) {
    MOE_TC_TRY(launch_pad_rows(a.x_disp, H, a.offsets, pad, E, L.npad, xP, s));
    MOE_TC_TRY(launch_pad_rows(a.dout, H, a.offsets, pad, E, L.npad, doutP, s));
  }
  cudaStream_t side = nullptr;
  cudaEvent_t fork = nullptr, join = nullptr;
  if (capture == cudaStreamCaptureStatusNone)
    MOE_TC_TRY(cudaStreamCreateWithFlags(&side, cudaStreamNonBlocking));
  if (side) {
    err = cudaEventCreateWithFlags(&fork, cudaEventDisableTiming);
    if (err == cudaSuccess) err = cudaEventCreateWithFlags(&join, cudaEventDisableTiming);
    if (err == cudaSuccess) err = cudaEventRecord(fork, s);
    if (err == cudaSuccess) err = cudaStreamWaitEvent(side, fork, 0);
    if (err == cudaSuccess) err = launch_pad_rows(a.x_disp, H, a.offsets, pad, E, L.npad, xP, side);
    if (err == cudaSuccess) err = launch_pad_rows(a.dout, H, a.offsets, pad, E, L.npad, doutP, side);
    if (err == cudaSuccess) err = cudaEventRecord(join, side);
    // destroying them now is legal: their resources go once the work is done
    cudaStreamDestroy(side);
    if (fork) cudaEventDestroy(fork);
  }
  struct EventGuard {
    cudaEvent_t e;
    ~EventGuard() {
      if (e) cudaEventDestroy(e);
    }
  } join_guard{join};
  if (err != cudaSuccess) return err;
  const bool pair = N >= (int64_t)BM * E;
  Params base{};
  base.offsets = a.offsets;
  base.E = E;
  base.status = a.status;
  base.wdt = (int)MOE_F32;
  base.pad = pad;
  // 1. da = dout W_down, stored in the 16-bit dtype
  Params p = base;
  p.mode = kDownPlain;
  p.b_form = kBMNmajor3d;
  p.k_blocks = (int)((H + BK - 1) / BK);
  p.cols_per_tile = 256;
  p.n_out = I;
  p.nb = (int)((I + 255) / 256);
  p.out = da;
  p.half_tails = 1;
  MOE_TC_TRY(launch_any<T>(pair, N, E, mDo, mWdMN, mWdMN, p, num_sms, s, &mDo64));
  // 2. g, u recomputed; epilogue: dg, du, a (padded rows)
  p = base;
  p.mode = kSwigluBwd;
  p.k_blocks = (int)((H + BK - 1) / BK);
  p.cols_per_tile = 128;
  p.b1_row_off = 0;
  p.n_out = I;
  p.nb = (int)((I + 127) / 128);
  p.out = dgduP;
  p.out2 = actP;
  p.da = da;
  p.half_tails = 1;
  p.b_inter = pair;  // gate/up staged as in the forward's CTA-pair product
  MOE_TC_TRY(launch_any<T>(pair, N, E, mX, pair ? w->gate64 : w->gate, pair ? w->up64 : w->up, p, num_sms, s,
                           &mX64));
  // 3. dinput
  const int kbI = (int)((I + BK - 1) / BK);
  p = base;
  p.mode = kDownPlain;
  p.b_form = kBMNmajor3d;
  p.a_row_pad = 1;
  p.kb_split = kbI;
  p.a_k2 = (int)I;
  p.k_blocks = 2 * kbI;
  p.cols_per_tile = 256;
  p.n_out = H;
  p.nb = (int)((H + 255) / 256);
  p.out = a.dinput;
  p.half_tails = 1;
  MOE_TC_TRY(launch_any<T>(pair, N, E, mDgduP, mWgMN, mWuMN, p, num_sms, s, &mDgduP64));
  // 4-5. weight gradients over the padded rows (after the side stream's copies)
  if (join) MOE_TC_TRY(cudaStreamWaitEvent(s, join, 0));
  constexpr int TM = Cfg<2>::TILE_M;
  p = base;
  p.mode = kWgrad;
  p.wgrad = 1;
  p.k_parts = 1;
  p.a_mn = 1;
  p.b_form = kBMNmajor2d;
  p.cols_per_tile = 256;
  p.m_total = 2 * I;
  p.split = I;
  p.mb = (int)((2 * I + TM - 1) / TM);
  p.n_out = H;
  p.nb = (int)((H + 255) / 256);
  p.out = a.dgate;
  p.out2 = a.dup;
  MOE_TC_TRY((launch_t<T, 2>(N, E, mDgduMN, mXMN, mXMN, p, num_sms, s)));
  p.m_total = H;
  p.split = H;
  p.mb = (int)((H + TM - 1) / TM);
  p.n_out = I;
  p.nb = (int)((I + 255) / 256);
  p.out = a.ddown;
  p.out2 = a.ddown;
  MOE_TC_TRY((launch_t<T, 2>(N, E, mDoMN, mActMN, mActMN, p, num_sms, s)));
#undef MOE_TC_TRY
  return cudaSuccess;
}

// The checkpointed backward: products 1 and 2 above become one (da stays in
// the accumulators, g and u come from the checkpoint), x's padded rows are read
// from its 8-bit tokens, and the weight gradients are stored in T.
struct CkLayout {
  int64_t npad;
  size_t pad, dgduP, actP, xP, tails, parts, total;
};

CkLayout ck_layout(int64_t N, int E, int64_t H, int64_t I, int num_sms) {
  CkLayout L{};
  L.npad = N + 63 * (int64_t)E;
  size_t off = 0;
  auto take = [&off](size_t bytes) {
    const size_t at = off;
    off += (bytes + 1023) & ~(size_t)1023;
    return at;
  };
  L.pad = take((size_t)(E + 1) * 4);
  L.dgduP = take((size_t)L.npad * 2 * I * 2);
  L.actP = take((size_t)L.npad * I * 2);
  L.xP = take((size_t)L.npad * H * 2);
  L.tails = take((size_t)E * BK * H * 2);
  L.parts = take((size_t)parts::room(N, E, H, I, num_sms) * 4);
  L.total = off;
  return L;
}

template <typename T>
cudaError_t backward_ck_t(const ExpertsCkBwdArgs& a, char* ws, int num_sms, cudaStream_t s) {
  const int64_t N = a.N, H = a.H, I = a.I;
  const int E = a.E;
  const moe_dtype dt = a.dt;
  const CkLayout L = ck_layout(N, E, H, I, num_sms);
  uint32_t* pad = reinterpret_cast<uint32_t*>(ws + L.pad);
  void* dgduP = ws + L.dgduP;
  void* actP = ws + L.actP;
  void* xP = ws + L.xP;
  void* tails = ws + L.tails;
  CUtensorMap mDo, mDo64, mDgduP, mDgduP64, mWdMN, mWgMN, mWuMN, mDgduMN, mXMN, mDoMN, mTailMN, mActMN;
  if (!encode_2d(&mDo, a.dout, dt, N, H) || !encode_2d(&mDo64, a.dout, dt, N, H, 64) ||
      !encode_2d(&mDgduP, dgduP, dt, L.npad, 2 * I) || !encode_2d(&mDgduP64, dgduP, dt, L.npad, 2 * I, 64) ||
      !encode_3d_mn(&mWdMN, a.down, dt, E, H, I) || !encode_3d_mn(&mWgMN, a.gate, dt, E, I, H) ||
      !encode_3d_mn(&mWuMN, a.up, dt, E, I, H) || !encode_2d_mn(&mDgduMN, dgduP, dt, L.npad, 2 * I) ||
      !encode_2d_mn(&mXMN, xP, dt, L.npad, H) || !encode_2d_mn(&mDoMN, a.dout, dt, N, H) || !encode_2d_mn(&mTailMN, tails, dt, (uint64_t)E * BK, H) ||
      !encode_2d_mn(&mActMN, actP, dt, L.npad, I))
    return cudaErrorInvalidValue;
  cudaError_t err;
#define MOE_TC_TRY(x) \
  if ((err = (x)) != cudaSuccess) return err
  MOE_TC_TRY(launch_check_offsets(a.offsets_in, E, N, a.offsets, a.status, pad, s));
  const bool pair = N >= (int64_t)BM * E;
  Params base{};
  base.offsets = a.offsets;
  base.E = E;
  base.status = a.status;
  base.wdt = (int)MOE_F32;
  base.pad = pad;
  base.half_tails = 1;
  base.b_form = kBMNmajor3d;
  base.cols_per_tile = 256;
  // dg, du, a from da = dout W_down
  Params p = base;
  p.mode = kSwigluBwd;
  p.k_blocks = (int)((H + BK - 1) / BK);
  p.n_out = I;
  p.nb = (int)((I + 255) / 256);
  p.out = dgduP;
  p.out2 = actP;
  p.ck_g = const_cast<uint8_t*>(a.g);
  p.ck_u = const_cast<uint8_t*>(a.u);
  p.ck_gs = const_cast<uint8_t*>(a.g_scales);
  p.ck_us = const_cast<uint8_t*>(a.u_scales);
  MOE_TC_TRY((launch_any<T, kUse>(pair, N, E, mDo, mWdMN, mWdMN, p, num_sms, s, &mDo64)));
  // dinput = dg W_gate + du W_up
  const int kbI = (int)((I + BK - 1) / BK);
  p = base;
  p.mode = kDownPlain;
  p.a_row_pad = 1;
  p.kb_split = kbI;
  p.a_k2 = (int)I;
  p.k_blocks = 2 * kbI;
  p.n_out = H;
  p.nb = (int)((H + 255) / 256);
  p.out = a.dinput;
  p.v8_out = H % 16 == 0 && reinterpret_cast<uintptr_t>(a.dinput) % 32 == 0;
  float* sums = reinterpret_cast<float*>(ws + L.parts);
  const int px = parts::dinput(N, E, H, I, num_sms);
  if (px > 1) {
    p.mode = kPartial;
    p.k_parts = px;
    p.m_total = N;
    p.out = sums;
    MOE_TC_TRY((launch_any<T, kUse>(pair, N, E, mDgduP, mWgMN, mWuMN, p, num_sms, s, &mDgduP64)));
    MOE_TC_TRY(launch_join_rows(sums, px, N, H, a.offsets, E, a.dinput, dt, s));
  } else {
    MOE_TC_TRY(launch_any<T>(pair, N, E, mDgduP, mWgMN, mWuMN, p, num_sms, s, &mDgduP64));
  }
  // weight gradients over the padded rows.  (On a stream beside the products
  // before, these copies take the same time off them: 2473 us against 2465 us
  // in order, headline shape.)
  MOE_TC_TRY(launch_pad_rows_mx8(a.x, a.x_scales, a.T, H, a.perm, a.k, a.offsets, pad, E, L.npad, xP, dt, s));
  MOE_TC_TRY(launch_tail_rows(a.dout, H, a.offsets, E, tails, s));
  constexpr int TM = Cfg<2>::TILE_M;
  p = base;
  p.half_tails = 0;
  p.mode = kWgrad;
  p.wgrad = 1;
  p.k_parts = 1;
  p.a_mn = 1;
  p.b_form = kBMNmajor2d;
  auto gradient = [&](const CUtensorMap& mA, const CUtensorMap& mB, const CUtensorMap* mTail, void* o1, void* o2) {
    p.mb = (int)((p.m_total + TM - 1) / TM);
    p.nb = (int)((p.n_out + 255) / 256);
    p.k_parts = parts::weight_gradient(N, E, p.m_total, p.n_out, num_sms);
    p.out = o1;
    p.out2 = o2;
    if (p.k_parts == 1) return launch_t<T, 2, 1, kUse>(N, E, mA, mB, mB, p, num_sms, s, mTail);
    const int64_t n1 = p.split * p.n_out, n2 = (p.m_total - p.split) * p.n_out;
    float* f2 = sums + (int64_t)p.k_parts * E * n1;
    p.out = sums;
    p.out2 = f2;
    cudaError_t e = launch_t<T, 2>(N, E, mA, mB, mB, p, num_sms, s, mTail);
    if (e == cudaSuccess) e = launch_join_parts(sums, E, p.k_parts, n1, o1, dt, s);
    if (e == cudaSuccess && n2 > 0) e = launch_join_parts(f2, E, p.k_parts, n2, o2, dt, s);
    return e;
  };
  p.m_total = 2 * I;
  p.split = I;
  p.n_out = H;
  MOE_TC_TRY(gradient(mDgduMN, mXMN, nullptr, a.dgate, a.dup));
  p.m_total = H;
  p.split = H;
  p.n_out = I;
  p.a_tail = 1;
  MOE_TC_TRY(gradient(mDoMN, mActMN, &mTailMN, a.ddown, a.ddown));
#undef MOE_TC_TRY
  return cudaSuccess;
}

}  // namespace tc

bool tc_supported(moe_dtype dt, int64_t I, int64_t H) {
  return (dt == MOE_BF16 || dt == MOE_F16) && I % 8 == 0 && H % 8 == 0;
}

TcWeights* tc_weights_create(const void* gate, const void* up, const void* down, moe_dtype dt,
                             int64_t E, int64_t I, int64_t H, const char** err) {
  if (!tc::encode_fn()) {
    *err = "cuTensorMapEncodeTiled is not available from the driver";
    return nullptr;
  }
  TcWeights* w = new TcWeights();
  w->E = E;
  w->I = I;
  w->H = H;
  if (!tc::encode_3d(&w->gate, gate, dt, E, I, H) || !tc::encode_3d(&w->up, up, dt, E, I, H) ||
      !tc::encode_3d(&w->down, down, dt, E, H, I) || !tc::encode_3d(&w->gate64, gate, dt, E, I, H, 64) ||
      !tc::encode_3d(&w->up64, up, dt, E, I, H, 64)) {
    *err = "cuTensorMapEncodeTiled rejected an expert weight tensor";
    delete w;
    return nullptr;
  }
  return w;
}

void tc_weights_destroy(TcWeights* w) { delete w; }

cudaError_t launch_bounded_wait_selftest(uint32_t* status, uint64_t limit_ns, cudaStream_t s) {
  tc::bounded_wait_selftest<<<1, 32, 0, s>>>(status, limit_ns);
  return cudaGetLastError();
}

cudaError_t launch_gemm_tc(const GemmArgs& a, const TcWeights* w, int num_sms, cudaStream_t s) {
  CUtensorMap mA, mA64;
  if (!tc::encode_2d(&mA, a.A, a.dt, (uint64_t)a.N, (uint64_t)a.K) ||
      !tc::encode_2d(&mA64, a.A, a.dt, (uint64_t)a.N, (uint64_t)a.K, 64))
    return cudaErrorInvalidValue;
  tc::Params p{};
  p.offsets = a.offsets;
  p.E = a.E;
  p.mode = a.mode;
  p.n_out = a.n_out;
  p.out = a.out;
  p.perm = a.perm;
  p.weights = a.weights;
  p.wdt = (int)a.wdt;
  p.status = a.status;
  p.k_blocks = (int)((a.K + tc::BK - 1) / tc::BK);
  p.half_tails = 1;
  p.ck_g = a.ck_g;
  p.ck_u = a.ck_u;
  p.ck_gs = a.ck_gs;
  p.ck_us = a.ck_us;
  const bool save = a.ck_g != nullptr;
  p.v8_out = a.n_out % 16 == 0 && reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
  // CTA pairs halve the B bytes each SM stages per k-block; they pay off when
  // experts hold at least a full 128-row tile on average.  With fewer rows per
  // expert (decode-sized batches) the GEMM streams weights from HBM and single
  // CTAs keep twice as many independent streams in flight.
  const bool pair = a.N >= (int64_t)tc::BM * a.E;
  const CUtensorMap* b0;
  const CUtensorMap* b1;
  if (a.mode == kGateUpSwiglu) {
    p.cols_per_tile = 128;
    p.b1_row_off = 0;
    p.b_inter = pair;
    b0 = pair ? &w->gate64 : &w->gate;
    b1 = pair ? &w->up64 : &w->up;
  } else {
    p.cols_per_tile = 256;
    p.b1_row_off = 128;
    b0 = &w->down;
    b1 = &w->down;
  }
  p.nb = (int)((a.n_out + p.cols_per_tile - 1) / p.cols_per_tile);
  if (pair && a.mode != kGateUpSwiglu && a.K > 4096) {
    // long-K down projection: six 64-deep stages rather than three 128-deep
    // ones (the same ring bytes); 0.5-5 % faster at K = 14336, 3 % slower at
    // K = 1408 (same-box A/B)
    if (a.dt == MOE_BF16) return tc::launch_t<__nv_bfloat16, 2>(a.N, a.E, mA, *b0, *b1, p, num_sms, s, &mA64);
    return tc::launch_t<__half, 2>(a.N, a.E, mA, *b0, *b1, p, num_sms, s, &mA64);
  }
  if (pair) {  // 128-deep k-blocks, two 64-deep sub-blocks per ring stage
    p.k_blocks = (int)((a.K + 2 * tc::BK - 1) / (2 * tc::BK));
    if (save)
      return a.dt == MOE_BF16
                 ? tc::launch_t<__nv_bfloat16, 2, 2, tc::kSave>(a.N, a.E, mA, *b0, *b1, p, num_sms, s, &mA64)
                 : tc::launch_t<__half, 2, 2, tc::kSave>(a.N, a.E, mA, *b0, *b1, p, num_sms, s, &mA64);
    if (a.dt == MOE_BF16)
      return tc::launch_t<__nv_bfloat16, 2, 2>(a.N, a.E, mA, *b0, *b1, p, num_sms, s, &mA64);
    return tc::launch_t<__half, 2, 2>(a.N, a.E, mA, *b0, *b1, p, num_sms, s, &mA64);
  }
  CUtensorMap mA32;
  if (!tc::encode_2d(&mA32, a.A, a.dt, (uint64_t)a.N, (uint64_t)a.K, 32)) return cudaErrorInvalidValue;
  p.thin_a = 1;
  if (save)
    return a.dt == MOE_BF16
               ? tc::launch_t<__nv_bfloat16, 1, 1, tc::kSave>(a.N, a.E, mA, *b0, *b1, p, num_sms, s, &mA32)
               : tc::launch_t<__half, 1, 1, tc::kSave>(a.N, a.E, mA, *b0, *b1, p, num_sms, s, &mA32);
  if (a.dt == MOE_BF16) return tc::launch_t<__nv_bfloat16, 1>(a.N, a.E, mA, *b0, *b1, p, num_sms, s, &mA32);
  return tc::launch_t<__half, 1>(a.N, a.E, mA, *b0, *b1, p, num_sms, s, &mA32);
}

size_t experts_backward_tc_workspace(int64_t N, int E, int64_t H, int64_t I) {
  return tc::bwd_layout(N, E, H, I).total;
}

cudaError_t launch_experts_backward_tc(const ExpertsBwdArgs& a, const TcWeights* w, void* ws,
                                       int num_sms, cudaStream_t s) {
  char* base = static_cast<char*>(ws);
  if (a.dt == MOE_BF16) return tc::backward_t<__nv_bfloat16>(a, w, base, num_sms, s);
  return tc::backward_t<__half>(a, w, base, num_sms, s);
}

size_t experts_backward_ck_workspace(int64_t N, int E, int64_t H, int64_t I, int num_sms) {
  return tc::ck_layout(N, E, H, I, num_sms).total;
}

cudaError_t launch_experts_backward_ck(const ExpertsCkBwdArgs& a, void* ws, int num_sms, cudaStream_t s) {
  char* base = static_cast<char*>(ws);
  if (a.dt == MOE_BF16) return tc::backward_ck_t<__nv_bfloat16>(a, base, num_sms, s);
  return tc::backward_ck_t<__half>(a, base, num_sms, s);
}

}  // namespace moe
