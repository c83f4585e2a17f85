// rows.cuh -- rows of router logits in registers, and packed sequences of rows.
//
// Shared by the router's training losses (balance.cu, distill.cu).  A row of
// E <= 1024 logits is held by `lpr` lanes (a power of two), NV vectors of VEC
// elements per lane: vector v of lane `sub` starts at element
// (v * lpr + sub) * VEC, so that one load reads contiguous pieces.  A warp holds
// 32 / lpr rows at once.
#pragma once

#include <math.h>

#include <atomic>
#include <type_traits>
#include <utility>

#include "common.cuh"

namespace moe {

// Calls f2(n) for pairs of 0..N-1 (f1(0) where N == 1).
template <int N, typename F2, typename F1>
__device__ __forceinline__ void pairwise(F2 f2, F1 f1) {
  if constexpr (N == 1) {
    f1(0);
  } else {
#pragma unroll
    for (int n = 0; n < N; n += 2) f2(n);
  }
}
template <int N>
__device__ __forceinline__ float2 pair(const float (&x)[N], int n) {
  return make_float2(x[n], x[n + 1]);
}
template <int N>
__device__ __forceinline__ void put(float (&x)[N], int n, float2 v) {
  x[n] = v.x;
  x[n + 1] = v.y;
}

// How the lanes of a warp are laid over rows: LPR lanes a row (0: `lpr` of them).
template <int LPR>
struct Lanes {
  int lpr, sub, grp, rows;  // lanes per row, lane in its row, row in the warp, rows per warp
  __device__ __forceinline__ explicit Lanes(int lpr_) {
    const int lane = threadIdx.x & 31;
    lpr = LPR ? LPR : lpr_;
    sub = lane & (lpr - 1);
    grp = lane / lpr;
    rows = 32 / lpr;
  }
  __device__ __forceinline__ unsigned mask() const {
    return lpr == 32 ? 0xffffffffu : ((1u << lpr) - 1u) << (grp * lpr);
  }
  // Butterflies over the lanes of a row: every lane gets the same bits.  All
  // lanes of the warp take part.
  template <typename V, typename F>
  __device__ __forceinline__ V all(V x, F f) const {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1)
      if (d < lpr) x = f(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
  }
  __device__ __forceinline__ float sum(float x) const {
    return all(x, [](float a, float b) { return a + b; });
  }
  __device__ __forceinline__ float max(float x) const {  // passes over NaN
    if constexpr (LPR == 32) {
      float y;
      asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
      return y;
    } else {
      return all(x, [](float a, float b) { return fmaxf(a, b); });
    }
  }
  // Does it hold on any lane of the row?
  __device__ __forceinline__ bool any(bool x) const { return (__ballot_sync(0xffffffffu, x) & mask()) != 0; }
};

// Blocks of 256 threads that a SM is to hold, by the bytes of a row that a lane
// holds, where a single element counts as two, in FP32 too.  Kernels that keep a
// list's entries as well hold three at most.  What else a lane holds (scores, sums)
// is not counted: of the 356 variants of the losses' kernels 107 spill registers, 71 of
// these among the 182 for single elements, 32 more than 100 bytes (one 832).  The balance loss
// of 524288 rows takes 95 us for 101 FP32 logits, single elements, and 48 for 100.
constexpr int blocks_for(int bytes, int most) {
  const int n = bytes <= 16 ? 4 : bytes <= 32 ? 3 : bytes <= 64 ? 2 : 1;
  return n < most ? n : most;
}
constexpr int kListBlocks = 3;
template <typename T, int VEC, int NV>
constexpr int blocks_per_sm(int most = 4) {
  return blocks_for(VEC == 1 ? NV * 2 : NV * 16, most);
}

// One row's elements of this lane.
template <typename T, int VEC, int NV>
struct RowRegs {
  static constexpr int N = VEC * NV;
  static __device__ __forceinline__ int elem(int n, int lpr, int sub) {
    return (n / VEC * lpr + sub) * VEC + n % VEC;
  }

  alignas(16) T raw[N];

  __device__ __forceinline__ void fill(T x) {
#pragma unroll
    for (int n = 0; n < N; ++n) raw[n] = x;
  }
  // `row` is the row at this lane's first element, of which `room` = E - sub * VEC
  // lie before the row's end.  Vectors behind it, and rows that are not loaded,
  // keep what they hold.  Plain loads: the kernel may write the row later on, and
  // the kernel before it may have written it (no data that stays as it is).
  __device__ __forceinline__ void load(const T* row, int room, int lpr, bool ok) {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (!ok || v * lpr * VEC >= room) continue;
      if constexpr (VEC > 1) {
        static_assert(VEC * sizeof(T) == 16, "16-byte vectors");
        *reinterpret_cast<uint4*>(raw + v * VEC) = *reinterpret_cast<const uint4*>(row + v * lpr * VEC);
      } else {
        raw[v] = row[v * lpr];
      }
    }
  }
  __device__ __forceinline__ void zero(int room, int lpr) {
#pragma unroll
    for (int n = 0; n < N; ++n)
      if (n / VEC * lpr * VEC < room) raw[n] = from_f32<T>(0.f);
  }
  __device__ __forceinline__ float operator[](int n) const { return to_f32<T>(raw[n]); }
  // This lane's maximum; passes over NaN.
  __device__ __forceinline__ float lane_max() const {
    if constexpr (sizeof(T) == 2 && VEC == 8) {  // two elements an instruction
      using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
      T2 m[N / 2];  // a tree: a chain of N / 2 would wait for itself
#pragma unroll
      for (int i = 0; i < N / 2; ++i) m[i] = reinterpret_cast<const T2*>(raw)[i];
#pragma unroll
      for (int w = N / 4; w > 0; w /= 2)
#pragma unroll
        for (int i = 0; i < w; ++i) m[i] = __hmax2(m[i], m[i + w]);
      return fmaxf(to_f32<T>(m[0].x), to_f32<T>(m[0].y));
    } else {
      float m[N];
#pragma unroll
      for (int n = 0; n < N; ++n) m[n] = (*this)[n];
#pragma unroll
      for (int w = N / 2; w > 0; w /= 2)
#pragma unroll
        for (int n = 0; n < w; ++n) m[n] = fmaxf(m[n], m[n + w]);
      return m[0];
    }
  }
};

// Stores a lane's values at `row` (as RowRegs::load has it), in 16-byte vectors
// or single elements.
template <typename T, int VEC, int NV>
__device__ __forceinline__ void store_row(T* row, int room, int lpr, const float (&f)[VEC * NV]) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
    if (v * lpr * VEC >= room) continue;
    if constexpr (VEC == 8) {
      *reinterpret_cast<uint4*>(row + v * lpr * VEC) = pack8<T>(f + v * VEC);
    } else if constexpr (VEC == 4) {
      *reinterpret_cast<float4*>(row + v * lpr * VEC) =
          make_float4(f[v * 4], f[v * 4 + 1], f[v * 4 + 2], f[v * 4 + 3]);
    } else {
      row[v * lpr] = from_f32<T>(f[v]);
    }
  }
}

// The rows of a warp, a batch of 32 / lpr consecutive rows after another, through a
// ring of kStages batches in the warp's shared memory by asynchronous copies, so
// that kStages - 1 batches are in flight without registers: 256 BF16 logits a row
// with one batch ahead in registers ran at 66 % of the copy bandwidth (16 warps of
// 128 registers on a SM do not cover the latency).
//
// Whole vectors (VEC > 1): a lane copies and reads the same 16 bytes, by vector and
// lane, so that no lane waits for another.  Single elements (VEC == 1: rows that
// start on any element): a batch is copied as it lies in memory, in the 16-byte
// pieces that hold it, and a lane reads its elements from there.
//
// cell(e) is element e of this lane's row in the current batch.  It may be written
// (each lane its own row's) until the next issue().
template <typename T, int VEC, int NV, int LPR>
struct RowStream {
  using Row = RowRegs<T, VEC, NV>;
  static constexpr bool kImage = VEC == 1;
  static constexpr int kStageBytes = 32 * VEC * NV * (int)sizeof(T) + (kImage ? 32 : 0);
  static constexpr int kStages = kStageBytes > 4096 ? 2 : 4;  // (two blocks of 64 KB fit a SM)
  static constexpr int kWarpBytes = (kStages * kStageBytes + 15) / 16 * 16;
  const Lanes<LPR>& L;
  char* ring;        // of this warp
  const T* logits;
  const T* p;        // next to issue: this lane's first element, or (kImage) the batch's
  int64_t step;      // elements between a warp's batches
  int64_t elements;  // of all rows
  int room, E, lpr_log;
  int head, tail;    // stages: current, issued next
  int shift;         // kImage: place of the current batch's first element in its stage

  __device__ __forceinline__ RowStream(const Lanes<LPR>& L_, void* smem, const void* logits_, int E_, int64_t T_rows)
      : L(L_), logits(static_cast<const T*>(logits_)), E(E_) {
    ring = static_cast<char*>(smem) + (threadIdx.x >> 5) * kWarpBytes;
    room = E - L.sub * VEC;
    lpr_log = 31 - __clz(L.lpr);
    elements = T_rows * E;
    if constexpr (!kImage) {  // vectors behind the row's end are never copied: they hold -inf
      Row low;
      low.fill(from_f32<T>(-INFINITY));
#pragma unroll
      for (int i = 0; i < kStages; ++i)
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (v * L.lpr * VEC >= room)
            *reinterpret_cast<uint4*>(ring + i * kStageBytes + (v * 32 + (threadIdx.x & 31)) * 16) =
                *reinterpret_cast<const uint4*>(low.raw);
    }
  }
  // `first`: the warp's first row; a batch every `rows` rows
  __device__ __forceinline__ void start(int64_t first, int64_t rows) {
    p = logits + (kImage ? first * E : (first + L.grp) * E + L.sub * VEC);
    step = rows * E;
    head = tail = 0;
  }
  static __device__ __forceinline__ int place(const T* q) {
    return (int)(reinterpret_cast<uintptr_t>(q) % 16 / sizeof(T));
  }
  // Rows that are not `ok` are not read (unless they lie beside others, kImage):
  // their cells hold anything, or (ZERO, vectors) zeros.
  template <bool ZERO = false>
  __device__ __forceinline__ void issue(bool ok) {
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(ring) + tail * kStageBytes;
    const int lane = threadIdx.x & 31;
    if constexpr (!kImage) {
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if ((ZERO || ok) && v * L.lpr * VEC < room)  // (a copy of 0 bytes writes zeros)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (v * 32 + lane) * 16),
                       "l"(p + v * L.lpr * VEC), "r"(ok ? 16 : 0)
                       : "memory");
    } else {
      __syncwarp();  // every lane has read what lay here
      if (__any_sync(0xffffffffu, ok)) {
        constexpr int C = 16 / (int)sizeof(T);
        const int at = place(p);
        const int64_t from = p - logits - at;  // element of the first piece (may lie before the first row)
        const int pieces = (at + L.rows * E + C - 1) / C;
        for (int c = lane; c < pieces; c += 32) {
          const int64_t e = from + c * C;
          if (e >= 0 && e + C <= elements) {
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + c * 16), "l"(logits + e) : "memory");
          } else {  // the first or the last piece of all rows: only what is theirs
            T* out = reinterpret_cast<T*>(ring + tail * kStageBytes) + c * C;
            for (int i = 0; i < C; ++i)
              if (e + i >= 0 && e + i < elements) out[i] = __ldg(logits + e + i);
          }
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    tail = tail + 1 == kStages ? 0 : tail + 1;
    p += step;
  }
  // The oldest batch issued becomes the current one: wait() lets it lie in shared
  // memory, get() reads this lane's elements.  Those behind a row's end are -inf.
  __device__ __forceinline__ void wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    head = tail == kStages - 1 ? 0 : tail + 1;  // issued kStages - 1 ago
    if constexpr (kImage) {
      shift = place(p - (kStages - 1) * step);
      __syncwarp();
    }
  }
  __device__ __forceinline__ void get(Row& cur) const {
    if constexpr (!kImage) {
      const T* from = stage() + (threadIdx.x & 31) * VEC;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        *reinterpret_cast<uint4*>(cur.raw + v * VEC) = *reinterpret_cast<const uint4*>(from + v * 32 * VEC);
    } else {
      const T* from = stage() + shift + L.grp * E + L.sub;
#pragma unroll
      for (int v = 0; v < NV; ++v) cur.raw[v] = v * L.lpr < room ? from[v * L.lpr] : from_f32<T>(-INFINITY);
    }
  }
  __device__ __forceinline__ void take(Row& cur) {
    wait();
    get(cur);
  }
  __device__ __forceinline__ void drain() { asm volatile("cp.async.wait_all;" ::: "memory"); }
  __device__ __forceinline__ T* stage() const { return reinterpret_cast<T*>(ring + head * kStageBytes); }
  __device__ __forceinline__ T& cell(int e) const {
    if constexpr (kImage) return stage()[shift + L.grp * E + e];
    const int q = e / VEC;
    return stage()[((q >> lpr_log) * 32 + L.grp * L.lpr + (q & (L.lpr - 1))) * VEC + e % VEC];
  }
  // Writes this lane's elements of the current batch.
  __device__ __forceinline__ void put(const Row& r) const {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (v * L.lpr * VEC >= room) continue;
      if constexpr (!kImage)
        *reinterpret_cast<uint4*>(stage() + (v * 32 + (threadIdx.x & 31)) * VEC) =
            *reinterpret_cast<const uint4*>(r.raw + v * VEC);
      else
        cell(v * L.lpr + L.sub) = r.raw[v];
    }
  }
  __device__ __forceinline__ void put(const float (&f)[VEC * NV]) const {
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      if (v * L.lpr * VEC >= room) continue;
      float g[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) g[i] = f[v * VEC + i];
      store_row<T, VEC, 1>(kImage ? &cell(v * L.lpr + L.sub) : stage() + (v * 32 + (threadIdx.x & 31)) * VEC, VEC, 1, g);
    }
  }
  // Stores the current batch, the first `left` rows from row t0 on, to `out`.  All
  // lanes take part; what they put() lies in shared memory (a __syncwarp before).
  __device__ __forceinline__ void store(T* out, int64_t t0, int left) const {
    const int lane = threadIdx.x & 31;
    if constexpr (!kImage) {
      if (L.grp >= left) return;
      T* row = out + (t0 + L.grp) * E + L.sub * VEC;
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (v * L.lpr * VEC < room)
          *reinterpret_cast<uint4*>(row + v * L.lpr * VEC) =
              *reinterpret_cast<const uint4*>(stage() + (v * 32 + lane) * VEC);
    } else {
      constexpr int C = 16 / (int)sizeof(T);
      T* to = out + t0 * E;
      const T* from = stage() + shift;
      const int n = min(L.rows, left) * E;
      if (place(to) == shift) {  // as the logits lie: whole pieces
        const int pieces = (shift + n + C - 1) / C;
        for (int c = lane; c < pieces; c += 32) {
          const int e = c * C - shift;
          if (e >= 0 && e + C <= n) {
            *reinterpret_cast<uint4*>(to + e) = *reinterpret_cast<const uint4*>(from + e);
          } else {
            for (int i = 0; i < C; ++i)
              if (e + i >= 0 && e + i < n) to[e + i] = from[e + i];
          }
        }
      } else {
        for (int e = lane; e < n; e += 32) to[e] = from[e];
      }
    }
  }
};

// exp((x - m) / tau) as 2^(x c - m c), c = log2(e) / tau, in one FMA an element.
// mc = m c is rounded, which leaves a factor 2^(m c - mc) on every element of the
// row: fix() takes it out of their sum (to first order: |m c - mc| < 2^-12).
// Rows that lie farther out (`wide`: masked with a large negative value, say; or
// infinite) form x - m first.
struct RowExp {
  float c, mc, m;
  __device__ __forceinline__ RowExp(float m_, float c_) : c(c_), mc(m_ * c_), m(m_) {}
  __device__ __forceinline__ bool wide() const { return !(fabsf(mc) <= 4096.f); }
  __device__ __forceinline__ float fix() const { return wide() ? 1.f : fmaf(fmaf(m, c, -mc), -kLn2, 1.f); }
  __device__ __forceinline__ float at(float x) const {
    return exp2_fast(wide() ? (x - m) * c : fmaf(x, c, -mc));
  }
  // p = the exponentials of a lane's elements
  template <typename Row>
  __device__ __forceinline__ void row(const Row& r, float (&p)[Row::N]) const {
    if (wide()) {
#pragma unroll
      for (int n = 0; n < Row::N; ++n) p[n] = exp2_fast((r[n] - m) * c);
    } else {
      pairwise<Row::N>(
          [&](int n) {
            const float2 x = fma2(make_float2(r[n], r[n + 1]), both(c), both(-mc));
            p[n] = exp2_fast(x.x);
            p[n + 1] = exp2_fast(x.y);
          },
          [&](int n) { p[n] = exp2_fast(fmaf(r[n], c, -mc)); });
    }
  }
};
template <int N>
__device__ __forceinline__ float lane_sum(const float (&p)[N]) {
  if constexpr (N == 1) {
    return p[0];
  } else {
    float2 s[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) s[i] = pair(p, 2 * i);
#pragma unroll
    for (int w = N / 4; w > 0; w /= 2)
#pragma unroll
      for (int i = 0; i < w; ++i) s[i] = add2(s[i], s[i + w]);
    return s[0].x + s[0].y;
  }
}

// A teacher's list in its own dtype.  An entry is kept as it was loaded (bits) and
// converted where it is used: a conversion next to the load would wait for it.
struct ListEntries {
  const void* logits;
  const uint32_t* idx;
  int dt;
  __device__ __forceinline__ uint32_t bits(int64_t i) const {
    if (dt == MOE_F32) return __ldg(static_cast<const uint32_t*>(logits) + i);
    return __ldg(static_cast<const uint16_t*>(logits) + i);
  }
  __device__ __forceinline__ uint32_t expert(int64_t i) const { return __ldg(idx + i); }
  // bits of -inf: no entry
  __device__ __forceinline__ uint32_t none() const {
    return dt == MOE_F32 ? 0xff800000u : dt == MOE_F16 ? 0xfc00u : 0xff80u;
  }
  __device__ __forceinline__ float value(uint32_t b) const {
    const float h = __half2float(__ushort_as_half((unsigned short)b));
    return dt == MOE_F16 ? h : __uint_as_float(b << (dt == MOE_F32 ? 0 : 16));
  }
};

// ---- packed sequences --------------------------------------------------------
// Sequence s holds the rows off[s] <= t < off[s+1] of a batch of T rows; a null
// `off` is one sequence of all rows.  Offsets come from the device and are
// clamped where they are used, so that no malformed entry leads outside.
struct Seqs {
  const uint32_t* off;
  int num;
  int64_t T;
  __device__ __forceinline__ int64_t at(int s) const {
    if (!off) return s == 0 ? 0 : T;
    const int64_t o = __ldg(off + s);
    return o < T ? o : T;
  }
  // How many of off[1..num] are <= row: the first sequence that ends behind it.
  // A whole warp searches, 32 entries a step.
  __device__ __forceinline__ int first(int64_t row) const {
    if (!off) return 0;
    int lo = 0, hi = num;  // the answer is in lo..hi
    const int lane = threadIdx.x & 31;
    while (lo < hi) {
      const int step = (hi - lo + 31) / 32;
      const int64_t i = (int64_t)lo + (int64_t)(lane + 1) * step;  // entry i, at most hi
      const bool le = i <= hi && at((int)i) <= row;
      const int n = __popc(__ballot_sync(0xffffffffu, le));
      hi = min(hi, lo + (n + 1) * step - 1);
      lo = min(hi, lo + n * step);
    }
    return lo;
  }
};

// Walks the rows [a, b): calls seq(s, lo, hi) for each piece that lies in a
// sequence and gap(lo, hi) for rows outside every sequence, in order, each row
// once whatever the offsets hold.
template <typename FSeq, typename FGap>
__device__ __forceinline__ void walk_sequences(const Seqs& q, int64_t a, int64_t b, FSeq seq, FGap gap) {
  int64_t cur = a;
  for (int s = q.first(a); cur < b; ++s) {
    if (s >= q.num) {
      gap(cur, b);
      break;
    }
    const int64_t lo = min(max(q.at(s), cur), b);
    const int64_t hi = min(max(q.at(s + 1), lo), b);
    if (lo > cur) gap(cur, lo);
    if (hi > lo) seq(s, lo, hi);
    cur = hi;
  }
}

// ---- variants by row length ------------------------------------------------------
// Vectors of 16 bytes where every row starts on a 16-byte boundary, else single
// elements.  Up to eight lanes a row (a copy then covers whole 128-byte lines), then
// up to 64 bytes or 32 single elements a lane, then more lanes.  Few lanes a row make
// its reductions and its scalar work cheap, since a warp does them for several rows
// at once: with it the balance loss of 524288 rows of 256 BF16 logits went from 84 to
// 65 us and the distillation loss from 438 to 163.
struct RowPlan {
  bool vec;
  int lpr;
  int nv;
};
inline RowPlan row_plan(const void* const* ptrs, int n_ptrs, moe_dtype dt, int E) {
  const int esz = (int)dtype_size(dt);
  bool vec = (E * esz) % 16 == 0;
  for (int i = 0; i < n_ptrs; ++i) vec = vec && reinterpret_cast<uintptr_t>(ptrs[i]) % 16 == 0;
  const int units = vec ? E * esz / 16 : E;
  RowPlan p{vec, 1, 1};
  while (p.lpr < 8 && p.lpr < units) p.lpr *= 2;
  if (!vec && p.lpr < units) p.nv = 4;  // (1, 4, 8, 16 or 32 elements a lane)
  while (p.nv < (vec ? 4 : 32) && p.lpr * p.nv < units) p.nv *= 2;
  while (p.lpr < 32 && p.lpr * p.nv < units) p.lpr *= 2;
  while (p.lpr * p.nv < units) p.nv *= 2;
  return p;
}

// Calls f.template run<T, VEC, NV, LPR>() for a plan.
template <typename T, typename F>
cudaError_t with_row_variant(const RowPlan& p, F&& f) {
  constexpr int V = 16 / sizeof(T);
  if (p.vec) {
    if (p.nv == 1) return f.template run<T, V, 1, 0>();
    if (p.nv == 2) return f.template run<T, V, 2, 8>();
    if (p.nv == 4) {
      if (p.lpr == 8) return f.template run<T, V, 4, 8>();
      if (p.lpr == 16) return f.template run<T, V, 4, 16>();
      return f.template run<T, V, 4, 32>();
    }
    if constexpr (V == 4) return f.template run<T, V, 8, 32>();
    return cudaErrorInvalidValue;
  }
  switch (p.nv) {
    case 1: return f.template run<T, 1, 1, 0>();
    case 4: return f.template run<T, 1, 4, 8>();
    case 8: return f.template run<T, 1, 8, 8>();
    case 16: return f.template run<T, 1, 16, 8>();
    default:
      if (p.lpr == 8) return f.template run<T, 1, 32, 8>();
      if (p.lpr == 16) return f.template run<T, 1, 32, 16>();
      return f.template run<T, 1, 32, 32>();
  }
}
template <typename F>
cudaError_t with_row_variant(moe_dtype dt, const RowPlan& p, F&& f) {
  if (dt == MOE_F32) return with_row_variant<float>(p, f);
  if (dt == MOE_F16) return with_row_variant<__half>(p, f);
  return with_row_variant<__nv_bfloat16>(p, f);
}
// Rows that a warp of a plan takes at once, and the blocks that a GPU of 152 SMs
// holds of its kernels (blocks_per_sm).
constexpr int kMaxBlocks = 152 * 4;
inline int plan_batch(const RowPlan& p) { return 32 / p.lpr; }
inline int plan_blocks(const RowPlan& p, int most = 4) { return 152 * blocks_for(p.nv * (p.vec ? 16 : 2), most); }

// Launches a kernel that may need more shared memory than the default, which is
// asked for once per kernel and device.
template <typename... KArgs, typename... Args>
cudaError_t launch_rows(void (*kernel)(KArgs...), int blocks, int threads, size_t smem, std::atomic<uint64_t>& asked,
                        cudaStream_t s, Args&&... args) {
  if (smem > 48 * 1024) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev > 63 || !(asked.load(std::memory_order_acquire) & bit)) {
      e = cudaFuncSetAttribute(reinterpret_cast<const void*>(kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                               220 * 1024);  // the kernels' own arrays take less than 7 KB
      if (e != cudaSuccess) return e;
      asked.fetch_or(bit, std::memory_order_release);
    }
  }
  return launch_pdl(kernel, dim3((unsigned)blocks), dim3((unsigned)threads), smem, s, std::forward<Args>(args)...);
}

// How a batch of rows is cut over blocks: `chunks` blocks of `rows` rows, whole
// rounds of a block's warps (`round` rows); one block where it has few rounds to
// make, since it then needs no second kernel: the balance loss of 64 rows of 256
// BF16 logits takes 4.6 us of the GPU, of 1024 rows in 32 blocks 8.6.
struct Chunks {
  int64_t rows;
  int chunks;
};
constexpr int64_t kRoundsAlone = 4;
inline Chunks cut_rows(int64_t T, int64_t round, int64_t max_chunks, int64_t alone = kRoundsAlone) {
  int64_t rounds = (T + round - 1) / round;
  if (rounds < 1) rounds = 1;
  const int64_t per = rounds <= alone ? rounds : (rounds + max_chunks - 1) / max_chunks;
  Chunks c;
  c.rows = per * round;
  c.chunks = (int)((rounds + per - 1) / per);
  return c;
}

}  // namespace moe
