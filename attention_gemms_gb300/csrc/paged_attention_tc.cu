// Paged grouped-query attention for chunks of new tokens, bf16, head_dim 64 or 128, on the
// tensor cores (tcgen05). One persistent CTA per SM; paged.cuh divides the work.
//
// A unit is 256 rows, two TMEM tiles of 128 rows (whole tokens x the query heads of one
// key/value head, so a key tile serves the whole group), keys in tiles of 128.
//   producer warp: page ids 32 at a time, one TMA box per page, 64-column half and tensor
//     into a ring of K and V tiles, V of a key tile and K of the next one to be multiplied
//     under one barrier (the operands of one turn); pages outside the cache or past the
//     unit's keys are boxes outside the tensor and arrive as zeros;
//   two MMA warps, one per tile: S = Q K^T into TMEM, and O += P V with P read from TMEM;
//   a warp that walks the CTA's work, publishes its segments and loads their Q;
//   eight softmax warps, four per tile, a thread per row: S out of TMEM, the running
//     maximum (moved lazily) and sum, P as bf16 back into TMEM, O rescaled there when the
//     maximum moves; at a segment's end O / l, or the piece for the join.
// A key tile flows in two halves of 64 keys, each with its own S, P and barriers: when a
// half's P arrives, its MMA warp issues O += P V of the half and the next key tile's S of the
// half, which lies over that P in TMEM (a thread's MMAs run in the order they were issued), so
// that the softmax finds the next half ready instead of waiting for both products. With
// whole tiles a row tile's period was softmax + 1024 cycles of products + the hand-overs
// (about 3500 cycles against the tensor cores' 2060 for both tiles); S in halves costs more
// tensor time (N = 64 reads Q twice as often: 2330) and still takes 3200.
// A unit of at most 128 rows (drafts, decoding requests beside a chunk, a chunk's end) would
// leave the second tile idle and the chain S, softmax, P V bare; then both tiles take the
// same rows, the first the even key tiles, the second the odd ones, and at the segment's end
// the first tile's warps read both O.
// What carries it: the walk's scalar work in one warp (in every role it cost more than a
// tile per unit: 525 -> 412 us for two chunks of 2048 tokens, 64 heads over 8, d = 128, 0 and
// 6000 cached), MMAs issued by an elected lane of a converged warp (a one-lane branch took
// 80 to 100 cycles per MMA in moves to uniform registers: 741 -> 650), a start cost per unit
// in the division of the work (none 721, one tile 640, two 576, three 526 before the walk was
// moved; now one 427, two 383, three 375, with three slower on the other shapes).
// Now: those chunks 400 us with new inputs each time, 1.35 PFLOP/s, 70 % of the card's matrix
// rate (373 with the same inputs again; bound by products and softmax in turn, tensor pipe 60 %
// of the launch); four chunks of 401 to 512 tokens, 32 heads over 8, d = 64: 65 us (no pipe is
// full: tensor 24 %, exponentials 25, ALU 29, issue 39; the chain of S, softmax and P V of two
// row tiles bounds it, and launch, schedule and join, 15 us); 33 requests of 2 to 7 drafts, 32
// heads over 8, d = 128 (347 MB): 77 us, 4.5 TB/s (the loads, the schedule and the join before
// and after them).
// Every wait is bounded; on a timeout the CTA records TP_ERR_TIMEOUT, stops issuing, waits
// (bounded) for its own copies and MMAs, frees TMEM and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace tp {
namespace {

constexpr int kTile = 128;  // rows of a TMEM tile, keys of a key tile
// The schedule's costs: a key tile of a unit with one tile of rows is bound by its softmax
// and its loads, and takes most of the time of one with two; a start costs about 2.4 tiles.
// At 1, 1 and a start of 2 a step of chunks and decodes (mixed-step) took 181 us against
// 163, two chunks of 2048 tokens 383 against 373;
// 7 / 6 / 17, 4 / 3 / 10 and 5 / 4 / 10 lie between.
constexpr int kTileCost = 5, kHalfTileCost = 4, kStartCost = 12;
constexpr int kOneStartCost = 3;  // where every unit has one row tile and tiles cost 1 (2 or 5: 1 % more)
// warps 0-3: softmax of tile 0, 4-7: of tile 1, 8: K and V loads, 9 and 10: MMA of tile 0
// and 1, 11: the walk over the CTA's work, and Q loads
constexpr int kProd = 8, kMma = 9, kWalk = 11, kThreads = 384;
// Registers: 384 threads launch with 168 each; the third warpgroup gives up its share
// (128 x 80 + 256 x 208 = 63488 of the launch's 64512) so that the softmax threads keep a
// half row's scores and weights in registers.
constexpr int kRegsLoad = 80, kRegsSoftmax = 208;
constexpr int kSegs = 4;            // segment descriptors in flight
constexpr int kSegReaders = 8 + 3;  // softmax warps, K/V loads, MMA
constexpr int kLoads = 16;  // barriers of loads in flight (at most a ring's tiles)
constexpr int kBadRing = 16;
constexpr uint64_t kDrainNs = 20000000ull;

struct PagedTcParams {
  CUtensorMap tk, tv;  // (n_pages * Hkv * page, d), box 64 x min(page, 128)
  CUtensorMap tq;      // (T, N blocks, hq heads, d) of the qkv rows, box: a row tile x 64
  PagedParams p;
  int cache_rows;
  int* status;
  uint64_t timeout_ns;
  int debug_hang;
};

// ONE: units of one row tile, for calls of at most 128 rows per request and key/value head.
// The second Q tile's place is a sixth place of the ring, and what such calls wait for is
// their loads: 33 requests of 2 to 7 drafts, 32 heads over 8, d = 128: 77 us against 83, 33 of
// 32 tokens 84 against 90. At d = 64 an eleventh place changed nothing (56 and 56).
template <int D, bool ONE>
struct Lay {
  static constexpr int kTiles = ONE ? 1 : 2, kUnit = kTiles * kTile;  // row tiles, rows
  static constexpr int kHalves = D / 64;
  static constexpr int kOp = kTile * D * 2;  // a Q, K or V tile
  static constexpr int kRing = (D == 128 ? 7 : 12) - kTiles;
  static constexpr int kOffRing = kTiles * kOp;
  static constexpr int kOffBar = kOffRing + kRing * kOp;
  static constexpr int kBars = 2 * kLoads + 18 + 2 * kSegs;  // even: 16-byte alignment after
  static constexpr int kOffJoin = kOffBar + kBars * 8 + kBadRing * 4 + 16;
  static constexpr int kOffSeg = kOffJoin + kTile * 8;
  static constexpr int kSmem = kOffSeg + kSegs * 64 + 1024;
  static constexpr uint32_t kO = 256, kOStep = D;                     // TMEM columns
  static constexpr uint32_t kP = 0, kPStep = 128, kPHalf = 64;  // over the half's own S
};

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
      "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// The products of one key tile, issued back to back. An MMA takes its operands from uniform
// registers: issued inside a one-lane branch, each cost 80 to 100 cycles of moves, more
// than the 64 that the tensor cores need for it. So the whole warp runs the MMA role on
// values that the compiler can see to be the same in every lane, and only the instruction
// itself is predicated to the leader; descriptors advance by constants in their low words
// (addresses in 16-byte units).
constexpr uint32_t kDescHi = 1024u >> 4 | 1u << 14 | 2u << 29;  // SBO 1024, version 1, SW128
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo) {
  return ((saddr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16);
}
// D[tmem] = A[smem] * B[smem], both K-major, 16 steps' k at 32-byte steps and 64-wide halves
template <int STEPS>
__device__ __forceinline__ void mma_qk(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t idesc) {
#pragma unroll
  for (int kk = 0; kk < STEPS; ++kk) {
    const uint32_t off = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\t"
        "mov.b64 da, {%1, %3};\n\tmov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %4, p;\n\t}" ::"r"(d),
        "r"(a_lo + off), "r"(b_lo + off), "n"(kDescHi), "r"(idesc), "r"(kk > 0 ? 1u : 0u)
        : "memory");
  }
}
// D[tmem] (+)= A[tmem] * B[smem]: A's row is the TMEM lane, two bf16 per column (8 columns
// per step of 16 keys); B MN-major, 16 keys are 2048 bytes
template <int STEPS>
__device__ __forceinline__ void mma_pv(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t idesc,
                                       uint32_t accumulate) {
#pragma unroll
  for (int kk = 0; kk < STEPS; ++kk)
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\t"
        "mov.b64 db, {%2, %3};\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %4, p;\n\t}" ::"r"(d),
        "r"(a + kk * 8), "r"(b_lo + kk * (2048 >> 4)), "n"(kDescHi), "r"(idesc),
        "r"(kk > 0 ? 1u : accumulate)
        : "memory");
}
// one lane of the converged warp, always the same one
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ int same(int v) { return __shfl_sync(0xFFFFFFFFu, v, 0); }
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* m, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z, int32_t w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}
// two fp32 values per instruction
__device__ __forceinline__ uint64_t pair_of(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {  // relative error about 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// P rounded to bf16 (relative 2^-8 of each weight), the operand of the second product
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// 4 x 4 transpose over the lanes of a quad: chunk i of lane y becomes chunk y of lane i
__device__ __forceinline__ void quad_transpose(uint32_t (&q)[4][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int s = 1; s <= 2; s <<= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i & s) continue;
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint32_t give = up ? q[i][y] : q[i | s][y];
        const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, give, s);
        if (up)
          q[i][y] = got;
        else
          q[i | s][y] = got;
      }
    }
  }
}

// A segment, as one warp works it out for all roles (through shared memory: the walk's scalar
// arithmetic in every role took longer than a key tile). pair: the row tiles hold different
// rows and tile t takes key tiles 0 .. n_t - 1 of the segment (n_1 = n); else both hold the
// same rows and tile t takes key tiles t, t + 2, ... of n.
struct __align__(16) Seg {
  int n, n0, pair, lo;              // n = 0: no more segments; lo: the first key tile
  int row0, tokens, pos0, kv_end;   // first token's row and position, tokens, the request's keys
                                    // that some row sees
  int head0, heads, j, kend;        // first query head, heads, key/value head, unit's keys
  int r, ends, last, pad;           // request; bit 0: the unit begins here, bit 1: it ends
                                    // here; else the CTA where it ends
  __device__ __forceinline__ int count(int t) const {  // row tile t's key tiles
    return pair ? (t ? n : n0) : (n + 1 - t) >> 1;
  }
};

template <class Walk>
__device__ __forceinline__ Seg make_seg(const PagedParams& p, const Walk& w, int tpt) {
  Seg g;  // tpt: tokens of a row tile
  const int j = w.vh / p.hs;
  g.n = w.hi - w.lo;
  g.lo = w.lo;
  g.tokens = min(p.tpu, w.q.rows - w.u * p.tpu);
  g.pair = g.tokens > tpt;
  g.row0 = w.q.row0 + w.u * p.tpu;
  g.pos0 = w.q.total - w.q.n + w.u * p.tpu;
  g.kv_end = w.q.kv_end;
  if (p.causal)  // rows past T do not exist, and nothing wrote their keys
    g.kv_end = max(0, min(g.kv_end, w.q.total - w.q.n + w.q.rows));
  g.head0 = j * p.G + (w.vh - j * p.hs) * p.Gv;
  g.heads = min(p.Gv, (j + 1) * p.G - g.head0);
  g.j = j;
  g.kend = paged_unit_kend(p, w.q, w.u);
  g.r = w.r;
  g.ends = (w.lo == 0 ? 1 : 0) | (w.hi == w.tiles ? 2 : 0);
  g.last = w.hi == w.tiles ? 0 : w.last_cta();
  g.n0 = g.n;
  if (g.pair && p.causal) {  // the first tile's rows see no key of the last tiles
    const int64_t end = min(static_cast<int64_t>(g.pos0) + tpt, static_cast<int64_t>(g.kv_end));
    g.n0 = static_cast<int>(min(static_cast<int64_t>(g.n),
                                max(((end + kTile - 1) >> 7) - g.lo, static_cast<int64_t>(0))));
  }
  return g;
}

template <int D, bool ONE>
__global__ void __launch_bounds__(kThreads, 1)
    paged_tc_kernel(const __grid_constant__ PagedTcParams tp_) {
  using L = Lay<D, ONE>;
  const PagedParams& p = tp_.p;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  volatile uint32_t* bad = reinterpret_cast<volatile uint32_t*>(bars + L::kBars);
  uint32_t* tmem_slot = const_cast<uint32_t*>(bad) + kBadRing;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](uint32_t l) { return bar0 + 8u * (l % kLoads); };
  auto empty = [&](uint32_t l) { return bar0 + 8u * (kLoads + l % kLoads); };
  auto round_of = [](uint32_t l) { return (l / kLoads) & 1u; };
  auto bar_at = [&](int i) { return bar0 + 8u * (2 * kLoads + i); };
  auto q_full = [&](int t) { return bar_at(t); };
  auto s_full = [&](int t, int h) { return bar_at((h ? 14 + 2 * kSegs : 2) + t); };
  auto p_full = [&](int t, int h) { return bar_at((h ? 16 + 2 * kSegs : 4) + t); };
  auto o_done = [&](int t) { return bar_at(6 + t); };
  const uint32_t j_full = bar_at(8), j_free = bar_at(9), drain = bar_at(10);
  auto q_empty = [&](int t) { return bar_at(11 + t); };
  const uint32_t q_other = bar_at(13 + 2 * kSegs);  // the second tile is done with the first's Q
  auto seg_full = [&](uint32_t i) { return bar_at(13 + i % kSegs); };
  auto seg_empty = [&](uint32_t i) { return bar_at(13 + kSegs + i % kSegs); };
  Seg* segs = reinterpret_cast<Seg*>(smem + L::kOffSeg);
  float2* join = reinterpret_cast<float2*>(smem + L::kOffJoin);  // the second tile's (m, l)
  PagedSched& sc = *reinterpret_cast<PagedSched*>(join);  // before any segment
  static_assert(sizeof(PagedSched) <= kTile * 8, "the schedule's scratch lies in the join's");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int l = 0; l < kLoads; ++l) {
      mbar_init(full(l), 1);
      mbar_init(empty(l), 2);  // one arrival per row tile
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(q_full(t), 1);
      mbar_init(q_empty(t), 1);
      for (int h = 0; h < 2; ++h) {
        mbar_init(s_full(t, h), 1);
        mbar_init(p_full(t, h), 4);
      }
      mbar_init(o_done(t), 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(seg_full(i), 1);
      mbar_init(seg_empty(i), kSegReaders);
    }
    mbar_init(j_full, 4);
    mbar_init(j_free, 4);
    mbar_init(q_other, 1);
    mbar_init(drain, 2);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == kMma) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(tmem_slot);
  pdl_wait();  // the set-up above overlaps the previous kernel
  pdl_trigger();
  auto tS = [&](int t) { return tmem + 128u * t; };
  auto tP = [&](int t) { return tmem + L::kP + L::kPStep * t; };
  auto tO = [&](int t) { return tmem + L::kO + L::kOStep * t; };
  auto w = paged_schedule<ONE ? 1 : kTileCost, ONE ? 1 : kHalfTileCost>(p, sc, blockIdx.x,
                                                                        gridDim.x);
  __syncthreads();  // the scratch has been read
  auto entry_at = [&](int e) { return sb + L::kOffRing + e * L::kOp; };
  auto timed_out = [&] {
    atomicCAS(tp_.status, 0, static_cast<int>(TP_ERR_TIMEOUT));
    atomicAdd(tp_.status + 1, 1);
  };
  // the i-th segment, read by a whole warp; false: none left, or a wait expired (ok = false)
  auto get_seg = [&](uint32_t i, Seg& g, bool& ok) -> bool {
    ok = __all_sync(0xFFFFFFFFu, mbar_wait(seg_full(i), (i / kSegs) & 1, tp_.timeout_ns,
                                           abort_flag)) != 0;
    if (!ok) return false;
    g = segs[i % kSegs];
    __syncwarp();
    if (lane == 0) mbar_arrive(seg_empty(i));
    return g.n > 0;
  };
  uint32_t issued = 0;        // K/V loads issued
  int issued_q[2] = {0, 0};   // Q loads: tiles issued

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLoad));
    if (warp == kProd) {
      // ---------------------------------------------------------------- TMA producer
      const int ps = 1 << p.ps_log2, box = min(ps, kTile), boxes = kTile / box;
      bool ok = true;
      uint32_t tiles = 0, slot = 0, freed = 0, sizes = 0;  // bit l % 32: load l has two tiles
      int room = L::kRing;
      Seg g;
      for (uint32_t i = 0; ok && get_seg(i, g, ok); ++i) {
        const int n = g.n, c = g.pair ? 1 : 2;
        const int32_t* tab = p.table + static_cast<int64_t>(g.r) * p.max_pages;
        const int npages = (g.kend + ps - 1) >> p.ps_log2;
        auto fetch = [&](int first) {
          const int i = first + lane;
          const int id = i < npages ? tab[i] : -1;
          return id >= 0 && id < p.n_pages ? id : -1;
        };
        int base = (g.lo * kTile) >> p.ps_log2;
        int ids = fetch(base), ahead = fetch(base + 32);
        int next = g.lo, y0 = 0, y1 = 0, y = 0;  // cache rows of this lane's page: the last tiles
        // the next key tile's rows (tiles are whole groups of at most 16 pages)
        auto locate = [&] {
          const int k0 = next * kTile, pg0 = k0 >> p.ps_log2;
          if (pg0 - base >= 32) {
            base += 32;
            ids = ahead;
            ahead = fetch(base + 32);
          }
          const int src = __shfl_sync(0xFFFFFFFFu, ids, (pg0 - base + min(lane, boxes - 1)) & 31);
          const uint32_t missing = __ballot_sync(0xFFFFFFFFu, lane < boxes && src < 0);
          if (lane == 0) bad[tiles % kBadRing] = missing;
          y0 = y1;
          y1 = y;
          y = src < 0 ? tp_.cache_rows
                      : (((src * p.Hkv + g.j) << p.ps_log2) + (k0 & (ps - 1)));
          ++next;
          ++tiles;
        };
        // room for a load's tiles, then its barrier's count
        auto begin = [&](int size) -> bool {
          while (room < size) {
            if (!__all_sync(0xFFFFFFFFu, mbar_wait(empty(freed), round_of(freed), tp_.timeout_ns,
                                                   abort_flag)))
              return false;
            room += 1 + ((sizes >> (freed % 32)) & 1);
            ++freed;
          }
          room -= size;
          sizes = (sizes & ~(1u << (issued % 32))) | static_cast<uint32_t>(size - 1) << (issued % 32);
          if (lane == 0) mbar_arrive_expect_tx(full(issued), size * L::kOp);
          __syncwarp();
          return true;
        };
        auto copy = [&](const CUtensorMap* m, int row) {
          if (lane < boxes)
#pragma unroll
            for (int h = 0; h < L::kHalves; ++h)
              tma_load_2d(entry_at(slot) + h * (kTile * 128) + lane * box * 128, m, full(issued),
                          h * 64, row);
          if (++slot == L::kRing) slot = 0;
        };
        const int lead = min(c, n);
        for (int i = 0; i < lead; ++i) locate();
        if (!(ok = begin(lead))) break;
        if (lead > 1) copy(&tp_.tk, y1);
        copy(&tp_.tk, y);
        ++issued;
        for (int m = 0; m < n; ++m) {
          const bool more = m + c < n;
          if (more) locate();  // its mask is written before the barrier's arrival
          if (!(ok = begin(more ? 2 : 1))) break;
          // V of tile m: c tiles (fewer at the end) before the last located one
          const int back = next - 1 - (g.lo + m);
          copy(&tp_.tv, back == 0 ? y : back == 1 ? y1 : y0);
          if (more) copy(&tp_.tk, y);
          ++issued;
        }
      }
      if (!ok && lane == 0) timed_out();
    } else if (warp != kWalk) {
      // ---------------------------------------------------------------- MMA issuers
      // One warp per row tile: the tensor cores' queue holds about five MMAs, so one warp's
      // waits and loop between two products would leave them idle; now the other tile's
      // products run meanwhile.
      const int t = same(warp - kMma);
      const uint32_t id_s = idesc_bf16_f32(128, kTile / 2, 0, 0);  // Q, K both K-major
      const uint32_t id_o = idesc_bf16_f32(128, D, 0, 1);      // P in TMEM, V MN-major
      const uint32_t tm = same(tmem), sbase = same(sb);
      const uint32_t ts = tm + 128 * t, to = tm + L::kO + L::kOStep * t;
      auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
        return same(mbar_wait(bar, parity, tp_.timeout_ns, abort_flag)) != 0;
      };
      bool ok = true;
      if (tp_.debug_hang) ok = wait(drain, 0);
      uint32_t q_par[2] = {0, 0}, p_par = 0;  // parities of the next Q tiles, the next P
      uint32_t load = 0, slot = 0;
      auto advance = [&](uint32_t n) {
        ++load;
        slot += n;
        if (slot >= L::kRing) slot -= L::kRing;
      };
      Seg g;
      for (uint32_t i = 0; same(ok && get_seg(i, g, ok)); ++i) {
        const int n = same(g.n), own = same(g.count(t));
        const bool pair = same(g.pair) != 0;
        const int c = pair ? 1 : 2, lead = min(c, n);
        const int qt = pair ? t : 0;  // the rows' Q: one for both tiles when they share rows
        const uint32_t q_done = qt == t ? q_empty(t) : q_other;
        auto s_of = [&](uint32_t ks, int h) {  // half h of S, by the elected lane
          mma_qk<D / 16>(ts + 64 * h, desc_lo(sbase + qt * L::kOp, 16),
                         desc_lo(sbase + L::kOffRing + ks * L::kOp + h * 8192, 16), id_s);
        };
        ok = wait(q_full(qt), q_par[qt]) && wait(full(load), round_of(load));
        q_par[0] ^= 1;  // every segment's first Q, whether this warp waited for it or not
        q_par[1] ^= pair;
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (own > 0) {
            uint32_t ks = slot + (pair ? 0 : t);
            if (ks >= L::kRing) ks = 0;
            s_of(ks, 0);
            mma_commit(s_full(t, 0));
            s_of(ks, 1);
            mma_commit(s_full(t, 1));
          }
          if (own < 2) mma_commit(q_done);
          mma_commit(empty(load));
        }
        __syncwarp();
        advance(lead);
        // Load m + 1: V of key tile m and K of tile m + c, the operands of one turn of the
        // tile (of both tiles for a pair): O += P V, then S of the row tile's next one.
        int left = own;
#pragma unroll 1
        for (int m = 0; m < n; ++m) {
          const uint32_t size = m + c < n ? 2 : 1;
          if (pair ? left == 0 : (m & 1) != t) {  // not this tile's
            if (elect_one()) mbar_arrive(empty(load));
            __syncwarp();
            advance(size);
            continue;
          }
          const uint32_t ks = slot + 1 < L::kRing ? slot + 1 : 0;
          ok = wait(full(load), round_of(load));
          if (!ok) break;
          // by halves of 64 keys: P V of the half, then the next S of the half, which lies over it
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            ok = wait(p_full(t, h), p_par);
            if (!ok) break;
            tc_fence_after();
            if (elect_one()) {
              mma_pv<4>(to, ts + L::kPHalf * h,
                        desc_lo(sbase + L::kOffRing + slot * L::kOp + h * 8192, kTile * 128), id_o,
                        left < own || h > 0);
              if (left > 1) s_of(ks, h);
              // committed after the last key tile's first half too: its P V is then complete
              if (left > 1 || h == 0) mma_commit(s_full(t, h));
              if (h == 1) {
                if (left == 2) mma_commit(q_done);
                // (the other order, in the loop's last turn alone, took 15 of 385 us more)
                if (left == 1) mma_commit(o_done(t));
                mma_commit(empty(load));
              }
            }
            __syncwarp();
          }
          if (!ok) break;
          p_par ^= 1;
          --left;
          advance(size);
        }
      }
      // behind every product and completion of this warp; waited for before the block ends
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      if (!ok && lane == 0) timed_out();
    } else {
      // ---------------------------------------------------------------- the walk, Q loads
      // Segment i + 1 is published before segment i's Q is loaded. A Q tile is tpt tokens x G
      // heads, in that order: a box of the qkv rows. Rows past the request's tokens are
      // other requests' or zeros; nothing of them is written.
      bool ok = true;
      const int tpt = p.tpu / L::kTiles;
      const uint32_t bytes = static_cast<uint32_t>(tpt) * p.G * D * 2;
      Seg g, next;
      g.n = 0;
      bool shared = false;  // the first Q tile in use serves both row tiles
      uint32_t other = 0;
      for (uint32_t i = 0; ok; ++i) {
        const bool more = w.valid();
        if (more) {
          next = make_seg(p, w, tpt);
          w.next(p);
        } else {
          next.n = 0;
        }
        if (i >= kSegs)
          ok = __all_sync(0xFFFFFFFFu, mbar_wait(seg_empty(i), (i / kSegs - 1) & 1, tp_.timeout_ns,
                                                 abort_flag)) != 0;
        if (!ok) break;
        if (lane == 0) {
          segs[i % kSegs] = next;
          mbar_arrive(seg_full(i));
        }
        __syncwarp();
        const int blk = g.head0 / p.hq;
        for (int t = 0; g.n > 0 && t < (g.pair ? 2 : 1); ++t) {
          if (issued_q[t] > 0)
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(q_empty(t), (issued_q[t] - 1) & 1,
                                                   tp_.timeout_ns, abort_flag)) != 0;
          if (ok && t == 0 && shared) {  // and the second tile has let go of it
            ok = __all_sync(0xFFFFFFFFu, mbar_wait(q_other, other, tp_.timeout_ns, abort_flag)) != 0;
            other ^= 1;
          }
          if (!ok) break;
          if (t == 0) shared = !g.pair;
          if (lane == 0) {
            mbar_arrive_expect_tx(q_full(t), bytes);
            for (int h = 0; h < L::kHalves; ++h)
              tma_load_4d(sb + t * L::kOp + h * (kTile * 128), &tp_.tq, q_full(t), h * 64,
                          g.head0 - blk * p.hq, blk, g.row0 + t * tpt);
          }
          __syncwarp();
          ++issued_q[t];
        }
        if (i > 0 && g.n == 0) break;
        g = next;
        if (i == 0 && !more) break;
      }
      if (!ok && lane == 0) timed_out();
    }
  } else {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int t = warp >> 2, x = threadIdx.x & 127;  // tile, row within it = TMEM lane
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const int tpt = p.tpu / L::kTiles, tt = x / p.Gv, hh = x - tt * p.Gv;
    PagedRec rec{0, 0, 0, 0, 0};
    int ns0 = 0, ns1 = 0, segs_o = 0, joined = 0;  // S halves' completions before the segment
    uint32_t tiles0 = 0;  // key tiles of earlier segments
    bool ok = true, taken = true;
    auto wait_all = [&](uint32_t bar, uint32_t parity) -> bool {
      return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, tp_.timeout_ns, abort_flag)) != 0;
    };
    Seg g;
    for (uint32_t i = 0; ok && get_seg(i, g, ok); ++i) {
      const int token = (g.pair ? t * tpt : 0) + tt, head = g.head0 + hh;  // of the unit's tokens
      const bool live = tt < tpt && hh < g.heads && token < g.tokens;
      const bool busy = __any_sync(0xFFFFFFFFu, live);  // a warp without rows computes nothing
      const int64_t row = static_cast<int64_t>(g.row0) + token;
      const int kv_end = g.kv_end;
      const int lim = live && p.causal ? min(kv_end, g.pos0 + token + 1) : kv_end;
      const int lim_min = __reduce_min_sync(0xFFFFFFFFu, lim);
      const int n = g.count(t);
      float m = -INFINITY, l = 0.0f;
      const uint64_t sc2 = pair_of(p.scale_log2, p.scale_log2);
#pragma unroll 1
      for (int s = 0; s < 2 * n; ++s) {  // half h of the tile's k-th key tile
        const int k = s >> 1, h = s & 1;
        const int mm = g.pair ? k : 2 * k + t, k0 = (g.lo + mm) * kTile + 64 * h;
        if (!wait_all(s_full(t, h), (h ? ns1 : ns0) + k & 1)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (h == 0 && k0 + kTile > kv_end) {
          // V rows of keys that no row of the request sees may hold anything and 0 * NaN would
          // spoil O
          const uint32_t ld = tiles0 + i + 1 + mm;  // V's load and place in the ring
          const uint32_t at =
              2 * tiles0 + (mm == g.n - 1 ? 2 * g.n - 1 : g.pair ? 1 + 2 * mm : 2 + 2 * mm);
          if (!wait_all(full(ld), round_of(ld))) {
            ok = false;
            break;
          }
          const uint32_t va = entry_at(at % L::kRing);
          if (k0 + x >= kv_end)
#pragma unroll
            for (int c = 0; c < D / 8; ++c)
              st_shared_v4(va + (c >> 3) * (kTile * 128) + x * 128 + ((c & 7) << 4), 0, 0, 0, 0);
          fence_proxy_async_smem();
        }
        if (busy) {
          const uint32_t miss = bad[(tiles0 + mm) % kBadRing];
          const bool masked = k0 + 64 > lim_min || miss;
          const uint32_t src = tS(t) + lanes + 64 * h;
          uint32_t v[64], pk[32];
          tmem_ld32(src, *reinterpret_cast<uint32_t(*)[32]>(v));
          tmem_ld32(src + 32, *reinterpret_cast<uint32_t(*)[32]>(v + 32));
          tmem_ld_wait();
          if (masked) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {  // bit y: key 32 c + y of the half is seen
              const int seen = min(max(lim - (k0 + 32 * c), 0), 32);
              uint32_t bits = seen == 32 ? ~0u : (1u << seen) - 1u;
              if (miss) {
                const int sh = min(p.ps_log2, 5), span = 32 >> sh;  // pages of the 32 keys
                for (int b = 0; b < span; ++b)
                  if ((miss >> ((64 * h + 32 * c + (b << sh)) >> min(p.ps_log2, 7))) & 1)
                    bits &= ~((sh == 5 ? ~0u : (1u << (1 << sh)) - 1u) << (b << sh));
              }
#pragma unroll
              for (int y = 0; y < 32; ++y)
                if (!(bits & (1u << y))) v[32 * c + y] = 0xff800000u;  // -inf
            }
          }
          // The weights from the maximum so far; this half's is searched for beside the
          // exponentials. They hold for every row of the warp unless one's maximum has to
          // move (by more than 8: weights up to 2^8 are harmless in bf16 and fp32, and o / l
          // does not depend on m); then they are formed again.
          // (A loop, so that the code is there once: a second copy of it slowed every tile.)
          float f = 1.0f;
          uint64_t sum[2];
          for (;;) {
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            const float mu = m == -INFINITY ? 0.0f : m;
            const uint64_t mu2 = pair_of(-mu, -mu);
            sum[0] = sum[1] = 0;
#pragma unroll
            for (int y = 0; y < 32; ++y) {
              const float s0 = __uint_as_float(v[2 * y]), s1 = __uint_as_float(v[2 * y + 1]);
              mx[y & 3] = max3(mx[y & 3], s0, s1);
              float a, b;
              split(fma2(pair_of(s0, s1), sc2, mu2), a, b);
              a = ex2(a);
              b = ex2(b);
              sum[y & 1] = add2(sum[y & 1], pair_of(a, b));
              pk[y] = pack2(a, b);
            }
            const float mb = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
            const bool move = mb > m + 8.0f;
            if (!__any_sync(0xFFFFFFFFu, move)) break;
            if (move) {
              f = ex2(m - mb);
              m = mb;
            }
            if (s > 0) {
              // all earlier P V of the tile have completed when the other half's next S has
              if (!wait_all(s_full(t, h ^ 1), (h ? ns0 + k + 1 : ns1 + k) & 1)) {
                ok = false;
                break;
              }
              tc_fence_after();
#pragma unroll 1
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO(t) + lanes + 32 * c, o);
                tmem_ld_wait();
#pragma unroll
                for (int y = 0; y < 32; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                tmem_st32(tO(t) + lanes + 32 * c, o);
              }
            }
          }
          if (!ok) break;
          tmem_st32(tP(t) + lanes + L::kPHalf * h, pk);
          float sa, sb2;
          split(add2(sum[0], sum[1]), sa, sb2);
          l = l * f + (sa + sb2);
          tmem_st_wait();
        }
        // the segment's first P V overwrites this tile's O: a join has read it
        if (!taken) {
          if (!wait_all(j_free, (joined - 1) & 1)) {
            ok = false;
            break;
          }
          taken = true;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full(t, h));
      }
      if (n > 0) {
        ns0 += n + 1;
        ns1 += n;
      }
      tiles0 += g.n;
      if (!ok) break;
      if (n > 0) {  // the last P V
        if (!wait_all(o_done(t), segs_o & 1)) {
          ok = false;
          break;
        }
        ++segs_o;
        tc_fence_after();
      }
      const bool begins = g.ends & 1, ends = g.ends & 2;
      if (begins && !ends) rec = {g.last, g.row0, g.tokens, g.head0, g.heads};
      const bool joins = !g.pair && g.count(1) > 0;
      if (!g.pair && t == 1) {
        if (joins) {
          // the first tile's warps read this tile's O, in the same TMEM lanes as their own
          join[x] = make_float2(m, l);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(j_full);
          ++joined;
          taken = false;
        }
        continue;
      }
      float mj = m, lj = l, fa = 1.0f, fb = 0.0f;
      if (joins) {
        if (!wait_all(j_full, joined & 1)) {
          ok = false;
          break;
        }
        ++joined;
        tc_fence_after();
        const float2 ml = join[x];
        mj = fmaxf(m, ml.x);
        const float mu = mj == -INFINITY ? 0.0f : mj;
        fa = ex2(m - mu);
        fb = ex2(ml.x - mu);
        lj = l * fa + ml.y * fb;
      }
      const bool whole = begins && ends;
      const float inv = paged_inv(lj);
      const float ga = whole ? fa * inv : fa, gb = whole ? fb * inv : fb;
      float* slot =
          p.part + static_cast<int64_t>(2 * blockIdx.x + (begins ? 1 : 0)) * L::kUnit * (D + 2);
      const int ur = (g.pair ? t : 0) * kTile + x;
      int64_t quad_dst[4];  // where the quad's rows go, -1: nowhere
      {
        const int64_t dst = live ? row * p.H * D + static_cast<int64_t>(head) * D : -1;
#pragma unroll
        for (int i = 0; i < 4; ++i) quad_dst[i] = __shfl_sync(0xFFFFFFFFu, dst, (lane & ~3) + i);
      }
#pragma unroll 1
      for (int c = 0; c < D / 32 && busy; ++c) {
        uint32_t o[32];
        __syncwarp();
        if (n > 0) {
          tmem_ld32(tO(t) + lanes + 32 * c, o);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * ga);
          if (joins) {
            uint32_t o2[32];
            tmem_ld32(tO(1) + lanes + 32 * c, o2);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i)
              o[i] = __float_as_uint(__uint_as_float(o[i]) + __uint_as_float(o2[i]) * gb);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0u;
        }
        if (live) {
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4*>(slot + 2 * L::kUnit + ((8 * c + i) * L::kUnit + ur) * 4) =
                  make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
          }
        }
        if (whole) {
          // Four lanes trade 16-byte chunks so that they store 64 bytes of one row at once:
          // a store instruction then touches 8 lines instead of 32, whose accesses cost a
          // unit's end about 5000 cycles.
          uint32_t q[4][4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int y = 0; y < 4; ++y)
              q[i][y] = pack2(__uint_as_float(o[8 * i + 2 * y]), __uint_as_float(o[8 * i + 2 * y + 1]));
          quad_transpose(q);
#pragma unroll
          for (int i = 0; i < 4; ++i)  // row of lane (lane & ~3) + i, its chunk lane & 3
            if (quad_dst[i] >= 0)
              *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + quad_dst[i] + 32 * c +
                                        8 * (lane & 3)) =
                  make_uint4(q[i][0], q[i][1], q[i][2], q[i][3]);
        }
      }
      if (joins) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(j_free);
      }
      if (live) {
        if (whole) {
          if (p.lse) p.lse[head * p.T + row] = paged_lse(mj, lj);
        } else {
          slot[ur] = mj;
          slot[L::kUnit + ur] = lj;
        }
      }
      tc_fence_before();  // O has been read before the next segment's P is handed over
    }
    if (!ok && lane == 0) timed_out();
    if (threadIdx.x == 0) p.rec[blockIdx.x] = rec;
  }

  // ------------------------------------------------------------------ teardown
  __syncthreads();
  if (*abort_flag) {
    volatile int no_abort = 0;
    if (warp == kWalk && lane == 0)  // the copies this CTA issued have landed
      for (int t = 0; t < 2; ++t)
        if (issued_q[t] > 0) mbar_wait(q_full(t), (issued_q[t] - 1) & 1, kDrainNs, &no_abort);
    if (warp == kProd && lane == 0)
      for (uint32_t l = issued > kLoads ? issued - kLoads : 0; l < issued; ++l)
        mbar_wait(full(l), round_of(l), kDrainNs, &no_abort);
  }
  if (warp == kMma || warp == kMma + 1) {  // the MMAs it issued, and their arrivals, are complete
    volatile int no_abort = 0;
    mbar_wait(drain, 0, kDrainNs, &no_abort);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool ONE>
tp_status tc_t(PagedTcParams& t, int N, cudaStream_t st) {
  using L = Lay<D, ONE>;
  paged_set_units(t.p, kTile, L::kUnit, 7, ONE ? kOneStartCost : kStartCost);
  TP_TRY(paged_q_map(&t.tq, t.p, D, N, t.p.tpu / L::kTiles));
  static std::atomic<uint64_t> attr_set{0};
  if (needs_setup(attr_set)) {
    TP_CUDA_TRY(cudaFuncSetAttribute(paged_tc_kernel<D, ONE>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem));
    mark_device(attr_set);
  }
  const int ctas = std::min(kPagedTcCtas, device_sm_count());
  TP_CUDA_TRY(launch_kernel(paged_tc_kernel<D, ONE>, dim3(ctas), dim3(kThreads),
                            static_cast<size_t>(L::kSmem), st, t));
  count_launch();
  return launch_paged_combine(t.p, D, L::kUnit, kTile, ctas, TP_BF16, st);
}

}  // namespace

tp_status launch_paged_tc(const PagedParams& p, int d, int N, bool one, cudaStream_t st) {
  PagedTcParams t{};
  t.p = p;
  const int64_t rows = (static_cast<int64_t>(p.n_pages) * p.Hkv) << p.ps_log2;
  t.cache_rows = static_cast<int>(rows);
  const int box = std::min(1 << p.ps_log2, kTile);
  TP_TRY(paged_cache_map(&t.tk, p.kc, rows, d, box));
  TP_TRY(paged_cache_map(&t.tv, p.vc, rows, d, box));
  t.status = device_status_word();
  if (!t.status) return fail(TP_ERR_CUDA, "device status word unavailable");
  t.timeout_ns = wait_timeout_ns();
  t.debug_hang = debug_hang_flag();
  if (d == 64) return tc_t<64, false>(t, N, st);
  return one ? tc_t<128, true>(t, N, st) : tc_t<128, false>(t, N, st);
}

size_t paged_tc_floats(int d) {
  return static_cast<size_t>(kPagedTcCtas) * 2 * Lay<64, false>::kUnit * (d + 2);
}

}  // namespace tp
