// Paged grouped-query attention for few rows per key/value head (decode, drafts), bf16.
//
// A unit is 16 rows (tokens x query heads of one key/value head) and its keys come in tiles
// of 64 (paged.cuh divides them over the GPU). Each K and V element is used for at most 16
// rows, so HBM bounds the kernel; everything else has to stay out of the loads' way:
//   one producer warp: page ids 32 at a time (the next 32 already on their way), then one
//     TMA box per page, 64-column half and tensor into a ring of stages; pages that are not
//     the cache's, or past the unit's keys, are boxes outside the tensor, which arrive as
//     zeros without any traffic;
//   four consumer warps, 16 keys each, with their own running maximum and sum, so that the
//     main loop has no exchange between warps: S = Q K^T and O += P V by mma.m16n8k16, Q,
//     P and O in registers (P's accumulator layout is the second product's operand layout),
//     K and V by ldmatrix out of the swizzled rows. tcgen05 would need 128 rows, or P
//     through shared memory with keys as rows; at 16 rows the legacy instruction takes about
//     a fifth of the loads' time (16 + 16 instructions of 4096 FLOP per 16 keys at d = 128).
// At a segment's end the warps' pieces join in shared memory, 32 columns at a time.
// Two CTAs per SM, 96 KB of loads in flight each (64 at d = 32, 32 at d = 16): one CTA's joins
// and unit changes overlap the other's stream. Measured: 61 requests of 1 to 8191 tokens, 64 heads over 8, d = 128,
// pages of 64 (1026 MB) 164 us, 6.2 TB/s, 92 % of what a copy reaches; three of 90001 to
// 131071, 32 heads over 4, pages of 128 (679 MB) 111 us, 6.1 TB/s; one of 701, 32 heads over
// 8, d = 64: 9.3 us, latency. At d = 16 and 32 the time goes by key tiles, not bytes: 64 requests
// of 2 to 8001 tokens, 32 heads over 8, pages of 16, 78 and 80 us (131 and 262 MB). Units of 32
// rows (twice the warps, one CTA per SM) took 90 us where the tcgen05 kernel took 82 (33
// requests of 8 to 28 rows; it takes 77 now).
// Every wait is bounded. A warp whose wait expired records TP_ERR_TIMEOUT and goes through
// the rest of its segments without waiting (the join's barrier needs all four warps); the
// producer waits, bounded, for the copies it issued.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <mutex>
#include <string>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace tp {
namespace {

constexpr int kRows = 16, kKT = 64;
constexpr int kConsumers = 4;
constexpr int kThreads = (kConsumers + 1) * 32;
constexpr uint64_t kDrainNs = 20000000ull;

struct DecodeParams {
  CUtensorMap tk, tv;  // (n_pages * Hkv * page, d), box min(64, d) x min(64, page)
  PagedParams p;
  int cache_rows;
  int* status;
  uint64_t timeout_ns;
  int debug_hang;
};

template <int D>
struct Lay {
  static constexpr int kTile = kKT * D * 2;  // K or V, bytes
  static constexpr int kStages = D == 128 ? 3 : D == 64 ? 6 : 8;
  static constexpr int kJoin = kStages * 2 * kTile;  // 4 warps x 16 rows x 32 floats
  static constexpr int kJoinCols = D < 32 ? D : 32;
  static constexpr int kMl = kJoin + kConsumers * kRows * kJoinCols * 4;  // (m, l) per warp and row
  static constexpr int kBar = kMl + kConsumers * kRows * 8;
  static constexpr int kSmem = kBar + 24 * 8 + 8 * 4 + 16 + 1024;
};

// byte offset of 16-byte chunk c of row r in a K or V tile, as TMA's swizzle leaves it
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (D >= 64)
    return (c >> 3) * (kKT * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
  else if constexpr (D == 32)
    return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  else
    return r * 32 + ((c ^ ((r >> 2) & 1)) << 4);
}

__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory");
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    paged_decode_kernel(const __grid_constant__ DecodeParams dp) {
  using L = Lay<D>;
  const PagedParams& p = dp.p;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_u32(smem);
  float* join = reinterpret_cast<float*>(smem + L::kJoin);
  float2* ml = reinterpret_cast<float2*>(smem + L::kMl);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::kBar);
  volatile uint32_t* bad = reinterpret_cast<volatile uint32_t*>(bars + 24);  // per stage
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 24) + 8;
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (8 + s); };
  const uint32_t never = bar0 + 8u * 16;
  __shared__ PagedSched sc;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kConsumers);
    }
    mbar_init(never, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();  // the set-up above overlaps the previous kernel
  pdl_trigger();
  auto w = paged_schedule(p, sc, blockIdx.x, gridDim.x);  // has block-wide barriers
  int it = 0;  // tiles so far: stage it % kStages, round it / kStages

  if (warp == kConsumers) {
    // ---------------------------------------------------------------- producer
    const int ps = 1 << p.ps_log2, box = min(ps, kKT), boxes = kKT / box;
    constexpr int kHalves = D >= 64 ? D / 64 : 1, kBoxCols = D >= 64 ? 64 : D;
    bool ok = true;
    for (; w.valid() && ok; w.next(p)) {
      const int j = w.vh / p.hs;
      const int kend = paged_unit_kend(p, w.q, w.u);
      const int32_t* tab = p.table + static_cast<int64_t>(w.r) * p.max_pages;
      // ids of 32 pages, one per lane; only pages that hold some of the unit's keys
      const int npages = (kend + ps - 1) >> p.ps_log2;
      auto fetch = [&](int first) {
        const int i = first + lane;
        const int id = i < npages ? tab[i] : -1;
        return id >= 0 && id < p.n_pages ? id : -1;
      };
      int base = (w.lo * kKT) >> p.ps_log2;
      int ids = fetch(base), ahead = fetch(base + 32);
      for (int tile = w.lo; tile < w.hi; ++tile, ++it) {
        const int st = it % L::kStages, round = it / L::kStages;
        if (round > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(empty(st), (round - 1) & 1,
                                                            dp.timeout_ns, abort_flag))) {
          ok = false;
          break;
        }
        const int k0 = tile * kKT;
        const int pg0 = k0 >> p.ps_log2;
        if (pg0 - base >= 32) {  // tiles are whole groups of at most 8 pages
          base += 32;
          ids = ahead;
          ahead = fetch(base + 32);
        }
        // box b of the tile: page pg0 + b (or a part of one page)
        const int src = __shfl_sync(0xFFFFFFFFu, ids, (pg0 - base + min(lane, boxes - 1)) & 31);
        const uint32_t missing = __ballot_sync(0xFFFFFFFFu, lane < boxes && src < 0);
        if (lane == 0) {
          bad[st] = missing;
          mbar_arrive_expect_tx(full(st), 2 * L::kTile);
        }
        __syncwarp();
        const int y = src < 0 ? dp.cache_rows
                              : (((src * p.Hkv + j) << p.ps_log2) + (k0 & (ps - 1)));
        for (int e = lane; e < 32 * 2 * kHalves; e += 32) {  // lane = box: every lane its own
          const int which = e >> 5;
          if (lane < boxes) {
            const int half = which % kHalves;
            const bool is_v = which >= kHalves;
            const uint32_t dst = sb + st * 2 * L::kTile + (is_v ? L::kTile : 0) +
                                 half * (kKT * 128) + lane * box * (kBoxCols * 2);
            tma_load_2d(dst, is_v ? &dp.tv : &dp.tk, full(st), half * 64, y);
          }
        }
      }
    }
    if (!ok && lane == 0) {
      atomicCAS(dp.status, 0, static_cast<int>(TP_ERR_TIMEOUT));
      atomicAdd(dp.status + 1, 1);
    }
  } else {
    // ---------------------------------------------------------------- consumers
    auto timed_out = [&] {
      atomicCAS(dp.status, 0, static_cast<int>(TP_ERR_TIMEOUT));
      atomicAdd(dp.status + 1, 1);
    };
    bool ok = true;
    if (dp.debug_hang && warp == 0) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(never, 0, dp.timeout_ns, abort_flag));
      if (!ok && lane == 0) timed_out();
    }
    const int row0 = lane >> 2, col = (lane & 3) * 2;
    PagedRec rec{0, 0, 0, 0, 0};
    for (; w.valid(); w.next(p)) {
      const int j = w.vh / p.hs;
      const int kend = paged_unit_kend(p, w.q, w.u);
      // this lane's two rows: token, query head and the first key they do not see
      int token[2], head[2], lim[2];
      bool live[2];
      uint32_t q[D / 16][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int x = row0 + 8 * i, tt = x / p.Gv, g = (w.vh - j * p.hs) * p.Gv + x - tt * p.Gv;
        token[i] = w.u * p.tpu + tt;
        head[i] = j * p.G + g;
        live[i] = tt < p.tpu && g < p.G && token[i] < w.q.rows;
        lim[i] = p.causal ? min(kend, w.q.total - w.q.n + token[i] + 1) : kend;
        if (!live[i]) lim[i] = kend;
        const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.qkv) +
                                   (static_cast<int64_t>(w.q.row0) + token[i]) * p.ldq +
                                   paged_qcol<D>(p, live[i] ? head[i] : 0) + col;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          q[kk][i] = live[i] ? *reinterpret_cast<const uint32_t*>(src + kk * 16) : 0u;
          q[kk][2 + i] = live[i] ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8) : 0u;
        }
      }
      const int lim_min = __reduce_min_sync(0xFFFFFFFFu, min(lim[0], lim[1]));
      float o[D / 8][4];
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[n][k] = 0.0f;
      float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
      for (int tile = w.lo; tile < w.hi; ++tile, ++it) {
        const int st = it % L::kStages, round = it / L::kStages;
        if (ok && !__all_sync(0xFFFFFFFFu, mbar_wait(full(st), round & 1, dp.timeout_ns, abort_flag))) {
          ok = false;
          if (lane == 0) timed_out();
        }
        if (!ok) continue;
        const uint32_t kt = sb + st * 2 * L::kTile, vt = kt + L::kTile;
        const int k0 = tile * kKT + warp * 16;  // this warp's 16 keys
        const int rbase = warp * 16;
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) s[n][k] = 0.0f;
        {
          // matrices: keys 0-7 / 8-15 (lane bit 4), dims 0-7 / 8-15 (lane bit 3)
          const int r = rbase + (lane & 7) + ((lane & 16) >> 1), c = (lane >> 3) & 1;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t b[4];
            ldmatrix_x4(b, kt + chunk_at<D>(r, 2 * kk + c));
            mma_16n8k16(s[0], q[kk], b[0], b[1]);
            mma_16n8k16(s[1], q[kk], b[2], b[3]);
          }
        }
        const uint32_t miss = bad[st];
        if (k0 + 16 > lim_min || miss) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int off = 8 * n + col + (k & 1);
              const bool hidden = k0 + off >= lim[k >> 1] ||
                                  ((miss >> ((rbase + off) >> min(p.ps_log2, 6))) & 1);
              if (hidden) s[n][k] = -INFINITY;
            }
          // V rows past the unit's keys may hold anything: 0 * NaN would spoil O
          if (k0 + 16 > kend) {
            for (int e = lane; e < 16 * (D / 8); e += 32) {
              const int r = e / (D / 8), c = e - r * (D / 8);
              if (k0 + r >= kend) st_shared_v4(vt + chunk_at<D>(rbase + r, c), 0, 0, 0, 0);
            }
            fence_proxy_async_smem();  // before the next TMA write of this stage
            __syncwarp();
          }
        }
        float mx[2] = {fmaxf(fmaxf(s[0][0], s[0][1]), fmaxf(s[1][0], s[1][1])),
                       fmaxf(fmaxf(s[0][2], s[0][3]), fmaxf(s[1][2], s[1][3]))};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 1));
          mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xFFFFFFFFu, mx[i], 2));
          mx[i] *= p.scale_log2;
        }
        // The maximum moves only when it grows by more than 8 (weights up to 2^8 are
        // harmless in bf16 and fp32): o / l does not depend on it.
        const bool move = mx[0] > m[0] + 8.0f || mx[1] > m[1] + 8.0f;
        if (__any_sync(0xFFFFFFFFu, move)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float m1 = fmaxf(m[i], mx[i]);
            const float f = m1 == -INFINITY ? 1.0f : ex2(m[i] - m1);
            m[i] = m1;
            l[i] *= f;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
              o[n][2 * i] *= f;
              o[n][2 * i + 1] *= f;
            }
          }
        }
        const float mu[2] = {m[0] == -INFINITY ? 0.0f : m[0], m[1] == -INFINITY ? 0.0f : m[1]};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s[n][k] = ex2(fmaf(s[n][k], p.scale_log2, -mu[k >> 1]));
            l[k >> 1] += s[n][k];
          }
        // P rounded to bf16 (relative 2^-8 of each weight), the operand of the second product
        const uint32_t a[4] = {pack_bf16x2(s[0][0], s[0][1]), pack_bf16x2(s[0][2], s[0][3]),
                               pack_bf16x2(s[1][0], s[1][1]), pack_bf16x2(s[1][2], s[1][3])};
        {
          // matrices (transposed): keys 0-7 / 8-15 (lane bit 3), dims 0-7 / 8-15 (lane bit 4)
          const int r = rbase + (lane & 15), c = lane >> 4;
#pragma unroll
          for (int n = 0; n < D / 16; ++n) {
            uint32_t b[4];
            ldmatrix_x4_trans(b, vt + chunk_at<D>(r, 2 * n + c));
            mma_16n8k16(o[2 * n], a, b[0], b[1]);
            mma_16n8k16(o[2 * n + 1], a, b[2], b[3]);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty(st));
      }
      // ---------------------------------------------------------------- the warps join
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 1);
        l[i] += __shfl_xor_sync(0xFFFFFFFFu, l[i], 2);
        if ((lane & 3) == 0) ml[warp * kRows + row0 + 8 * i] = make_float2(m[i], l[i]);
      }
      consumers_sync();
      float f[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float M = -INFINITY;
#pragma unroll
        for (int v = 0; v < kConsumers; ++v) M = fmaxf(M, ml[v * kRows + row0 + 8 * i].x);
        f[i] = M == -INFINITY ? 0.0f : ex2(m[i] - M);
      }
      // thread: one row and 4 columns of each group of 32
      constexpr int JC = L::kJoinCols, TPR = JC / 4;
      const int tid = threadIdx.x, jr = tid / TPR, jc = (tid % TPR) * 4;
      const bool begins = w.lo == 0, ends = w.hi == w.tiles;
      if (begins && !ends) paged_tail(p, rec, w);
      float M = -INFINITY, lsum = 0.0f;
      int jtoken = 0, jhead = 0;
      bool jlive = false;
      if (jr < kRows) {
#pragma unroll
        for (int v = 0; v < kConsumers; ++v) M = fmaxf(M, ml[v * kRows + jr].x);
        // (M = -inf: all sums are 0, or NaN where the scores are)
        const float mu = M == -INFINITY ? 0.0f : M;
#pragma unroll
        for (int v = 0; v < kConsumers; ++v)
          lsum += ml[v * kRows + jr].y * ex2(ml[v * kRows + jr].x - mu);
        const int tt = jr / p.Gv, g = (w.vh - j * p.hs) * p.Gv + jr - tt * p.Gv;
        jtoken = w.u * p.tpu + tt;
        jhead = j * p.G + g;
        jlive = tt < p.tpu && g < p.G && jtoken < w.q.rows;
      }
      const int64_t t = static_cast<int64_t>(w.q.row0) + jtoken;
      float* slot =
          p.part + static_cast<int64_t>(2 * blockIdx.x + (begins ? 1 : 0)) * kRows * (D + 2);
      const float inv = paged_inv(lsum);
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += JC) {
#pragma unroll
        for (int n = 0; n < JC / 8; ++n)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            *reinterpret_cast<float2*>(join + (warp * kRows + row0 + 8 * i) * JC + 8 * n + col) =
                make_float2(o[c0 / 8 + n][2 * i] * f[i], o[c0 / 8 + n][2 * i + 1] * f[i]);
        consumers_sync();
        if (jlive) {
          float4 v = *reinterpret_cast<const float4*>(join + jr * JC + jc);
#pragma unroll
          for (int k = 1; k < kConsumers; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(join + (k * kRows + jr) * JC + jc);
            v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
          }
          if (begins && ends)
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.o) + t * p.H * D +
                                      static_cast<int64_t>(jhead) * D + c0 + jc) =
                make_uint2(pack_bf16x2(v.x * inv, v.y * inv), pack_bf16x2(v.z * inv, v.w * inv));
          else
            *reinterpret_cast<float4*>(slot + 2 * kRows + jr * D + c0 + jc) = v;
        }
        consumers_sync();
      }
      if (jlive && jc == 0) {
        if (begins && ends) {
          if (p.lse) p.lse[jhead * p.T + t] = paged_lse(M, lsum);
        } else {
          slot[jr] = M;
          slot[kRows + jr] = lsum;
        }
      }
    }
    if (threadIdx.x == 0) p.rec[blockIdx.x] = rec;
  }
  // a role that gave up may have left copies in flight (whenever it did): they land first
  __syncthreads();
  if (*abort_flag && warp == kConsumers) {
    volatile int no_abort = 0;
    for (int s = 0; s < L::kStages; ++s) {
      const int n = it > s ? (it - 1 - s) / L::kStages : -1;  // last round of stage s
      if (n >= 0) mbar_wait(full(s), n & 1, kDrainNs, &no_abort);
    }
  }
  __syncthreads();
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeFn encoder() {
  static EncodeFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeFn>(f);
  });
  return fn;
}

template <int D>
tp_status decode_t(DecodeParams& dp, cudaStream_t st) {
  using L = Lay<D>;
  static std::atomic<uint64_t> attr_set{0};
  if (needs_setup(attr_set)) {
    TP_CUDA_TRY(cudaFuncSetAttribute(paged_decode_kernel<D>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem));
    mark_device(attr_set);
  }
  const int ctas = std::min(kPagedMaxCtas, 2 * device_sm_count());
  TP_CUDA_TRY(launch_kernel(paged_decode_kernel<D>, dim3(ctas), dim3(kThreads),
                            static_cast<size_t>(L::kSmem), st, dp));
  count_launch();
  return launch_paged_combine(dp.p, D, kRows, kRows, ctas, TP_BF16, st);
}

}  // namespace

tp_status paged_cache_map(CUtensorMap* m, const void* cache, int64_t rows, int d, int box_rows) {
  EncodeFn enc = encoder();
  if (!enc) return fail(TP_ERR_CUDA, "cuTensorMapEncodeTiled entry point not available");
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(d) * 2};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(std::min(d, 64)),
                             static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUtensorMapSwizzle sw = d >= 64   ? CU_TENSOR_MAP_SWIZZLE_128B
                                : d == 32 ? CU_TENSOR_MAP_SWIZZLE_64B
                                          : CU_TENSOR_MAP_SWIZZLE_32B;
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(cache), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(TP_ERR_CUDA, "cuTensorMapEncodeTiled failed (code " + std::to_string(r) + ")");
  return TP_OK;
}

tp_status paged_q_map(CUtensorMap* m, const PagedParams& p, int d, int N, int tokens) {
  EncodeFn enc = encoder();
  if (!enc) return fail(TP_ERR_CUDA, "cuTensorMapEncodeTiled entry point not available");
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(p.hq),
                              static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(p.T)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, static_cast<cuuint64_t>(p.S) * 2,
                                 static_cast<cuuint64_t>(p.ldq) * 2};
  const int heads = std::min(p.G, p.hq);  // of one shard block
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(heads),
                             static_cast<cuuint32_t>(p.G / heads),
                             static_cast<cuuint32_t>(tokens)};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(p.qkv), dims,
                         strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(TP_ERR_CUDA, "cuTensorMapEncodeTiled failed (code " + std::to_string(r) + ")");
  return TP_OK;
}

tp_status launch_paged_decode(const PagedParams& p, int d, cudaStream_t st) {
  DecodeParams dp{};
  dp.p = p;
  // start cost of a unit, in tiles: none 184 us, one 174, two 170 (the 61 requests above, before
  // the join was changed)
  paged_set_units(dp.p, kRows, kRows, 6, 2);
  const int64_t rows = (static_cast<int64_t>(p.n_pages) * p.Hkv) << p.ps_log2;
  dp.cache_rows = static_cast<int>(rows);
  const int box = std::min(1 << p.ps_log2, kKT);
  TP_TRY(paged_cache_map(&dp.tk, p.kc, rows, d, box));
  TP_TRY(paged_cache_map(&dp.tv, p.vc, rows, d, box));
  dp.status = device_status_word();
  if (!dp.status) return fail(TP_ERR_CUDA, "device status word unavailable");
  dp.timeout_ns = wait_timeout_ns();
  dp.debug_hang = debug_hang_flag();
  switch (d) {
    case 16: return decode_t<16>(dp, st);
    case 32: return decode_t<32>(dp, st);
    case 64: return decode_t<64>(dp, st);
    default: return decode_t<128>(dp, st);
  }
}

}  // namespace tp
