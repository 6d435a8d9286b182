// Grouped-query attention of each request's new tokens over a paged key/value cache in fp32,
// on CUDA cores (no TF32), and the join of the partial results of all paged kernels. The
// division of the work is paged.cuh's.
//
//   o_i = sum_k softmax_k(q_i . K_k / sqrt(d)) V_k over the keys that row i sees, in one
//   pass: for each tile of keys the scores s (base 2), the running maximum m and sum l,
//     m' = max(m, max s), w = 2^(m - m'), l' = w l + sum 2^(s - m'), O' = w O + 2^(s - m') V,
//   and o = O / l, lse = ln 2 (m + log2 l). Statistics and O are fp32.
// Pieces (m_j, l_j, O_j) of one row join the same way: M = max m_j, o = sum 2^(m_j - M) O_j
// / sum 2^(m_j - M) l_j, in the order of their keys, so a call's result does not depend on
// which CTA finished first.
// Three causal chunks of 2400 tokens over 0, 300 and 600 cached ones, 8 heads over 2, d = 128 /
// 64: 2.03 ms / 966 us, 22 / 23 TFLOP/s of products that are used. No pipe is full (FMA 35 / 38
// % of its peak, shared memory 43 / 58, issue 49 / 60): the 8 / 16 warps that fit an SM wait for
// operands out of shared memory. Nine requests, one with 130 new tokens, d = 64: 32 us; shared
// memory 60 %, FMA 28 % (each key tile is read for two rows at a time), and five tiles per block.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "internal.h"
#include "paged.cuh"
#include "ptx.cuh"

namespace tp {
namespace {

constexpr int kThreads = 256;
constexpr int kKT = 64;  // keys per tile

__device__ __forceinline__ void load4(const float* src, float (&f)[4]) {
  const float4 v = *reinterpret_cast<const float4*>(src);
  f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
}
__device__ __forceinline__ void store4(float* dst, const float (&f)[4]) {
  *reinterpret_cast<float4*>(dst) = make_float4(f[0], f[1], f[2], f[3]);
}
// the output's one rounding: to nearest
__device__ __forceinline__ void store4(__nv_bfloat16* dst, const float (&f)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
  *reinterpret_cast<uint2*>(dst) = make_uint2(*reinterpret_cast<const uint32_t*>(&a),
                                              *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ void store8(__nv_bfloat16* dst, const float (&a)[4], const float (&b)[4]) {
  const __nv_bfloat162 v[4] = {__floats2bfloat162_rn(a[0], a[1]), __floats2bfloat162_rn(a[2], a[3]),
                               __floats2bfloat162_rn(b[0], b[1]), __floats2bfloat162_rn(b[2], b[3])};
  const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
  *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
}


// 16 bytes of global into shared memory, zeros unless `live` (the address is valid either way)
__device__ __forceinline__ void copy16(float* dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src), "r"(live ? 16 : 0)
               : "memory");
}

// Row i of a unit (tiles of tile_rows rows, each of whole tokens): its token and query
// head; false when the row is none.
__device__ __forceinline__ bool unit_row(const PagedParams& p, const PagedReq& q, int u, int vh,
                                         int tile_rows, int i, int* token, int* head) {
  const int tpt = tile_rows / p.Gv;
  const int tile = i / tile_rows, x = i - tile * tile_rows;
  const int tt = x / p.Gv, hh = x - tt * p.Gv;
  const int j = vh / p.hs, g = (vh - j * p.hs) * p.Gv + hh;
  *token = u * p.tpu + tile * tpt + tt;
  *head = j * p.G + g;
  return tt < tpt && g < p.G && *token < q.rows;
}

// RT rows per unit: 16 for a token or a few, 64 for chunks (a key tile is then read from
// L2 once per 64 rows instead of 16).
template <int D, int RT>
struct SimtLayout {
  static constexpr int LD = D + 4;  // padded row: float4 accesses of 8 rows hit 32 banks
  // Q | two stages of K and V | P | m, l, weight per row | key flags per stage
  static constexpr int kQ = 0, kKV = RT * LD, kStage = 2 * kKT * LD, kP = kKV + 2 * kStage,
                       kStat = kP + RT * (kKT + 4), kEnd = kStat + 3 * RT + 2 * kKT;
  static constexpr int kSmem = kEnd * 4;
  static constexpr int kCtas = kSmem <= 112 * 1024 ? 2 : 1;  // per SM
};

template <int D, int RT>
__global__ void __launch_bounds__(kThreads, SimtLayout<D, RT>::kCtas)
    paged_simt_kernel(const PagedParams p) {
  using Lay = SimtLayout<D, RT>;
  constexpr int LD = Lay::LD, PLD = kKT + 4;
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm + Lay::kQ, *Ps = sm + Lay::kP;
  float *ms = sm + Lay::kStat, *ls = ms + RT, *ws = ls + RT;
  int* oks = reinterpret_cast<int*>(ws + RT);  // key is in the cache, per stage
  __shared__ PagedSched sc;
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Scores: a warp has 8 lanes of keys x 4 of rows, a thread SK keys and SR rows of the tile,
  // so that each 16-byte operand access of the warp is one or a half pass over the banks (16
  // x 2 lanes read four times the bytes and took 2.5 times as long). Likewise the output: CL
  // lanes of 4 columns x RL of rows.
  constexpr int RG = RT / 16, SR = 4, SK = kKT / (8 / RG) / 8;  // RG groups of 16 rows
  const int kx = lane & 7, sk0 = (warp / RG) * 8 * SK + kx, sr0 = (warp % RG) * 16 + (lane >> 3);
  constexpr int CG = D / 4, CL = CG < 8 ? CG : 8, RL = 32 / CL, CW = CG / CL, RW = 8 / CW;
  constexpr int OY = RL * RW < RT ? RL * RW : RT, OR = RT / OY;
  // 16 rows: each warp has its own two; 64: the block's warps share all
  constexpr bool kOwn = RT == 16;
  constexpr int CPL = D >= 32 ? D / 32 : 1;
  const int cg = (warp % CW) * CL + lane % CL, oy = (warp / CW) * RL + lane / CL;
  PagedRec rec{0, 0, 0, 0, 0};
  auto w = paged_schedule(p, sc, blockIdx.x, gridDim.x);
  for (; w.valid(); w.next(p)) {
    const int j = w.vh / p.hs;
    const int32_t* tab = p.table + static_cast<int64_t>(w.r) * p.max_pages;
    const int kend = paged_unit_kend(p, w.q, w.u);
    // rows of the unit that are any: a decoding request beside chunks has few of the 64
    const int rows = min(p.tpu, w.q.rows - w.u * p.tpu) * p.Gv;
    // A key tile's loads run beside the work on the one before it (the first's beside Q's):
    // copies into shared memory that occupy no registers; missing keys are zeros.
    auto fetch = [&](int tile) {
      const int k0 = tile * kKT, stage = (tile - w.lo) & 1;
      float* Ks = sm + Lay::kKV + stage * Lay::kStage;
#pragma unroll 4
      for (int e = tid; e < kKT * CG; e += kThreads) {
        const int k = e / CG, c = (e - k * CG) * 4;
        const int64_t row = k0 + k < kend ? paged_row(p, tab, j, k0 + k) : -1;
        const int64_t at = row < 0 ? 0 : row * D + c;
        copy16(Ks + k * LD + c, static_cast<const float*>(p.kc) + at, row >= 0);
        copy16(Ks + (kKT + k) * LD + c, static_cast<const float*>(p.vc) + at, row >= 0);
        if (c == 0) oks[stage * kKT + k] = row >= 0;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    __syncthreads();  // the previous segment's readers are done
    fetch(w.lo);
    for (int e = tid; e < RT * CG; e += kThreads) {
      const int i = e / CG, c = (e - i * CG) * 4;
      int token, head;
      float f[4] = {0.f, 0.f, 0.f, 0.f};
      if (unit_row(p, w.q, w.u, w.vh, RT, i, &token, &head)) {
        load4(static_cast<const float*>(p.qkv) + (static_cast<int64_t>(w.q.row0) + token) * p.ldq +
                  paged_qcol<D>(p, head) + c, f);
      }
      store4(Qs + i * LD + c, f);
    }
    for (int i = tid; i < RT; i += kThreads) {
      ms[i] = -INFINITY;
      ls[i] = ws[i] = 0.0f;
    }
    int lim[SR];  // keys a row's token sees: all, or up to its own position
#pragma unroll
    for (int a = 0; a < SR; ++a)
      lim[a] = p.causal ? static_cast<int>(
                              min(static_cast<int64_t>(w.q.kv_end),
                                  static_cast<int64_t>(w.q.total) - w.q.n + w.u * p.tpu +
                                      (sr0 + 4 * a) / p.Gv + 1))
                        : w.q.kv_end;
    int own_lim[2];
    float own_m[2], own_l[2], own_o[2][CPL];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      own_lim[r] = p.causal ? static_cast<int>(
                                  min(static_cast<int64_t>(w.q.kv_end),
                                      static_cast<int64_t>(w.q.total) - w.q.n + w.u * p.tpu +
                                          (2 * warp + r) / p.Gv + 1))
                            : w.q.kv_end;
      own_m[r] = -INFINITY;
      own_l[r] = 0.0f;
#pragma unroll
      for (int y = 0; y < CPL; ++y) own_o[r][y] = 0.0f;
    }
    float acc[OR][4];
#pragma unroll
    for (int i = 0; i < OR; ++i)
#pragma unroll
      for (int k = 0; k < 4; ++k) acc[i][k] = 0.0f;
    for (int tile = w.lo; tile < w.hi; ++tile) {
      const int k0 = tile * kKT, stage = (tile - w.lo) & 1;
      const float *Ks = sm + Lay::kKV + stage * Lay::kStage, *Vs = Ks + kKT * LD;
      const int* ok = oks + stage * kKT;
      if (tile + 1 < w.hi) {
        if (tile > w.lo) __syncthreads();  // the other stage's readers are done
        fetch(tile + 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      __syncthreads();
      if constexpr (kOwn) {
        // Two rows per warp, a lane two keys' scores and CPL columns of the output: nothing but
        // the key tile is shared, so no warp waits for another within a tile.
        const int r0 = 2 * warp;
        if (r0 < rows) {
          float s[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
#pragma unroll 4
          for (int c = 0; c < D; c += 4) {
            const float4 ka = *reinterpret_cast<const float4*>(Ks + lane * LD + c);
            const float4 kb = *reinterpret_cast<const float4*>(Ks + (lane + 32) * LD + c);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              const float4 q = *reinterpret_cast<const float4*>(Qs + (r0 + r) * LD + c);
              s[r][0] = fmaf(q.w, ka.w, fmaf(q.z, ka.z, fmaf(q.y, ka.y, fmaf(q.x, ka.x, s[r][0]))));
              s[r][1] = fmaf(q.w, kb.w, fmaf(q.z, kb.z, fmaf(q.y, kb.y, fmaf(q.x, kb.x, s[r][1]))));
            }
          }
          const bool oa = ok[lane], ob = ok[lane + 32];
          float mx[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            s[r][0] = oa && k0 + lane < own_lim[r] ? s[r][0] * p.scale_log2 : -INFINITY;
            s[r][1] = ob && k0 + lane + 32 < own_lim[r] ? s[r][1] * p.scale_log2 : -INFINITY;
            mx[r] = fmaxf(s[r][0], s[r][1]);
          }
#pragma unroll
          for (int o = 16; o; o >>= 1)
#pragma unroll
            for (int r = 0; r < 2; ++r) mx[r] = fmaxf(mx[r], __shfl_xor_sync(0xFFFFFFFFu, mx[r], o));
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float m1 = fmaxf(own_m[r], mx[r]), mu = m1 == -INFINITY ? 0.0f : m1;
            const float wt = ex2(own_m[r] - mu), ea = ex2(s[r][0] - mu), eb = ex2(s[r][1] - mu);
            own_m[r] = m1;
            own_l[r] = own_l[r] * wt + (ea + eb);  // this lane's keys
            Ps[(r0 + r) * PLD + lane] = ea;
            Ps[(r0 + r) * PLD + lane + 32] = eb;
#pragma unroll
            for (int y = 0; y < CPL; ++y) own_o[r][y] *= wt;
          }
          __syncwarp();
          if (lane * CPL < D) {
#pragma unroll 2
            for (int k = 0; k < kKT; k += 4) {
              float e[2][4];
              load4(Ps + r0 * PLD + k, e[0]);
              load4(Ps + (r0 + 1) * PLD + k, e[1]);
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                const float* v = Vs + (k + z) * LD + lane * CPL;
                float vv[CPL];
                if constexpr (CPL == 4) {
                  load4(v, vv);
                } else {
#pragma unroll
                  for (int y = 0; y < CPL; ++y) vv[y] = v[y];
                }
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                  for (int y = 0; y < CPL; ++y) own_o[r][y] = fmaf(e[r][z], vv[y], own_o[r][y]);
              }
            }
          }
        }
        continue;
      }
      {
        float s[SR][SK];
#pragma unroll
        for (int a = 0; a < SR; ++a)
#pragma unroll
          for (int b = 0; b < SK; ++b) s[a][b] = 0.0f;
        const int rows_here = rows - (warp % RG) * 16;
        if (rows_here > 0) {
          auto dot = [&](auto sr) {  // the first sr of this thread's rows
            constexpr int N = decltype(sr)::value;
#pragma unroll 4
            for (int c = 0; c < D; c += 4) {
              float4 kv[SK];
#pragma unroll
              for (int b = 0; b < SK; ++b)
                kv[b] = *reinterpret_cast<const float4*>(Ks + (sk0 + 8 * b) * LD + c);
#pragma unroll
              for (int a = 0; a < N; ++a) {
                const float4 q = *reinterpret_cast<const float4*>(Qs + (sr0 + 4 * a) * LD + c);
#pragma unroll
                for (int b = 0; b < SK; ++b) {
                  s[a][b] = fmaf(q.x, kv[b].x, s[a][b]);
                  s[a][b] = fmaf(q.y, kv[b].y, s[a][b]);
                  s[a][b] = fmaf(q.z, kv[b].z, s[a][b]);
                  s[a][b] = fmaf(q.w, kv[b].w, s[a][b]);
                }
              }
            }
          };
          if (rows_here > 4)
            dot(std::integral_constant<int, SR>{});
          else
            dot(std::integral_constant<int, 1>{});
#pragma unroll
          for (int b = 0; b < SK; ++b) {
            const int k = sk0 + 8 * b;
            const bool there = ok[k];
#pragma unroll
            for (int a = 0; a < SR; ++a)
              Ps[(sr0 + 4 * a) * PLD + k] =
                  there && k0 + k < lim[a] ? s[a][b] * p.scale_log2 : -INFINITY;
          }
        }
      }
      __syncthreads();
      {
        // a warp's rows side by side: one row's shuffles wait behind another's
        constexpr int NR = RT / 8;
        float a[NR], b[NR], mx[NR];
        auto each = [&](auto f) {
#pragma unroll
          for (int y = 0; y < NR; ++y)
            if (warp + 8 * y < rows) f(y, warp + 8 * y);
        };
        each([&](int y, int i) {
          a[y] = Ps[i * PLD + lane];
          b[y] = Ps[i * PLD + lane + 32];
          mx[y] = fmaxf(a[y], b[y]);
        });
#pragma unroll
        for (int o = 16; o; o >>= 1)
          each([&](int y, int) { mx[y] = fmaxf(mx[y], __shfl_xor_sync(0xFFFFFFFFu, mx[y], o)); });
        each([&](int y, int i) {
          const float m0 = ms[i], m1 = fmaxf(m0, mx[y]), mu = m1 == -INFINITY ? 0.0f : m1;
          a[y] = ex2(a[y] - mu);
          b[y] = ex2(b[y] - mu);
          Ps[i * PLD + lane] = a[y];
          Ps[i * PLD + lane + 32] = b[y];
          a[y] += b[y];
          b[y] = ex2(m0 - mu);
          mx[y] = m1;
        });
#pragma unroll
        for (int o = 16; o; o >>= 1)
          each([&](int y, int) { a[y] += __shfl_xor_sync(0xFFFFFFFFu, a[y], o); });
        __syncwarp();
        each([&](int y, int i) {
          if (lane == 0) {
            ws[i] = b[y];
            ls[i] = ls[i] * b[y] + a[y];
            ms[i] = mx[y];
          }
        });
      }
      __syncthreads();
      if (oy < OY) {
#pragma unroll
        for (int i = 0; i < OR; ++i) {
          if (i * OY >= rows) break;
          const float wt = ws[oy + i * OY];
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[i][k] *= wt;
        }
#pragma unroll 2
        for (int k = 0; k < kKT; k += 4) {
          float4 v[4];
#pragma unroll
          for (int z = 0; z < 4; ++z)
            v[z] = *reinterpret_cast<const float4*>(Vs + (k + z) * LD + cg * 4);
#pragma unroll
          for (int i = 0; i < OR; ++i) {
            if (i * OY >= rows) break;
            const float4 e = *reinterpret_cast<const float4*>(Ps + (oy + i * OY) * PLD + k);
            acc[i][0] += e.x * v[0].x + e.y * v[1].x + e.z * v[2].x + e.w * v[3].x;
            acc[i][1] += e.x * v[0].y + e.y * v[1].y + e.z * v[2].y + e.w * v[3].y;
            acc[i][2] += e.x * v[0].z + e.y * v[1].z + e.z * v[2].z + e.w * v[3].z;
            acc[i][3] += e.x * v[0].w + e.y * v[1].w + e.z * v[2].w + e.w * v[3].w;
          }
        }
      }
    }
    const bool begins = w.lo == 0, ends = w.hi == w.tiles;
    if (begins && !ends) paged_tail(p, rec, w);
    float* slot = p.part + static_cast<int64_t>(2 * blockIdx.x + (begins ? 1 : 0)) * RT * (D + 2);
    if constexpr (kOwn) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 2 * warp + r;
        float l = own_l[r];
#pragma unroll
        for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xFFFFFFFFu, l, o);
        int token, head;
        if (!unit_row(p, w.q, w.u, w.vh, RT, row, &token, &head)) continue;
        const int64_t t = static_cast<int64_t>(w.q.row0) + token;
        const float inv = paged_inv(l);
        const bool whole = begins && ends;
        float* dst = whole ? static_cast<float*>(p.o) + t * p.H * D + static_cast<int64_t>(head) * D
                           : slot + 2 * RT + row * D;
        if (lane * CPL < D)
#pragma unroll
          for (int y = 0; y < CPL; ++y) dst[lane * CPL + y] = own_o[r][y] * (whole ? inv : 1.0f);
        if (lane == 0) {
          if (!whole) {
            slot[row] = own_m[r];
            slot[RT + row] = l;
          } else if (p.lse) {
            p.lse[head * p.T + t] = paged_lse(own_m[r], l);
          }
        }
      }
    } else if (oy < OY) {
#pragma unroll
      for (int i = 0; i < OR; ++i) {
        const int row = oy + i * OY;
        int token, head;
        if (!unit_row(p, w.q, w.u, w.vh, RT, row, &token, &head)) continue;
        if (begins && ends) {
          const float l = ls[row], inv = paged_inv(l);
          float f[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] = acc[i][k] * inv;
          const int64_t t = static_cast<int64_t>(w.q.row0) + token;
          store4(static_cast<float*>(p.o) + t * p.H * D + static_cast<int64_t>(head) * D + cg * 4, f);
          if (cg == 0 && p.lse) p.lse[head * p.T + t] = paged_lse(ms[row], l);
        } else {
          store4(slot + 2 * RT + row * D + cg * 4, acc[i]);
          if (cg == 0) {
            slot[row] = ms[row];
            slot[RT + row] = ls[row];
          }
        }
      }
    }
  }
  if (tid == 0) p.rec[blockIdx.x] = rec;
}

// CTA (i, y) joins a part of the unit whose first piece is CTA i's tail: that piece, then the
// heads of the following CTAs up to the one where the unit ends. A thread has PER groups of
// 4 columns of one row and every G-th piece: the maximum over its pieces first, then weights,
// sums and outputs, whose loads do not wait for one another; the G threads of a row and
// columns join in shared memory. G = 4 for the slots of few rows, where a long context has
// tens of pieces, and 1 for those of 256, which have two or three. Slots of 128: 4 where a
// unit has about ten pieces or more (8 drafts, 32 heads over 8, d = 128, us, with 1 / 4: one
// request of 3000 tokens 24.7 / 24.0, of 30000 47 / 45; three of 100000 213 / 216).
// Slots of 128-row tiles hold O by groups of 4 columns, (d / 4, rows, 4), as their kernel has a
// thread per row; the others by rows. Threads follow the slots' order.
template <typename T, int D, int PER, int G>
__global__ void __launch_bounds__(kThreads) paged_combine_kernel(const PagedParams p,
                                                                 const int unit_rows,
                                                                 const int tile_rows) {
  static_assert(G == 1 || PER == 1, "");
  constexpr int kPer = kThreads / G;  // threads of a group of pieces
  __shared__ float join[G > 1 ? G : 1][6][G > 1 ? kPer : 1];
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  constexpr int CG = D / 4;
  const int i = blockIdx.x;
  const PagedRec rec = p.rec[i];
  if (rec.tail <= i) return;
  const int pieces = min(rec.tail, static_cast<int>(gridDim.x) - 1) - i + 1;
  const int group = threadIdx.x / kPer, et = threadIdx.x % kPer;
  const int e = blockIdx.y * kPer + et;
  int row, cg, step;  // this thread's first group of columns, and to its next one
  if (tile_rows >= 128) {
    row = e % unit_rows;
    cg = e / unit_rows * PER;
    step = unit_rows;
  } else {
    row = e / CG;
    cg = e % CG;
    step = 0;
  }
  const int tile = row / tile_rows, x = row - tile * tile_rows, tpt = tile_rows / p.Gv;
  const int tt = x / p.Gv, hh = x - tt * p.Gv, token = tile * tpt + tt;
  const bool live =
      row < unit_rows && cg < CG && tt < tpt && hh < rec.heads && token < rec.tokens;
  if (G == 1 && !live) return;
  const int64_t floats = static_cast<int64_t>(unit_rows) * (D + 2);
  // piece 0 is CTA i's tail (its second slot), piece k CTA i + k's head
  const float* base = p.part + 2 * static_cast<int64_t>(i) * floats;
  auto slot_of = [&](int k) { return base + (2 * static_cast<int64_t>(k) + (k == 0)) * floats; };
  const int count = live ? pieces : 0;
  float M = -INFINITY;
#pragma unroll 8
  for (int k = group; k < count; k += G) M = fmaxf(M, slot_of(k)[row]);
  float mu = M == -INFINITY ? 0.0f : M;
  const int64_t at = 2 * unit_rows + 4 * (step ? static_cast<int64_t>(cg) * step + row
                                               : static_cast<int64_t>(row) * CG + cg);
  float l = 0.0f, f[PER][4];
#pragma unroll
  for (int g = 0; g < PER; ++g)
#pragma unroll
    for (int y = 0; y < 4; ++y) f[g][y] = 0.0f;
#pragma unroll 4
  for (int k = group; k < count; k += G) {
    const float* s = slot_of(k);
    const float w = exp2f(s[row] - mu);
    l += s[unit_rows + row] * w;
#pragma unroll
    for (int g = 0; g < PER; ++g) {
      float o[4];
      load4(s + at + 4 * g * static_cast<int64_t>(step), o);
#pragma unroll
      for (int y = 0; y < 4; ++y) f[g][y] += o[y] * w;
    }
  }
  if constexpr (G > 1) {
    join[group][0][et] = M;
    join[group][1][et] = l;
#pragma unroll
    for (int y = 0; y < 4; ++y) join[group][2 + y][et] = f[0][y];
    __syncthreads();
    if (group > 0 || !live) return;
#pragma unroll
    for (int g = 1; g < G; ++g) M = fmaxf(M, join[g][0][et]);
    mu = M == -INFINITY ? 0.0f : M;
    l = 0.0f;
#pragma unroll
    for (int y = 0; y < 4; ++y) f[0][y] = 0.0f;
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const float w = exp2f(join[g][0][et] - mu);
      l += join[g][1][et] * w;
#pragma unroll
      for (int y = 0; y < 4; ++y) f[0][y] += join[g][2 + y][et] * w;
    }
  }
  const float inv = paged_inv(l);
  const int64_t t = static_cast<int64_t>(rec.row0) + token;
  const int head = rec.head0 + hh;
  T* dst = static_cast<T*>(p.o) + t * p.H * D + static_cast<int64_t>(head) * D + 4 * cg;
#pragma unroll
  for (int g = 0; g < PER; ++g)
#pragma unroll
    for (int y = 0; y < 4; ++y) f[g][y] *= inv;
  if constexpr (PER % 2 == 0 && sizeof(T) == 2) {
#pragma unroll
    for (int g = 0; g < PER; g += 2) store8(dst + 4 * g, f[g], f[g + 1]);
  } else {
#pragma unroll
    for (int g = 0; g < PER; ++g) store4(dst + 4 * g, f[g]);
  }
  if (cg == 0 && p.lse) p.lse[head * p.T + t] = paged_lse(M, l);
}

template <typename T, int D>
tp_status combine_t(const PagedParams& p, int unit_rows, int tile_rows, int ctas, cudaStream_t st) {
  const bool few_units = unit_rows == 128 && 10 * static_cast<int64_t>(p.R) * p.Hv <= ctas;
  if (tile_rows >= 128 && !few_units) {
    constexpr int PER = 4;
    TP_CUDA_TRY(launch_kernel(paged_combine_kernel<T, D, PER, 1>,
                              dim3(ctas, unit_rows * (D / 4 / PER) / kThreads), dim3(kThreads), 0,
                              st, p, unit_rows, tile_rows));
  } else {
    constexpr int G = 4;
    TP_CUDA_TRY(launch_kernel(paged_combine_kernel<T, D, 1, G>,
                              dim3(ctas, std::max(1, unit_rows * (D / 4) / (kThreads / G))),
                              dim3(kThreads), 0, st, p, unit_rows, tile_rows));
  }
  count_launch();
  return TP_OK;
}

template <int D, int RT>
tp_status simt_t(PagedParams& p, cudaStream_t st) {
  using Lay = SimtLayout<D, RT>;
  paged_set_units(p, RT, RT, 6, 1);
  static std::atomic<uint64_t> attr_set{0};
  if (needs_setup(attr_set)) {
    TP_CUDA_TRY(cudaFuncSetAttribute(paged_simt_kernel<D, RT>,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize, Lay::kSmem));
    mark_device(attr_set);
  }
  const int ctas = std::min(kPagedMaxCtas, device_sm_count() * Lay::kCtas);
  TP_CUDA_TRY(launch_kernel(paged_simt_kernel<D, RT>, dim3(ctas), dim3(kThreads),
                            static_cast<size_t>(Lay::kSmem), st, p));
  count_launch();
  return launch_paged_combine(p, D, RT, RT, ctas, TP_F32, st);
}

}  // namespace

tp_status launch_paged_simt(PagedParams p, int d, bool wide, cudaStream_t st) {
  switch (d) {
    case 16: return wide ? simt_t<16, 64>(p, st) : simt_t<16, 16>(p, st);
    case 32: return wide ? simt_t<32, 64>(p, st) : simt_t<32, 16>(p, st);
    case 64: return wide ? simt_t<64, 64>(p, st) : simt_t<64, 16>(p, st);
    default: return wide ? simt_t<128, 64>(p, st) : simt_t<128, 16>(p, st);
  }
}

tp_status launch_paged_combine(const PagedParams& p, int d, int unit_rows, int tile_rows, int ctas,
                               tp_dtype dt, cudaStream_t st) {
  auto go = [&](auto dim) -> tp_status {
    constexpr int D = decltype(dim)::value;
    return dt == TP_BF16 ? combine_t<__nv_bfloat16, D>(p, unit_rows, tile_rows, ctas, st)
                         : combine_t<float, D>(p, unit_rows, tile_rows, ctas, st);
  };
  switch (d) {
    case 16: return go(std::integral_constant<int, 16>{});
    case 32: return go(std::integral_constant<int, 32>{});
    case 64: return go(std::integral_constant<int, 64>{});
    default: return go(std::integral_constant<int, 128>{});
  }
}

void paged_set_units(PagedParams& p, int tile_rows, int unit_rows, int kt_log2, int unit_cost) {
  p.hs = (p.G + tile_rows - 1) / tile_rows;
  p.Gv = (p.G + p.hs - 1) / p.hs;
  p.Hv = p.Hkv * p.hs;
  p.tpu = tile_rows / p.Gv * (unit_rows / tile_rows);
  p.kt_log2 = kt_log2;
  p.tpu_log2 = -1;
  for (int k = 0; k < 16; ++k)
    if (p.tpu == 1 << k) p.tpu_log2 = k;
  p.unit_cost = unit_cost;
}

size_t paged_workspace_bytes(int d, tp_dtype dt) {
  const int rows = dt == TP_F32 ? 64 : 16;  // of a unit of the fp32, the few-row kernel
  size_t floats = static_cast<size_t>(kPagedMaxCtas) * 2 * rows * (d + 2);
  if (dt == TP_BF16 && d >= 64) floats = std::max(floats, paged_tc_floats(d));
  return align_up(kPagedMaxCtas * sizeof(PagedRec), 256) + floats * 4;
}

}  // namespace tp
