// fp32 GEMM engine on CUDA cores (FFMA, no TF32: TF32's 10-bit mantissa would not
// hold the fp32 path to 1e-5). Same problem descriptor and epilogues as the
// tensor-core engine; 64 x 64 output tile per CTA, 4 x 4 per thread, K in steps of 32.
// Each thread gathers a whole K step of A and B into registers before storing it to
// shared memory, and the next step's loads are issued before the current step's FMAs,
// so one load latency per step is hidden behind the arithmetic instead of several
// being paid in a row (the small fp32 GEMMs are latency-bound).
// When the output has few tiles (fewer than half the SMs), the K steps of a tile are
// split over the CTAs of a thread-block cluster (2, 4 or 8): each CTA accumulates its
// share, parks the partial tile in shared memory, and after a cluster barrier CTA r
// sums row slice r of the tile over the cluster's CTAs in rank order (distributed
// shared memory) and runs the epilogue on it. The order of the sum is fixed, so the
// result is deterministic; no workspace is needed.
#include <cuda_runtime.h>

#include <atomic>

#include <algorithm>

#include "epi_math.cuh"
#include "internal.h"
#include "ptx.cuh"

namespace tp {
namespace {

constexpr int TM = 64, TN = 64, TK = 32;
constexpr int kPer = TM * TK / 256;  // elements of A (and of each B) per thread per K step

struct SimtParams {
  const float* A[3];
  const float* B[3];
  int64_t lda[3], ldb[3], k0[3];
  int64_t M, N, K;
  int a_mn, b_mn, nseg, paired;
  float* out0;
  float* out1;
  float* out2;
  const float* in0;
  const float* in1;
  int64_t ldo, out_group_stride;
  CeEpi ce;   // EPI_LSE, EPI_DCE
  int split;  // CTAs of a cluster sharing one output tile's K steps (1: no split)
};


template <int EPI>
__device__ __forceinline__ void epi1(const SimtParams& p, int g, int64_t r, int64_t c, float a,
                                     float b) {
  const int64_t i = r * p.ldo + c;
  if constexpr (EPI == EPI_STORE) {
    p.out0[g * p.out_group_stride + i] = a + (p.in0 ? p.in0[i] : 0.0f);
  } else if constexpr (EPI == EPI_GELU) {
    if (p.out0) p.out0[i] = a;
    p.out1[i] = gelu_f(a);
  } else if constexpr (EPI == EPI_SWIGLU) {
    if (p.out0) p.out0[i] = a;
    if (p.out1) p.out1[i] = b;
    p.out2[i] = silu_f(a) * b;
  } else if constexpr (EPI == EPI_DGELU) {
    p.out0[i] = a * gelu_prime_f(p.in0[i]);
  } else if constexpr (EPI == EPI_DSWIGLU) {
    float du;
    p.out0[i] = dswiglu_f(a, p.in0[i], p.in1[i], du);
    p.out1[i] = du;
  } else if constexpr (EPI == EPI_PAIR) {
    p.out0[i] = a;
    p.out1[i] = b;
  }
}

// The gradient by one logit of a row with target t and this lse
__device__ __forceinline__ float ce_grad(const SimtParams& p, float a, int64_t t, float lse, int64_t c) {
  const float q = expf(a - lse) - (t == p.ce.col0 + c ? 1.0f : 0.0f);
  return t >= 0 && t < p.ce.vocab ? q * p.ce.scale : 0.0f;
}

// EPI_LSE of the `rows` rows of the tile's logits in sm (TN floats each), rows r0 .. of the
// product with these targets, columns c0 ..: a warp per row, two columns per lane; expf and the sum in
// 32 bits.
__device__ __forceinline__ void lse_rows(const SimtParams& p, const float* sm, const int32_t* target,
                                         int rows, int64_t r0, int64_t c0, int64_t slot) {
  static_assert(TN == 64, "two columns per lane");
  const int lane = threadIdx.x & 31;
  for (int rr = threadIdx.x >> 5; rr < rows; rr += 8) {
    const int64_t r = r0 + rr;
    if (r >= p.M) break;
    const int64_t ca = c0 + lane, cb = ca + 32;
    const float a = ca < p.N ? sm[rr * TN + lane] : -INFINITY;
    const float b = cb < p.N ? sm[rr * TN + lane + 32] : -INFINITY;
    const int64_t t = target[rr];
    if (t == ca && ca < p.N) p.ce.hit[r] = a;
    if (t == cb && cb < p.N) p.ce.hit[r] = b;
    float m = fmaxf(a, b);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    float s = expf(a - m) + expf(b - m);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0) p.ce.part[slot * p.M + r] = make_float2(m, s);
  }
}

// A and B staging; reused for the partial tile of a split (unpaired only: TM x TN fits)
constexpr int simt_floats(bool paired) { return TK * (TM + 4) + (paired ? 2 : 1) * TK * (TN + 4); }
static_assert(simt_floats(false) >= TM * TN, "partial tile must fit the staging buffers");

// row slice `rank` of the tile: the partial tiles of the CTAs `base` .. `base` + SPLIT - 1 of the
// cluster added in that order, four columns at a time, every load of a thread in flight at once;
// put(row of the tile, column, sum)
template <int SPLIT, class F>
__device__ __forceinline__ void add_partials(const float* sm, int rank, int base, F&& put) {
  constexpr int rows = TM / SPLIT, kVecs = rows * TN / 4 / 256;  // 2, 1 and (8 ranks) half a vector
  float4 v[kVecs > 0 ? kVecs : 1][SPLIT];
#pragma unroll
  for (int i = 0; i < (kVecs > 0 ? kVecs : 1); ++i) {
    const int e = (threadIdx.x + i * 256) * 4;
    if (e < rows * TN) {
      const uint32_t off = smem_u32(sm + rank * rows * TN + e);
#pragma unroll
      for (int q = 0; q < SPLIT; ++q) v[i][q] = ld_cluster_v4(mapa_shared(off, static_cast<uint32_t>(base + q)));
    }
  }
#pragma unroll
  for (int i = 0; i < (kVecs > 0 ? kVecs : 1); ++i) {
    const int e = (threadIdx.x + i * 256) * 4;
    if (e < rows * TN) {
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int q = 0; q < SPLIT; ++q) {
        a.x += v[i][q].x; a.y += v[i][q].y; a.z += v[i][q].z; a.w += v[i][q].w;
      }
      const int rr = rank * rows + e / TN, cc = e % TN;
      put(rr, cc, a.x);
      put(rr, cc + 1, a.y);
      put(rr, cc + 2, a.z);
      put(rr, cc + 3, a.w);
    }
  }
}

// Output tile (bx, by) of group g; sm: simt_floats(PAIRED) floats of shared memory. The p.split CTAs
// of a tile are consecutive ranks of a cluster, which may hold several tiles (exchange: it has more
// than one CTA, all of which meet at its barriers).
template <int EPI, bool PAIRED>
__device__ __forceinline__ void simt_tile(const SimtParams& p, int bx, int by, int g, float* sm,
                                          bool exchange) {
  constexpr int NB = PAIRED ? 2 : 1;
  auto As = reinterpret_cast<float(*)[TM + 4]>(sm);
  auto Bs = reinterpret_cast<float(*)[TK][TN + 4]>(sm + TK * (TM + 4));
  const int split = p.split;
  const int in_cluster = exchange ? static_cast<int>(cluster_ctarank()) : 0;
  const int rank = in_cluster % split, base = in_cluster - rank;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = static_cast<int64_t>(by) * TM;
  const int64_t n0 = static_cast<int64_t>(bx) * TN;
  // the rows' targets and lse, asked for before the product (read after its barriers)
  constexpr bool kCe = EPI == EPI_LSE || EPI == EPI_DCE;
  __shared__ int32_t row_t[kCe ? TM : 1];
  __shared__ float row_lse[kCe ? TM : 1];
  if constexpr (kCe) {
    if (threadIdx.x < TM) {
      const bool in = m0 + threadIdx.x < p.M;
      row_t[threadIdx.x] = in ? p.ce.targets[m0 + threadIdx.x] : -1;
      if constexpr (EPI == EPI_DCE) row_lse[threadIdx.x] = in ? p.ce.lse[m0 + threadIdx.x] : 0.0f;
    }
    if (EPI == EPI_LSE && bx == 0 && by == 0 && rank == 0 && threadIdx.x == 0) *p.ce.counter = 0;
  }
  float acc[4][4] = {}, acc2[4][4] = {};
  float ra[kPer], rb[NB][kPer];
  // element e of a step: consecutive threads walk the contiguous storage dimension
  auto a_idx = [&](int e, int& mm, int& kk) {
    mm = p.a_mn ? e % TM : e / TK;
    kk = p.a_mn ? e / TM : e % TK;
  };
  auto b_idx = [&](int e, int& nn, int& kk) {
    nn = p.b_mn ? e % TN : e / TK;
    kk = p.b_mn ? e / TN : e % TK;
  };
  // a thread's elements of an operand's tile and K step (a_idx, b_idx): one pointer, a fixed distance
  // apart (K-major: 8 rows, MN-major: 4 values of k)
  static_assert(TM == 64 && TN == 64 && TK == 32, "distances below");
  auto fetch = [&](const float* X, int64_t ld, bool mn, int64_t x0, int64_t x_end, int64_t kg,
                   int64_t k0, float* r) {
    const int t = threadIdx.x;
    const float* q = X + (mn ? (kg + t / 64) * ld + x0 + t % 64 : (x0 + t / 32) * ld + kg + t % 32);
    const int64_t step = mn ? 4 * ld : 8 * ld;
    const bool in = mn ? x0 + t % 64 < x_end : k0 + t % 32 < p.K;
    // how many of them there are
    const int64_t n = !in ? 0 : mn ? (p.K - k0 - t / 64 + 3) / 4 : (x_end - x0 - t / 32 + 7) / 8;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      r[i] = i < n ? *q : 0.0f;
      q += step;
    }
  };
  auto load = [&](int s, int64_t k0) {  // one K step of segment s: global -> registers
    const int64_t kg = p.k0[s] + g * p.K + k0;
    fetch(p.A[s], p.lda[s], p.a_mn, m0, p.M, kg, k0, ra);
#pragma unroll
    for (int h = 0; h < NB; ++h)
      fetch(p.B[PAIRED ? h : s], p.ldb[PAIRED ? h : s], p.b_mn, n0, p.N, kg, k0, rb[h]);
  };
  const int64_t steps = (p.K + TK - 1) / TK, total = steps * p.nseg;
  const int64_t per = (total + split - 1) / split;  // this CTA's K steps: [it0, it1)
  const int64_t it0 = rank * per, it1 = it0 + per < total ? it0 + per : total;
  int seg = 0;  // the segment and its step that are loaded next
  int64_t ks = it0;
  while (ks >= steps && seg + 1 < p.nseg) {
    ks -= steps;
    ++seg;
  }
  auto load_next = [&]() {
    load(seg, ks * TK);
    if (++ks == steps) {
      ks = 0;
      ++seg;
    }
  };
  if (it0 < it1) load_next();
  for (int64_t it = it0; it < it1; ++it) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {  // registers -> shared (the previous step's reads ended
      int mm, kk;                     // at the __syncthreads below)
      a_idx(threadIdx.x + i * 256, mm, kk);
      As[kk][mm] = ra[i];
#pragma unroll
      for (int h = 0; h < NB; ++h) {
        int nn, kb;
        b_idx(threadIdx.x + i * 256, nn, kb);
        Bs[h][kb][nn] = rb[h][i];
      }
    }
    __syncthreads();
    if (it + 1 < it1) load_next();  // the next step's loads fly while this step's FMAs run
#pragma unroll
    for (int kk = 0; kk < TK; ++kk) {
      float a[4], b[4], b2[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = As[kk][ty * 4 + i];
        b[i] = Bs[0][kk][tx * 4 + i];
        if constexpr (PAIRED) b2[i] = Bs[NB - 1][kk][tx * 4 + i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
          if constexpr (PAIRED) acc2[i][j] = fmaf(a[i], b2[j], acc2[i][j]);
        }
    }
    __syncthreads();
  }
  if (EPI == EPI_LSE && split == 1) {
    if constexpr (EPI == EPI_LSE) {  // the tile through shared memory, whose last reads have ended
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) sm[(ty * 4 + i) * TN + tx * 4 + j] = acc[i][j];
      __syncthreads();
      lse_rows(p, sm, row_t, TM, m0, n0, n0 / TN);
    }
    return;
  }
  if (split == 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t r = m0 + ty * 4 + i, c = n0 + tx * 4 + j;
        if (r < p.M && c < p.N) {
          if constexpr (EPI == EPI_DCE)
            p.out0[r * p.ldo + c] = ce_grad(p, acc[i][j], row_t[ty * 4 + i], row_lse[ty * 4 + i], c);
          else
            epi1<EPI>(p, g, r, c, acc[i][j], acc2[i][j]);
        }
      }
    if (exchange) {  // other tiles of the cluster do exchange theirs
      cluster_sync_all();
      cluster_sync_all();
    }
    return;
  }
  if constexpr (!PAIRED) {  // split K (the host splits unpaired problems only)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sm[(ty * 4 + i) * TN + tx * 4 + j] = acc[i][j];
    cluster_sync_all();  // every CTA's partial tile is in its shared memory
    const int rows = TM / split;
    auto put = [&](int rr, int cc, float v) {
      const int64_t r = m0 + rr, c = n0 + cc;
      if constexpr (EPI == EPI_LSE) {
        sm[rr * TN + cc] = v;  // read by this thread alone
      } else if (r < p.M && c < p.N) {
        if constexpr (EPI == EPI_DCE) p.out0[r * p.ldo + c] = ce_grad(p, v, row_t[rr], row_lse[rr], c);
        else epi1<EPI>(p, g, r, c, v, 0.0f);
      }
    };
    if (split == 2) add_partials<2>(sm, rank, base, put);
    else if (split == 4) add_partials<4>(sm, rank, base, put);
    else add_partials<8>(sm, rank, base, put);
    if constexpr (EPI == EPI_LSE) {
      __syncthreads();
      lse_rows(p, sm + rank * rows * TN, row_t + rank * rows, rows, m0 + rank * rows, n0, n0 / TN);
    }
    cluster_sync_all();  // no CTA leaves while another still reads its tile
  }
}

template <int EPI, bool PAIRED>
__global__ void __launch_bounds__(256) gemm_simt_kernel(const SimtParams p) {
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  __shared__ __align__(16) float sm[simt_floats(PAIRED)];
  simt_tile<EPI, PAIRED>(p, blockIdx.x / p.split, blockIdx.y, blockIdx.z, sm, p.split > 1);
}

// Two plain products that do not depend on one another, the second's CTAs (from ctas0 on) after the
// first's: one launch instead of two, which at small sizes is most of their time. Each has a split of
// its own that divides the cluster's size; a cluster's last tiles may lie past the product.
__global__ void __launch_bounds__(256)
    gemm_simt_two_kernel(const SimtParams p0, const SimtParams p1, int ctas0, int gx0, int gx1,
                         int cluster) {
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  __shared__ __align__(16) float sm[simt_floats(false)];
  const bool first = blockIdx.x < ctas0;
  const SimtParams& p = first ? p0 : p1;
  const int gx = first ? gx0 : gx1, t = (blockIdx.x - (first ? 0 : ctas0)) / p.split;
  simt_tile<EPI_STORE, false>(p, t % gx, t / gx, 0, sm, cluster > 1);
}

// ---- large products: 128 x 128 tile, 8 x 8 per thread (two 4 x 4 blocks each way, 64 apart, so that
// a warp's operand reads are whole 16-byte words without bank conflicts), K in steps of 16, two
// stages: the next step's loads fly while this step's 1024 FMAs per thread run, one barrier a step.
// Four 16-byte reads of shared memory feed 64 FMAs, where the 64 x 64 tile needs two for 16. Every
// element is the same chain of FMAs over k as there: the same bits. 8192 x 8192 x 2048: 59 TFLOP/s (the
// library product 68, 64 x 64 tiles 27; 50 with single FMAs); the cross-entropy of 4096 x 32000 x 1024
// 5.1 ms (9.9 with 64 x 64 tiles), its gradients 15.4 (30.0).
constexpr int BT = 128, BTK = 16, BPAD = 4;

// a thread's share of a step's operand tile (128 x 16): two vectors of four, along k (K-major) or
// along the tile (MN-major)
struct BigLoad {
  float4 v[2];
};
__device__ __forceinline__ BigLoad big_load(const float* X, int64_t ld, bool mn, bool vec, int64_t x0,
                                            int64_t X_end, int64_t k0, int64_t K) {
  BigLoad r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = threadIdx.x + i * 256;
    const int64_t x = x0 + (mn ? e % 32 * 4 : e / 4), k = k0 + (mn ? e / 32 : e % 4 * 4);
    const float* p = mn ? X + k * ld + x : X + x * ld + k;
    float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const int64_t left = mn ? (k < K ? X_end - x : 0) : (x < X_end ? K - k : 0);  // of the vector
    if (vec && left >= 4) {
      f = *reinterpret_cast<const float4*>(p);
    } else {
      if (left > 0) f.x = p[0];
      if (left > 1) f.y = p[1];
      if (left > 2) f.z = p[2];
      if (left > 3) f.w = p[3];
    }
    r.v[i] = f;
  }
  return r;
}
__device__ __forceinline__ void big_put(float (*S)[BT + BPAD], bool mn, const BigLoad& r) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = threadIdx.x + i * 256;
    if (mn) {
      *reinterpret_cast<float4*>(&S[e / 32][e % 32 * 4]) = r.v[i];
    } else {
      const int x = e / 4, k = e % 4 * 4;
      S[k][x] = r.v[i].x;
      S[k + 1][x] = r.v[i].y;
      S[k + 2][x] = r.v[i].z;
      S[k + 3][x] = r.v[i].w;
    }
  }
}

template <int EPI>
__global__ void __launch_bounds__(256, 2)
    gemm_simt_big_kernel(const SimtParams p, int tiles_m, int tiles_n, int vec_a, int vec_b) {
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  __shared__ __align__(16) float As[2][BTK][BT + BPAD], Bs[2][BTK][BT + BPAD];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  // eight tiles down, then across: CTAs that run together share operands in L2
  const int per = 8 * tiles_n, grp = blockIdx.x / per, rem = blockIdx.x % per;
  const int down = min(8, tiles_m - grp * 8);
  const int64_t m0 = static_cast<int64_t>(grp * 8 + rem % down) * BT;
  const int64_t n0 = static_cast<int64_t>(rem / down) * BT;
  if constexpr (EPI == EPI_LSE) {
    if (blockIdx.x == 0 && threadIdx.x == 0) *p.ce.counter = 0;
  }
  uint64_t acc2[8][4] = {};  // pairs of columns
  const int64_t steps = (p.K + BTK - 1) / BTK;
  BigLoad la = big_load(p.A[0], p.lda[0], p.a_mn, vec_a, m0, p.M, 0, p.K);
  BigLoad lb = big_load(p.B[0], p.ldb[0], p.b_mn, vec_b, n0, p.N, 0, p.K);
  big_put(As[0], p.a_mn, la);
  big_put(Bs[0], p.b_mn, lb);
  __syncthreads();
  for (int64_t it = 0; it < steps; ++it) {
    const int st = it & 1;
    if (it + 1 < steps) {
      la = big_load(p.A[0], p.lda[0], p.a_mn, vec_a, m0, p.M, (it + 1) * BTK, p.K);
      lb = big_load(p.B[0], p.ldb[0], p.b_mn, vec_b, n0, p.N, (it + 1) * BTK, p.K);
    }
#pragma unroll
    for (int kk = 0; kk < BTK; ++kk) {
      float a[8];
      uint64_t b[4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<float4*>(a + 4 * h) = *reinterpret_cast<const float4*>(&As[st][kk][64 * h + ty * 4]);
        const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(&Bs[st][kk][64 * h + tx * 4]);
        b[2 * h] = q.x;
        b[2 * h + 1] = q.y;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint64_t aa = pair_of(a[i], a[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) acc2[i][j] = fma2(aa, b[j], acc2[i][j]);
      }
    }
    if (it + 1 < steps) {  // the other stage: its reads ended before the last barrier
      big_put(As[st ^ 1], p.a_mn, la);
      big_put(Bs[st ^ 1], p.b_mn, lb);
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = m0 + 64 * (i / 4) + ty * 4 + i % 4;
    float acc[8];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      split_pair(acc2[i][j], acc[2 * j], acc[2 * j + 1]);
    if constexpr (EPI == EPI_LSE) {  // the row's 128 columns lie in 16 lanes of the warp
      const int64_t t = r < p.M ? p.ce.targets[r] : -1;
      float m = -INFINITY;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t c = n0 + 64 * (j / 4) + tx * 4 + j % 4;
        if (c >= p.N) acc[j] = -INFINITY;
        else if (c == t) p.ce.hit[r] = acc[j];
        m = fmaxf(m, acc[j]);
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      float s = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += expf(acc[j] - m);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
      if (tx == 0 && r < p.M) p.ce.part[n0 / BT * p.M + r] = make_float2(m, s);
    } else {
      const int64_t t = EPI == EPI_DCE && r < p.M ? p.ce.targets[r] : -1;
      const float lse = EPI == EPI_DCE && r < p.M ? p.ce.lse[r] : 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int64_t c = n0 + 64 * (j / 4) + tx * 4 + j % 4;
        if (r < p.M && c < p.N) {
          if constexpr (EPI == EPI_DCE) p.out0[r * p.ldo + c] = ce_grad(p, acc[j], t, lse, c);
          else epi1<EPI>(p, 0, r, c, acc[j], 0.0f);
        }
      }
    }
  }
}

// Whether 128 x 128 tiles give every SM one and hold no more than the product (a plain product of one
// segment and one group, or a cross-entropy epilogue)
bool simt_big(const GemmDesc& d) {
  const int64_t tiles = (d.M + BT - 1) / BT * ((d.N + BT - 1) / BT);
  return !d.paired && d.nseg == 1 && d.groups == 1 && d.M >= BT && d.N >= BT &&
         tiles >= device_sm_count() && tiles < 2147483647ll &&
         (d.epi == EPI_STORE || d.epi == EPI_LSE || d.epi == EPI_DCE);
}

// Whether the device can place a cluster of `split` CTAs of this kernel: asked once per
// device and cluster size (cudaOccupancyMaxActiveClusters), before the first launch.
template <auto kKernel>
bool cluster_fits(int split) {
  static std::atomic<int> known[64][4];  // 0 unknown, 1 fits, 2 does not
  const int slot = split == 2 ? 0 : split == 4 ? 1 : split == 8 ? 2 : 3;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = -1;
  if (dev >= 0 && known[dev][slot].load() != 0) return known[dev][slot].load() == 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(split), 1, 1);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  const bool fits = cudaOccupancyMaxActiveClusters(&n, kKernel, &cfg) ==
                        cudaSuccess && n > 0;
  if (!fits) cudaGetLastError();  // the query's own error, not a launch's
  if (dev >= 0) known[dev][slot].store(fits ? 1 : 2);
  return fits;
}

// `grid` without the split, which multiplies its x and is the cluster's size
template <auto kKernel, typename... Args>
cudaError_t launch_split(int split, dim3 grid, cudaStream_t st, const Args&... args) {
  if (split == 1) return launch_kernel(kKernel, grid, 256, 0, st, args...);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(split);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see launch_kernel
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid.x * static_cast<unsigned>(split), grid.y, grid.z);
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kKernel, args...);
}

template <int EPI, bool PAIRED>
cudaError_t launch_k(SimtParams p, dim3 grid, cudaStream_t st) {
  // unsplit: one CTA per tile (also when the device cannot place the cluster)
  if (p.split > 1 && !cluster_fits<gemm_simt_kernel<EPI, PAIRED>>(p.split)) p.split = 1;
  return launch_split<gemm_simt_kernel<EPI, PAIRED>>(p.split, grid, st, p);
}

// split K over a cluster while the tiles (times the split) stay within `most` CTAs (half the SMs) and
// every CTA keeps at least one K step: at these sizes a K step is a global-load latency, so fewer steps
// per CTA is a shorter launch
int simt_split(int64_t tiles, int64_t ksteps, int64_t most) {
  int split = 1;
  while (split < 8 && tiles * split * 2 <= most && ksteps >= 2 * split) split *= 2;
  return split;
}

int64_t simt_ksteps(const GemmDesc& d) { return (d.K + TK - 1) / TK * d.nseg; }

SimtParams simt_params(const GemmDesc& d) {
  SimtParams p{};
  for (int s = 0; s < 3; ++s) {
    const int sa = s < d.nseg ? s : 0;
    const int sb = s < (d.paired ? 2 : d.nseg) ? s : 0;
    p.k0[s] = d.seg_k0[s];
    p.A[s] = static_cast<const float*>(d.A[sa].ptr);
    p.lda[s] = d.A[sa].ld;
    p.B[s] = static_cast<const float*>(d.B[sb].ptr);
    p.ldb[s] = d.B[sb].ld;
  }
  p.M = d.M;
  p.N = d.N;
  p.K = d.K;
  p.a_mn = d.a_mn;
  p.b_mn = d.b_mn;
  p.nseg = d.nseg;
  p.paired = d.paired;
  p.out0 = static_cast<float*>(d.out[0]);
  p.out1 = static_cast<float*>(d.out[1]);
  p.out2 = static_cast<float*>(d.out[2]);
  // out_acc: the output is its own residual (each element is read by the thread that writes it)
  p.in0 = static_cast<const float*>(d.out_acc ? d.out[0] : d.in[0]);
  p.in1 = static_cast<const float*>(d.in[1]);
  p.ldo = d.ldo;
  p.out_group_stride = d.out_group_stride;
  p.ce = d.ce;
  return p;
}

}  // namespace

tp_status launch_gemm_simt(const GemmDesc& d, cudaStream_t st) {
  if (d.M <= 0 || d.N <= 0 || d.K <= 0) return TP_OK;
  if (d.nseg < 1 || d.nseg > 3) return fail(TP_ERR_INVALID_ARG, "1 to 3 K segments");
  SimtParams p = simt_params(d);
  if (simt_big(d)) {
    const int tm = static_cast<int>((d.M + BT - 1) / BT), tn = static_cast<int>((d.N + BT - 1) / BT);
    auto vec = [](const Operand& o) { return reinterpret_cast<uintptr_t>(o.ptr) % 16 == 0 && o.ld % 4 == 0; };
    auto launch = [&](auto kern) {
      p.A[0] += p.k0[0] * (d.a_mn ? p.lda[0] : 1);
      p.B[0] += p.k0[0] * (d.b_mn ? p.ldb[0] : 1);
      return launch_kernel(kern, static_cast<unsigned>(static_cast<int64_t>(tm) * tn), 256, 0, st, p, tm, tn,
                           vec(d.A[0]) && p.k0[0] % 4 == 0 ? 1 : 0, vec(d.B[0]) && p.k0[0] % 4 == 0 ? 1 : 0);
    };
    if (d.epi == EPI_LSE) *d.ce.slots = tn;
    const cudaError_t e = d.epi == EPI_STORE ? launch(gemm_simt_big_kernel<EPI_STORE>)
                          : d.epi == EPI_LSE ? launch(gemm_simt_big_kernel<EPI_LSE>)
                                             : launch(gemm_simt_big_kernel<EPI_DCE>);
    count_launch();
    TP_CUDA_TRY(e);
    return TP_OK;
  }
  const int64_t gx = (d.N + TN - 1) / TN, gy = (d.M + TM - 1) / TM;
  if (gx > 2147483647ll || gy > 65535 || d.groups > 65535)
    return fail(TP_ERR_SHAPE, "fp32 GEMM grid too large");
  dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>(gy), static_cast<unsigned>(d.groups));
  const bool pr = d.paired;
  // (the cross-entropy's products, whose tiles end in exponentials: up to two CTAs per SM)
  const bool ce = d.epi == EPI_LSE || d.epi == EPI_DCE;
  p.split = pr ? 1 : simt_split(gx * gy * d.groups, simt_ksteps(d), ce ? 2 * device_sm_count() : device_sm_count() / 2);
  cudaError_t e = cudaSuccess;
  switch (d.epi) {
    case EPI_STORE: e = launch_k<EPI_STORE, false>(p, grid, st); break;
    case EPI_GELU: e = launch_k<EPI_GELU, false>(p, grid, st); break;
    case EPI_SWIGLU:
      if (!pr) return fail(TP_ERR_INVALID_ARG, "SwiGLU epilogue needs a paired problem");
      e = launch_k<EPI_SWIGLU, true>(p, grid, st);
      break;
    case EPI_DGELU: e = launch_k<EPI_DGELU, false>(p, grid, st); break;
    case EPI_DSWIGLU: e = launch_k<EPI_DSWIGLU, false>(p, grid, st); break;
    case EPI_PAIR:
      if (!pr) return fail(TP_ERR_INVALID_ARG, "pair epilogue needs a paired problem");
      e = launch_k<EPI_PAIR, true>(p, grid, st);
      break;
    case EPI_LSE:
      *d.ce.slots = static_cast<int>(gx);
      e = launch_k<EPI_LSE, false>(p, grid, st);
      break;
    case EPI_DCE: e = launch_k<EPI_DCE, false>(p, grid, st); break;
    default: return fail(TP_ERR_INVALID_ARG, "unknown epilogue");
  }
  count_launch();
  TP_CUDA_TRY(e);
  return TP_OK;
}

tp_status launch_gemm_simt_two(const GemmDesc& a, const GemmDesc& b, cudaStream_t st) {
  const GemmDesc* d[2] = {&a, &b};
  int64_t gx[2], tiles[2], steps[2], split[2] = {1, 1};
  bool here[2];
  for (int i = 0; i < 2; ++i) {
    here[i] = !simt_big(*d[i]);
    if (!here[i] && d[i]->out[0]) TP_TRY(launch_gemm_simt(*d[i], st));
    gx[i] = (d[i]->N + TN - 1) / TN;
    tiles[i] = here[i] ? gx[i] * ((d[i]->M + TM - 1) / TM) : 0;
    steps[i] = here[i] ? simt_ksteps(*d[i]) : 0;
    here[i] = here[i] && d[i]->out[0];
  }
  if (!here[0] && !here[1]) return TP_OK;
  // the longer sum per CTA is halved while it has two steps (one takes a CTA 2 us) and four CTAs of an
  // SM hold them all
  while (true) {
    int i = -1;
    for (int j = 0; j < 2; ++j)
      if (split[j] < 8 && steps[j] >= 2 * split[j] &&
          tiles[0] * split[0] + tiles[1] * split[1] + tiles[j] * split[j] <= 4 * device_sm_count() &&
          (i < 0 || steps[j] * split[i] > steps[i] * split[j]))
        i = j;
    if (i < 0) break;
    split[i] *= 2;
  }
  int64_t cluster = std::max(split[0], split[1]);
  if (cluster > 1 && !cluster_fits<gemm_simt_two_kernel>(static_cast<int>(cluster)))
    cluster = split[0] = split[1] = 1;
  SimtParams p[2];
  int64_t clusters[2];
  for (int i = 0; i < 2; ++i) {
    p[i] = simt_params(*d[i]);
    p[i].split = static_cast<int>(split[i]);
    clusters[i] = here[i] ? (tiles[i] * split[i] + cluster - 1) / cluster : 0;
  }
  if ((clusters[0] + clusters[1]) * cluster > 2147483647ll)
    return fail(TP_ERR_SHAPE, "fp32 GEMM grid too large");
  const cudaError_t e = launch_split<gemm_simt_two_kernel>(
      static_cast<int>(cluster), static_cast<unsigned>(clusters[0] + clusters[1]), st, p[0], p[1],
      static_cast<int>(clusters[0] * cluster), static_cast<int>(gx[0]), static_cast<int>(gx[1]),
      static_cast<int>(cluster));
  count_launch();
  TP_CUDA_TRY(e);
  return TP_OK;
}

}  // namespace tp
