// The output layer and its cross-entropy without the logits, l = x E^T (M, v) with x (M, h) and
// the shared embedding E (v, h) [张量并行 notes, §损失计算层的并行化; the tied output layer of the
// Megatron-LM 实战 04 listing, 核心实现, SmallGPT]:
//   lse_r = log sum_c exp(l_rc),  loss_r = lse_r - l_{r, t_r}
//   q_rc = exp(l_rc - lse_r) - [c = t_r],  dx = scale q E,  dE = scale q^T x
// Forward: one product whose epilogue (EPI_LSE of the GEMM engines) keeps, per row and column
// tile, the largest logit and the sum of exponentials, and the target's logit; the tiles of all
// vocabulary shards are then joined as the pages' two all-reduces join the shards. A logit lives in
// the accumulator only.
// Backward: the vocabulary goes by in pieces. Of each piece the logits are formed again and leave
// the accumulator as q (EPI_DCE, in the element type: the operand of the next two products), which
// gives the piece's rows of dE and its share of dx. One piece's q is all that is kept. In bf16 q is
// rounded without the scale, which the products' sums get in 32 bits: rounded with it, a scale that
// is no power of two shifts every target's term alike (1/1003 by 2.4e-3; dx of 1003 rows was 2.9e-3 off
// in the 2-norm, and is 1.9e-3 this way, a rounded perfect result 1.7e-3).
// The products bound both: 2 M v h operations forward, 6 backward. bf16, 8192 rows, v = 50304: h = 2048
// 0.96 ms (1756 TFLOP/s, the rate that a library product sustains under the power cap) and 3.1 ms (1630),
// h = 4096 backward 5.98 ms (1694). The exponentials hide: 6 % of their pipe, 17 % of the issue slots,
// an epilogue of 3.5 k cycles in a tile's 17 k at h = 1032. For few rows HBM does: 37 rows of h = 4096
// read E at 6 TB/s (74 us with the join).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"

namespace tp {
namespace {

constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
constexpr int64_t kSms = 152;
constexpr int kSumShards = 32;    // most shards whose losses the join adds up itself
constexpr float kLog2e = 1.4426950408889634f;  // log2(e)

// (m, s) pairs: s exp(m) summed
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float mm = fmaxf(m, m2);
  // an empty side (-inf, 0) adds nothing; NaN in either sum stays
  s = (m == mm ? s : s * exp2f((m - mm) * kLog2e)) + (m2 == mm ? s2 : s2 * exp2f((m2 - mm) * kLog2e));
  m = mm;
}

// A CTA joins ROWS rows: its threads, consecutive ones on consecutive rows, share the slots, shuffles
// join a warp's, and a thread per row the warps'. The CTA that ends last adds the CTAs' losses up (in an
// order of their own, whichever CTA that is): a launch less than a kernel of its own. early: launched
// ahead of its predecessor's end, and the next kernel ahead of its own (may_go_early).
template <int ROWS>
__global__ void __launch_bounds__(kJoinThreads) vocab_linear_join_kernel(
    const float2* __restrict__ part, const float* __restrict__ hit,
    const int32_t* __restrict__ targets, float* __restrict__ lse, float* __restrict__ row_loss,
    float* __restrict__ shard_loss, float* __restrict__ loss, float* cta_loss, int32_t* counter,
    int slots, int64_t M, int64_t v, int N, int early) {
  pdl_wait();  // the previous kernel's results are complete and visible
  if (early) pdl_trigger();
  // pairs that are left of a row: one of each warp, or of each thread where a warp has 32 rows
  constexpr int kPairs = ROWS <= 32 ? kJoinWarps : kJoinThreads / ROWS;
  __shared__ float2 sm[kPairs][ROWS];
  __shared__ float losses[ROWS];
  __shared__ int shard[ROWS];
  __shared__ float sum[kSumShards];
  __shared__ int last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t own = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x;  // the row that it ends
  const bool ends = threadIdx.x < ROWS && own < M;
  int64_t t = ends ? targets[own] : -1;
  if (t >= v) t = -1;
  const float at = t >= 0 ? hit[own] : 0.0f;
  float m = -INFINITY, s = 0.0f;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x % ROWS;
  if (row < M) {
#pragma unroll 8
    for (int i = threadIdx.x / ROWS; i < slots; i += kJoinThreads / ROWS) {
      const float2 p = part[i * M + row];
      join(m, s, p.x, p.y);
    }
  }
#pragma unroll
  for (int o = ROWS; o < 32; o *= 2)
    join(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o));
  if (ROWS > 32 || lane < ROWS)
    sm[ROWS <= 32 ? warp : threadIdx.x / ROWS][threadIdx.x % ROWS] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x < ROWS) {
    float2 p[kPairs];
#pragma unroll
    for (int w = 0; w < kPairs; ++w) p[w] = sm[w][threadIdx.x];
    m = p[0].x;
#pragma unroll
    for (int w = 1; w < kPairs; ++w) m = fmaxf(m, p[w].x);
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kPairs; ++w) s += p[w].y * exp2f((p[w].x - m) * kLog2e);
    // m is a logit and s >= 1: the loss does not go by way of lse, whose rounding is the logits' size,
    // and is never below 0
    const float log_s = logf(s);
    const float l = t >= 0 ? (m - at) + log_s : 0.0f;
    if (ends) {
      lse[own] = m + log_s;
      row_loss[own] = l;
    }
    losses[threadIdx.x] = l;
    shard[threadIdx.x] = t >= 0 ? static_cast<int>(t / (v / N)) : -1;
  }
  if (N > kSumShards) return;
  __syncthreads();
  for (int i = warp; i < N; i += kJoinWarps) {
    float a = 0.0f;
#pragma unroll
    for (int r = 0; r < ROWS; r += 32)
      if (lane + r < ROWS) a += shard[lane + r] == i ? losses[lane + r] : 0.0f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    if (lane == 0) {
      sum[i] = a;
      if (gridDim.x > 1) {
        cta_loss[static_cast<int64_t>(blockIdx.x) * N + i] = a;
        __threadfence();
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    last = gridDim.x == 1 || atomicAdd(counter, 1) == static_cast<int>(gridDim.x) - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  if (gridDim.x > 1)
    for (int i = warp; i < N; i += kJoinWarps) {
      float a = 0.0f;
#pragma unroll 8
      for (int64_t c = lane; c < gridDim.x; c += 32) a += __ldcg(cta_loss + c * N + i);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
      if (lane == 0) sum[i] = a;
    }
  __syncthreads();
  if (threadIdx.x == 0) {
    float total = 0.0f;
    for (int i = 0; i < N; ++i) {
      if (shard_loss) shard_loss[i] = sum[i];
      total += sum[i];
    }
    loss[0] = total / static_cast<float>(M);
  }
}

// ---- dE = q^T x of up to 64 rows (bf16): next to no arithmetic, every byte of dE written. A CTA keeps
// 256 columns of x in shared memory and walks over 64-entry pieces of the vocabulary, q's next piece
// loading while one is worked on; a warp takes 16 entries x 128 columns by mma.m16n8k16 (the tcgen05
// engine's tiles of a single K block are bound by their hand-over), and the lanes of a quad exchange
// their pairs, so that each stores 16 bytes. The whole backward, engine -> this: 50304 x 2048, 1 row 150
// -> 123 us, 16 rows 149 -> 125, 64 rows 156 -> 152; 50257 x 4096, 37 rows 268 -> 243; 128000 x 4096, 64
// rows 647 -> 621. It is a launch more, in plain stream order: 30000 x 1024, 64 rows 61 -> 59, but 8000 x
// 512, 64 rows 24.5 -> 24.8 and 1000 x 256, 16 rows 17.1 -> 18.6, so it takes dE from 2^24 elements.
constexpr int kOuterRows = 64;     // most rows of x
constexpr int64_t kOuterLeast = 1ll << 24;  // least elements of dE
constexpr int kOuterCols = 256;    // columns of a CTA
constexpr int kOuterEntries = 64;  // vocabulary entries of a step
constexpr int kXPitch = kOuterCols + 8, kQPitch = kOuterEntries + 8;  // no bank conflicts of ldmatrix
constexpr int kOuterSmem = (kOuterRows * kXPitch + 2 * kOuterRows * kQPitch) * 2;

// p[j] of lane t of a quad becomes p[t] of its lane j
__device__ __forceinline__ void transpose_quad(uint32_t (&p)[4], int t) {
#pragma unroll
  for (int s = 1; s <= 2; s *= 2) {
    const bool up = (t & s) != 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (j & s) continue;
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, up ? p[j] : p[j + s], s);
      if (up) p[j] = got;
      else p[j + s] = got;
    }
  }
}

// blockIdx: column block fastest; q (M, n) with pitch ldq, x (M, h), dE (n, h); h % 8 == 0, ldq % 64 == 0
__global__ void __launch_bounds__(256, 2)
    vocab_outer_kernel(const __nv_bfloat16* __restrict__ q, const __nv_bfloat16* __restrict__ x,
                       __nv_bfloat16* __restrict__ dE, int M, int64_t n, int64_t h, int64_t ldq,
                       int col_blocks, float scale) {
  extern __shared__ __align__(16) uint8_t outer_smem[];
  __nv_bfloat16* xs = reinterpret_cast<__nv_bfloat16*>(outer_smem);
  __nv_bfloat16* qs = xs + kOuterRows * kXPitch;  // two stages
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t j0 = static_cast<int64_t>(blockIdx.x % col_blocks) * kOuterCols;
  const int64_t steps = (n + kOuterEntries - 1) / kOuterEntries;
  const int64_t stride = gridDim.x / col_blocks;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int i = threadIdx.x; i < kOuterRows * (kOuterCols / 8); i += 256) {
    const int r = i / (kOuterCols / 8), c = i % (kOuterCols / 8) * 8;
    *reinterpret_cast<uint4*>(xs + r * kXPitch + c) =
        r < M && j0 + c < h ? *reinterpret_cast<const uint4*>(x + r * h + j0 + c) : zero;
  }
  // q's piece `step`: 64 rows x 8 vectors, two of them a thread's (entries past n, which no row of dE
  // takes, are whatever the pitch leaves there)
  auto load = [&](int64_t step, uint4 (&v)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = threadIdx.x + 256 * i, r = e / 8;
      v[i] = r < M ? *reinterpret_cast<const uint4*>(q + r * ldq + step * kOuterEntries + e % 8 * 8) : zero;
    }
  };
  auto put = [&](int st, const uint4 (&v)[2]) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int e = threadIdx.x + 256 * i;
      *reinterpret_cast<uint4*>(qs + (st * kOuterRows + e / 8) * kQPitch + e % 8 * 8) = v[i];
    }
  };
  const int64_t first = blockIdx.x / col_blocks;
  uint4 next[2];
  if (first < steps) {
    load(first, next);
    put(0, next);
  }
  __syncthreads();
  const uint64_t by = pair_of(scale, scale);
  const int ksteps = (M + 15) / 16, c0 = warp / 2 * 16, w0 = warp % 2 * 128;
  const uint32_t xa = smem_u32(xs), qa = smem_u32(qs);
  int st = 0;
  for (int64_t step = first; step < steps; step += stride, st ^= 1) {
    const bool more = step + stride < steps;
    if (more) load(step + stride, next);
    float acc[16][4] = {};
    for (int k = 0; k < ksteps; ++k) {
      uint32_t a[4];  // 16 entries x 16 rows of q^T
      ldmatrix_x4_trans(a, qa + ((st * kOuterRows + k * 16 + lane / 16 * 8 + lane % 8) * kQPitch + c0 +
                                 lane / 8 % 2 * 8) * 2);
#pragma unroll
      for (int j = 0; j < 16; j += 2) {
        uint32_t b[4];  // 16 rows x two tiles of 8 columns of x
        ldmatrix_x4_trans(b, xa + ((k * 16 + lane / 8 % 2 * 8 + lane % 8) * kXPitch + w0 + j * 8 +
                                   lane / 16 * 8) * 2);
        mma_16n8k16(acc[j], a, b[0], b[1]);
        mma_16n8k16(acc[j + 1], a, b[2], b[3]);
      }
    }
    const int t = lane % 4;
    const int64_t c = step * kOuterEntries + c0 + lane / 4;
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      const int64_t col = j0 + w0 + (j + t) * 8;  // the tile that this lane stores of the four
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo, hi;
          split_pair(mul2(pair_of(acc[j + i][2 * hf], acc[j + i][2 * hf + 1]), by), lo, hi);
          p[i] = pack_bf16x2(lo, hi);
        }
        transpose_quad(p, t);
        if (c + 8 * hf < n && col < h)
          *reinterpret_cast<uint4*>(dE + (c + 8 * hf) * h + col) = make_uint4(p[0], p[1], p[2], p[3]);
      }
    }
    if (more) put(st ^ 1, next);  // the other stage, whose reads ended before the last barrier
    __syncthreads();
  }
}

size_t a256(size_t x) { return align_up(x, 256); }

// ---- forward: partials of every row (a slot for 64 columns at the least), the targets' logits,
// the CTAs' losses, the counter of the CTAs that have ended
struct FwdLayout {
  size_t part, hit, cta, counter, total;
};
// Rows of a CTA of the join where they have many slots. Two with up to a CTA per SM, eight while 32
// threads of a row count (1300 x 50304 x 64 51 us, 59 with 32 rows; 4864 rows 125 and 134), 32 beyond,
// where the sums of the CTAs' losses do (8192 rows x 5000 33.0 us, 34.8 with eight; 60000 x 3000 107 and
// 127).
int join_rows(int64_t M) { return M <= 2 * kSms ? 2 : M <= 32 * kSms ? 8 : 32; }
int64_t join_ctas(int64_t M) { return (M + join_rows(M) - 1) / join_rows(M); }
FwdLayout fwd_layout(int64_t M, int64_t v) {
  FwdLayout L{};
  size_t o = 0;
  L.part = o;    o += a256(static_cast<size_t>((v + 63) / 64) * M * sizeof(float2));
  L.hit = o;     o += a256(M * sizeof(float));
  // join_ctas or more, and never less for more rows
  const int64_t ctas = std::max({kSms, join_ctas(std::min(M, 32 * kSms)), (M + 31) / 32});
  L.cta = o;     o += a256(ctas * kSumShards * sizeof(float));
  L.counter = o; o += 256;
  L.total = o;
  return L;
}

// ---- backward: q of one piece, and (bf16) the fp32 sums of dx where one product does not make it
// Fewer pieces are faster (8192 x 50304 x 2048: 4 of 256 MiB 3.03 ms, 2 of 512 2.92, one of 1 GiB
// 2.76), but keep more of q: half of it here.
constexpr int64_t kPieceBytes = 512ll << 20;
struct BwdPlan {
  int64_t piece;  // vocabulary entries of a piece, whole 256-column tiles; also q's pitch
  int pieces;
  int x_parts, e_parts;  // parts of the sums of dx (over a piece) and of dE (over the rows)
  bool x_direct;         // dx leaves one product
  size_t q, dx, dE, total;
};
// Parts of the sum over K of a product with (rows, cols) outputs, where its tiles alone would leave
// SMs idle: the number that takes the least time by whole waves of the tiles (256 x 512 or 256 x 256
// on an SM pair, as the engine takes them, else about 128 x 128 on an SM) and by the fp32 partials,
// written, read and added up by a launch more. No part of fewer than 256 products, none that holds
// nothing, no more than 512 MiB of partials; `partials`: one part is a partial too. (dx of 8192 x 4096,
// tiles of 3.4 waves, in two parts: 5.55 ms with the other products, 5.75 in one.)
int64_t part_length(int64_t K, int64_t parts) {  // whole K blocks, where there is more than one part
  return parts == 1 ? K : ((K + parts - 1) / parts + 63) / 64 * 64;
}
int sum_parts(int64_t rows, int64_t cols, int64_t K, bool partials) {
  const bool pair = rows >= 256 && cols >= 256;
  const int64_t tw = pair ? 256 : 128, at_once = pair ? kSms / 2 : kSms;
  const int64_t down = (rows + tw - 1) / tw, tiles = down * ((cols + tw - 1) / tw);
  auto waves = [&](int64_t n) { return (n + at_once - 1) / at_once; };
  int best = 1;
  double least = 0.0;
  for (int g = 1; g <= 32; ++g) {
    if (g > 1 && (K / g < 256 || g * rows * cols * 4 > (512ll << 20))) break;
    const int64_t k = part_length(K, g);
    if ((g - 1) * k >= K) continue;  // the last part would hold nothing
    double w = static_cast<double>(waves(tiles * g));
    if (pair && cols % 512 == 0 && k >= 4096) {
      const int64_t wide = down * (cols / 512) * g;  // a tile of two, at 10 % more of its work
      if (wide >= 4 * at_once || 18 * waves(wide) < 10 * waves(tiles * g))
        w = 1.8 * static_cast<double>(waves(wide));
    }
    // seconds: a wave's products at 1.7e15 / (152 SMs), the partials at 5e12 bytes, their launch
    const double t = w * (2.0 * tw * tw * k) * at_once / 1.7e15 +
                     (g > 1 || partials ? g * rows * cols * 8.0 / 5e12 + 3e-6 : 0.0);
    if (g == 1 || t < least) {
      best = g;
      least = t;
    }
  }
  return best;
}
BwdPlan bwd_plan(int64_t M, int64_t v, int64_t h, tp_dtype dt) {
  BwdPlan P{};
  const int64_t e = static_cast<int64_t>(elem_size(dt));
  const int64_t most = std::max<int64_t>(kPieceBytes / (std::max<int64_t>(M, 1) * e) / 256 * 256, 256);
  const int64_t n = (v + most - 1) / most;
  P.piece = ((v + n - 1) / n + 255) / 256 * 256;
  P.pieces = static_cast<int>((v + P.piece - 1) / P.piece);
  P.x_parts = dt == TP_BF16 ? sum_parts(M, h, std::min(P.piece, v), P.pieces > 1) : 1;
  P.e_parts = dt == TP_BF16 ? sum_parts(std::min(P.piece, v), h, M, false) : 1;
  P.x_direct = dt != TP_BF16 || (P.pieces == 1 && P.x_parts == 1);
  P.q = a256(M * P.piece * e);
  P.dx = P.x_direct ? 0 : a256(static_cast<size_t>(P.x_parts) * M * h * sizeof(float));
  P.dE = P.e_parts == 1 ? 0 : a256(static_cast<size_t>(P.e_parts) * P.piece * h * sizeof(float));
  P.total = P.q + P.dx + P.dE;
  return P;
}

// a product's sum over K in `parts` parts (1: as it is), each a partial of its own at out
void split_sum(GemmDesc& d, int parts) {
  if (parts == 1) return;
  d.K = part_length(d.K, parts);
  d.groups = parts;
  d.out_group_stride = d.M * d.N;
}

tp_status launch_outer(const void* q, const void* x, void* dE, int64_t M, int64_t n, int64_t h,
                       int64_t ldq, float scale, cudaStream_t st) {
  static std::atomic<uint64_t> attr_set{0};
  if (needs_setup(attr_set)) {
    TP_CUDA_TRY(cudaFuncSetAttribute(vocab_outer_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     kOuterSmem));
    mark_device(attr_set);
  }
  const int64_t blocks = (h + kOuterCols - 1) / kOuterCols, steps = (n + kOuterEntries - 1) / kOuterEntries;
  const int64_t walkers = std::min(steps, std::max<int64_t>(2 * kSms / blocks, 1));  // of a column block
  // plain stream order: two CTAs fill an SM's registers, which leaves no room beside a GEMM's
  vocab_outer_kernel<<<static_cast<unsigned>(blocks * walkers), 256, kOuterSmem, st>>>(
      static_cast<const __nv_bfloat16*>(q), static_cast<const __nv_bfloat16*>(x),
      static_cast<__nv_bfloat16*>(dE), static_cast<int>(M), n, h, ldq, static_cast<int>(blocks),
      scale);
  TP_CUDA_TRY(cudaGetLastError());
  count_launch();
  return TP_OK;
}

tp_status product(const GemmDesc& d, cudaStream_t st) {
  return d.dtype == TP_BF16 ? launch_gemm_tc(d, st) : launch_gemm_simt(d, st);
}

}  // namespace

size_t vocab_linear_ce_ws_bytes(bool fwd, int64_t M, int64_t v, int64_t h, tp_dtype dt) {
  return fwd ? fwd_layout(M, v).total : bwd_plan(M, v, h, dt).total;
}

tp_status launch_vocab_linear_ce_fwd(const void* x, const void* E, const int32_t* targets,
                                     float* lse, float* row_loss, float* shard_loss, float* loss,
                                     int64_t M, int64_t v, int64_t h, int N, tp_dtype dt, void* ws,
                                     cudaStream_t st) {
  const FwdLayout L = fwd_layout(M, v);
  char* base = static_cast<char*>(ws);
  float* hit = reinterpret_cast<float*>(base + L.hit);
  int32_t* counter = reinterpret_cast<int32_t*>(base + L.counter);
  int slots = 0;
  GemmDesc d;
  d.dtype = dt;
  d.M = M;
  d.N = v;
  d.K = h;
  d.A[0] = {x, M, h, h};
  d.B[0] = {E, v, h, h};  // E (v, h) read as B(k = h, n = v): K-major
  d.epi = EPI_LSE;
  d.ce.targets = targets;
  d.ce.vocab = v;
  d.ce.part = reinterpret_cast<float2*>(base + L.part);
  d.ce.hit = hit;
  d.ce.counter = counter;
  d.ce.slots = &slots;
  TP_TRY(product(d, st));
  // 128 rows of few slots: one CTA, which has no other to wait for
  const bool one = M <= 128 && slots <= 32;
  const unsigned grid = one ? 1u : static_cast<unsigned>(join_ctas(M));
  const bool early = may_go_early(grid, kJoinThreads, device_sm_count());
  auto join = [&](auto kern) {
    return launch_kernel_if(early, kern, grid, kJoinThreads, 0, st, d.ce.part, hit, targets, lse, row_loss,
                            shard_loss, loss, reinterpret_cast<float*>(base + L.cta), counter, slots, M,
                            v, N, early ? 1 : 0);
  };
  TP_CUDA_TRY(one                 ? join(vocab_linear_join_kernel<128>)
              : join_rows(M) == 2 ? join(vocab_linear_join_kernel<2>)
              : join_rows(M) == 8 ? join(vocab_linear_join_kernel<8>)
                                  : join(vocab_linear_join_kernel<32>));
  count_launch();
  return N > kSumShards ? launch_vocab_ce_loss(row_loss, targets, shard_loss, loss, M, v, N, st)
                        : TP_OK;
}

tp_status launch_vocab_linear_ce_bwd(const void* x, const void* E, const int32_t* targets,
                                     const float* lse, void* dx, void* dE, int64_t M, int64_t v,
                                     int64_t h, float scale, tp_dtype dt, void* ws,
                                     cudaStream_t st) {
  const BwdPlan P = bwd_plan(M, v, h, dt);
  const int64_t e = static_cast<int64_t>(elem_size(dt));
  void* q = ws;
  float* xs = reinterpret_cast<float*>(static_cast<char*>(ws) + P.q);
  float* es = reinterpret_cast<float*>(static_cast<char*>(ws) + P.q + P.dx);
  for (int i = 0; i < P.pieces; ++i) {
    const int64_t c0 = i * P.piece, n = std::min(P.piece, v - c0);
    const char* Ei = static_cast<const char*>(E) + c0 * h * e;
    {  // q
      GemmDesc d;
      d.dtype = dt;
      d.M = M;
      // whole 8-column stores in bf16: columns past n (rows past E's end read as zeros) are not used
      d.N = dt == TP_BF16 ? (n + 7) / 8 * 8 : n;
      d.K = h;
      d.A[0] = {x, M, h, h};
      d.B[0] = {Ei, n, h, h};
      d.ldo = P.piece;
      d.epi = EPI_DCE;
      d.out[0] = q;
      d.ce.targets = targets;
      d.ce.vocab = v;
      d.ce.col0 = c0;
      d.ce.lse = lse;
      d.ce.scale = scale;
      TP_TRY(product(d, st));
    }
    GemmDesc gx, ge;
    // dx (+)= q E
    gx.dtype = dt;
    gx.M = M;
    gx.N = h;
    gx.K = n;
    gx.A[0] = {q, M, n, P.piece};
    gx.B[0] = {Ei, n, h, h};
    gx.b_mn = true;
    gx.ldo = h;
    gx.epi = dt == TP_BF16 ? EPI_SCALE : EPI_STORE;
    gx.ce.scale = scale;
    gx.out[0] = P.x_direct || !dx ? dx : xs;
    gx.out_f32 = dt == TP_F32 || !P.x_direct;
    gx.out_acc = i > 0;
    split_sum(gx, P.x_parts);
    // dE = q^T x, the piece's rows
    char* dEi = dE ? static_cast<char*>(dE) + c0 * h * e : nullptr;
    ge.dtype = dt;
    ge.M = n;
    ge.N = h;
    ge.K = M;
    ge.A[0] = {q, M, n, P.piece};  // q (M, n) read as A(m = n, k = M): MN-major
    ge.a_mn = true;
    ge.B[0] = {x, M, h, h};
    ge.b_mn = true;
    ge.ldo = h;
    ge.epi = gx.epi;
    ge.ce.scale = scale;
    ge.out[0] = P.e_parts > 1 && dE ? static_cast<void*>(es) : dEi;
    ge.out_f32 = dt == TP_F32 || P.e_parts > 1;
    split_sum(ge, P.e_parts);
    if (dt == TP_F32) {
      TP_TRY(launch_gemm_simt_two(gx, ge, st));
      continue;
    }
    if (M <= kOuterRows && n * h >= kOuterLeast) {
      if (dx) TP_TRY(launch_gemm_tc(gx, st));
      if (dE) TP_TRY(launch_outer(q, x, dEi, M, n, h, P.piece, scale, st));
      continue;
    }
    if (dx && dE) TP_TRY(launch_gemm_tc_two(gx, ge, st));
    else TP_TRY(launch_gemm_tc(dx ? gx : ge, st));
    if (dE && P.e_parts > 1) TP_TRY(launch_shard_reduce(es, nullptr, dEi, P.e_parts, n, h, dt, st));
  }
  if (dx && !P.x_direct) return launch_shard_reduce(xs, nullptr, dx, P.x_parts, M, h, dt, st);
  return TP_OK;
}

}  // namespace tp
