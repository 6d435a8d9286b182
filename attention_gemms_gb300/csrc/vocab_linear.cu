// The output layer and its cross-entropy without the logits, l = x E^T (M, v) with x (M, h) and
// the shared embedding E (v, h) [张量并行 notes, §损失计算层的并行化; the tied output layer of the
// Megatron-LM 实战 04 listing, 核心实现, SmallGPT]:
//   lse_r = log sum_c exp(l_rc),  loss_r = lse_r - l_{r, t_r}
//   q_rc = scale (exp(l_rc - lse_r) - [c = t_r]),  dx = q E,  dE = q^T x
// Forward: one product whose epilogue (EPI_LSE of the GEMM engines) keeps, per row and column
// tile, the largest logit and the sum of exponentials, and the target's logit; the tiles of all
// vocabulary shards are then joined as the pages' two all-reduces join the shards. A logit lives in
// the accumulator only.
// Backward: the vocabulary goes by in pieces. Of each piece the logits are formed again and leave
// the accumulator as q (EPI_DCE, in the element type: the operand of the next two products), which
// gives the piece's rows of dE and its share of dx. One piece's q is all that is kept.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"

namespace tp {
namespace {

constexpr int kRows = 8;          // rows of a CTA of the join at the least
constexpr int kJoinThreads = 1024;
constexpr int64_t kSms = 152;
constexpr int kSumShards = 8;     // shards whose losses the join adds up itself
constexpr float kLn2 = 0.6931471805599453f;

// (m, s) pairs, m in base 2: s 2^m summed
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float mm = fmaxf(m, m2);
  // an empty side (-inf, 0) adds nothing; NaN in either sum stays
  s = (m == mm ? s : s * exp2f(m - mm)) + (m2 == mm ? s2 : s2 * exp2f(m2 - mm));
  m = mm;
}

// A CTA joins ROWS rows: its 1024 threads, consecutive ones on consecutive rows, share the slots,
// warps join by shuffles and warp 0 joins the warps in order. The CTA that ends last adds the losses
// up (in the order of the CTAs' rows, so the sum does not depend on which one that is): a launch
// less than a kernel of its own. 32 rows where that gives every SM a CTA (8192 rows x 197 slots: 8
// us, 11 with 8 rows), else 8 (37 rows x 393 slots: 5 us against 8).
template <int ROWS>
__global__ void __launch_bounds__(kJoinThreads) vocab_linear_join_kernel(
    const float2* __restrict__ part, const float* __restrict__ hit,
    const int32_t* __restrict__ targets, float* __restrict__ lse, float* __restrict__ row_loss,
    float* __restrict__ shard_loss, float* __restrict__ loss, float* cta_loss, int32_t* counter,
    int slots, int64_t M, int64_t v, int N) {
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  __shared__ float2 sm[32][32];
  __shared__ int last;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mine = lane % ROWS;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + mine;
  float m = -INFINITY, s = 0.0f;
  if (row < M) {
#pragma unroll 4
    for (int i = threadIdx.x / ROWS; i < slots; i += kJoinThreads / ROWS) {
      const float2 p = part[i * M + row];
      join(m, s, p.x, p.y);
    }
  }
#pragma unroll
  for (int o = ROWS; o < 32; o *= 2)
    join(m, s, __shfl_xor_sync(0xFFFFFFFFu, m, o), __shfl_xor_sync(0xFFFFFFFFu, s, o));
  sm[warp][lane] = make_float2(m, s);
  __syncthreads();
  if (warp == 0) {
    for (int w = 1; w < 32; ++w) join(m, s, sm[w][lane].x, sm[w][lane].y);
    float l = 0.0f;
    int64_t t = -1;
    if (row < M && lane < ROWS) {
      const float z = (m + log2f(s)) * kLn2;
      t = targets[row];
      if (t >= 0 && t < v) l = z - hit[row];
      else t = -1;
      lse[row] = z;
      row_loss[row] = l;
    }
    if (N <= kSumShards) {
      const int64_t vs = v / N;
      for (int i = 0; i < N; ++i) {
        float a = t >= i * vs && t < (i + 1) * vs ? l : 0.0f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
        if (lane == 0) cta_loss[static_cast<int64_t>(blockIdx.x) * N + i] = a;
      }
      if (lane == 0) {
        __threadfence();
        last = atomicAdd(counter, 1) == static_cast<int>(gridDim.x) - 1;
      }
    }
  }
  if (N > kSumShards) return;
  __syncthreads();
  if (!last) return;
  __threadfence();
  float* red = reinterpret_cast<float*>(sm);  // [N][32 warps]
  for (int i = 0; i < N; ++i) {
    float a = 0.0f;
    for (int64_t c = threadIdx.x; c < gridDim.x; c += kJoinThreads) a += __ldcg(cta_loss + c * N + i);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
    if (lane == 0) red[i * 32 + warp] = a;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    float total = 0.0f;
    for (int i = 0; i < N; ++i) {
      float a = 0.0f;
      for (int w = 0; w < 32; ++w) a += red[i * 32 + w];
      if (shard_loss) shard_loss[i] = a;
      total += a;
    }
    loss[0] = total / static_cast<float>(M);
  }
}

size_t a256(size_t x) { return align_up(x, 256); }

// ---- forward: partials of every row (a slot for 64 columns at the least), the targets' logits,
// the CTAs' losses, the counter of the CTAs that have ended
struct FwdLayout {
  size_t part, hit, cta, counter, total;
};
FwdLayout fwd_layout(int64_t M, int64_t v) {
  FwdLayout L{};
  size_t o = 0;
  L.part = o;    o += a256(static_cast<size_t>((v + 63) / 64) * M * sizeof(float2));
  L.hit = o;     o += a256(M * sizeof(float));
  L.cta = o;     o += a256((M + kRows - 1) / kRows * kSumShards * sizeof(float));
  L.counter = o; o += 256;
  L.total = o;
  return L;
}

// ---- backward: q of one piece, and (bf16) the fp32 sums of dx where one product does not make it
constexpr int64_t kPieceBytes = 512ll << 20;
struct BwdPlan {
  int64_t piece;  // vocabulary entries of a piece, whole 256-column tiles; also q's pitch
  int pieces;
  int groups;     // parts of dx's sum over a piece, each a partial of its own
  bool direct;    // dx leaves one product: no partials
  size_t q, dx, total;
};
// Parts of dx's sum over a piece, where its tiles alone would leave SMs idle: the number that
// takes the least time, whole waves of the tiles (256 x 256 on an SM pair, 128 x 128 on an SM where
// there are fewer than 256 rows) against the fp32 partials written and read.
int dx_groups(int64_t M, int64_t h, int64_t piece) {
  const int64_t tw = M >= 256 ? 256 : 128, at_once = M >= 256 ? kSms / 2 : kSms;
  const int64_t tiles = (M + tw - 1) / tw * ((h + tw - 1) / tw);
  if (tiles >= 2 * at_once) return 1;
  int best = 1;
  double least = 0.0;
  for (int g = 1; g <= 32 && (g == 1 || piece / g >= 512); ++g) {
    const double waves = static_cast<double>((tiles * g + at_once - 1) / at_once);
    // seconds: a wave's products at 1.7e15 / (152 SMs), the partials at 5e12 bytes
    const double t = waves * (2.0 * tw * tw * (piece / g)) * at_once / 1.7e15 +
                     (g > 1 ? g * M * h * 8.0 / 5e12 : 0.0);
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
  P.groups = dt == TP_BF16 ? dx_groups(M, h, P.piece) : 1;
  P.direct = dt != TP_BF16 || (P.pieces == 1 && P.groups == 1);
  P.q = a256(M * P.piece * e);
  P.dx = P.direct ? 0 : a256(static_cast<size_t>(P.groups) * M * h * sizeof(float));
  P.total = P.q + P.dx;
  return P;
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
  const int rows = M >= 32 * kSms ? 32 : kRows;
  TP_CUDA_TRY(launch_kernel(rows == 32 ? vocab_linear_join_kernel<32> : vocab_linear_join_kernel<kRows>,
                            static_cast<unsigned>((M + rows - 1) / rows), kJoinThreads, 0, st,
                            d.ce.part, hit, targets, lse, row_loss, shard_loss, loss,
                            reinterpret_cast<float*>(base + L.cta), counter, slots, M, v, N));
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
  float* sums = reinterpret_cast<float*>(static_cast<char*>(ws) + P.q);
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
    if (dx) {  // dx (+)= q E
      GemmDesc d;
      d.dtype = dt;
      d.M = M;
      d.N = h;
      d.K = P.groups > 1 ? ((n + P.groups - 1) / P.groups + 63) / 64 * 64 : n;
      d.groups = P.groups;
      d.A[0] = {q, M, n, P.piece};
      d.B[0] = {Ei, n, h, h};
      d.b_mn = true;
      d.ldo = h;
      d.epi = EPI_STORE;
      d.out[0] = P.direct ? dx : sums;
      d.out_f32 = dt == TP_F32 || !P.direct;
      d.out_acc = i > 0;
      d.out_group_stride = P.groups > 1 ? M * h : 0;
      TP_TRY(product(d, st));
    }
    if (dE) {  // dE = q^T x, the piece's rows
      GemmDesc d;
      d.dtype = dt;
      d.M = n;
      d.N = h;
      d.K = M;
      d.A[0] = {q, M, n, P.piece};  // q (M, n) read as A(m = n, k = M): MN-major
      d.a_mn = true;
      d.B[0] = {x, M, h, h};
      d.b_mn = true;
      d.ldo = h;
      d.epi = EPI_STORE;
      d.out[0] = static_cast<char*>(dE) + c0 * h * e;
      d.out_f32 = dt == TP_F32;
      TP_TRY(product(d, st));
    }
  }
  if (dx && !P.direct) return launch_shard_reduce(sums, nullptr, dx, P.groups, M, h, dt, st);
  return TP_OK;
}

}  // namespace tp
