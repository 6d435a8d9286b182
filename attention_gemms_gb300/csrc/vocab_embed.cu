// Scaled embedding lookup and its gradient by sorted tokens [张量并行 notes, §嵌入层的并行化]:
//   x_t = scale E[id_t],   dE[c] (+)= scale sum_{t: id_t = c} dx_t  (tokens in order)
// An id lies in one vocabulary shard, whose rows are consecutive rows of E: the shards' sum is the
// row itself. Ids outside [0, v) give a zero row and no gradient.
//
// The gradient takes three launches.
//  * Sort: every CTA owns a range of vocabulary rows and reads all ids (4 M bytes out of L2). It
//    counts its own per row and warp, and the ids below its range, which is where its part of the
//    sorted list begins: no exchange between CTAs, no order left to chance. It also cuts the line
//    (row 0's tokens, row 0, row 1's tokens, row 1, ...) into equal units.
//  * Sum: a group of threads walks a unit, 16 bytes of the columns each, several tokens' loads in
//    flight whatever rows they belong to, and writes the rows that end in it, those without a token
//    too. A row of many tokens can lie in several units, which then leave fp32 partials.
//  * Join: the partials of such rows in order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "internal.h"

namespace tp {
namespace {

constexpr int kThreads = 256;
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxRange = 1408;   // rows of a sorting CTA: 32 counters each in shared memory
constexpr int kWhole = 16;        // a row of at most so many tokens is not split
constexpr int kInFlight = 8;      // tokens whose loads a thread of the sum issues together

// VEC consecutive elements of T in fp32
template <typename T, int VEC>
struct Vec;
template <>
struct Vec<__nv_bfloat16, 8> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void load_rw(const __nv_bfloat16* p) {
    u = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void get(float* v) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float* v) {
    uint4 r;
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = r;
  }
};
template <>
struct Vec<float, 4> {
  float4 u;
  __device__ __forceinline__ void load(const float* p) { u = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ __forceinline__ void load_rw(const float* p) { u = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
  }
  __device__ __forceinline__ static void store(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Vec<__nv_bfloat16, 1> {
  __nv_bfloat16 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(p); }
  __device__ __forceinline__ void load_rw(const __nv_bfloat16* p) { u = *p; }
  __device__ __forceinline__ void get(float* v) const { v[0] = __bfloat162float(u); }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float* v) {
    *p = __float2bfloat16_rn(v[0]);
  }
};
template <>
struct Vec<float, 1> {
  float u;
  __device__ __forceinline__ void load(const float* p) { u = __ldg(p); }
  __device__ __forceinline__ void load_rw(const float* p) { u = *p; }
  __device__ __forceinline__ void get(float* v) const { v[0] = u; }
  __device__ __forceinline__ static void store(float* p, const float* v) { *p = v[0]; }
};

// ------------------------------------------------------------------ lookup

// blockDim (threads of a row, rows): VEC elements per thread and step, four steps' loads in flight
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) vocab_embed_scaled_fwd_kernel(
    const int32_t* __restrict__ ids, const T* __restrict__ E, T* __restrict__ x, int64_t M,
    int64_t v, int64_t h, float scale) {
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  if (row >= M) return;
  const int64_t id = ids[row];
  const bool in = id >= 0 && id < v;
  const T* src = E + (in ? id : 0) * h;
  T* dst = x + row * h;
  const int64_t step = static_cast<int64_t>(blockDim.x) * VEC;
  for (int64_t c = static_cast<int64_t>(threadIdx.x) * VEC; c < h; c += 4 * step) {
    Vec<T, VEC> a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (in && c + i * step < h) a[i].load(src + c + i * step);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (c + i * step < h) {
        float f[VEC];
        a[i].get(f);
#pragma unroll
        for (int k = 0; k < VEC; ++k) f[k] = in ? f[k] * scale : 0.0f;
        Vec<T, VEC>::store(dst + c + i * step, f);
      }
  }
}

// ------------------------------------------------------------------ sort

// Where a unit begins: at token `tok` of the sorted list, in row `row`; mid: after the row's first
// token, else before the whole row.
struct Border {
  int32_t row, tok, mid, pad;
};

__global__ void __launch_bounds__(kSortThreads) vocab_embed_sort_kernel(
    const int32_t* __restrict__ ids, int2* __restrict__ sorted, Border* __restrict__ border,
    int64_t M, int64_t v, int range, int units, int row_weight) {
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  extern __shared__ int32_t cnt[];           // [warp][range], then the rows' starts
  int32_t* start = cnt + kSortWarps * range;  // [range + 1]
  __shared__ int32_t red[2][kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t lo = static_cast<int64_t>(blockIdx.x) * range;
  const int n = static_cast<int>(min(static_cast<int64_t>(range), v - lo));
  for (int i = threadIdx.x; i < kSortWarps * range; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  // warp w takes tokens [w seg, (w + 1) seg), in order
  const int64_t seg = ((M + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
  const int64_t t0 = warp * seg, t1 = min(t0 + seg, M);
  int32_t* mine = cnt + warp * range;
  int below = 0, total = 0;
#pragma unroll 8
  for (int64_t t = t0 + lane; t < t1; t += 32) {
    const int64_t id = ids[t];
    const bool in = id >= 0 && id < v;
    total += in;
    below += in && id < lo;
    if (id >= lo && id < lo + n) atomicAdd(mine + (id - lo), 1);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    below += __shfl_xor_sync(0xFFFFFFFFu, below, o);
    total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  }
  if (lane == 0) {
    red[0][warp] = below;
    red[1][warp] = total;
  }
  __syncthreads();
  below = red[0][lane];
  total = red[1][lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    below += __shfl_xor_sync(0xFFFFFFFFu, below, o);
    total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  }
  // each row's tokens before each warp's, and the rows' counts
  for (int r = threadIdx.x; r < n; r += kSortThreads) {
    int run = 0;
    for (int w = 0; w < kSortWarps; ++w) {
      const int c = cnt[w * range + r];
      cnt[w * range + r] = run;
      run += c;
    }
    start[r + 1] = run;
  }
  __syncthreads();
  if (warp == 0) {  // running sum of the counts
    int run = below;
    if (lane == 0) start[0] = run;
    for (int r = 0; r < n; r += 32) {
      int c = r + lane < n ? start[r + lane + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, c, o);
        if (lane >= o) c += y;
      }
      if (r + lane < n) start[r + lane + 1] = run + c;
      run += __shfl_sync(0xFFFFFFFFu, c, 31);
    }
  }
  __syncthreads();
  // the tokens to their places, each warp its own in order
  for (int64_t tb = t0; tb < t1; tb += 32) {
    const int64_t t = tb + lane;
    const int64_t id = t < t1 ? ids[t] : -1;
    const bool in = id >= lo && id < lo + n;
    const unsigned any = __ballot_sync(0xFFFFFFFFu, in);
    if (any == 0) continue;
    if (in) {
      const int r = static_cast<int>(id - lo);
      const unsigned same = __match_any_sync(any, r);
      const int before = __popc(same & ((1u << lane) - 1u));
      const int at = start[r] + mine[r] + before;
      sorted[at] = make_int2(static_cast<int>(t), static_cast<int>(id));
      __syncwarp(any);
      if (before == 0) mine[r] += __popc(same);
      __syncwarp(any);
    }
  }
  // the units' borders that fall into this range's part of the line
  const int64_t len = row_weight * v + total;
  for (int r = threadIdx.x; r < n; r += kSortThreads) {
    const int64_t f = row_weight * (lo + r) + start[r];
    const int c = start[r + 1] - start[r], items = c + row_weight;
    if (items == 0) continue;
    for (int64_t u = (f * units + len - 1) / len; u < units && u * len / units < f + items; ++u) {
      const int off = static_cast<int>(u * len / units - f);
      Border b;
      b.pad = 0;
      if (off == 0 || c <= kWhole) b = {static_cast<int32_t>(lo + r), start[r], 0, 0};
      else if (off >= c) b = {static_cast<int32_t>(lo + r + 1), start[r + 1], 0, 0};
      else b = {static_cast<int32_t>(lo + r), start[r] + off, 1, 0};
      border[u] = b;
    }
  }
  if (blockIdx.x == gridDim.x - 1)  // the end, and the borders of a line without items
    for (int u = (len == 0 ? 0 : units) + threadIdx.x; u <= units; u += kSortThreads)
      border[u] = {static_cast<int32_t>(v), total, 0, 0};
}

// ------------------------------------------------------------------ sum

// blockDim (threads of a unit, units); blockIdx.y: slice of the columns. part: [unit][2][h] fp32
// sums of rows that the unit does not hold whole: 0 a row begun before it, 1 one begun in it.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads) vocab_embed_sum_kernel(
    const int2* __restrict__ sorted, const Border* __restrict__ border, const T* __restrict__ dx,
    T* dE, float* __restrict__ part, int64_t h, int units, float scale, int accumulate) {
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  const int u = blockIdx.x * blockDim.y + threadIdx.y;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * VEC;
  if (u >= units || c >= h) return;
  const Border b0 = border[u], b1 = border[u + 1];
  int row = b0.row;
  bool lead = b0.mid != 0, any = false;
  float acc[VEC];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
  };
  auto partial = [&](int which) {
    float* o = part + (static_cast<int64_t>(u) * 2 + which) * h + c;
#pragma unroll
    for (int i = 0; i < VEC; ++i) o[i] = acc[i];
  };
  auto flush = [&]() {  // the row's end
    if (lead) {
      partial(0);
    } else if (any || !accumulate) {
      T* o = dE + row * h + c;
      float f[VEC], g[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) f[i] = acc[i] * scale;
      if (accumulate) {
        Vec<T, VEC> a;
        a.load_rw(o);
        a.get(g);
#pragma unroll
        for (int i = 0; i < VEC; ++i) f[i] += g[i];
      }
      Vec<T, VEC>::store(o, f);
    }
    lead = any = false;
    clear();
  };
  auto zeros = [&](int from, int to) {  // rows without a token
    if (accumulate) return;
    for (int r = from; r < to; ++r) Vec<T, VEC>::store(dE + r * h + c, acc);
  };
  clear();
  for (int k = b0.tok; k < b1.tok; k += kInFlight) {
    Vec<T, VEC> a[kInFlight];
    int r[kInFlight];
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      r[i] = -1;
      if (k + i < b1.tok) {
        const int2 s = __ldg(sorted + k + i);
        r[i] = s.y;
        a[i].load(dx + s.x * h + c);
      }
    }
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) {
      if (r[i] < 0) break;
      if (r[i] != row) {
        flush();
        zeros(row + 1, r[i]);
        row = r[i];
      }
      float f[VEC];
      a[i].get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] += f[j];
      any = true;
    }
  }
  if (row < b1.row) {
    flush();
    zeros(row + 1, b1.row);
  } else if (b1.mid) {
    partial(lead ? 0 : 1);
  }
}

// ------------------------------------------------------------------ join

// Rows begun in a unit and ended in a later one: partial 1 of the unit, then partials 0 of the
// following ones up to the row's end. A CTA takes (row, 32 columns); eight warps share the
// partials, the warps' sums are added in order.
template <typename T>
__global__ void __launch_bounds__(kThreads) vocab_embed_join_kernel(
    const Border* __restrict__ border, const float* __restrict__ part, T* dE, int64_t h, int units,
    float scale, int accumulate) {
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  __shared__ float sm[kThreads / 32][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t slices = (h + 31) / 32;
  for (int u = blockIdx.x; u < units; u += gridDim.x) {
    const Border b0 = border[u], b1 = border[u + 1];
    if (!b1.mid || (b0.mid && b0.row == b1.row)) continue;  // no row is begun here and left open
    int last = u + 1;  // the last unit with tokens of the row
    while (last + 1 < units && border[last + 1].mid && border[last + 1].row == b1.row) ++last;
    for (int64_t sl = blockIdx.y; sl < slices; sl += gridDim.y) {
      const int64_t c = sl * 32 + lane;
      float a = 0.0f;
      if (c < h) {
#pragma unroll 4
        for (int k = u + warp; k <= last; k += kThreads / 32)
          a += part[(static_cast<int64_t>(k) * 2 + (k == u ? 1 : 0)) * h + c];
      }
      __syncthreads();
      sm[warp][lane] = a;
      __syncthreads();
      if (warp == 0 && c < h) {
        a = 0.0f;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) a += sm[w][lane];
        T* o = dE + b1.row * h + c;
        float f = a * scale;
        if (accumulate) {
          float g;
          Vec<T, 1> old;
          old.load_rw(o);
          old.get(&g);
          f += g;
        }
        Vec<T, 1>::store(o, &f);
      }
    }
  }
}

// ------------------------------------------------------------------ host side

struct SumPlan {
  int vec, tx, ty, slices;  // elements per thread, threads of a unit, units of a CTA, column slices
  int units;
  size_t sorted, border, part, total;
};
SumPlan sum_plan(int64_t M, int64_t v, int64_t h, tp_dtype dt) {
  SumPlan P{};
  const int64_t wide = 16 / static_cast<int64_t>(elem_size(dt));
  P.vec = static_cast<int>(h % wide == 0 ? wide : 1);
  const int64_t nv = h / P.vec;
  P.tx = 4;
  while (P.tx < kThreads && P.tx < nv) P.tx *= 2;
  P.ty = kThreads / P.tx;
  P.slices = static_cast<int>((nv + P.tx - 1) / P.tx);
  // four CTAs per SM at once (152 SMs), but no unit of fewer than 16 items
  const int64_t most = std::max<int64_t>(4 * 152 / P.slices, 1) * P.ty;
  P.units = static_cast<int>(std::max<int64_t>(std::min(most, (M + v) / 16), 1));
  size_t o = 0;
  P.sorted = o; o += align_up(M * sizeof(int2), 256);
  P.border = o; o += align_up((P.units + 1) * sizeof(Border), 256);
  P.part = o;   o += align_up(static_cast<size_t>(P.units) * 2 * h * 4, 256);
  P.total = o;
  return P;
}

template <typename T, int VEC>
tp_status embed_fwd(const int32_t* ids, const void* E, void* x, int64_t M, int64_t v, int64_t h,
                    float scale, cudaStream_t st) {
  int tx = 4;
  while (tx < kThreads && tx * VEC < h) tx *= 2;
  const int ty = kThreads / tx;
  TP_CUDA_TRY(launch_kernel(vocab_embed_scaled_fwd_kernel<T, VEC>,
                            dim3(static_cast<unsigned>((M + ty - 1) / ty)), dim3(tx, ty), 0, st, ids,
                            static_cast<const T*>(E), static_cast<T*>(x), M, v, h, scale));
  count_launch();
  return TP_OK;
}

template <typename T, int VEC>
tp_status embed_sum(const SumPlan& P, const void* dx, void* dE, int64_t h, float scale,
                    bool accumulate, char* ws, cudaStream_t st) {
  const Border* border = reinterpret_cast<const Border*>(ws + P.border);
  float* part = reinterpret_cast<float*>(ws + P.part);
  TP_CUDA_TRY(launch_kernel(
      vocab_embed_sum_kernel<T, VEC>,
      dim3(static_cast<unsigned>((P.units + P.ty - 1) / P.ty), static_cast<unsigned>(P.slices)),
      dim3(P.tx, P.ty), 0, st, reinterpret_cast<const int2*>(ws + P.sorted), border,
      static_cast<const T*>(dx), static_cast<T*>(dE), part, h, P.units, scale, accumulate ? 1 : 0));
  count_launch();
  if (P.units > 1) {
    const unsigned gx = static_cast<unsigned>(std::min(P.units, 608));
    TP_CUDA_TRY(launch_kernel(vocab_embed_join_kernel<T>, dim3(gx, 4), kThreads, 0, st, border, part,
                              static_cast<T*>(dE), h, P.units, scale, accumulate ? 1 : 0));
    count_launch();
  }
  return TP_OK;
}

}  // namespace

size_t vocab_embed_scaled_ws_bytes(int64_t M, int64_t v, int64_t h, tp_dtype dt) {
  return sum_plan(M, v, h, dt).total;
}

tp_status launch_vocab_embed_scaled_fwd(const int32_t* ids, const void* E, void* x, int64_t M,
                                        int64_t v, int64_t h, float scale, tp_dtype dt,
                                        cudaStream_t st) {
  if (dt == TP_BF16)
    return h % 8 == 0 ? embed_fwd<__nv_bfloat16, 8>(ids, E, x, M, v, h, scale, st)
                      : embed_fwd<__nv_bfloat16, 1>(ids, E, x, M, v, h, scale, st);
  return h % 4 == 0 ? embed_fwd<float, 4>(ids, E, x, M, v, h, scale, st)
                    : embed_fwd<float, 1>(ids, E, x, M, v, h, scale, st);
}

tp_status launch_vocab_embed_scaled_bwd(const int32_t* ids, const void* dx, void* dE, int64_t M,
                                        int64_t v, int64_t h, float scale, bool accumulate,
                                        tp_dtype dt, void* ws, cudaStream_t st) {
  const SumPlan P = sum_plan(M, v, h, dt);
  char* base = static_cast<char*>(ws);
  // at most one CTA per SM, and no range of fewer than 32 rows
  const int64_t ctas = std::min<int64_t>((v + 31) / 32, 152);
  const int range = static_cast<int>(std::min<int64_t>((v + ctas - 1) / ctas, kMaxRange));
  const size_t smem = (static_cast<size_t>(kSortWarps) * range + range + 1) * 4;
  static std::atomic<uint64_t> attr_set{0};
  if (needs_setup(attr_set)) {
    TP_CUDA_TRY(cudaFuncSetAttribute(vocab_embed_sort_kernel,
                                     cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (kSortWarps * kMaxRange + kMaxRange + 1) * 4));
    mark_device(attr_set);
  }
  TP_CUDA_TRY(launch_kernel(vocab_embed_sort_kernel, static_cast<unsigned>((v + range - 1) / range),
                            kSortThreads, smem, st, ids, reinterpret_cast<int2*>(base + P.sorted),
                            reinterpret_cast<Border*>(base + P.border), M, v, range, P.units,
                            accumulate ? 0 : 1));
  count_launch();
  if (dt == TP_BF16)
    return P.vec == 8 ? embed_sum<__nv_bfloat16, 8>(P, dx, dE, h, scale, accumulate, base, st)
                      : embed_sum<__nv_bfloat16, 1>(P, dx, dE, h, scale, accumulate, base, st);
  return P.vec == 4 ? embed_sum<float, 4>(P, dx, dE, h, scale, accumulate, base, st)
                    : embed_sum<float, 1>(P, dx, dE, h, scale, accumulate, base, st);
}

}  // namespace tp
