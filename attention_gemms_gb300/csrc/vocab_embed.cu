// Scaled embedding lookup and its gradient by sorted tokens [张量并行 notes, §嵌入层的并行化]:
//   x_t = scale E[id_t],   dE[c] (+)= scale sum_{t: id_t = c} dx_t
// the sums in fp32, in an order that the ids alone decide.
// An id lies in one vocabulary shard, whose rows are consecutive rows of E: the shards' sum is the
// row itself. Ids outside [0, v) give a zero row and no gradient.
//
// The gradient takes two launches.
//  * Sort: CTA g of G (a power of two) owns the rows c with c mod G = g, so that frequent ids that
//    lie together, as a tokeniser's do, fall to different CTAs. It reads all ids (4 M bytes out of
//    L2), counts its own per row and warp, and the ids of the CTAs before it, which is where its
//    part of the sorted list begins: no exchange between CTAs, no order left to chance. It also
//    cuts the list into equal units, and notes its rows without a token.
//  * Sum: a group of threads walks a unit, 16 bytes of the columns each, four tokens' loads in
//    flight whatever rows they belong to, and writes the rows that end in it. A row of many tokens
//    can lie in several units, which then leave fp32 partials; the thread that leaves a column's
//    last one adds them up, in the units' order. Rows without a token are written beside.
// HBM bounds the sum, latency the sort, which moves next to nothing. bf16, ids whose frequency falls
// as 1 / (id + 1): 8192 tokens of 50304 x 2048 47.5 us (5.0 TB/s, 75 % of a copy's rate; the sort some 6
// of it), 65536 of 50257 x 4096 169 us (5.6 TB/s). With contiguous ranges of rows for the sorting CTAs,
// empty rows written by the sort, and a launch of its own for the partials: 54 and 251.
// The lookup: 8192 rows of 4096 16 us (95 MB that it cannot do without, 5.8 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "internal.h"

namespace tp {
namespace {

constexpr int kThreads = 256;
// warps of a sorting CTA: 8 for few tokens, whose launch overlaps its predecessor (may_go_early), 32
// beyond. us: 128 tokens of 256 x 128 7.6 and 10.3, 1000 of 5000 x 512 10.1 and 12.5, 4096 of 50304 x
// 2048 44 either way, 8192 50 and 47.
constexpr int kFewWarps = 8, kManyWarps = 32;
constexpr int64_t kFewTokens = 4096;
constexpr int kMaxRange = 1152;   // rows of a sorting CTA: a counter for each warp in shared memory
constexpr int kKept = 512;        // tokens of its own that a sorting warp remembers
constexpr int kWhole = 8;         // a row of at most so many tokens is not split
constexpr int kGroup = 32;        // units whose partials of one row are added up on the way
// tokens whose loads a thread of the sum issues together, at four CTAs of 256 per SM: 65536 x 4096 179
// us, 190 with 8 at three CTAs (more registers), 214 with 4 at six (spills)
constexpr int kInFlight = 4;

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
struct Vec<__nv_bfloat16, 2> {
  uint32_t u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint32_t*>(p)); }
  __device__ __forceinline__ void load_rw(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = __uint_as_float(u << 16);
    v[1] = __uint_as_float(u & 0xFFFF0000u);
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float* v) {
    *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v[0], v[1]);
  }
};
template <>
struct Vec<float, 2> {
  float2 u;
  __device__ __forceinline__ void load(const float* p) { u = __ldg(reinterpret_cast<const float2*>(p)); }
  __device__ __forceinline__ void load_rw(const float* p) { u = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = u.x; v[1] = u.y;
  }
  __device__ __forceinline__ static void store(float* p, const float* v) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
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

// Where unit u begins: at token `tok` of the sorted list, in row `row`, which has tokens start ..
// end - 1. Units have L = ceil(total / units) tokens, so tok is u L, or the row's start where the
// row is short enough to be left whole.
struct Border {
  int32_t row, tok, start, end;
  __device__ __forceinline__ bool mid() const { return tok > start; }
};

// Row c is row c >> log2_ctas of CTA c mod ctas; the list goes by CTA, then by row, then by warp and
// the order in which a warp meets its tokens (four at a time per lane: a fixed order).
// ahead: the sums, which come next on the stream, may start ahead of its end: with no more than a CTA for
// each SM all of its own are placed by then, and none of them waits for another.
template <int kSortWarps>
__global__ void __launch_bounds__(32 * kSortWarps) vocab_embed_sort_kernel(
    const int32_t* __restrict__ ids, int2* __restrict__ sorted, Border* __restrict__ border,
    int32_t* __restrict__ arrived, uint32_t* __restrict__ absent, int32_t M, int32_t v,
    int log2_ctas, int range, int units, int columns, int ahead) {
  constexpr int kSortThreads = 32 * kSortWarps;
  pdl_wait();  // the previous kernel's results are complete and visible
  if (ahead) pdl_trigger();
  extern __shared__ int32_t cnt[];              // [warp][range]
  int32_t* start = cnt + kSortWarps * range;    // [range + 1] the rows' starts
  uint32_t* kept = reinterpret_cast<uint32_t*>(start + range + 1);  // [warp][kKept]
  __shared__ int32_t red[2][kSortWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned lower = (1u << lane) - 1u;
  const int me = blockIdx.x, mask = (1 << log2_ctas) - 1;
  const int n = (v - me + mask) >> log2_ctas;  // rows of this CTA
  for (int i = threadIdx.x; i < kSortWarps * range; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
  // warp w takes tokens [w seg, (w + 1) seg), 128 at a time: lane l tokens 4 l .. 4 l + 3
  const int seg = ((M + kSortWarps - 1) / kSortWarps + 127) / 128 * 128;
  const int64_t t0 = min(static_cast<int64_t>(warp) * seg, static_cast<int64_t>(M));
  const int64_t t1 = min(t0 + seg, static_cast<int64_t>(M));
  int32_t* mine = cnt + warp * range;
  uint32_t* list = kept + warp * kKept;
  const bool quads = reinterpret_cast<uintptr_t>(ids) % 16 == 0;
  auto load = [&](int64_t tb, int (&id)[4]) {  // -1: outside the vocabulary, or no token
    const int64_t t = tb + 4 * lane;
    if (quads && t + 4 <= t1) {
      const int4 q = *reinterpret_cast<const int4*>(ids + t);
      id[0] = q.x; id[1] = q.y; id[2] = q.z; id[3] = q.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) id[j] = t + j < t1 ? ids[t + j] : -1;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) id[j] = id[j] < v ? id[j] : -1;
  };
  // counts; the tokens that are this CTA's are kept, 16 bits of token and of row, while they fit
  int below = 0, total = 0, have = 0;
  for (int64_t tb = t0; tb < t1; tb += 512) {
    int id[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) load(tb + 128 * i, id[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (tb + 128 * i >= t1) break;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int x = id[i][j], g = x & mask;
        total += x >= 0;
        below += x >= 0 && g < me;
        const bool in = x >= 0 && g == me;
        const unsigned any = __ballot_sync(0xFFFFFFFFu, in);
        if (any == 0) continue;
        if (in) {
          const int r = x >> log2_ctas, at = have + __popc(any & lower);
          atomicAdd(mine + r, 1);
          if (at < kKept)
            list[at] = static_cast<uint32_t>(tb + 128 * i + 4 * lane + j - t0) << 16 | r;
        }
        have += __popc(any);
      }
    }
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
  below = lane < kSortWarps ? red[0][lane] : 0;
  total = lane < kSortWarps ? red[1][lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    below += __shfl_xor_sync(0xFFFFFFFFu, below, o);
    total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  }
  // each row's tokens before each warp's, and the running sum of the rows' counts
  if (threadIdx.x == 0) start[0] = below;
  int carry = below;
  for (int r0 = 0; r0 < n; r0 += kSortThreads) {
    const int r = r0 + threadIdx.x;
    int run = 0;
    if (r < n) {
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        const int c = cnt[w * range + r];
        cnt[w * range + r] = run;
        run += c;
      }
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, run, o);
      if (lane >= o) run += y;
    }
    __syncthreads();  // red has been read
    if (lane == 31) red[0][warp] = run;
    __syncthreads();
    int all = lane < kSortWarps ? red[0][lane] : 0, before = lane < warp ? all : 0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      before += __shfl_xor_sync(0xFFFFFFFFu, before, o);
      all += __shfl_xor_sync(0xFFFFFFFFu, all, o);
    }
    if (r < n) start[r + 1] = carry + before + run;
    carry += all;
  }
  __syncthreads();
  // the tokens to their places, each warp its own in order: up to 32 of them, in the lanes `any`
  auto place = [&](unsigned any, bool in, int64_t t, int r) {
    if (in) {
      const unsigned same = __match_any_sync(any, r);
      const int before = __popc(same & lower);
      const int base = mine[r];
      sorted[start[r] + base + before] = make_int2(static_cast<int>(t), (r << log2_ctas) + me);
      __syncwarp(any);
      if (before == 0) mine[r] = base + __popc(same);
      __syncwarp(any);
    }
  };
  if (have <= kKept && seg <= 65536) {
    for (int k = 0; k < have; k += 32) {
      const bool in = k + lane < have;
      const uint32_t x = in ? list[k + lane] : 0u;
      place(__ballot_sync(0xFFFFFFFFu, in), in, t0 + (x >> 16), static_cast<int>(x & 0xFFFFu));
    }
  } else {
    for (int64_t tb = t0; tb < t1; tb += 128) {
      int id[4];
      load(tb, id);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = id[j] >= 0 && (id[j] & mask) == me;
        const unsigned any = __ballot_sync(0xFFFFFFFFu, in);
        if (any) place(any, in, tb + 4 * lane + j, id[j] >> log2_ctas);
      }
    }
  }
  // the units' borders that fall into this CTA's part of the list
  const int len = max((total + units - 1) / units, 1);
  for (int u = (start[0] + len - 1) / len + threadIdx.x; u < units; u += kSortThreads) {
    const int64_t at = static_cast<int64_t>(u) * len;
    if (at >= start[n]) break;
    int lo = 0, hi = n;  // the row that holds token `at`: start[lo] <= at < start[lo + 1]
    while (hi - lo > 1) {
      const int m = (lo + hi) / 2;
      if (start[m] <= at) lo = m;
      else hi = m;
    }
    const int s = start[lo], end = start[lo + 1];
    border[u] = {(lo << log2_ctas) + me, end - s > kWhole ? static_cast<int>(at) : s, s, end};
  }
  if (blockIdx.x == gridDim.x - 1)  // borders past the last token
    for (int u = (total + len - 1) / len + threadIdx.x; u <= units; u += kSortThreads)
      border[u] = {v, total, total, total};
  // the counters of rows that several units share: at the first unit, and at each group's
  for (int r = warp; r < n; r += kSortWarps) {
    const int s = start[r], e = start[r + 1];
    if (e - s <= kWhole || s / len == (e - 1) / len) continue;
    for (int u = s / len; u <= (e - 1) / len; u = (u / kGroup + 1) * kGroup)
      for (int i = lane; i < 3 * columns; i += 32) arrived[static_cast<int64_t>(u) * 3 * columns + i] = 0;
  }
  // rows without a token, a bit each
  const int words = (range + 31) / 32;
  for (int w = warp; w < words; w += kSortWarps) {
    const int r = 32 * w + lane;
    const unsigned bits = __ballot_sync(0xFFFFFFFFu, r < n && start[r + 1] == start[r]);
    if (lane == 0) absent[static_cast<int64_t>(me) * words + w] = bits;
  }
}

// ------------------------------------------------------------------ sum

// blockDim (threads of a unit, units); blockIdx.y: slice of the columns. part: [unit][2][h] fp32
// sums of rows that the unit does not hold whole: 0 a row begun before it, 1 one begun in it.
// arrived: [unit][3][thread's columns]: 0 the partials that are written of the row begun in the unit
// (of its first group of 32 units, where it has more); 1 the groups of that row that are added up; 2 the
// partials of the group that begins at the unit, of a row begun before it. 0 and 2 are two rows' where
// the one ends in the unit in which the other begins.
// Blocks past the units' write the rows without a token (not where dE is accumulated into), a word of
// `absent` each: they fill the memory's time while the units wait for their loads.
template <typename T, int VEC>
__global__ void __launch_bounds__(kThreads, 4) vocab_embed_sum_kernel(
    const int2* __restrict__ sorted, const Border* __restrict__ border, const T* __restrict__ dx,
    T* dE, float* part, int32_t* arrived, const uint32_t* __restrict__ absent, int64_t h, int units,
    int unit_blocks, int columns, int log2_ctas, int words, float scale, int accumulate, int ahead) {
  pdl_wait();  // the sort's results are complete and visible
  if (ahead) pdl_trigger();
  const int col = blockIdx.y * blockDim.x + threadIdx.x;
  const int64_t c = static_cast<int64_t>(col) * VEC;
  if (blockIdx.x >= unit_blocks) {
    const unsigned w = blockIdx.x - unit_blocks;
    const uint32_t bits = absent[w];
    const int64_t first = static_cast<int64_t>(w % words * 32) << log2_ctas | w / words;
    if constexpr (VEC * sizeof(T) == 16) {
      const float zero[VEC] = {};
      for (int i = threadIdx.y; i < 32 && c < h; i += blockDim.y)
        if (bits >> i & 1u)
          Vec<T, VEC>::store(dE + (first + (static_cast<int64_t>(i) << log2_ctas)) * h + c, zero);
    } else if (blockIdx.y == 0) {  // rows that begin between 16-byte words: their inside by words
      constexpr int kWord = 16 / sizeof(T);
      const int tid = threadIdx.x;
      for (int i = threadIdx.y; i < 32; i += blockDim.y) {
        if (!(bits >> i & 1u)) continue;
        T* o = dE + (first + (static_cast<int64_t>(i) << log2_ctas)) * h;
        const int64_t head = min(h, static_cast<int64_t>((16 - reinterpret_cast<uintptr_t>(o) % 16) % 16 / sizeof(T)));
        const int64_t inside = (h - head) / kWord, tail = head + inside * kWord;
        for (int64_t k = tid; k < head; k += blockDim.x) o[k] = T(0.0f);
        for (int64_t k = tid; k < inside; k += blockDim.x)
          reinterpret_cast<uint4*>(o + head)[k] = make_uint4(0u, 0u, 0u, 0u);
        for (int64_t k = tail + tid; k < h; k += blockDim.x) o[k] = T(0.0f);
      }
    }
    return;
  }
  if (c >= h) return;
  const int u = blockIdx.x * blockDim.y + threadIdx.y;
  if (u >= units) return;
  const Border b0 = border[u], b1 = border[u + 1];
  const int total = border[units].tok;
  int row = b0.row;
  bool lead = b0.mid(), any = false;
  float acc[VEC];
  auto clear = [&]() {
#pragma unroll
    for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
  };
  auto write = [&]() {
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
  };
  auto part_at = [&](int unit, int which) { return part + (static_cast<int64_t>(unit) * 2 + which) * h + c; };
  auto leave = [&](int unit, int which) {
    float* p = part_at(unit, which);
    if constexpr (VEC >= 4) {
#pragma unroll
      for (int i = 0; i < VEC; i += 4)
        __stcg(reinterpret_cast<float4*>(p + i), make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]));
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i) __stcg(p + i, acc[i]);
    }
  };
  auto flush = [&]() {  // the row's end
    if (lead) leave(u, 0);
    else if (any) write();
    lead = any = false;
    clear();
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
        row = r[i];
      }
      float f[VEC];
      a[i].get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) acc[j] += f[j];
      any = true;
    }
  }
  const bool open = b1.mid() && row == b1.row;
  if (open) leave(u, lead ? 0 : 1);
  else if (any) flush();
  // The rows left in parts, the one begun before this unit and the one left open: whoever leaves a
  // row's last part in these columns adds them up; where there are many, a group's last adds up the
  // group's in the place of its first, and the last group's the groups' (1520 tokens of one row in
  // 380 units: 18 us, 42 in one go).
  auto add_up = [&](int first, int from, int to, auto step) {
    clear();
#pragma unroll 4
    for (int k = from; k <= to; k = (k / step + 1) * step) {
      const float* p = part_at(k, k == first ? 1 : 0);
      if constexpr (VEC >= 4) {
#pragma unroll
        for (int i = 0; i < VEC; i += 4) {
          const float4 f = __ldcg(reinterpret_cast<const float4*>(p + i));
          acc[i] += f.x; acc[i + 1] += f.y; acc[i + 2] += f.z; acc[i + 3] += f.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] += __ldcg(p + i);
      }
    }
  };
  auto arrive = [&](int unit, int which, int of) {  // whether this is the last of `of`
    __threadfence();
    const bool is = atomicAdd(arrived + (static_cast<int64_t>(unit) * 3 + which) * columns + col, 1) == of - 1;
    __threadfence();
    return is;
  };
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (which == 0 ? !b0.mid() : !open || (b0.mid() && b0.row == b1.row)) continue;
    const Border& b = which == 0 ? b0 : b1;
    const int len = (total + units - 1) / units, first = b.start / len, last = (b.end - 1) / len;
    const bool grouped = last - first >= kGroup;
    const int lo = grouped ? max(first, u / kGroup * kGroup) : first;
    const int hi = grouped ? min(last, u / kGroup * kGroup + kGroup - 1) : last;
    if (!arrive(lo, lo == first ? 0 : 2, hi - lo + 1)) continue;
    add_up(first, lo, hi, std::integral_constant<int, 1>());
    if (grouped) {
      leave(lo, lo == first ? 1 : 0);
      if (!arrive(first, 1, last / kGroup - first / kGroup + 1)) continue;
      add_up(first, first, last, std::integral_constant<int, kGroup>());
    }
    row = b.row;
    write();
  }
}

// ------------------------------------------------------------------ host side

struct SumPlan {
  int vec, tx, ty, slices;  // elements per thread, threads of a unit, units of a CTA, column slices
  int units, columns;       // columns: threads that share a row
  int log2_ctas, range;     // of the sort
  size_t sorted, border, arrived, absent, part, total;
};
SumPlan sum_plan(int64_t M, int64_t v, int64_t h, tp_dtype dt) {
  SumPlan P{};
  const int64_t wide = 16 / static_cast<int64_t>(elem_size(dt));
  P.vec = static_cast<int>(h % wide == 0 ? wide : h % 2 == 0 ? 2 : 1);
  const int64_t nv = h / P.vec;
  P.tx = 4;
  while (P.tx < kThreads && P.tx < nv) P.tx *= 2;
  P.ty = kThreads / P.tx;
  P.slices = static_cast<int>((nv + P.tx - 1) / P.tx);
  // 16 tokens of a unit, and up to 8 CTAs of units per SM, more than run at once: rows end in some
  // units and not in others. Few tokens: 4, whose loads are in flight together (1000 tokens, 5000
  // rows of 512: 16 us, 20 with 16).
  P.units = static_cast<int>(std::max<int64_t>(
      1, std::max(std::min<int64_t>(M / 4, 512), std::min<int64_t>(M / 16, 8 * 152))));
  size_t o = 0;
  P.sorted = o; o += align_up(M * sizeof(int2), 256);
  P.border = o; o += align_up((P.units + 1) * sizeof(Border), 256);
  P.columns = P.tx * P.slices;
  // 128 sorting CTAs (one per SM, of 152), fewer where they would have less than 32 rows each, more
  // where their counters would not fit in shared memory
  while ((P.log2_ctas < 7 && v >> P.log2_ctas > 32) || (v - 1) >> P.log2_ctas >= kMaxRange)
    ++P.log2_ctas;
  P.range = static_cast<int>((v - 1) >> P.log2_ctas) + 1;
  P.absent = o; o += align_up((static_cast<size_t>((P.range + 31) / 32) << P.log2_ctas) * 4, 256);
  P.arrived = o; o += align_up(static_cast<size_t>(P.units) * 3 * P.columns * 4, 256);
  P.part = o;   o += align_up(static_cast<size_t>(P.units) * 2 * h * 4, 256);
  P.total = o;
  return P;
}

template <typename T, int VEC>
tp_status embed_fwd(const int32_t* ids, const void* E, void* x, int64_t M, int64_t v, int64_t h,
                    float scale, cudaStream_t st) {
  // four vectors of a row per thread (65536 rows of 1024, bf16: 31 us, 56 with one; 8192 of 4096: 21
  // and 25)
  int tx = 4;
  while (tx < kThreads && tx * VEC * 4 < h) tx *= 2;
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
  const int words = (P.range + 31) / 32, unit_blocks = (P.units + P.ty - 1) / P.ty;
  const int64_t blocks = unit_blocks + (accumulate ? 0 : static_cast<int64_t>(words) << P.log2_ctas);
  // behind the sort, and ahead of what comes next only where may_go_early has it: its CTAs fill an SM's
  // registers, and there are more of them than fit at once
  const bool ahead = may_go_early(blocks * P.slices, kThreads, device_sm_count());
  TP_CUDA_TRY(launch_kernel(
      vocab_embed_sum_kernel<T, VEC>,
      dim3(static_cast<unsigned>(blocks), static_cast<unsigned>(P.slices)), dim3(P.tx, P.ty), 0, st,
      reinterpret_cast<const int2*>(ws + P.sorted), reinterpret_cast<const Border*>(ws + P.border),
      static_cast<const T*>(dx), static_cast<T*>(dE), reinterpret_cast<float*>(ws + P.part),
      reinterpret_cast<int32_t*>(ws + P.arrived), reinterpret_cast<const uint32_t*>(ws + P.absent), h,
      P.units, unit_blocks, P.columns, P.log2_ctas, words, scale, accumulate ? 1 : 0, ahead ? 1 : 0));
  count_launch();
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
    return h % 8 == 0   ? embed_fwd<__nv_bfloat16, 8>(ids, E, x, M, v, h, scale, st)
           : h % 2 == 0 ? embed_fwd<__nv_bfloat16, 2>(ids, E, x, M, v, h, scale, st)
                        : embed_fwd<__nv_bfloat16, 1>(ids, E, x, M, v, h, scale, st);
  return h % 4 == 0   ? embed_fwd<float, 4>(ids, E, x, M, v, h, scale, st)
         : h % 2 == 0 ? embed_fwd<float, 2>(ids, E, x, M, v, h, scale, st)
                      : embed_fwd<float, 1>(ids, E, x, M, v, h, scale, st);
}

tp_status launch_vocab_embed_scaled_bwd(const int32_t* ids, const void* dx, void* dE, int64_t M,
                                        int64_t v, int64_t h, float scale, bool accumulate,
                                        tp_dtype dt, void* ws, cudaStream_t st) {
  const SumPlan P = sum_plan(M, v, h, dt);
  char* base = static_cast<char*>(ws);
  const unsigned ctas = 1u << P.log2_ctas;
  auto sort = [&](auto warps) -> tp_status {
    constexpr int kWarps = decltype(warps)::value;
    auto kern = vocab_embed_sort_kernel<kWarps>;
    static std::atomic<uint64_t> attr_set{0};  // per kernel and device
    if (needs_setup(attr_set)) {
      TP_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (kWarps * (kMaxRange + kKept) + kMaxRange + 1) * 4));
      mark_device(attr_set);
    }
    const size_t smem = (static_cast<size_t>(kWarps) * (P.range + kKept) + P.range + 1) * 4;
    const bool early = may_go_early(ctas, 32 * kWarps, device_sm_count());
    TP_CUDA_TRY(launch_kernel_if(early, kern, ctas, 32 * kWarps, smem, st, ids,
                                 reinterpret_cast<int2*>(base + P.sorted),
                                 reinterpret_cast<Border*>(base + P.border),
                                 reinterpret_cast<int32_t*>(base + P.arrived),
                                 reinterpret_cast<uint32_t*>(base + P.absent), static_cast<int32_t>(M),
                                 static_cast<int32_t>(v), P.log2_ctas, P.range, P.units, P.columns,
                                 ctas <= static_cast<unsigned>(device_sm_count()) ? 1 : 0));
    return TP_OK;
  };
  if (M <= kFewTokens) TP_TRY(sort(std::integral_constant<int, kFewWarps>()));
  else TP_TRY(sort(std::integral_constant<int, kManyWarps>()));
  count_launch();
  if (dt == TP_BF16)
    return P.vec == 8   ? embed_sum<__nv_bfloat16, 8>(P, dx, dE, h, scale, accumulate, base, st)
           : P.vec == 2 ? embed_sum<__nv_bfloat16, 2>(P, dx, dE, h, scale, accumulate, base, st)
                        : embed_sum<__nv_bfloat16, 1>(P, dx, dE, h, scale, accumulate, base, st);
  return P.vec == 4   ? embed_sum<float, 4>(P, dx, dE, h, scale, accumulate, base, st)
         : P.vec == 2 ? embed_sum<float, 2>(P, dx, dE, h, scale, accumulate, base, st)
                      : embed_sum<float, 1>(P, dx, dE, h, scale, accumulate, base, st);
}

}  // namespace tp
