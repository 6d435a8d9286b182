// The paged key/value cache's set-up and write.
//
// kv_tables: from the requests' cached and new lengths, the pages that the new tokens
// need (taken off a free list in request order), the rows' offsets, slots and positions.
// Two prefix sums over the requests (rows, new pages) and a binary search per row. A few
// hundred KB at most, so latency bounds it: one launch, one block for a decode step, more
// for many rows, each of which forms both sums on its own. A step that updates its lengths
// or list position in place takes at most kTableCtas blocks of one cluster, whose barrier
// stands between the last read of the inputs and the first write of the same buffers.
//
// kv_append: the new rows' K and V columns of the packed QKV rows into their slots. It
// reads and writes each element once and HBM bounds it; 16-byte accesses, two in flight per
// thread (7999 rows of 2 x 8 x 128 bf16: 12.6 us, 5.2 TB/s; one 12.9, four 15.6).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "internal.h"
#include "ptx.cuh"

namespace tp {
namespace {

constexpr int kTableThreads = 1024;  // at most; a decode step's few rows take fewer
constexpr int kTableCtas = 8;
constexpr int kMaxLen = 1 << 30;  // a length, as the sums take it

struct TablesParams {
  const int32_t *ctx, *add, *free_pages, *head;
  int32_t *head_out, *table, *total, *cu, *slots, *pos, *counts;
  int64_t T;
  int R, n_free, ps_log2, max_pages;
  bool clustered;
};

__global__ void __launch_bounds__(kTableThreads) kv_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t sm[];
  int32_t *cu_s = sm, *base_s = cu_s + p.R + 1, *ctx_s = base_s + p.R + 1;
  __shared__ int64_t wr[32], wp[32];
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int cta = blockIdx.x, ctas = gridDim.x, threads = blockDim.x;
  auto pages_of = [&](int64_t len) {
    const int64_t n = (len + (static_cast<int64_t>(1) << p.ps_log2) - 1) >> p.ps_log2;
    return static_cast<int>(min(n, static_cast<int64_t>(p.max_pages)));
  };
  const int head = min(max(*p.head, 0), p.n_free);
  const int per = (p.R + threads - 1) / threads;
  const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
  int64_t rows = 0, pages = 0;
  for (int r = r0; r < r1; ++r) {
    const int c = min(max(p.ctx[r], 0), kMaxLen), n = min(max(p.add[r], 0), kMaxLen);
    ctx_s[r] = c;
    rows += n;
    pages += pages_of(static_cast<int64_t>(c) + n) - pages_of(c);
  }
  int64_t ir = rows, ip = pages;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t a = __shfl_up_sync(0xFFFFFFFFu, ir, o), b = __shfl_up_sync(0xFFFFFFFFu, ip, o);
    if (lane >= o) ir += a, ip += b;
  }
  if (lane == 31) wr[warp] = ir, wp[warp] = ip;
  __syncthreads();
  int64_t sr = ir - rows, sp = ip - pages, all_rows = 0, all_pages = 0;
#pragma unroll 4
  for (int w = 0; w < threads / 32; ++w) {
    if (w < warp) sr += wr[w], sp += wp[w];
    all_rows += wr[w], all_pages += wp[w];
  }
  constexpr int64_t kTop = 2147483647;
  for (int r = r0; r < r1; ++r) {
    const int n = min(max(p.add[r], 0), kMaxLen);
    cu_s[r] = static_cast<int32_t>(min(sr, kTop));
    base_s[r] = static_cast<int32_t>(min(sp, kTop));
    sr += n;
    sp += pages_of(static_cast<int64_t>(ctx_s[r]) + n) - pages_of(ctx_s[r]);
  }
  if (tid == 0) {
    cu_s[p.R] = static_cast<int32_t>(min(all_rows, kTop));
    base_s[p.R] = static_cast<int32_t>(min(all_pages, kTop));
  }
  // past this point only shared memory, the free list and old table entries are read
  if (p.clustered)
    cluster_sync_all();
  else
    __syncthreads();
  auto fresh_page = [&](int r, int k) -> int {  // k-th new page of request r
    const int64_t i = static_cast<int64_t>(head) + base_s[r] + k;
    return i < p.n_free ? p.free_pages[i] : -1;
  };
  // lengths and offsets; the pages of request r: one warp
  const int gt = cta * threads + tid, step = ctas * threads;
  for (int r = gt; r <= p.R; r += step) {
    p.cu[r] = cu_s[r];
    if (r < p.R)
      p.total[r] = static_cast<int32_t>(
          min(static_cast<int64_t>(ctx_s[r]) + (cu_s[r + 1] - cu_s[r]), kTop));
  }
  for (int r = gt >> 5; r < p.R; r += step >> 5) {
    const int have = pages_of(ctx_s[r]), need = base_s[r + 1] - base_s[r];
    for (int k = lane; k < need; k += 32)
      p.table[static_cast<int64_t>(r) * p.max_pages + have + k] = fresh_page(r, k);
  }
  const int live = cu_s[p.R];
  // four rows at a time: their searches and page loads overlap
  constexpr int kBatch = 4;
  for (int64_t t0 = gt; t0 < p.T; t0 += kBatch * static_cast<int64_t>(step)) {
    int at[kBatch], req[kBatch];
    int64_t page[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t t = t0 + i * static_cast<int64_t>(step);
      at[i] = -1;
      page[i] = -1;
      if (t >= live) continue;
      int lo = 0, hi = p.R;  // cu[lo] <= t < cu[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (cu_s[mid] <= t) lo = mid;
        else hi = mid;
      }
      req[i] = lo;
      at[i] = ctx_s[lo] + static_cast<int>(t - cu_s[lo]);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int pg = at[i] >> p.ps_log2;
      if (at[i] < 0 || pg >= p.max_pages || t0 + i * static_cast<int64_t>(step) >= p.T) continue;
      const int have = pages_of(ctx_s[req[i]]);
      page[i] = pg < have ? p.table[static_cast<int64_t>(req[i]) * p.max_pages + pg]
                          : fresh_page(req[i], pg - have);
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int64_t t = t0 + i * static_cast<int64_t>(step);
      if (t >= p.T) break;
      const int64_t s = (page[i] << p.ps_log2) + (at[i] & ((1 << p.ps_log2) - 1));
      p.slots[t] = page[i] >= 0 && s <= kTop ? static_cast<int>(s) : -1;
      if (p.pos) p.pos[t] = at[i];
    }
  }
  if (gt == 0) {
    const int64_t left = p.n_free - head;
    const int taken = static_cast<int>(min(all_pages, left));
    *p.head_out = head + taken;
    if (p.counts) {
      p.counts[0] = live;
      p.counts[1] = taken;
      p.counts[2] = static_cast<int>(min(all_pages - taken, kTop));
      p.counts[3] = static_cast<int>(max(static_cast<int64_t>(live) - p.T, static_cast<int64_t>(0)));
    }
  }
}

struct AppendParams {
  const uint4* qkv;  // 16-byte vectors
  uint4 *kc, *vc;
  const int32_t* slots;
  int64_t T, ld, S, KO, VO;  // row pitch, shard block, K and V offsets: in vectors
  int Hkv, hkv, rep, dv_log2;  // vectors per head: 2^dv_log2
  int ps_log2;
  int64_t n_slots;
};

// vector v of a row's 2 Hkv heads (K heads, then V heads)
constexpr int kAppendUnroll = 2;
template <typename I>  // uint32_t where it holds every index, whose division is a tenth of int64_t's
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendParams p) {
  pdl_wait();  // the previous kernel's results are complete and visible
  pdl_trigger();
  const I per_row = static_cast<I>(2 * p.Hkv) << p.dv_log2;
  const I n = static_cast<I>(p.T) * per_row;
  const I step = static_cast<I>(gridDim.x) * blockDim.x;
  for (I e0 = blockIdx.x * static_cast<I>(blockDim.x) + threadIdx.x; e0 < n;
       e0 += step * kAppendUnroll) {
    uint4 val[kAppendUnroll];
    uint4* dst[kAppendUnroll];
#pragma unroll
    for (int i = 0; i < kAppendUnroll; ++i) {
      const I e = e0 + i * step;
      dst[i] = nullptr;
      if (e >= n) continue;
      const int64_t t = e / per_row;
      const int v = static_cast<int>(e - static_cast<I>(t) * per_row);
      const int head = v >> p.dv_log2, c = v & ((1 << p.dv_log2) - 1);
      const bool is_k = head < p.Hkv;
      const int j = is_k ? head : head - p.Hkv;
      const int slot = p.slots[t];
      if (slot < 0 || slot >= p.n_slots) continue;
      const int blk = j / p.hkv;
      val[i] = p.qkv[t * p.ld + static_cast<int64_t>(blk) * p.rep * p.S + (is_k ? p.KO : p.VO) +
                     (static_cast<int64_t>(j - blk * p.hkv) << p.dv_log2) + c];
      const int64_t page = slot >> p.ps_log2, off = slot & ((1 << p.ps_log2) - 1);
      dst[i] = (is_k ? p.kc : p.vc) +
               (((((page * p.Hkv + j) << p.ps_log2) + off) << p.dv_log2) + c);
    }
#pragma unroll
    for (int i = 0; i < kAppendUnroll; ++i)
      if (dst[i]) *dst[i] = val[i];
  }
}

}  // namespace

tp_status launch_kv_tables(const int32_t* ctx, const int32_t* add, const int32_t* free_pages,
                           int n_free, const int32_t* head, int32_t* head_out, int32_t* table,
                           int32_t* total, int32_t* cu, int32_t* slots, int32_t* pos,
                           int32_t* counts, int64_t R, int64_t T, int ps_log2, int max_pages,
                           cudaStream_t st) {
  TablesParams p{ctx, add, free_pages, head, head_out, table, total, cu, slots, pos, counts, T,
                 static_cast<int>(R), n_free, ps_log2, max_pages, false};
  const size_t smem = (3 * R + 2) * sizeof(int32_t);
  static std::atomic<uint64_t> attr_set{0};
  if (needs_setup(attr_set)) {
    TP_CUDA_TRY(cudaFuncSetAttribute(kv_tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>((3 * kKvMaxRequests + 2) * sizeof(int32_t))));
    mark_device(attr_set);
  }
  // 33000 rows of 333 requests: 10.3 us with the cluster's 8 blocks (41 with one), 6.9 us
  // with as many as there are 2048 rows, 4.2 us with 512 rows to a block of 512
  const bool in_place = total == ctx || head_out == head;
  const int64_t most = std::max(T, R), work = std::max(T, 32 * R);
  const int threads = static_cast<int>(
      std::clamp<int64_t>((most + 31) / 32 * 32, 128, in_place ? kTableThreads : 512));
  const int ctas = static_cast<int>(
      in_place ? std::clamp<int64_t>((work + 2047) / 2048, 1, kTableCtas)
               : std::clamp<int64_t>((work + 511) / 512, 1, device_sm_count()));
  p.clustered = in_place && ctas > 1;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int na = 0;
  if (pdl_enabled()) {
    attr[na].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[na++].val.programmaticStreamSerializationAllowed = 1;
  }
  if (p.clustered) {
    attr[na].id = cudaLaunchAttributeClusterDimension;
    attr[na].val.clusterDim.x = ctas;
    attr[na].val.clusterDim.y = attr[na].val.clusterDim.z = 1;
    ++na;
  }
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = na;
  TP_CUDA_TRY(cudaLaunchKernelEx(&cfg, kv_tables_kernel, p));
  count_launch();
  return TP_OK;
}

tp_status launch_kv_append(const void* qkv, const int32_t* slots, void* kc, void* vc, int64_t T,
                           int d, int Hkv, int hkv, int hq, int rep, int64_t W, int64_t n_slots,
                           int ps_log2, tp_dtype dt, cudaStream_t st) {
  const int per_head = static_cast<int>(d * elem_size(dt) / 16);  // 2 .. 32, a power of two
  AppendParams p{};
  p.qkv = static_cast<const uint4*>(qkv);
  p.kc = static_cast<uint4*>(kc);
  p.vc = static_cast<uint4*>(vc);
  p.slots = slots;
  p.T = T;
  p.ld = W / d * per_head;
  p.S = static_cast<int64_t>(hq + 2 * hkv) * per_head;
  p.KO = static_cast<int64_t>(hq) * per_head;
  p.VO = static_cast<int64_t>(hq + hkv) * per_head;
  p.Hkv = Hkv;
  p.hkv = hkv;
  p.rep = rep;
  while ((1 << p.dv_log2) < per_head) ++p.dv_log2;
  p.ps_log2 = ps_log2;
  p.n_slots = n_slots;
  const int64_t n = T * 2 * Hkv * per_head;
  const unsigned grid = static_cast<unsigned>(
      std::clamp<int64_t>((n + 255) / 256, 1, 8ll * device_sm_count()));
  // the largest index a thread forms stays below n + 2 kAppendUnroll grid-wide steps
  if (n < (1ll << 31))
    TP_CUDA_TRY(launch_kernel(kv_append_kernel<uint32_t>, dim3(grid), dim3(256), 0, st, p));
  else
    TP_CUDA_TRY(launch_kernel(kv_append_kernel<int64_t>, dim3(grid), dim3(256), 0, st, p));
  count_launch();
  return TP_OK;
}

}  // namespace tp
