// C ABI of the paged key/value cache and the grouped-query attention that reads it: the
// decode attention against a KV cache of the 20260402-parallelism page (Decode 阶段) and
// the chunked prefill before it, over the sharded QKV rows of the tp_gqa_* entry points.
#include <cuda_runtime.h>

#include <algorithm>

#include "internal.h"
#include "paged.cuh"

namespace tp {
namespace {

struct PagedGqa {
  int hq, hkv, rep, d;
  int64_t S, W;
};

tp_status paged_shape(int64_t h, int32_t H, int32_t Hkv, int32_t N, PagedGqa* g) {
  TP_TRY(need(h >= 1 && H >= 1 && Hkv >= 1 && N >= 1, TP_ERR_INVALID_ARG,
              "need h, n_heads, n_kv_heads, N >= 1"));
  TP_TRY(need(h <= (1 << 24) && N <= 65536, TP_ERR_SHAPE, "h or N too large"));
  TP_TRY(need(h % H == 0, TP_ERR_SHAPE, "h must be divisible by n_heads"));
  TP_TRY(need(H % Hkv == 0, TP_ERR_SHAPE, "n_heads must be divisible by n_kv_heads"));
  TP_TRY(need(H % N == 0, TP_ERR_SHAPE, "n_heads must be divisible by N (N <= n_heads)"));
  TP_TRY(need(N <= Hkv ? Hkv % N == 0 : N % Hkv == 0, TP_ERR_SHAPE,
              "N must divide n_kv_heads, or be a multiple of it (replicated key/value heads)"));
  const int64_t d = h / H;
  TP_TRY(need(d == 16 || d == 32 || d == 64 || d == 128, TP_ERR_SHAPE,
              "head_dim must be 16, 32, 64 or 128"));
  g->d = static_cast<int>(d);
  g->hq = H / N;
  g->hkv = N <= Hkv ? Hkv / N : 1;
  g->rep = N <= Hkv ? 1 : N / Hkv;
  g->S = static_cast<int64_t>(g->hq + 2 * g->hkv) * d;
  g->W = N * g->S;
  return TP_OK;
}

int log2_of(int64_t x) {
  int k = 0;
  while ((1ll << k) < x) ++k;
  return k;
}

tp_status check_pages(int64_t n_pages, int64_t page_size, int64_t max_pages, int32_t Hkv) {
  TP_TRY(need(n_pages >= 1 && max_pages >= 1, TP_ERR_INVALID_ARG, "need n_pages, max_pages >= 1"));
  TP_TRY(need(page_size >= 8 && page_size <= 256 && (page_size & (page_size - 1)) == 0,
              TP_ERR_SHAPE, "page_size must be a power of two from 8 to 256"));
  TP_TRY(need(n_pages < (1ll << 31) && n_pages * page_size <= 2147482623ll / Hkv, TP_ERR_SHAPE,
              "n_pages * page_size * n_kv_heads must be below 2^31 - 1024"));
  return need(max_pages <= (1ll << 30) / page_size, TP_ERR_SHAPE,
              "max_pages * page_size must be at most 2^30");
}

// lengths, tables, offsets and lse: 4-byte elements read one by one
tp_status check_words(std::initializer_list<const void*> ptrs) {
  for (const void* q : ptrs)
    TP_TRY(need(reinterpret_cast<uintptr_t>(q) % 4 == 0, TP_ERR_ALIGNMENT,
                "int32 and fp32 arrays must be 4-byte aligned"));
  return TP_OK;
}

struct PagedArgs {
  const void* qkv;
  const void *kc, *vc;
  const int32_t *table, *total, *cu;
  void* o;
  float* lse;
  int64_t T, R, h;
  int32_t H, Hkv, N;
  int64_t n_pages, page_size, max_pages, max_new;
  int causal;
  tp_dtype dt;
};

tp_status check_rows(int64_t T, int64_t R, int64_t max_new) {
  TP_TRY(need(T >= 0 && R >= 0 && max_new >= 0, TP_ERR_INVALID_ARG, "need T, R, max_new >= 0"));
  TP_TRY(need(T < (1ll << 31), TP_ERR_SHAPE, "T must be below 2^31"));
  return need(R <= (1 << 20), TP_ERR_SHAPE, "at most 2^20 requests");
}

tp_status launch_paged(const PagedArgs& a, const PagedGqa& g, void* ws, cudaStream_t st) {
  PagedParams p{};
  p.qkv = a.qkv;
  p.kc = a.kc;
  p.vc = a.vc;
  p.table = a.table;
  p.total = a.total;
  p.cu = a.cu;
  p.o = a.o;
  p.lse = a.lse;
  p.rec = static_cast<PagedRec*>(ws);
  p.part = reinterpret_cast<float*>(static_cast<char*>(ws) +
                                    align_up(kPagedMaxCtas * sizeof(PagedRec), 256));
  p.T = a.T;
  p.R = static_cast<int>(a.R);
  p.ldq = g.W;
  p.S = g.S;
  p.H = a.H;
  p.Hkv = a.Hkv;
  p.G = a.H / a.Hkv;
  p.hq = g.hq;
  p.n_pages = static_cast<int>(a.n_pages);
  p.ps_log2 = log2_of(a.page_size);
  p.max_pages = static_cast<int>(a.max_pages);
  p.causal = a.causal != 0;
  p.scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(g.d));
  // most rows of a request per key/value head (no request has more than T tokens)
  const int64_t rows = std::min(a.max_new, a.T) * p.G;
  // The kernel for few rows reads K and V once per 16 rows, the tcgen05 one per 128 or 256. 33
  // requests over 100 to 5000 tokens, 8 key/value heads, us (few rows / tcgen05): d = 128, 16
  // rows 67 / 78, 20 rows 99 / 79, 64 rows 204 / 80; d = 64, 16 rows 44 / 56, 20 rows 63 / 57,
  // 32 rows 69 / 57. One token each: 161 / 166 (61 requests), 9 / 16 (one).
  if (a.dt == TP_BF16)
    return rows > 16 && g.d >= 64 && p.G <= 128 ? launch_paged_tc(p, g.d, a.N, rows <= 128, st)
                                                : launch_paged_decode(p, g.d, st);
  // 64-row units where there are many rows, else 16 (three requests of 8 heads over 2,
  // head_dim 64 / 128, us, 16-row against 64-row units: 4800 rows over all heads 44 / 81
  // against 51 / 84, 19200 rows 202 / 436 against 184 / 351)
  return launch_paged_simt(p, g.d, rows > 16 && a.T * a.H >= 8192, st);
}

}  // namespace
}  // namespace tp

using namespace tp;

extern "C" {

tp_status tp_kv_tables(const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* free_pages,
                       int64_t n_free, const int32_t* free_head, int32_t* free_head_out,
                       int32_t* block_table, int32_t* total_lens, int32_t* cu_new, int32_t* slots,
                       int32_t* positions, int32_t* counts, int64_t R, int64_t T,
                       int64_t page_size, int64_t max_pages, void* stream) {
  TP_TRY(need(ctx_lens && new_lens && free_head && free_head_out && block_table && total_lens &&
                  cu_new && (slots || T == 0) && (free_pages || n_free == 0),
              TP_ERR_INVALID_ARG, "lengths, list, table, cu_new and slots are required"));
  TP_TRY(need(n_free >= 0, TP_ERR_INVALID_ARG, "need n_free >= 0"));
  TP_TRY(check_rows(T, R, 0));
  TP_TRY(need(R <= kKvMaxRequests, TP_ERR_SHAPE, "at most 8192 requests"));
  TP_TRY(need(n_free < (1ll << 31), TP_ERR_SHAPE, "n_free must be below 2^31"));
  TP_TRY(check_pages(1, page_size, max_pages, 1));
  TP_TRY(check_words({ctx_lens, new_lens, free_pages, free_head, free_head_out, block_table,
                      total_lens, cu_new, slots, positions, counts}));
  TP_TRY(check_device());
  return launch_kv_tables(ctx_lens, new_lens, free_pages, static_cast<int>(n_free), free_head,
                          free_head_out, block_table, total_lens, cu_new, slots, positions, counts,
                          R, T, log2_of(page_size), static_cast<int>(max_pages),
                          static_cast<cudaStream_t>(stream));
}

tp_status tp_kv_append(const void* qkv, const int32_t* slots, void* kcache, void* vcache, int64_t T,
                       int64_t h, int32_t n_heads, int32_t n_kv_heads, int32_t N, int64_t n_pages,
                       int64_t page_size, tp_dtype dtype, void* stream) {
  TP_TRY(check_dtype(dtype));
  TP_TRY(need(qkv && slots && kcache && vcache, TP_ERR_INVALID_ARG,
              "qkv, slots, kcache and vcache are required"));
  TP_TRY(check_rows(T, 0, 0));
  PagedGqa g;
  TP_TRY(paged_shape(h, n_heads, n_kv_heads, N, &g));
  TP_TRY(check_pages(n_pages, page_size, 1, n_kv_heads));
  TP_TRY(check_aligned({qkv, kcache, vcache}));
  TP_TRY(check_words({slots}));
  if (T == 0) return TP_OK;
  TP_TRY(check_device());
  return launch_kv_append(qkv, slots, kcache, vcache, T, g.d, n_kv_heads, g.hkv, g.hq, g.rep, g.W,
                          n_pages * page_size, log2_of(page_size), dtype,
                          static_cast<cudaStream_t>(stream));
}

size_t tp_gqa_paged_attention_workspace_size(int64_t h, int32_t n_heads, int32_t n_kv_heads,
                                             int32_t N, tp_dtype dtype) {
  PagedGqa g;
  if ((dtype != TP_BF16 && dtype != TP_F32) ||
      paged_shape(h, n_heads, n_kv_heads, N, &g) != TP_OK)
    return 0;
  return paged_workspace_bytes(g.d, dtype);
}

tp_status tp_gqa_paged_attention_fwd(const void* qkv, const void* kcache, const void* vcache,
                                     const int32_t* block_table, const int32_t* total_lens,
                                     const int32_t* cu_new, void* o, float* lse, int64_t T,
                                     int64_t R, int64_t h, int32_t n_heads, int32_t n_kv_heads,
                                     int32_t N, int64_t n_pages, int64_t page_size,
                                     int64_t max_pages, int64_t max_new, int causal,
                                     tp_dtype dtype, void* ws, size_t ws_bytes, void* stream) {
  TP_TRY(check_dtype(dtype));
  TP_TRY(need(qkv && kcache && vcache && block_table && total_lens && cu_new && o,
              TP_ERR_INVALID_ARG,
              "qkv, kcache, vcache, block_table, total_lens, cu_new and o are required"));
  TP_TRY(check_rows(T, R, max_new));
  PagedGqa g;
  TP_TRY(paged_shape(h, n_heads, n_kv_heads, N, &g));
  TP_TRY(check_pages(n_pages, page_size, max_pages, n_kv_heads));
  TP_TRY(check_aligned({qkv, kcache, vcache, o, ws}));
  TP_TRY(check_words({block_table, total_lens, cu_new, lse}));
  if (T == 0 || R == 0) return TP_OK;
  TP_TRY(need(ws && ws_bytes >= paged_workspace_bytes(g.d, dtype), TP_ERR_WORKSPACE,
              "workspace smaller than tp_gqa_paged_attention_workspace_size"));
  TP_TRY(check_device());
  return launch_paged({qkv, kcache, vcache, block_table, total_lens, cu_new, o, lse, T, R, h,
                       n_heads, n_kv_heads, N, n_pages, page_size, max_pages, max_new, causal,
                       dtype},
                      g, ws, static_cast<cudaStream_t>(stream));
}

size_t tp_gqa_paged_workspace_size(int64_t T, int64_t h, int32_t n_heads, int32_t n_kv_heads,
                                   int32_t N, tp_dtype dtype, tp_reduce mode) {
  PagedGqa g;
  if (T < 0 || (dtype != TP_BF16 && dtype != TP_F32) ||
      paged_shape(h, n_heads, n_kv_heads, N, &g) != TP_OK || !extents_ok(T, h, N))
    return 0;
  return std::max(paged_workspace_bytes(g.d, dtype), partial_bytes(T, h, N, mode));
}

tp_status tp_gqa_paged_attn_proj_fwd(
    const void* x, const float* gamma, const float* beta, const void* Wqkv, const void* Wo,
    void* xn, float* mean, float* rstd, void* qkv, void* kcache, void* vcache,
    const int32_t* block_table, const int32_t* total_lens, const int32_t* cu_new,
    const int32_t* slots, void* o, float* lse, void* out, int64_t T, int64_t R, int64_t h,
    int32_t n_heads, int32_t n_kv_heads, int32_t N, int64_t n_pages, int64_t page_size,
    int64_t max_pages, int64_t max_new, int causal, tp_dtype dtype, tp_reduce mode, void* ws,
    size_t ws_bytes, void* stream) {
  TP_TRY(check_dtype(dtype));
  TP_TRY(need(mode == TP_REDUCE_BUFFERS || mode == TP_REDUCE_SPLITK, TP_ERR_INVALID_ARG,
              "unknown reduce mode"));
  TP_TRY(need(x && gamma && beta && Wqkv && Wo && xn && qkv && kcache && vcache && block_table &&
                  total_lens && cu_new && slots && o && out,
              TP_ERR_INVALID_ARG,
              "every tensor of tp_gqa_paged_attn_proj_fwd but mean, rstd and lse is required"));
  TP_TRY(check_rows(T, R, max_new));
  PagedGqa g;
  TP_TRY(paged_shape(h, n_heads, n_kv_heads, N, &g));
  TP_TRY(check_pages(n_pages, page_size, max_pages, n_kv_heads));
  TP_TRY(check_extents(T, h, N));
  TP_TRY(check_extents(T, g.W, 1));
  TP_TRY(check_extents(h, g.W, 1));
  if (dtype == TP_BF16) {
    TP_TRY(need(g.S % 64 == 0, TP_ERR_SHAPE,
                "bf16 path: each shard's QKV block ((hq + 2 hkv) * head_dim) must be a multiple of 64"));
    TP_TRY(need((h / N) % 64 == 0, TP_ERR_SHAPE, "bf16 path: h/N must be a multiple of 64"));
  }
  TP_TRY(check_aligned({x, gamma, beta, Wqkv, Wo, xn, mean, rstd, qkv, kcache, vcache, o, out, ws}));
  TP_TRY(check_words({block_table, total_lens, cu_new, slots, lse}));
  if (T == 0) return TP_OK;
  TP_TRY(need(ws && ws_bytes >= tp_gqa_paged_workspace_size(T, h, n_heads, n_kv_heads, N, dtype, mode),
              TP_ERR_WORKSPACE, "workspace smaller than tp_gqa_paged_workspace_size"));
  TP_TRY(check_device());
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TP_TRY(launch_layernorm_fwd(x, gamma, beta, xn, mean, rstd, T, h, 1e-5f, dtype, st));
  {  // column-parallel projection: shard i's block of S columns
    GemmDesc d;
    d.dtype = dtype;
    d.M = T;
    d.N = g.W;
    d.K = h;
    d.A[0] = {xn, T, h, h};
    d.B[0] = {Wqkv, h, g.W, g.W};
    d.b_mn = true;
    d.ldo = g.W;
    d.shards = N;
    d.shard_axis = 1;
    d.epi = EPI_STORE;
    d.out[0] = qkv;
    d.out_f32 = dtype == TP_F32;
    TP_TRY(launch_gemm(d, st));
  }
  TP_TRY(launch_kv_append(qkv, slots, kcache, vcache, T, g.d, n_kv_heads, g.hkv, g.hq, g.rep, g.W,
                          n_pages * page_size, log2_of(page_size), dtype, st));
  if (R > 0)
    TP_TRY(launch_paged({qkv, kcache, vcache, block_table, total_lens, cu_new, o, lse, T, R, h,
                         n_heads, n_kv_heads, N, n_pages, page_size, max_pages, max_new, causal,
                         dtype},
                        g, ws, st));
  // shard i's O_i (its query heads) feeds row block i of W_o; sum + residual
  return row_impl(o, Wo, x, out, T, h, h, N, dtype, mode, ws, st);
}

}  // extern "C"
