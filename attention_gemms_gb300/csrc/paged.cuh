// Work division of the paged attention kernels (paged_attention.cu and the kernels beside
// it): which request, key/value head, query rows and keys each CTA takes.
//
// The work of one call is a line of key tiles. Request r with n new tokens has, for each
// of Hv head groups, ceil(n / tpu) units of tpu tokens x Gv query heads that share a
// key/value head; a unit's tiles are the KT-key tiles that its last token may see (at
// least one, so that rows that see no key are written too), each at the cost that it has in
// a unit that is more or at most half full, after the unit's start cost (queries, first
// loads, the output). CTA i of g takes [i total / g, (i + 1) total / g) of the line,
// whatever units that falls into (a tile belongs to the CTA that holds its end): every CTA
// gets the same work for any mix of lengths, and a long context is split over the whole GPU
// without a setting. A unit that lies in one CTA is finished there; else
// each CTA leaves its rows' (maximum, sum, unnormalised output) in its slot of the
// workspace and the combine kernel joins them in key order. At most one unit begins and
// one ends inside other CTAs' ranges, so two slots per CTA are enough for any lengths.
//
// Lengths live on the device (a captured step replays with new ones), so each CTA finds
// its own place: one pass over the lengths with a block-wide scan, and within a request
// by the closed form of the tile counts' sum. Nothing is planned ahead, so no plan can go
// stale. Lengths and page ids are not trusted: rows end at T, keys at the table's width,
// and a page id outside the cache is a page of masked keys.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"

namespace tp {

struct PagedParams {
  const void *qkv, *kc, *vc;
  const int32_t *table, *total, *cu;
  void* o;
  float* lse;              // (H, T), may be null
  float* part;             // partial results: per slot m (rows), l (rows), O (rows x d)
  struct PagedRec* rec;    // one per CTA
  int64_t T;               // rows of qkv, o, lse
  int64_t ldq, S;          // qkv row pitch, shard block width (elements)
  int R, H, Hkv, G, hq;    // G = H / Hkv; hq query heads per shard block
  int n_pages, ps_log2, max_pages;
  int causal;
  float scale_log2;        // log2(e) / sqrt(d)
  int hs, Gv, Hv;          // head groups per key/value head, heads per group, Hkv * hs
  int tpu, kt_log2;        // tokens per unit, keys per tile
  int tpu_log2;            // -1: not a power of two
  int unit_cost;           // of a unit, beside its tiles
};

// CTA i's two slots: the first holds its piece of a unit that began in an earlier CTA (its
// head), the second the first piece of a unit that goes on after it (its tail). What the join
// needs to know of the tail: the CTA where the unit ends (0: no tail), the unit's first row,
// its tokens, its first query head and their number.
struct PagedRec {
  int tail, row0, tokens, head0, heads;
};

#ifdef __CUDACC__

struct PagedReq {
  int row0, n, rows, total, kv_end;  // rows: those below T; kv_end: keys the table can hold
};

__device__ __forceinline__ PagedReq paged_req(const PagedParams& p, int r) {
  PagedReq q;
  const int c0 = p.cu[r], c1 = p.cu[r + 1];
  q.row0 = c0;
  q.n = (c0 >= 0 && c1 > c0) ? c1 - c0 : 0;
  q.rows = static_cast<int>(min(static_cast<int64_t>(q.n), max(p.T - c0, static_cast<int64_t>(0))));
  q.total = max(p.total[r], 0);
  q.kv_end = static_cast<int>(
      min(static_cast<int64_t>(q.total), static_cast<int64_t>(p.max_pages) << p.ps_log2));
  return q;
}

__device__ __forceinline__ int paged_units(const PagedParams& p, const PagedReq& q) {
  const int n = q.rows + p.tpu - 1;
  return p.tpu_log2 >= 0 ? n >> p.tpu_log2 : n / p.tpu;
}

// first key that no row of unit u sees
__device__ __forceinline__ int paged_unit_kend(const PagedParams& p, const PagedReq& q, int u) {
  if (!p.causal) return q.kv_end;
  const int64_t tokens = min(static_cast<int64_t>(u + 1) * p.tpu, static_cast<int64_t>(q.rows));
  const int64_t end = static_cast<int64_t>(q.total) - q.n + tokens;
  return static_cast<int>(max(static_cast<int64_t>(0), min(end, static_cast<int64_t>(q.kv_end))));
}
__device__ __forceinline__ int paged_unit_tiles(const PagedParams& p, const PagedReq& q, int u) {
  return max(1, static_cast<int>((static_cast<int64_t>(paged_unit_kend(p, q, u)) +
                                  (1 << p.kt_log2) - 1) >> p.kt_log2));
}

// division by a small number, in 32 bits where that holds it (64 bits: a long call)
__device__ __forceinline__ int64_t div_by(int64_t a, int b) {
  return (static_cast<uint64_t>(a) >> 32) == 0
             ? static_cast<int64_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b))
             : a / b;
}

// sum over i < n of floor((a i + b) / 2^k), b >= 0: whole parts by their closed form, the rest
// by the reciprocity of such sums (the lattice points under a line, counted along the other
// axis: Graham, Knuth, Patashnik, Concrete Mathematics, section 3.5), as in Euclid's algorithm
__device__ __forceinline__ int64_t floor_sum(int64_t n, int k, int a, int64_t b) {
  int64_t ans = 0;
  int m = 1 << k;
  while (n > 0) {
    if (a >= m) {
      ans += (n - 1) * n / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      const int64_t d = div_by(b, m);
      ans += n * d;
      b -= d * m;
    }
    const int64_t y = a * n + b;
    if (y < m) break;
    n = div_by(y, m);
    b = y - n * m;
    const int t = m;
    m = a;
    a = t;
  }
  return ans;
}

// The costs of a tile of a unit with more than (full) and at most (half) tpu / 2 tokens are
// constants of the kernel: at 1 and 1 nothing is left of them.
template <int FULL, int HALF>
__device__ __forceinline__ bool paged_half(const PagedParams& p, const PagedReq& q, int u) {
  return FULL != HALF && 2 * static_cast<int64_t>(min(p.tpu, q.rows - u * p.tpu)) <= p.tpu;
}

// cost of unit u's tiles
template <int FULL, int HALF>
__device__ __forceinline__ int paged_unit_cost(const PagedParams& p, const PagedReq& q, int u) {
  return paged_unit_tiles(p, q, u) * (paged_half<FULL, HALF>(p, q, u) ? HALF : FULL);
}

// cost of the first `u` units of a request's head group
template <int FULL, int HALF>
__device__ __forceinline__ int64_t paged_prefix(const PagedParams& p, const PagedReq& q, int u) {
  if (u <= 0) return 0;
  const int64_t starts = static_cast<int64_t>(u) * p.unit_cost;
  if (u == 1) return starts + paged_unit_cost<FULL, HALF>(p, q, 0);
  const int units = paged_units(p, q);
  const int64_t full = min(u, units - 1);  // the last unit may hold fewer tokens
  const int last = u > full ? paged_unit_cost<FULL, HALF>(p, q, units - 1) : 0;
  const int c = q.total - q.n;
  int64_t s = 0;  // tiles of the full units
  if (!p.causal) {
    s = full * paged_unit_tiles(p, q, 0);
  } else if (c < 0 || q.kv_end < q.total) {  // tokens outside the cache: no closed form, rare
    for (int i = 0; i < full; ++i) s += paged_unit_tiles(p, q, i);
  } else {
    const int64_t b = static_cast<int64_t>(c) + p.tpu + (1 << p.kt_log2) - 1;
    if (p.tpu_log2 >= p.kt_log2) {  // a whole number of tiles more per unit
      s = ((full * (full - 1) / 2) << (p.tpu_log2 - p.kt_log2)) + full * (b >> p.kt_log2);
    } else if (p.tpu_log2 >= 0) {  // a tile more every 2^k units
      const int k = p.kt_log2 - p.tpu_log2;
      auto below = [&](int64_t n) {  // sum over x < n of x >> k
        const int64_t a = n >> k, r = n & ((1 << k) - 1);
        return ((a * (a - 1) / 2) << k) + a * r;
      };
      const int64_t x = b >> p.tpu_log2;
      s = below(x + full) - below(x);
    } else {
      s = floor_sum(full, p.kt_log2, p.tpu, b);
    }
  }
  return starts + s * FULL + last;
}

// A CTA's walk over its work: segment by segment, a segment being tiles [lo, hi) of unit u
// (never none of them: a share that ends before a unit's first tile does leaves it to the next).
template <int FULL, int HALF>
struct PagedWalk {
  int64_t left;  // work left after the current segment
  int64_t stop, total;  // the CTA's end on the line, the line's
  int ctas;             // those with work
  int rest;             // cost of the segment's unit after it
  PagedReq q;
  int r, vh, u, units, tiles, lo, hi;

  __device__ __forceinline__ bool valid() const { return hi > lo; }
  // from `x` on, counted from the unit's beginning
  __device__ __forceinline__ void take(const PagedParams& p, int x) {
    tiles = paged_unit_tiles(p, q, u);
    const bool half = paged_half<FULL, HALF>(p, q, u);
    const int all = tiles * (half ? HALF : FULL) + p.unit_cost;
    const int end = static_cast<int>(min(static_cast<int64_t>(all), x + left));
    left -= end - x;
    rest = all - end;
    const int a = max(x - p.unit_cost, 0), b = max(end - p.unit_cost, 0);
    lo = half ? a / HALF : a / FULL;
    hi = half ? b / HALF : b / FULL;
  }
  // of a segment that does not end its unit (it is the CTA's last one): where the unit ends
  __device__ __forceinline__ int last_cta() const {
    return static_cast<int>(((stop + rest) * ctas + total - 1) / total) - 1;
  }
  __device__ __forceinline__ void next(const PagedParams& p) {
    if (left <= 0) {
      lo = hi = 0;
      return;
    }
    if (++u >= units) {
      u = 0;
      if (++vh >= p.Hv) {
        vh = 0;
        do {
          if (++r >= p.R) {  // lengths changed under the call: nothing left
            left = 0;
            lo = hi = 0;
            return;
          }
          q = paged_req(p, r);
        } while (q.rows == 0);
        units = paged_units(p, q);
      }
    }
    take(p, 0);
  }
};

// Scratch of the schedule (shared memory).
struct PagedSched {
  int64_t warp_sum[32];
  int64_t x, per_head;  // the CTA's first work, from the beginning of request r; its heads' cost
  PagedReq q;
  int r, units;
};

// Every thread of the CTA (blockDim.x a multiple of 32, at most 1024) calls it; returns
// the CTA's first segment. Two block-wide barriers. (By one warp it took as long for a few
// requests and grew with their number.)
template <int FULL = 1, int HALF = 1>
__device__ __forceinline__ PagedWalk<FULL, HALF> paged_schedule(const PagedParams& p,
                                                                PagedSched& sc, int cta, int ctas) {
  const int tid = threadIdx.x, nt = blockDim.x, lane = tid & 31, warp = tid >> 5;
  const int per = (p.R + nt - 1) / nt;
  const int r0 = min(tid * per, p.R), r1 = min(r0 + per, p.R);
  int64_t sum = 0, head_cost = 0;
  PagedReq q;
  for (int r = r0; r < r1; ++r) {
    q = paged_req(p, r);
    head_cost = q.rows > 0 ? paged_prefix<FULL, HALF>(p, q, paged_units(p, q)) : 0;
    sum += p.Hv * head_cost;
  }
  int64_t inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc += v;
  }
  if (lane == 31) sc.warp_sum[warp] = inc;
  if (tid == 0) sc.r = -1;
  __syncthreads();
  int64_t before = 0, total = 0;
  for (int w = 0; w < (nt >> 5); ++w) {
    const int64_t v = sc.warp_sum[w];
    before += w < warp ? v : 0;
    total += v;
  }
  // a share holds the end of a tile at least, so that a unit's pieces lie in consecutive CTAs
  const int64_t shares = max(total / (FULL > HALF ? FULL : HALF), static_cast<int64_t>(1));
  const int n = static_cast<int>(min(static_cast<int64_t>(ctas), shares));
  const int64_t begin = cta < n ? div_by(total * cta, n) : total;
  const int64_t end = cta < n ? div_by(total * (cta + 1), n) : total;
  const int64_t mine = before + inc - sum;  // tiles before this thread's requests
  if (end > begin && begin >= mine && begin < mine + sum) {
    int64_t x = begin - mine;
    int r = r0;
    if (per > 1)  // with one request per thread, it is still at hand
      for (; r < r1; ++r) {
        q = paged_req(p, r);
        head_cost = q.rows > 0 ? paged_prefix<FULL, HALF>(p, q, paged_units(p, q)) : 0;
        if (x < p.Hv * head_cost) break;
        x -= p.Hv * head_cost;
      }
    sc.r = r;
    sc.x = x;
    sc.q = q;
    sc.per_head = head_cost;
    sc.units = paged_units(p, q);
  }
  __syncthreads();
  PagedWalk<FULL, HALF> w;
  w.lo = w.hi = 0;
  w.left = end - begin;
  w.stop = end;
  w.total = total;
  w.ctas = n;
  w.r = sc.r;
  if (w.left <= 0 || w.r < 0 || w.r >= p.R) {
    w.left = 0;
    return w;
  }
  // every warp finds the unit on its own (32 candidates at a time)
  w.q = sc.q;
  w.units = sc.units;
  const int64_t per_head = sc.per_head;
  int64_t x = sc.x;
  w.vh = static_cast<int>((static_cast<uint64_t>(x) | static_cast<uint64_t>(per_head)) >> 32
                              ? x / per_head
                              : static_cast<uint32_t>(x) / static_cast<uint32_t>(per_head));
  x -= w.vh * per_head;
  int lo = 0, hi = w.units;  // prefix(lo) <= x < prefix(hi)
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int cand = min(lo + lane * step, hi);
    const bool le = cand < hi && paged_prefix<FULL, HALF>(p, w.q, cand) <= x;
    const int k = __popc(__ballot_sync(0xFFFFFFFFu, le)) - 1;  // lane 0 always holds
    const int base = lo;
    lo = base + k * step;
    hi = min(hi, base + (k + 1) * step);
  }
  w.u = lo;
  w.take(p, static_cast<int>(x - paged_prefix<FULL, HALF>(p, w.q, lo)));
  return w;
}

// the tail entry of the walk's segment
template <class Walk>
__device__ __forceinline__ void paged_tail(const PagedParams& p, PagedRec& rec, const Walk& w) {
  const int j = w.vh / p.hs;
  rec.tail = w.last_cta();
  rec.row0 = w.q.row0 + w.u * p.tpu;
  rec.tokens = min(p.tpu, w.q.rows - w.u * p.tpu);
  rec.head0 = j * p.G + (w.vh - j * p.hs) * p.Gv;
  rec.heads = min(p.Gv, (j + 1) * p.G - rec.head0);
}

// column of query head t in a qkv row
template <int D>
__device__ __forceinline__ int64_t paged_qcol(const PagedParams& p, int t) {
  const int i = t / p.hq;
  return i * p.S + static_cast<int64_t>(t - i * p.hq) * D;
}

// cache row (of D elements) of key `key` of the request whose table row is `tab`, head j;
// -1 when its page id is not one of the cache's
__device__ __forceinline__ int64_t paged_row(const PagedParams& p, const int32_t* tab, int j,
                                             int key) {
  const int page = tab[key >> p.ps_log2];
  if (page < 0 || page >= p.n_pages) return -1;
  return (((static_cast<int64_t>(page) * p.Hkv + j) << p.ps_log2)) + (key & ((1 << p.ps_log2) - 1));
}

// What a row's sum l and maximum m (base 2) give: the factor of its output, and its lse. A
// row that sees no key has l = 0; one whose scores are NaN has l = NaN, which stays NaN.
__device__ __forceinline__ float paged_inv(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float paged_lse(float m, float l) {
  return l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

#endif  // __CUDACC__

// fp32 on CUDA cores (wide: chunks), and the join of the partial results (paged_attention.cu)
constexpr int kPagedMaxCtas = 304;
tp_status launch_paged_simt(PagedParams p, int d, bool wide, cudaStream_t st);
// unit_rows: rows of a slot; tile_rows: rows of its tiles (whole tokens each)
tp_status launch_paged_combine(const PagedParams& p, int d, int unit_rows, int tile_rows, int ctas,
                               tp_dtype dt, cudaStream_t st);
// units of unit_rows rows in tiles of tile_rows, 2^kt_log2 keys per tile
void paged_set_units(PagedParams& p, int tile_rows, int unit_rows, int kt_log2, int unit_cost);
// bf16, few rows per key/value head (paged_decode.cu)
tp_status launch_paged_decode(const PagedParams& p, int d, cudaStream_t st);
// bf16, head_dim 64 or 128, chunks, at most 128 query heads per key/value head
// (paged_attention_tc.cu)
constexpr int kPagedTcCtas = 152;
// one: at most 128 rows per request and key/value head are expected
tp_status launch_paged_tc(const PagedParams& p, int d, int N, bool one, cudaStream_t st);
// tensor map of the queries: rows, shard blocks, heads, dims; box: `tokens` tokens x the
// query heads of one key/value head x 64
tp_status paged_q_map(CUtensorMap* m, const PagedParams& p, int d, int N, int tokens);
size_t paged_tc_floats(int d);  // partial results it may leave
// tensor map of a cache (rows of d bf16, swizzled): boxes of box_rows x min(64, d)
tp_status paged_cache_map(CUtensorMap* m, const void* cache, int64_t rows, int d, int box_rows);
size_t paged_workspace_bytes(int d, tp_dtype dt);

}  // namespace tp
