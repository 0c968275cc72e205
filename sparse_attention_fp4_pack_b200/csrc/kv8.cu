// The paged 8-bit KV cache: block tables and slot maps from request lengths
// (csa2_paged_plan), their inverse (csa2_paged_release), and the write side of the cache
// (csa2_kv8_append).  Formats and rules are in include/csa2.h.
//
// plan / release are one launch each: a cluster of CTAs reads the requests in chunks of 1024,
// every CTA scans the whole chunk for itself (the arrays are a few KB), and the tokens, new
// pages and rows behind them are shared out over the cluster.  In-place use (seq_len is
// ctx_len, n_free_out is n_free) is safe because a cluster barrier stands between the last
// read of a chunk and the first write of it.  Both are bound by latency: a launch, two
// dependent loads, one or two block-wide scans.  Per call (back to back): plan of 256 requests
// of one token 4.6 us, of 48 with 24K rows 7.1; release of 8 of 61 requests 4.7, of 256 of 1024
// with 254K pages 13.8 (20 instructions per page before, 6 now; 18.2).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "csa2_device.cuh"
#include "kv8.cuh"
#include "tc.cuh"

namespace csa2 {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

__device__ __forceinline__ void cluster_sync_all() {
  tc::cluster_arrive();
  tc::cluster_wait();
}

// Exclusive sum of v over the CTA's threads, and the total.  `warp_sums` holds one value per
// warp; the trailing barrier lets the caller reuse it.
__device__ __forceinline__ int64_t block_exclusive(int64_t v, int64_t* warp_sums, int64_t* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int64_t s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += y;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  const int64_t before = warp ? warp_sums[warp - 1] : 0;
  *total = warp_sums[kPlanWarps - 1];
  __syncthreads();
  return before + x - v;
}

// The last i with a[i] <= x, for ascending a[0..n) with a[0] <= x.
template <typename T>
__device__ __forceinline__ int last_at_most(const T* a, int n, T x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

struct PlanArgs {
  const int32_t* ctx_len;
  const int32_t* new_len;
  int R, page_log2;
  int32_t* table;
  int max_pages;
  const int32_t* free_pages;
  int64_t free_cap;
  const int32_t* n_free;
  int64_t n_pages;
  int32_t* seq_len;
  int32_t* n_free_out;
  int32_t* q_start;
  int64_t* slot_map;
  int64_t* pos;
  int64_t t_cap;
  uint32_t* status;
};

__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(PlanArgs a) {
  __shared__ int64_t s_sums[32];
  __shared__ int64_t s_start[kPlanThreads + 1];  // first token of each request of the chunk
  __shared__ int64_t s_page[kPlanThreads + 1];   // first new page of each, counted from the call's first
  __shared__ int32_t s_ctx[kPlanThreads];
  __shared__ int32_t s_have[kPlanThreads];       // pages held before
  chain_enter();
  const int tid = threadIdx.x;
  const unsigned rank = blockIdx.x, ranks = gridDim.x;  // one cluster
  const int page = 1 << a.page_log2;
  uint32_t bad = 0;
  int64_t n_free = *a.n_free;
  if (n_free < 0 || n_free > a.free_cap) {
    bad |= CSA2_DEV_BAD_COUNT;
    n_free = n_free < 0 ? 0 : a.free_cap;
  }
  int64_t tok0 = 0, page0 = 0;  // tokens and new pages of the chunks before
  for (int r0 = 0; r0 < a.R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    int64_t c = 0, n = 0;
    if (r < a.R) {
      c = a.ctx_len[r];
      n = a.new_len[r];
      if (c < 0 || n < 0) bad |= CSA2_DEV_BAD_COUNT;
      c = c < 0 ? 0 : c;
      n = n < 0 ? 0 : n;
      if (c + n > 0x7FFFFFFF) {
        bad |= CSA2_DEV_BAD_COUNT;
        n = 0x7FFFFFFF - c;
      }
    }
    int64_t n_total;
    int64_t start = tok0 + block_exclusive(n, s_sums, &n_total);
    if (start + n > a.t_cap) {  // what does not fit the token arrays is cut off
      if (n > 0) bad |= CSA2_DEV_BAD_COUNT;
      n = a.t_cap > start ? a.t_cap - start : 0;
      start = start < a.t_cap ? start : a.t_cap;
    }
    int64_t have = (c + page - 1) >> a.page_log2, want = (c + n + page - 1) >> a.page_log2;
    if (want > a.max_pages) bad |= CSA2_DEV_BAD_COUNT;
    have = have < a.max_pages ? have : a.max_pages;
    want = want < a.max_pages ? want : a.max_pages;
    int64_t need_total;
    const int64_t off = page0 + block_exclusive(want - have, s_sums, &need_total);
    s_start[tid] = start;
    s_page[tid] = off;
    s_ctx[tid] = (int32_t)c;
    s_have[tid] = (int32_t)have;
    const int64_t tok1 = tok0 + n_total < a.t_cap ? tok0 + n_total : a.t_cap;
    const int64_t page1 = page0 + need_total;
    if (tid == kPlanThreads - 1) {
      s_start[kPlanThreads] = tok1;
      s_page[kPlanThreads] = page1;
    }
    // every CTA has read this chunk's inputs: they may be written (also a barrier for s_*)
    if (ranks > 1) cluster_sync_all();
    else __syncthreads();
    const int live = a.R - r0 < kPlanThreads ? a.R - r0 : kPlanThreads;
    if (r < a.R && (unsigned)(tid >> 5) % ranks == rank) {
      a.seq_len[r] = (int32_t)(c + n);
      a.q_start[r] = (int32_t)start;
    }
    // new pages of the chunk: the list's last entries first
    for (int64_t p = page0 + rank * kPlanThreads + tid; p < page1; p += (int64_t)ranks * kPlanThreads) {
      const int i = last_at_most(s_page, live, p);
      int32_t id = -1;
      if (p < n_free) {
        id = a.free_pages[n_free - 1 - p];
        if (id < 0 || id >= a.n_pages) {
          bad |= CSA2_DEV_BAD_INDEX;
          id = -1;
        }
      } else {
        bad |= CSA2_DEV_NO_PAGES;
      }
      a.table[(int64_t)(r0 + i) * a.max_pages + s_have[i] + (p - s_page[i])] = id;
    }
    for (int64_t t = tok0 + rank * kPlanThreads + tid; t < tok1; t += (int64_t)ranks * kPlanThreads) {
      const int i = last_at_most(s_start, live, t);
      const int64_t at = s_ctx[i] + (t - s_start[i]), j = at >> a.page_log2;
      int64_t id = -1;
      if (j < s_have[i]) {
        id = a.table[(int64_t)(r0 + i) * a.max_pages + j];
        if (id < 0 || id >= a.n_pages) {
          bad |= CSA2_DEV_BAD_INDEX;
          id = -1;
        }
      } else if (j < a.max_pages) {
        const int64_t p = s_page[i] + (j - s_have[i]);
        if (p < n_free) {
          id = a.free_pages[n_free - 1 - p];
          if (id >= a.n_pages) id = -1;  // flagged where the page is entered
        }
      }
      a.slot_map[t] = id < 0 ? -1 : (id << a.page_log2) + (at & (page - 1));
      a.pos[t] = at;
    }
    tok0 = tok1;
    page0 = page1;
    __syncthreads();
  }
  for (int64_t t = tok0 + rank * kPlanThreads + tid; t < a.t_cap; t += (int64_t)ranks * kPlanThreads) {
    a.slot_map[t] = -1;
    a.pos[t] = -1;
  }
  if (ranks > 1) cluster_sync_all();  // n_free is read by every CTA before it may change
  if (rank == 0 && tid == 0) {
    a.q_start[a.R] = (int32_t)tok0;
    *a.n_free_out = (int32_t)(n_free > page0 ? n_free - page0 : 0);
  }
  if (bad) flag(a.status, bad);
}

cudaError_t launch_paged_plan(const int32_t* ctx_len, const int32_t* new_len, int R, int page, int32_t* table,
                              int max_pages, const int32_t* free_pages, int64_t free_cap, const int32_t* n_free,
                              int64_t n_pages, int32_t* seq_len, int32_t* n_free_out, int32_t* q_start,
                              int64_t* slot_map, int64_t* pos, int64_t t_cap, uint32_t* status,
                              cudaStream_t stream) {
  PlanArgs a{ctx_len, new_len, R, log2_of(page), table, max_pages, free_pages, free_cap, n_free, n_pages,
             seq_len, n_free_out, q_start, slot_map, pos, t_cap, status};
  // one CTA or a cluster of eight: 4.3 against 4.7 us at 1,224 rows, 5.8 against 4.8 at 3,815, 14.0
  // against 6.0 at 14,169
  const unsigned ranks = t_cap > 2 * kPlanThreads ? 8 : 1;
  cudaError_t e = launch_chained(paged_plan_kernel, dim3(ranks), dim3(kPlanThreads), 0, stream, ranks, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------------------------------
// Release.  Every CTA scans the rows' page counts; the pages, laid end to end, are shared out
// over the cluster's warps and read, 32 loads per lane in flight; when all are valid, each is
// written at its place.  Only when one is not, valid pages are counted row by row instead.
// ------------------------------------------------------------------------------------
struct ReleaseArgs {
  const int32_t* seq_len;
  const int32_t* table;
  const uint8_t* release;
  int R, page_log2, max_pages;
  int32_t* free_pages;
  int64_t free_cap;
  const int32_t* n_free;
  int64_t n_pages;
  int32_t* seq_len_out;
  int32_t* n_free_out;
  uint32_t* status;
};

constexpr int kMaxRanks = 8;

__global__ void __launch_bounds__(kPlanThreads) paged_release_kernel(ReleaseArgs a) {
  __shared__ int64_t s_sums[32];
  __shared__ int32_t s_count[kPlanThreads];
  __shared__ int32_t s_first[kPlanThreads];  // first page of each row, counted from the chunk's first
  __shared__ int64_t s_at[kPlanThreads];     // place of each row's first valid page in the list
  __shared__ int32_t s_rows[kPlanThreads];  // pages of each released row of the chunk, else 0
  __shared__ uint32_t s_bad[2][kMaxRanks];  // by chunk parity: a rank may be a chunk ahead of another's reads
  chain_enter();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const unsigned rank = blockIdx.x, ranks = gridDim.x;  // one cluster
  // a peer's shared memory may be written only when the peer has started: each says so here, and
  // the wait stands before the first store into a peer, behind the scan and the page loads
  if (ranks > 1) tc::cluster_arrive();
  const int page = 1 << a.page_log2;
  uint32_t bad = 0;
  int64_t n_free = *a.n_free;
  if (n_free < 0 || n_free > a.free_cap) {
    bad |= CSA2_DEV_BAD_COUNT;
    n_free = n_free < 0 ? 0 : a.free_cap;
  }
  int64_t pushed = 0;
  for (int r0 = 0; r0 < a.R; r0 += kPlanThreads) {
    const int r = r0 + tid;
    bool gone = false;
    int32_t len = 0;
    int64_t rows = 0;
    if (r < a.R) {
      len = a.seq_len[r];
      gone = a.release[r] != 0;
      if (gone) {
        if (len < 0) bad |= CSA2_DEV_BAD_COUNT;
        rows = len < 0 ? 0 : ((int64_t)len + page - 1) >> a.page_log2;
        if (rows > a.max_pages) {
          bad |= CSA2_DEV_BAD_COUNT;
          rows = a.max_pages;
        }
      }
    }
    s_rows[tid] = (int32_t)rows;
    int64_t total;
    const int64_t before = block_exclusive(rows, s_sums, &total);
    s_first[tid] = (int32_t)before;  // used when the chunk's pages count in 32 bits
    __syncthreads();
    const int live = a.R - r0 < kPlanThreads ? a.R - r0 : kPlanThreads;
    // a warp takes consecutive pages
    const bool fits = total <= INT32_MAX - (1 << 16);
    const int warps = ranks * kPlanWarps;
    const int each = fits ? (((int)total + warps - 1) / warps + 31) & ~31 : 0;
    const int p_beg = (int)(rank * kPlanWarps + warp) * each;
    const int p_end = !fits ? p_beg : p_beg + each < (int)total ? p_beg + each : (int)total;
    // a batch of the warp's pages from p on, kBatch per lane: their loads are all in flight
    constexpr int kBatch = 32;
    int32_t id[kBatch];
    const auto read = [&](int p) {
      int i = last_at_most(s_first, live, p), until;
      const int32_t* row;  // where position 0 would be if the list were this row's
      const auto open = [&] {
        row = a.table + (int64_t)(r0 + i) * a.max_pages - s_first[i];
        until = i + 1 < live ? s_first[i + 1] : INT32_MAX;
      };
      open();
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        if (x % 8 == 0 && p + x * 32 >= p_end) break;  // the same for the whole warp
        const int q = p + x * 32 + lane;
        if (q < p_end) {
          while (q >= until) {
            ++i;
            open();
          }
          id[x] = row[q];
        }
      }
    };
    bool all = true;
    for (int p = p_beg; p < p_end; p += kBatch * 32) {
      read(p);
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        if (x % 8 == 0 && p + x * 32 >= p_end) break;
        all &= p + x * 32 + lane >= p_end || (id[x] >= 0 && id[x] < a.n_pages);
      }
    }
    uint32_t some = __syncthreads_or(!all);
    if (ranks > 1) {
      if (r0 == 0) tc::cluster_wait();  // every peer has started (a cluster has requests: it is chosen by their number)
      if (tid < ranks) {
        const uint32_t at = tc::mapa(tc::smem_u32(&s_bad[r0 / kPlanThreads & 1][rank]), tid);
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(some) : "memory");
      }
      cluster_sync_all();  // also: this chunk's inputs are read everywhere
      some = 0;
      for (unsigned k = 0; k < ranks; ++k) some |= s_bad[r0 / kPlanThreads & 1][k];
    }
    if (!some && fits) {
      int32_t* to = a.free_pages + n_free + pushed;
      const int64_t room = a.free_cap - n_free - pushed;
      for (int p = p_beg; p < p_end; p += kBatch * 32) {
        if (p_beg + kBatch * 32 < p_end) read(p);  // one batch is still there
#pragma unroll
        for (int x = 0; x < kBatch; ++x) {
          if (x % 8 == 0 && p + x * 32 >= p_end) break;
          const int q = p + x * 32 + lane;
          if (q < p_end && q < room) to[q] = id[x];
        }
      }
    } else {  // the valid pages of each row, counted by one warp for every CTA
      __syncthreads();
      s_count[tid] = 0;
      if (ranks > 1) cluster_sync_all();
      else __syncthreads();
      for (int i = rank * kPlanWarps + warp; i < live; i += ranks * kPlanWarps) {
        const int m = s_rows[i];
        if (m == 0) continue;
        const int32_t* row = a.table + (int64_t)(r0 + i) * a.max_pages;
        int cnt = 0;
        for (int j = lane; j < m; j += 32) {
          const int32_t id = row[j];
          cnt += id >= 0 && id < a.n_pages;
        }
        cnt = __reduce_add_sync(0xffffffffu, cnt);
        if (cnt != m) bad |= CSA2_DEV_BAD_INDEX;
        if (lane < ranks) {
          if (ranks > 1) {
            const uint32_t at = tc::mapa(tc::smem_u32(&s_count[i]), lane);
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"(cnt) : "memory");
          } else {
            s_count[i] = cnt;
          }
        }
      }
      if (ranks > 1) cluster_sync_all();
      else __syncthreads();
      s_at[tid] = n_free + pushed + block_exclusive(s_count[tid], s_sums, &total);
      __syncthreads();
      for (int i = rank * kPlanWarps + warp; i < live; i += ranks * kPlanWarps) {
        const int m = s_rows[i];
        const int32_t* row = a.table + (int64_t)(r0 + i) * a.max_pages;
        int64_t at = s_at[i];
        for (int j0 = 0; j0 < m; j0 += 32) {
          const int j = j0 + lane;
          const int32_t id = j < m ? row[j] : -1;
          const bool ok = id >= 0 && id < a.n_pages;
          const unsigned mask = __ballot_sync(0xffffffffu, ok);
          const int64_t to = at + __popc(mask & ((1u << lane) - 1u));
          if (ok && to < a.free_cap) a.free_pages[to] = id;
          at += __popc(mask);
        }
      }
    }
    if (r < a.R && (unsigned)warp % ranks == rank) a.seq_len_out[r] = gone ? 0 : len;
    pushed += total;
    __syncthreads();
  }
  if (ranks > 1) cluster_sync_all();
  if (rank == 0 && tid == 0) {
    int64_t n = n_free + pushed;
    if (n > a.free_cap) {
      bad |= CSA2_DEV_BAD_COUNT;
      n = a.free_cap;
    }
    *a.n_free_out = (int32_t)n;
  }
  if (bad) flag(a.status, bad);
}

cudaError_t launch_paged_release(const int32_t* seq_len, const int32_t* table, const uint8_t* release, int R,
                                 int page, int max_pages, int32_t* free_pages, int64_t free_cap,
                                 const int32_t* n_free, int64_t n_pages, int32_t* seq_len_out, int32_t* n_free_out,
                                 uint32_t* status, cudaStream_t stream) {
  ReleaseArgs a{seq_len, table, release, R, log2_of(page), max_pages, free_pages, free_cap, n_free, n_pages,
                seq_len_out, n_free_out, status};
  // by what may be released: 4.8 against 5.9 us at 4K pages of 16K entries, 8.0 against 6.2 at 16K of 64K
  const unsigned ranks = (int64_t)R * max_pages > 16 * kPlanThreads ? kMaxRanks : 1;
  cudaError_t e = launch_chained(paged_release_kernel, dim3(ranks), dim3(kPlanThreads), 0, stream, ranks, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------------------------------------------
// Append.  A unit is (page touched by the call, head, K or V): GW = page / 16 warps, 16 page
// rows per warp, a lane 8 channels of a row (16 bytes), so a warp's loads of new rows are
// whole 128 to 256 byte rows and all of them are in registers between the amax and the
// encoding: one pass over the input.  Pages are found from the slot map alone: a token leads
// a unit when the token before it lies in another page.  A unit walks the leaders of `win`
// consecutive tokens.  Measured: single tokens of 32 sequences and 8 heads 4.9 us per call, 9.5K
// rows of a fused projection 12.75 us (4.6 TB/s of 58.6 MB; HBM's floor is 8.9).  Finding the
// leaders by ballot, packed 16-bit maxima and 64 registers (twice the warps) brought 33 -> 17,
// one branch instead of a select between the two divisions 17 -> 12.
// ------------------------------------------------------------------------------------
struct AppendArgs {
  const uint8_t* x[2];  // keys, values (16-bit elements)
  int64_t stride[2];    // bytes from token to token
  uint8_t* cache[2];
  float* scale[2];
  const int64_t* slot;
  int64_t T, n_pages;
  int Hk, win;
  uint32_t* status;
};

// The smallest power of two s >= 2^-64 with amax <= 448 s.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - ((b & 0x7FFFFFu) <= 0x600000u ? 8 : 7);  // 448 = 1.75 * 2^8
  return __uint_as_float((uint32_t)(e < 63 ? 63 : e) << 23);
}

__device__ __forceinline__ uint2 encode8(const float (&y)[8]) {
  return make_uint2(e4m3x2_sat(y[0], y[1]) | (e4m3x2_sat(y[2], y[3]) << 16),
                    e4m3x2_sat(y[4], y[5]) | (e4m3x2_sat(y[6], y[7]) << 16));
}

template <typename T>
struct PairOf;
template <>
struct PairOf<__nv_bfloat16> { using type = __nv_bfloat162; };
template <>
struct PairOf<__half> { using type = __half2; };
template <typename T>
using Pair = typename PairOf<T>::type;
template <typename T>
__device__ __forceinline__ Pair<T> zero_pair() {
  Pair<T> z;
  *reinterpret_cast<uint32_t*>(&z) = 0;
  return z;
}
__device__ __forceinline__ float larger(__nv_bfloat162 v) { return fmaxf(__low2float(v), __high2float(v)); }
__device__ __forceinline__ float larger(__half2 v) { return fmaxf(__low2float(v), __high2float(v)); }

template <int HD, typename T, int GW>
__global__ void __launch_bounds__(256, 4) kv8_append_kernel(AppendArgs a) {
  constexpr int kPage = GW * 16, kUnits = 8 / GW;
  constexpr int kLanes = HD / 8;         // lanes per row
  constexpr int kRowsAt = 32 / kLanes;   // rows per warp load
  constexpr int kLoads = 16 / kRowsAt;
  __shared__ float s_amax[8];
  chain_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int unit = warp / GW, g = warp % GW;
  const int64_t u = (int64_t)blockIdx.x * kUnits + unit;
  const int h = (int)(u % a.Hk);
  const int kv = blockIdx.y;
  const uint8_t* x_all = kv ? a.x[1] : a.x[0];
  const int64_t stride = kv ? a.stride[1] : a.stride[0];
  uint8_t* cache = kv ? a.cache[1] : a.cache[0];
  float* scale = kv ? a.scale[1] : a.scale[0];
  const int64_t w0 = u / a.Hk * a.win;
  const int64_t w1 = w0 + a.win < a.T ? w0 + a.win : a.T;
  const int64_t n_slots = a.n_pages * kPage;
  uint32_t bad = 0;
  for (int64_t t0 = w0; t0 < w1; t0 += 32) {  // the same for every warp of the unit
    int64_t slots = -1;
    bool first = false;  // this lane's token is the first of its page
    bool behind = false;  // it is, and what is in front of it is skipped
    if (t0 + lane < w1) {
      slots = a.slot[t0 + lane];
      const int64_t prev = t0 + lane > 0 ? a.slot[t0 + lane - 1] : -1;
      if (slots < 0 || slots >= n_slots) {
        if (slots != -1) bad = CSA2_DEV_BAD_INDEX;
      } else if (prev >= 0 && prev < n_slots && prev / kPage == slots / kPage) {
        if (prev + 1 != slots) bad = CSA2_DEV_BAD_INDEX;
      } else {
        first = true;
        behind = (prev < 0 || prev >= n_slots) && t0 + lane > 0;
      }
    }
    unsigned firsts = __ballot_sync(0xffffffffu, first);
    // Skipped rows inside a page would give it two units, which would write its scale and rows at the
    // same time: the nearest row in front that has a slot, however far, must lie in another page.
    for (unsigned todo = __ballot_sync(0xffffffffu, behind); todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      for (int64_t at = t0 + from - 2; at >= 0; at -= 32) {
        const int64_t before = at >= lane ? a.slot[at - lane] : -1;
        const unsigned valid = __ballot_sync(0xffffffffu, before >= 0 && before < n_slots);
        if (valid) {
          if (__shfl_sync(0xffffffffu, before, __ffs(valid) - 1) / kPage == __shfl_sync(0xffffffffu, slots, from) / kPage) {
            bad = CSA2_DEV_BAD_INDEX;
            firsts &= ~(1u << from);
          }
          break;
        }
      }
    }
    for (unsigned todo = firsts; todo; todo &= todo - 1) {
      const int from = __ffs(todo) - 1;
      const int64_t t = t0 + from, slot = __shfl_sync(0xffffffffu, slots, from);
      const int64_t pid = slot / kPage;
      const int off = (int)(slot % kPage);
      int n = 1;  // tokens of this page: consecutive slots
      {
        const int most = kPage - off;
#pragma unroll
        for (int i0 = 0; i0 < kPage; i0 += 32) {
          const int i = i0 + lane;
          const bool in = i < most && t + i < a.T && a.slot[t + i] == slot + i;
          const unsigned m = __ballot_sync(0xffffffffu, in);
          if (n >= i0) n = i0 + (m == 0xffffffffu ? 32 : __ffs(~m) - 1);
          if (m != 0xffffffffu) break;
        }
      }
      float* sp = scale + pid * a.Hk + h;
      const float s_old = off > 0 ? *sp : 0.0f;
      const uint8_t* x0 = x_all + t * stride + (int64_t)h * (HD * 2) + (lane % kLanes) * 16;
      uint4 raw[kLoads];
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const int i = g * 16 + k * kRowsAt + lane / kLanes - off;  // token of the run
        raw[k] = make_uint4(0u, 0u, 0u, 0u);
        if (i >= 0 && i < n) raw[k] = __ldcs(reinterpret_cast<const uint4*>(x0 + i * stride));
      }
      Pair<T> top = zero_pair<T>();  // largest magnitudes so far; NaN counts for nothing
#pragma unroll
      for (int k = 0; k < kLoads; ++k) {
        const uint32_t v[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) top = __hmax2(top, __habs2(*reinterpret_cast<const Pair<T>*>(&v[i])));
      }
      float amax = larger(top);
      amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));  // >= 0: ordered as integers
      if (GW > 1) {
        if (lane == 0) s_amax[warp] = amax;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + unit), "n"(GW * 32) : "memory");
#pragma unroll
        for (int i = 0; i < GW; ++i) amax = fmaxf(amax, s_amax[unit * GW + i]);
      }
      const float s = fmaxf(block_scale(amax), s_old);
      const bool pow2 = (__float_as_uint(s) & 0x7FFFFFu) == 0;
      uint8_t* c0 = cache + (pid * a.Hk + h) * (int64_t)(kPage * HD) + (lane % kLanes) * 8;
      if (off > 0 && s != s_old) {  // earlier rows under the larger scale
        const float ratio = __fdiv_rn(s_old, s);
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int row = g * 16 + k * kRowsAt + lane / kLanes;
          if (row < off) {
            uint2* p = reinterpret_cast<uint2*>(c0 + row * HD);
            const uint2 c = *p;
            float x[8];
            e4m3x4_f32(c.x, x);
            e4m3x4_f32(c.y, x + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= ratio;
            *p = encode8(x);
          }
        }
      }
      // a power of two (every scale this call chooses) divides exactly by its reciprocal; a page's
      // earlier scale may be any fp32
      const auto store = [&](auto over) {
#pragma unroll
        for (int k = 0; k < kLoads; ++k) {
          const int row = g * 16 + k * kRowsAt + lane / kLanes;
          if (row >= off && row < off + n) {
            float x[8];
            unpack8<T>(raw[k], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = over(x[i]);
            *reinterpret_cast<uint2*>(c0 + row * HD) = encode8(x);
          }
        }
      };
      if (pow2) {
        const float inv = __fdiv_rn(1.0f, s);
        store([&](float x) { return x * inv; });
      } else {
        store([&](float x) { return __fdiv_rn(x, s); });
      }
      if (g == 0 && lane == 0) *sp = s;
      if (GW > 1)  // s_amax is free again
        asm volatile("bar.sync %0, %1;" ::"r"(1 + unit), "n"(GW * 32) : "memory");
    }
  }
  if (bad && h == 0 && kv == 0 && g == 0) flag(a.status, bad);
}

template <int HD, typename T>
static cudaError_t launch_append_t(const AppendArgs& a, int page, unsigned blocks, cudaStream_t stream) {
  const dim3 grid(blocks, 2), block(256);
  switch (page) {
    case 16: return launch_chained(kv8_append_kernel<HD, T, 1>, grid, block, 0, stream, 0, a);
    case 32: return launch_chained(kv8_append_kernel<HD, T, 2>, grid, block, 0, stream, 0, a);
    case 64: return launch_chained(kv8_append_kernel<HD, T, 4>, grid, block, 0, stream, 0, a);
    default: return launch_chained(kv8_append_kernel<HD, T, 8>, grid, block, 0, stream, 0, a);
  }
}

cudaError_t launch_kv8_append(const void* k, const void* v, int64_t k_stride, int64_t v_stride, int f16, int64_t T,
                              int Hk, int hd, const int64_t* slot, uint8_t* k_cache, uint8_t* v_cache, float* k_scale,
                              float* v_scale, int64_t n_pages, int page, uint32_t* status, cudaStream_t stream,
                              int num_sms) {
  AppendArgs a;
  a.x[0] = static_cast<const uint8_t*>(k);
  a.x[1] = static_cast<const uint8_t*>(v);
  a.stride[0] = k_stride * 2;
  a.stride[1] = v_stride * 2;
  a.cache[0] = k_cache;
  a.cache[1] = v_cache;
  a.scale[0] = k_scale;
  a.scale[1] = v_scale;
  a.slot = slot;
  a.T = T;
  a.n_pages = n_pages;
  a.Hk = Hk;
  a.status = status;
  const int gw = page / 16, units = 8 / gw;
  // tokens per unit: one while the units' warps fit the GPU at once (a unit then has one page
  // at most), more beyond that, up to a page (most units of a long chunk then have one or two)
  int64_t win = (T * Hk * 2 * gw + (int64_t)num_sms * 64 - 1) / ((int64_t)num_sms * 64);
  win = win < 1 ? 1 : (win > page ? page : win);
  a.win = (int)win;
  const int64_t n_units = (T + win - 1) / win * Hk;
  const unsigned blocks = (unsigned)((n_units + units - 1) / units);
  cudaError_t e;
  if (hd == 64)
    e = f16 ? launch_append_t<64, __half>(a, page, blocks, stream)
            : launch_append_t<64, __nv_bfloat16>(a, page, blocks, stream);
  else
    e = f16 ? launch_append_t<128, __half>(a, page, blocks, stream)
            : launch_append_t<128, __nv_bfloat16>(a, page, blocks, stream);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace csa2
