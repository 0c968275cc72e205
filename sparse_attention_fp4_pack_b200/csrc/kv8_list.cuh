// What the attention kernels of the paged 8-bit KV cache share: their arguments, the list of key
// tiles that the CTAs split evenly, bounded waits, and the kernel that joins split items.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "csa2_device.cuh"
#include "kv8.cuh"
#include "tc.cuh"

namespace csa2 {

constexpr int kKeys = 128;             // keys per tile
constexpr int kMaxTilePages = 8;       // pages of 16 rows
constexpr float kSlack = 2.0f;         // the running maximum is raised when exceeded by more (base 2)
constexpr uint32_t kKvPolls = 1u << 22;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct KvAttnArgs {
  const uint8_t* q;
  int64_t q_stride;  // bytes from token to token
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* q_start;
  const int32_t* seq_len;
  int R, Hq, Hk, max_pages, page_log2;
  int64_t n_pages;
  int64_t T;
  float sm_scale;
  int window;
  float softcap;
  uint8_t* out;
  float* lse;
  float* part;    // [CTA][2][NC][hd + 2]
  int32_t* meta;  // [CTA][8]
  uint32_t* status;
};

// Partial results of CTA c, each an output over the piece's own sum, its maximum and its sum: slot 0
// the piece that continues an item, slot 1 the one that starts an item and does not end it.  meta:
// [0] slot 1 is used; then [1] the CTA whose slot 0 ends the item, [2] key head * head blocks + head
// block, [3] query block, [4] first row and [5] number of queries of the request.
constexpr int kMetaInts = 8;

// Rows of hd bytes from `row` on (a box of the map) into shared memory.
__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int row, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
          dst),
      "l"(map), "r"(0), "r"(row), "r"(bar)
      : "memory");
}
// Bounded wait that also ends when another role of the CTA has given up (*abort != 0).
__device__ __forceinline__ bool kv_wait(int* abort, uint64_t& bar, uint32_t parity) {
  const uint32_t b = tc::smem_u32(&bar);
  uint64_t t0 = 0;
  for (uint32_t i = 0; i < kKvPolls; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(b), "r"(parity)
        : "memory");
    if (ok) return true;
    if ((i & 63u) == 63u) {
      if (*reinterpret_cast<volatile int*>(abort)) return false;
      const uint64_t now = tc::globaltimer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > tc::kWaitLimitNs) break;
    }
  }
  *reinterpret_cast<volatile int*>(abort) = 1;
  return false;
}

// Lane 0's value, known to be the same in the whole warp.
template <typename T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }

// Products and their completion, issued by the lane where `on` holds.  The whole warp runs the
// issuing loop: descriptors then stay in uniform registers, where a lone thread's would be
// moved there one by one before every product.
__device__ __forceinline__ void mma_ss(bool on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)on));
}
__device__ __forceinline__ void mma_ts(bool on, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)on));
}
__device__ __forceinline__ void mma_f8(bool on, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate), "r"((uint32_t)on));
}
__device__ __forceinline__ void commit_if(bool on, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"((uint32_t)on)
      : "memory");
}
// kv_wait of a whole warp.
template <class Sh>
__device__ __forceinline__ bool kv_wait_all(Sh& sh, uint64_t& bar, uint32_t parity) {
  return __all_sync(0xffffffffu, kv_wait(&sh.abort, bar, parity));
}
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh by an odd polynomial near zero and by the exponential beyond.  Up to kTanhSmall x + x^3 q(x^2)
// with q fitted at Chebyshev points: relative error 2^-26 and the roundings of its steps.  Beyond,
// 1 - 2 / (1 + e^2x): an absolute error near 2^-22, which would be a relative 2^-17 of a score of a
// thirtieth of the cap.
constexpr float kTanhSmall = 0.625f;
constexpr float kTanh1 = -0.3333326280117035f, kTanh2 = 0.13331149518489838f, kTanh3 = -0.05372267961502075f,
                kTanh4 = 0.020595679059624672f, kTanh5 = -0.005664775148034096f;
__device__ __forceinline__ float tanh_small(float x) {
  const float z = x * x;
  const float q = fmaf(fmaf(fmaf(fmaf(kTanh5, z, kTanh4), z, kTanh3), z, kTanh2), z, kTanh1);
  return fmaf(x * z, q, x);
}
__device__ __forceinline__ float tanh_large(float x) {
  const float y = x * (2.0f * kLog2e);
  return 1.0f - __fdividef(2.0f, 1.0f + exp2_approx(y > 126.0f ? 126.0f : y));  // NaN stays NaN
}
__device__ __forceinline__ float tanh_any(float x) {
  const float small = tanh_small(x), large = tanh_large(x);
  return fabsf(x) <= kTanhSmall ? small : large;
}

// The least power of two that is not below a positive normal x, and its exponent.
__device__ __forceinline__ int pow2_above_exp(float x) {
  const uint32_t b = __float_as_uint(x);
  return (int)(b >> 23) - 127 + ((b & 0x7FFFFFu) != 0);
}
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }  // -126 <= e <= 127
__device__ __forceinline__ float pow2_inverse(float x) { return __uint_as_float(0x7F000000u - __float_as_uint(x)); }
// What value scales count as at least (csa2_kv8_append goes no lower), and log2 of it.
constexpr float kLeastScale = 5.421010862427522e-20f;
constexpr int kLeastExp = -64;

template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ __half from_float<__half>(float x) { return __float2half_rn(x); }

// ---- the list of key tiles -------------------------------------------------------------
struct Request {
  int q0, n;     // first query row, queries
  int pos0;      // position of the first query
  int cap;       // keys: min(seq_len, what the table holds)
  int nqb;       // query blocks
};
struct Shape {   // how a request's columns are cut
  int G, QB, HB, nhb;
};
template <int NC>
__device__ __forceinline__ Shape shape_of(const KvAttnArgs& a) {
  Shape s;
  s.G = a.Hq / a.Hk;
  s.HB = s.G < NC ? s.G : NC;
  s.QB = s.G < NC ? NC / s.G : 1;
  s.nhb = (s.G + NC - 1) / NC;
  return s;
}
__device__ __forceinline__ Request request_of(const KvAttnArgs& a, const Shape& s, int r, uint32_t* bad) {
  Request x;
  const int64_t b = a.q_start[r], e = a.q_start[r + 1];
  int len = a.seq_len[r];
  const int64_t q0 = b < 0 ? 0 : (b < a.T ? b : a.T), q1 = e < q0 ? q0 : (e < a.T ? e : a.T);
  if (q0 != b || q1 != e || len < 0) *bad |= CSA2_DEV_BAD_COUNT;
  if (len < 0) len = 0;
  x.q0 = (int)q0;
  x.n = (int)(q1 - q0);
  if (x.n > len) *bad |= CSA2_DEV_BAD_COUNT;
  x.pos0 = len - x.n;
  const int64_t held = (int64_t)a.max_pages << a.page_log2;
  if (len > held) *bad |= CSA2_DEV_BAD_COUNT;
  x.cap = len < held ? len : (int)held;
  x.nqb = (x.n + s.QB - 1) / s.QB;
  return x;
}
// Keys [lo, hi) that any query of block qb sees, and its first tile and number of tiles (at
// least one: a block that sees nothing still writes its rows).
struct Range {
  int lo, hi, tile, tiles;
};
__device__ __forceinline__ Range range_of(const KvAttnArgs& a, const Shape& s, const Request& x, int qb) {
  Range g;
  const int i0 = qb * s.QB, i1 = i0 + s.QB < x.n ? i0 + s.QB : x.n;
  const int64_t hi = (int64_t)x.pos0 + i1;
  g.hi = hi < 0 ? 0 : (hi < x.cap ? (int)hi : x.cap);
  const int64_t lo = a.window > 0 ? (int64_t)x.pos0 + i0 + 1 - a.window : 0;
  g.lo = lo < 0 ? 0 : (lo < g.hi ? (int)lo : g.hi);
  g.tile = g.lo / kKeys;
  const int end = (g.hi + kKeys - 1) / kKeys;
  g.tiles = end > g.tile ? end - g.tile : 1;
  return g;
}
// Tiles of one (request, key head, head block).
__device__ __forceinline__ int64_t row_tiles(const KvAttnArgs& a, const Shape& s, const Request& x, int first, int step) {
  int64_t n = 0;
  for (int qb = first; qb < x.nqb; qb += step) n += range_of(a, s, x, qb).tiles;
  return n;
}
__device__ __forceinline__ int64_t warp_sum(int64_t v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// row_tiles of request r for each lane (r < R where live), long requests by the whole warp.
__device__ __forceinline__ int64_t lane_row_tiles(const KvAttnArgs& a, const Shape& s, int r, bool live, int lane,
                                                  uint32_t* bad) {
  Request x = {};
  if (live) x = request_of(a, s, r, bad);
  const bool big = x.nqb > 8;
  int64_t n = big ? 0 : row_tiles(a, s, x, 0, 1);
  unsigned todo = __ballot_sync(0xffffffffu, big);
  while (todo) {
    const int src = __ffs(todo) - 1;
    todo &= todo - 1;
    Request y;
    y.q0 = __shfl_sync(0xffffffffu, x.q0, src);
    y.n = __shfl_sync(0xffffffffu, x.n, src);
    y.pos0 = __shfl_sync(0xffffffffu, x.pos0, src);
    y.cap = __shfl_sync(0xffffffffu, x.cap, src);
    y.nqb = __shfl_sync(0xffffffffu, x.nqb, src);
    const int64_t m = warp_sum(row_tiles(a, s, y, lane, 32));
    if (lane == src) n = m;
  }
  return n;
}

// This CTA's share of the list: its length, and where it begins.
struct Share {
  int64_t left;
  int64_t t0, total;   // first tile of the share, tiles of the list
  int r, hh, qb, off;  // request, key head * nhb + head block, query block, tile inside the item
};

// A walk over a share's pieces; every role keeps its own.
struct Walk {
  int64_t left;
  int r, hh, qb, off;
  Request x;
  Range g;
  int take;        // tiles of this piece
  bool first, last;
  __device__ __forceinline__ void open(const KvAttnArgs& a, const Shape& s) {
    g = range_of(a, s, x, qb);
    const int rest = g.tiles - off;
    take = left < rest ? (int)left : rest;
    first = off == 0;
    last = off + take == g.tiles;
  }
  __device__ __forceinline__ void start(const KvAttnArgs& a, const Shape& s, const Share& w) {
    left = w.left;
    r = w.r;
    hh = w.hh;
    qb = w.qb;
    off = w.off;
    if (left <= 0) return;
    uint32_t bad = 0;
    x = request_of(a, s, r, &bad);
    open(a, s);
  }
  __device__ __forceinline__ void next(const KvAttnArgs& a, const Shape& s) {
    left -= take;
    off = 0;
    if (left <= 0) return;
    if (++qb < x.nqb) {
      open(a, s);
      return;
    }
    qb = 0;
    if (++hh < a.Hk * s.nhb) {
      open(a, s);
      return;
    }
    hh = 0;
    uint32_t bad = 0;
    do {
      if (++r >= a.R) {  // cannot happen while left > 0
        left = 0;
        return;
      }
      x = request_of(a, s, r, &bad);
    } while (x.n == 0);
    open(a, s);
  }
};

// a / b of nonnegative numbers, which mostly fit 32 bits (64-bit divisions take far longer).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// Sum of the lanes' values up to and including this one's.
__device__ __forceinline__ int64_t warp_upto(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

// First tile of CTA c's share.  With fewer tiles than CTAs the first CTAs take one each, so the
// pieces of an item are always neighbours.
__device__ __forceinline__ int64_t share_ctas(int64_t total) { return total < gridDim.x ? total : gridDim.x; }
__device__ __forceinline__ int64_t share_start(int64_t total, int64_t c) {
  const int64_t C = share_ctas(total);
  return c < C ? quotient(total * c, C) : total;  // at most 2^31 items of 2^23 tiles: below 2^63
}
// Notes the item that this CTA starts with `w` and does not end.
__device__ __forceinline__ void note_item(const KvAttnArgs& a, const Share& share, const Walk& w) {
  const int64_t last = share_start(share.total, blockIdx.x + 1) + (w.g.tiles - w.off - w.take) - 1;  // its last tile
  // the largest c with total * c / C <= last
  const int c = (int)quotient((last + 1) * share_ctas(share.total) - 1, share.total);
  int32_t* meta = a.meta + (int64_t)blockIdx.x * kMetaInts;
  meta[0] = 1;
  meta[1] = c;
  meta[2] = w.hh;
  meta[3] = w.qb;
  meta[4] = w.x.q0;
  meta[5] = w.x.n;
}

// Computed by the whole CTA (kThreads threads); `sums` holds a value per warp.
template <int kThreads>
__device__ void find_share(const KvAttnArgs& a, const Shape& s, int64_t* sums, Share* out, uint32_t* bad) {
  constexpr int kWarps = kThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.R + kThreads - 1) / kThreads;  // requests per thread, consecutive
  const int heads = a.Hk * s.nhb;
  int64_t mine = 0;
  for (int i = 0; i < per; ++i) {
    const int r = tid * per + i;
    mine += lane_row_tiles(a, s, r, r < a.R, lane, bad);
  }
  mine *= heads;
  int64_t upto = warp_upto(mine, lane);
  if (lane == 31) sums[warp] = upto;
  __syncthreads();
  const int64_t of_warps = warp_upto(lane < kWarps ? sums[lane] : 0, lane);
  const int64_t total = __shfl_sync(0xffffffffu, of_warps, kWarps - 1);
  const int64_t warps_before = __shfl_sync(0xffffffffu, of_warps, warp > 0 ? warp - 1 : 0);
  if (warp > 0) upto += warps_before;
  const int64_t t0 = share_start(total, blockIdx.x), left = share_start(total, blockIdx.x + 1) - t0;
  if (tid == 0) {
    out->left = left;
    out->t0 = t0;
    out->total = total;
  }
  // the thread whose requests hold tile t0: its warp finds the request (32 at a time) ...
  const unsigned holder = __ballot_sync(0xffffffffu, left > 0 && upto - mine <= t0 && t0 < upto);
  if (holder) {
    const int src = __ffs(holder) - 1;
    int64_t rest = t0 - __shfl_sync(0xffffffffu, upto - mine, src), row = __shfl_sync(0xffffffffu, mine, src);
    int r = (warp * 32 + src) * per;
    if (per > 1) {
      for (;;) {
        const int64_t n = lane_row_tiles(a, s, r + lane, r + lane < a.R, lane, bad) * heads, in = warp_upto(n, lane);
        const unsigned hit = __ballot_sync(0xffffffffu, in > rest);
        if (hit) {
          const int l = __ffs(hit) - 1;
          rest -= __shfl_sync(0xffffffffu, in - n, l);
          row = __shfl_sync(0xffffffffu, n, l);
          r += l;
          break;
        }
        rest -= __shfl_sync(0xffffffffu, in, 31);
        r += 32;
      }
    }
    row = quotient(row, heads);
    const Request x = request_of(a, s, r, bad);
    const int hh = (int)quotient(rest, row);
    rest -= (int64_t)hh * row;
    // ... and the query block
    int qb = 0;
    while (x.nqb > 1) {
      const int64_t n = qb + lane < x.nqb ? range_of(a, s, x, qb + lane).tiles : 0, in = warp_upto(n, lane);
      const unsigned hit = __ballot_sync(0xffffffffu, in > rest);
      if (hit) {
        const int l = __ffs(hit) - 1;
        rest -= __shfl_sync(0xffffffffu, in - n, l);
        qb += l;
        break;
      }
      rest -= __shfl_sync(0xffffffffu, in, 31);
      qb += 32;
      if (qb >= x.nqb) break;  // cannot happen
    }
    if (lane == 0) {
      out->r = r;
      out->hh = hh;
      out->qb = qb;
      out->off = (int)rest;
    }
  }
  __syncthreads();
}

// Joins the pieces of the item that CTA blockIdx.x starts and does not end.  A piece left its own
// output O (over its own sum l, so it is of the values' size whatever their scales), its maximum m
// and l: with M the largest m and w = 2^(m - M) l, out = sum w O / sum w.  A warp joins one column:
// its lanes first hold the statistics of 32 pieces, then 4 (2 of 64) channels each, so the loads of
// all pieces are independent.
constexpr int kMergeThreads = 256;  // 8 columns
// 2^24 keys of at most 2^10 (the larger of the kernels' slacks) sum up to 2^34: with 2^-34 the weighted
// values stay in fp32 up to its largest, and the smallest (2^-73, a scale of 2^-64) normal.
constexpr float kMergeShift = 34.0f;

template <int NC, int HD, typename T>
__global__ void __launch_bounds__(kMergeThreads) kv8_merge_kernel(const KvAttnArgs a) {
  constexpr int kPart = NC * (HD + 2), kPer = HD / 32;
  using Vec = std::conditional_t<kPer == 4, float4, float2>;
  chain_enter();
  const int cta = blockIdx.x, lane = threadIdx.x & 31, c = blockIdx.y * 8 + (threadIdx.x >> 5);
  const int4 m0 = *reinterpret_cast<const int4*>(a.meta + (int64_t)cta * kMetaInts);
  const int2 m1 = *reinterpret_cast<const int2*>(a.meta + (int64_t)cta * kMetaInts + 4);
  if (m0.x == 0) return;
  const Shape s = shape_of<NC>(a);
  const int hh = m0.z, qb = m0.w, q0 = m1.x, nq = m1.y, hb = hh % s.nhb;
  const int qi = c / s.HB, head = c - qi * s.HB, i = qb * s.QB + qi;
  if (qi >= s.QB || i >= nq || head >= s.G - hb * s.HB) return;  // no query in this column
  const int n = m0.y + 1 - cta;                                  // piece k is CTA cta + k's
  const float* part = a.part + (int64_t)cta * 2 * kPart;
  const auto piece = [&](int k) { return part + (k == 0 ? kPart : (int64_t)k * 2 * kPart); };
  const auto stats = [&](int k) {  // maximum and sum; a piece that saw no key has sum 0 and no maximum
    return k < n ? *reinterpret_cast<const float2*>(piece(k) + NC * HD + 2 * c) : make_float2(0.0f, 0.0f);
  };
  float M = -INFINITY;
  for (int k = lane; k < n; k += 32) {
    const float2 v = stats(k);
    if (v.y != 0.0f) M = fmaxf(M, v.x);
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  M += kMergeShift;
  float l = 0.0f, acc[kPer];
#pragma unroll
  for (int d = 0; d < kPer; ++d) acc[d] = 0.0f;
  for (int k0 = 0; k0 < n; k0 += 32) {
    const float2 v = stats(k0 + lane);
    const float w = v.y != 0.0f ? v.y * exp2f(v.x - M) : 0.0f;
    l += w;
    const int in = n - k0 < 32 ? n - k0 : 32;
#pragma unroll 8
    for (int k = 0; k < in; ++k) {
      const Vec o = *reinterpret_cast<const Vec*>(piece(k0 + k) + c * HD + lane * kPer);
      const float wk = __shfl_sync(0xffffffffu, w, k);
      const float* x = reinterpret_cast<const float*>(&o);
#pragma unroll
      for (int d = 0; d < kPer; ++d) acc[d] = fmaf(x[d], wk, acc[d]);
    }
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  const int64_t to = (int64_t)(q0 + i) * a.Hq + hh / s.nhb * s.G + hb * s.HB + head;
  T* out = reinterpret_cast<T*>(a.out) + to * HD + lane * kPer;
#pragma unroll
  for (int d = 0; d < kPer; ++d) out[d] = from_float<T>(l != 0.0f ? __fdiv_rn(acc[d], l) : 0.0f);
  if (a.lse && lane == 0) a.lse[to] = l != 0.0f ? (M + log2f(l)) * kLn2 : -INFINITY;
}

// kv8_wide.cu: the kernel for many rows per key head.
// rows: 128 or 256, the most of an item.
size_t kv8_wide_workspace_bytes(int hd, int rows, int num_sms);
cudaError_t launch_kv8_wide(const KvAttnArgs& a, int f16, int hd, int rows, const CUtensorMap& km, const CUtensorMap& vm, void* ws,
                            int num_sms, cudaStream_t stream);

}  // namespace csa2
