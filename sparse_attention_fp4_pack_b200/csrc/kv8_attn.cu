// Attention over the paged 8-bit KV cache (csa2_kv8_attn), on the sm_100a tensor cores.
//
// Both products run as tcgen05.mma kind::f8f6f4 with the cache's E4M3 codes as the A operand,
// exactly as TMA brings them from their pages: nothing is dequantised.  The 16-bit operand of
// each product is written as a sum of 8-bit digits instead:
//   * a query row times a power of two that brings its largest element into [128, 256): E4M3 digits
//     of weights 1, 1/16 (and 1/256 for fp16).  Elements from 2^-13 of the row's largest on are held
//     exactly, smaller ones to 2^-21 of it (bf16) or 2^-25 (fp16);
//   * a weight p * v_scale (at most 2^15 after its shift) is rounded to f16 and held exactly, down to
//     f16's smallest, by four E5M2 digits of weights 1, 1/8, 1/64, 1/512.  E5M2 has f16's exponents,
//     so a digit is the upper byte of what is left: three bits of eleven, no conversion.  Three E4M3
//     digits, as the queries have, would end at 2^-17 of 2^8: a weight e^-12 of the largest was 1% off
//     and one of e^-17 gone, which shows where the largest meets only zeros in V.
// Digits are extra columns of the same product (N), so they cost no extra reads of the keys.
// A page's scale multiplies the score of its keys (K) and the probability of its keys (V): with
// p = exp2(score * log2 e - running maximum), p is the key's share of the softmax sum and
// p * v_scale the weight of its V codes, in units of the largest v_scale so far (a power of two).
// The sum is of the scores alone: no value scale, however large, takes a key out of it.
//
// S^T[128 keys x N] = K_tile . Q^T, O^T[hd x N] += V_tile^T . P^T.  Keys are the M rows (TMEM
// lanes), a column is one (query, head of the group); up to NC columns share a tile's keys.
// The work of the whole call is one list of key tiles: requests, key heads, column blocks, and
// the tiles each block sees.  CTA c takes the c-th of equal shares of it; an item cut by a
// share's border leaves partial sums in the workspace and kv8_merge_kernel joins them.
//
// Bound by HBM when the sequences are long (32 of 64K-128K tokens, 4 key heads: 476 us, 6.3 TB/s;
// 520 where the 1000 W cap lowers the clock; 16 of 32K-64K 132 us in bf16 and in fp16), by the latency
// of a tile's softmax (about 1 us) and of an item's start and end (3 us) when they are short or
// windowed (61 of up to 8191 tokens, window 1024, 8 key heads of 64: 50 us against a floor of 9); one
// sequence of 4096 takes 15.4 us, of which the joining of its pieces is 3.
//
// Roles: warps 0-3 softmax, then one producer warp (TMA, page ids, scales, queries)
// and one warp that issues the products.  The producer works ahead: a piece's tiles, query rows
// and description are on their way while the one before is computed, and the softmax warps turn
// the rows into digits before they write the previous piece's output.  Every wait is bounded: on
// expiry the CTA flags CSA2_DEV_TIMEOUT, drains its copies and products, frees its tensor memory
// and returns.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "csa2_device.cuh"
#include "kv8.cuh"
#include "kv8_list.cuh"
#include "tc.cuh"

namespace csa2 {

// Weights p v_scale count in 2^-13 of the largest v_scale's power of two: with p at most 2^2 (kSlack) they
// end at 2^15, below E5M2's 57344, and f16 holds them to half a step down to 2^-27 of that power.
constexpr int kLift = 13;
constexpr int kDigitsP = 4;
constexpr float kDigitP = 0.125f;  // weight of a digit over the one before

__host__ __device__ constexpr int round16(int n) { return (n + 15) / 16 * 16; }
constexpr uint32_t pow2_cols(int n) { return n <= 32 ? 32u : n <= 64 ? 64u : n <= 128 ? 128u : n <= 256 ? 256u : 512u; }

// CTAs per SM.  A tile of 64 channels is half the bytes for the same softmax, so three are needed
// to hide it: 143 us against 164 for 16 sequences of 64K-128K tokens, 49 against 56 for 61 windowed
// ones (four: 141 and 53).  With 128 channels two leave each more copies in flight: 135 against
// 145 us for 16 of 32K-64K.
__host__ __device__ constexpr int kv8_ctas(int nc, int hd) { return nc == 8 && hd == 64 ? 3 : 2; }

template <int HD, int NC_, int DQ_, bool CAP_>
struct KvCfg {
  static constexpr int kHD = HD, NC = NC_, DQ = DQ_;
  static constexpr bool CAP = CAP_;
  static constexpr int NS = round16(NC * DQ);   // columns of S
  static constexpr int NP = round16(NC * kDigitsP);  // columns of O
  static constexpr int kSoft = 128, kThreads = kSoft + 64;
  static constexpr uint32_t kTile = kKeys * HD;  // bytes of a K or V tile
  static constexpr uint32_t kQBytes = (NS * HD + 1023) / 1024 * 1024;
  static constexpr uint32_t kPBytes = NP * kKeys;
  static constexpr uint32_t kRawBytes = NC * HD * 2;  // query rows as they come
  static constexpr int kCtas = kv8_ctas(NC, HD);  // per SM
  static constexpr uint32_t kBudget = (kCtas == 3 ? 75u : 112u) * 1024u - 4096u;
  static constexpr int kFit = (int)((kBudget - 2 * kQBytes - kPBytes - 2 * kRawBytes) / (2 * kTile));
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr uint32_t kOffK = 0, kOffV = kStages * kTile, kOffQ = 2 * kStages * kTile, kOffP = kOffQ + 2 * kQBytes;
  static constexpr uint32_t kOffRaw = kOffP + kPBytes;
  static constexpr uint32_t kSmem = kOffRaw + 2 * kRawBytes + 1024;  // + alignment slack
  static constexpr uint32_t kColS = 0, kColO = 2 * NS;
  static constexpr uint32_t kCols = pow2_cols(2 * NS + NP);
  static constexpr uint32_t kSwz = tc::swizzle_code(HD);
};

// ---- primitives ------------------------------------------------------------------------
// A is E4M3, B E4M3 or E5M2.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, bool a_mn, bool b_mn, bool b_e5m2) {
  return (1u << 4) | ((b_e5m2 ? 1u : 0u) << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t addr, uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16, "columns of a tile");
  if constexpr (N == 8) tc::tmem_ld8(addr, r);
  else tc::tmem_ld16(addr, r);
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t addr, const uint32_t (&r)[N]) {
  if constexpr (N == 8) tc::tmem_st8_nowait(addr, r);
  else tc::tmem_st16_nowait(addr, r);
}
// N values per lane -> lane i holds value i mod N reduced over the warp (N - 1 exchanges, then
// the remaining whole-warp ones).
template <int N, bool kMax>
__device__ __forceinline__ float warp_columns(float (&v)[N], int lane) {
#pragma unroll
  for (int n = N / 2; n >= 1; n >>= 1) {
    const bool upper = (lane & n) != 0;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float send = upper ? v[j] : v[j + n];
      const float keep = upper ? v[j + n] : v[j];
      const float recv = __shfl_xor_sync(0xffffffffu, send, n);
      v[j] = kMax ? fmaxf(keep, recv) : keep + recv;
    }
  }
  float x = v[0];
#pragma unroll
  for (int o = N; o <= 16; o <<= 1) {
    const float y = __shfl_xor_sync(0xffffffffu, x, o);
    x = kMax ? fmaxf(x, y) : x + y;
  }
  return x;
}

// What the leading digits of two weights (their upper bytes) leave, times 8, exactly: three bits fewer.
__device__ __forceinline__ uint32_t next_digit(uint32_t p) {
  const uint32_t d = p & 0xFF00FF00u;
  const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&p), *reinterpret_cast<const __half2*>(&d)),
                            __floats2half2_rn(8.0f, 8.0f));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// ---- shared state of a CTA -----------------------------------------------------------------
template <class C>
struct KvShared {
  uint64_t kfull[C::kStages], kempty[C::kStages], vfull[C::kStages], vempty[C::kStages];
  uint64_t sfull[2], sfree[2], rows[2], qfull[2], qfree[2], pfull, pvdone, drain;
  uint32_t tmem;
  int abort;
  Share share;
  int64_t sums[C::kThreads / 32];
  float ks[C::kStages][kMaxTilePages], vs[C::kStages][kMaxTilePages];
  struct Piece {           // two are kept, the next one's description comes early
    int take, tile;        // its tiles, and the first one's place in the request
    int lo, hi;            // keys that any of its columns sees,
    int all_lo, all_hi;    // that every column sees
    int first, whole;      // it starts its item, it is all of it
    int q0, n, i0, pos0;   // first row and number of queries of the request, the block's first query, its position
    int cap;               // keys of the request
    int head0, heads;      // first query head of the block, number of them
  } piece[2];
  struct Column {  // of the queries of a piece
    float qscale;
    int lo, hi;    // keys it sees
    int row;       // of out / lse (token * Hq + head), -1 for padding columns
  } col[2][C::NC];
  float red[4][C::NC];
  uint32_t top_v[4];  // largest value scale of the warps' keys (bits)
  float linv[C::NC];
};

// ---- queries -----------------------------------------------------------------------------
// One warp: a piece's description, and its query rows on their way.
template <class C>
__device__ __forceinline__ void fetch_queries(const KvAttnArgs& a, const Shape& s, KvShared<C>& sh, uint32_t smem,
                                              const Walk& w, int buf) {
  constexpr int kChunks = C::kHD / 8;  // of 16 bytes per row
  const int lane = threadIdx.x & 31;
  const int h = w.hh / s.nhb, hb = w.hh - h * s.nhb;
  const int nh = s.G - hb * s.HB < s.HB ? s.G - hb * s.HB : s.HB, head0 = h * s.G + hb * s.HB, i0 = w.qb * s.QB;
#pragma unroll 1
  for (int x = lane; x < C::NC * kChunks; x += 32) {
    const int c = x / kChunks, qi = c / s.HB, hd = c - qi * s.HB;
    if (qi < s.QB && i0 + qi < w.x.n && hd < nh)
      tc::cp_async16(smem + C::kOffRaw + buf * C::kRawBytes + x * 16,
                     a.q + (int64_t)(w.x.q0 + i0 + qi) * a.q_stride + (int64_t)(head0 + hd) * (C::kHD * 2) + (x % kChunks) * 16);
  }
  const uint32_t bar = tc::smem_u32(&sh.rows[buf]);
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
  if (lane == 0) {
    // the block's first query ends soonest, its last starts latest
    const int last_q = i0 + s.QB < w.x.n ? i0 + s.QB - 1 : w.x.n - 1;
    const int64_t all_hi = (int64_t)w.x.pos0 + i0 + 1;
    const int64_t all_lo = a.window > 0 ? (int64_t)w.x.pos0 + last_q + 1 - a.window : 0;
    auto& p = sh.piece[buf];
    p.take = w.take;
    p.tile = w.g.tile + w.off;
    p.lo = w.g.lo;
    p.hi = w.g.hi;
    p.all_hi = all_hi < 0 ? 0 : (all_hi < w.x.cap ? (int)all_hi : w.x.cap);
    p.all_lo = all_lo < 0 ? 0 : (all_lo < 0x7FFFFFFF ? (int)all_lo : 0x7FFFFFFF);
    p.first = w.first;
    p.whole = w.first && w.last;
    p.q0 = w.x.q0;
    p.n = w.x.n;
    p.i0 = i0;
    p.pos0 = w.x.pos0 + i0;
    p.cap = w.x.cap;
    p.head0 = head0;
    p.heads = nh;
    tc::mbar_arrive(bar);
    if (w.first && !w.last) note_item(a, sh.share, w);
  }
}

// The softmax warps: the piece's query rows as E4M3 digits (row d * NC + column of the Q
// operand), and what each column needs later.  A warp's columns do not wait for one another.
template <class C, typename T>
__device__ __forceinline__ bool prepare_queries(const KvAttnArgs& a, const Shape& s, KvShared<C>& sh, uint32_t smem,
                                                uint32_t piece) {
  constexpr int kPer = C::kHD / 32, kCols = C::NC / 4;  // elements per lane, columns per warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, buf = (int)(piece & 1u);
  if (!kv_wait(&sh.abort, sh.rows[buf], (piece >> 1) & 1u)) return false;
  const auto& p = sh.piece[buf];
  const int i0 = p.i0, n = p.n, heads = p.heads;
  float x[kCols][kPer], amax[kCols];
  int qi[kCols], hd[kCols];
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    const int c = k * 4 + warp;
    qi[k] = c / s.HB;
    hd[k] = c - qi[k] * s.HB;
    uint32_t raw[kPer / 2];
    const uint32_t at = smem + C::kOffRaw + buf * C::kRawBytes + c * (C::kHD * 2) + lane * (kPer * 2);
    if constexpr (kPer == 4)
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(raw[0]), "=r"(raw[1]) : "r"(at) : "memory");
    else raw[0] = tc::ld_shared_u32(at);
    if (!(qi[k] < s.QB && i0 + qi[k] < n && hd[k] < heads)) {
      qi[k] = -1;  // a padding column: its row was not brought
#pragma unroll
      for (int e = 0; e < kPer / 2; ++e) raw[e] = 0;
    }
    float top = 0.0f;
#pragma unroll
    for (int e = 0; e < kPer / 2; ++e) {
      if constexpr (std::is_same<T, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&raw[e]));
        x[k][2 * e] = f.x;
        x[k][2 * e + 1] = f.y;
      } else {
        x[k][2 * e] = bf16_lo(raw[e]);
        x[k][2 * e + 1] = bf16_hi(raw[e]);
      }
      top = fmaxf(top, fmaxf(fabsf(x[k][2 * e]), fabsf(x[k][2 * e + 1])));
    }
    amax[k] = top;
  }
#pragma unroll
  for (int k = 0; k < kCols; ++k) amax[k] = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax[k])));
#pragma unroll
  for (int k = 0; k < kCols; ++k) {
    const int c = k * 4 + warp;
    int e = (int)(__float_as_uint(amax[k]) >> 23) - 127;  // amax in [2^e, 2^(e+1))
    e = e < -118 ? -118 : e;  // both powers of two below are normal
    const float up = __uint_as_float((uint32_t)(127 + 7 - e) << 23);
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[k][i] *= up;
#pragma unroll
    for (int d = 0; d < C::DQ; ++d) {
      uint32_t word = 0;
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) {
        const uint32_t b = e4m3x2_sat(x[k][2 * i], x[k][2 * i + 1]);
        word |= b << (16 * i);
        const uint32_t back = f16x2_of_e4m3x2(b);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&back));
        x[k][2 * i] = (x[k][2 * i] - f.x) * 16.0f;
        x[k][2 * i + 1] = (x[k][2 * i + 1] - f.y) * 16.0f;
      }
      const uint32_t at = smem + C::kOffQ + buf * C::kQBytes + tc::swz(d * C::NC + c, lane * kPer, C::kHD);
      if constexpr (kPer == 4) asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(word) : "memory");
      else asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)word) : "memory");
    }
    if (lane == 0) {
      const float per = a.sm_scale * __uint_as_float((uint32_t)(127 + e - 7) << 23);
      auto& col = sh.col[buf][c];
      // an infinite element leaves no digits of the others: the row's scores are NaN
      col.qscale = isinf(amax[k]) ? __int_as_float(0x7FFFFFFF) : C::CAP ? per / a.softcap : per * kLog2e;
      const int64_t hi = (int64_t)p.pos0 + qi[k] + 1, lo = a.window > 0 ? hi - a.window : 0;
      col.hi = qi[k] < 0 || hi < 0 ? 0 : (hi < p.cap ? (int)hi : p.cap);
      col.lo = lo < 0 ? 0 : (lo < 0x7FFFFFFF ? (int)lo : 0x7FFFFFFF);
      col.row = qi[k] < 0 ? -1 : (p.q0 + i0 + qi[k]) * a.Hq + p.head0 + hd[k];
    }
  }
  tc::fence_async_smem();
  __syncwarp();
  if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.qfull[buf]));
  return true;
}

// ---- producer --------------------------------------------------------------------------
template <class C>
__device__ void produce(const KvAttnArgs& a, const Shape& s, KvShared<C>& sh, uint32_t smem, const CUtensorMap* kmap,
                        const CUtensorMap* vmap) {
  const int lane = threadIdx.x & 31;
  const int page = 1 << a.page_log2, ppt = kKeys >> a.page_log2;
  const uint32_t page_bytes = (uint32_t)page * C::kHD;
  uint32_t bad = 0;
  int64_t nk = 0, nv = 0;  // tiles of K and of V whose copies were issued
  bool ok = true;
  uint32_t piece = 0;
  Walk w;
  if (lane == 0) a.meta[(int64_t)blockIdx.x * kMetaInts] = 0;
  for (w.start(a, s, sh.share); ok && w.left > 0; w.next(a, s), ++piece) {
    const int h = w.hh / s.nhb;
    const int32_t* row = a.table + (int64_t)w.r * a.max_pages;
    const int p_end = (w.g.hi + page - 1) >> a.page_log2, p_beg = w.g.lo >> a.page_log2;
    int base = -1;       // first page of the 32 ids held, one per lane
    int32_t ids = -1, ahead = -1;
    for (int i = 0; i < w.take; ++i) {
      const int p0 = (w.g.tile + w.off + i) * ppt;
      if (base < 0 || p0 >= base + 32) {
        const bool next = base >= 0;
        base = p0;
        ids = next ? ahead : (base + lane >= p_beg && base + lane < p_end ? row[base + lane] : -1);
        ahead = base + 32 + lane < p_end ? row[base + 32 + lane] : -1;
      }
      const int32_t id = __shfl_sync(0xffffffffu, ids, (p0 - base + lane) & 31);
      const int p = p0 + lane;
      const bool in = lane < ppt && p >= p_beg && p < p_end && w.g.lo < w.g.hi;
      const bool valid = in && id >= 0 && id < a.n_pages;
      if (in && !valid) bad |= CSA2_DEV_BAD_INDEX;
      const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, valid)) * page_bytes;
      const int st = (int)(nk % C::kStages);
      const uint32_t parity = (uint32_t)(nk / C::kStages + 1) & 1u;
      const int head = id * a.Hk + h, at = head << a.page_log2;  // rows of a cache are below 2^31
      ok = __all_sync(0xffffffffu, kv_wait(&sh.abort, sh.kempty[st], parity));
      if (!ok) break;
      const uint32_t kb = tc::smem_u32(&sh.kfull[st]);
      if (lane == 0) tc::mbar_arrive_expect_tx(kb, bytes);
      __syncwarp();
      if (valid) tma_rows(smem + C::kOffK + st * C::kTile + lane * page_bytes, kmap, at, kb);
      ++nk;
      ok = __all_sync(0xffffffffu, kv_wait(&sh.abort, sh.vempty[st], parity));
      if (!ok) break;
      const uint32_t vb = tc::smem_u32(&sh.vfull[st]);
      if (lane == 0) tc::mbar_arrive_expect_tx(vb, bytes);
      __syncwarp();
      if (valid) {
        tma_rows(smem + C::kOffV + st * C::kTile + lane * page_bytes, vmap, at, vb);
        tc::cp_async4(tc::smem_u32(&sh.ks[st][lane]), a.k_scale + head);
        tc::cp_async4(tc::smem_u32(&sh.vs[st][lane]), a.v_scale + head);
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(vb) : "memory");
      } else {
        if (lane < ppt) {  // no page: its rows are masked
          sh.ks[st][lane] = 0.0f;
          sh.vs[st][lane] = -1.0f;
        }
        tc::mbar_arrive(vb);
      }
      ++nv;
      if (i == 0) {  // behind the first tile's copies
        ok = kv_wait_all(sh, sh.qfree[piece & 1u], ((piece >> 1) & 1u) ^ 1u);
        if (!ok) break;
        fetch_queries<C>(a, s, sh, smem, w, (int)(piece & 1u));
      }
    }
  }
  if (!ok) {  // given up: no copy may land after the CTA has gone
    for (int64_t n = nk > C::kStages ? nk - C::kStages : 0; n < nk; ++n)
      tc::mbar_wait(tc::smem_u32(&sh.kfull[n % C::kStages]), (uint32_t)(n / C::kStages) & 1u, kKvPolls);
    for (int64_t n = nv > C::kStages ? nv - C::kStages : 0; n < nv; ++n)
      tc::mbar_wait(tc::smem_u32(&sh.vfull[n % C::kStages]), (uint32_t)(n / C::kStages) & 1u, kKvPolls);
  }
  if (bad) flag(a.status, bad);
}

// ---- products (one warp) ----------------------------------------------------------------
template <class C>
__device__ void multiply(KvShared<C>& sh, uint32_t smem, uint32_t tmem) {
  constexpr uint32_t kIdS = idesc_f8(kKeys, C::NS, false, false, false);
  constexpr uint32_t kIdO = idesc_f8(128, C::NP, true, true, true);
  // K tile and queries: rows of HD bytes, K-major.  V tile: the same bytes read MN-major (with
  // 64 channels the second half of the 128 M rows repeats the first: leading offset 0).  P:
  // granules of 16 columns x 128 keys, 16 bytes per key, MN-major, no swizzle.
  const uint64_t dk0 = tc::smem_desc(smem + C::kOffK, 16, 8 * C::kHD, C::kSwz);
  const uint64_t dq0 = tc::smem_desc(smem + C::kOffQ, 16, 8 * C::kHD, C::kSwz);
  const uint64_t dv0 = tc::smem_desc(smem + C::kOffV, 0, 8 * C::kHD, C::kSwz);
  const uint64_t dp = tc::smem_desc(smem + C::kOffP, 128, 16 * kKeys, 0);
  int64_t n = 0;
  uint32_t piece = 0;
  const bool on = (threadIdx.x & 31) == 0;
  bool ok = true;
  auto scores = [&](int64_t m) {  // S of tile m
    const int st = (int)(m % C::kStages);
    ok = kv_wait_all(sh, sh.kfull[st], (uint32_t)(m / C::kStages) & 1u) &&
         kv_wait_all(sh, sh.sfree[m & 1], ((uint32_t)(m >> 1) & 1u) ^ 1u);
    if (!ok) return;
    tc::fence_after_sync();
    const uint64_t dk = tc::desc_add(dk0, st * C::kTile), dq = tc::desc_add(dq0, (piece & 1u) * C::kQBytes);
    const uint32_t d = tmem + C::kColS + (uint32_t)(m & 1) * C::NS;
#pragma unroll
    for (int k = 0; k < C::kHD / 32; ++k)
      mma_f8(on, d, tc::desc_add(dk, 32 * k), tc::desc_add(dq, 32 * k), kIdS, k > 0);
    commit_if(on, tc::smem_u32(&sh.sfull[m & 1]));
    commit_if(on, tc::smem_u32(&sh.kempty[st]));
  };
  int take = 0;
  for (int64_t left = uniform(sh.share.left); ok && left > 0; left -= take, ++piece) {
    ok = kv_wait_all(sh, sh.qfull[piece & 1u], (piece >> 1) & 1u);
    if (!ok) break;
    take = uniform(sh.piece[piece & 1u].take);
    scores(n);
    for (int i = 0; ok && i < take; ++i, ++n) {
      if (i + 1 < take) scores(n + 1);
      const int st = (int)(n % C::kStages);
      ok = ok && kv_wait_all(sh, sh.vfull[st], (uint32_t)(n / C::kStages) & 1u) &&
           kv_wait_all(sh, sh.pfull, (uint32_t)n & 1u);
      if (!ok) break;
      tc::fence_after_sync();
      const uint64_t dv = tc::desc_add(dv0, st * C::kTile);
#pragma unroll
      for (int k = 0; k < kKeys / 32; ++k)
        mma_f8(on, tmem + C::kColO, tc::desc_add(dv, 32 * k * C::kHD), tc::desc_add(dp, 32 * k * 16), kIdO,
                 i > 0 || k > 0);
      commit_if(on, tc::smem_u32(&sh.vempty[st]));
      commit_if(on, tc::smem_u32(&sh.pvdone));
    }
  }
  if (!ok) {  // given up: no product may run after the tensor memory is freed
    commit_if(on, tc::smem_u32(&sh.drain));
    tc::mbar_wait(tc::smem_u32(&sh.drain), 0, kKvPolls);
  }
}

// ---- softmax -----------------------------------------------------------------------------
template <class C, typename T>
__device__ void soften(const KvAttnArgs& a, const Shape& s, KvShared<C>& sh, uint8_t* smem_p, uint32_t tmem) {
  constexpr int CW = C::NC;
  const uint32_t smem = tc::smem_u32(smem_p);
  const int tid = threadIdx.x, lane = tid & 31, wq = tid >> 5, row = tid;
  const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
  const float cap2 = C::CAP ? a.softcap * kLog2e : 0.0f;
  bool bad = false;
  int64_t n = 0;
  uint32_t piece = 0;
  int take;
  if (sh.share.left > 0) bad = !prepare_queries<C, T>(a, s, sh, smem, 0);
  if (tc::named_sync_or(1, 128, bad)) return;  // the columns are known to every softmax thread
  for (int64_t left = sh.share.left; left > 0; left -= take, ++piece) {
    const int buf = (int)(piece & 1u);
    const auto& w = sh.piece[buf];
    take = w.take;
    const int lo = w.lo, hi = w.hi, all_lo = w.all_lo, all_hi = w.all_hi, tile = w.tile;
    float qs[CW], m[CW], l[CW];
#pragma unroll
    for (int c = 0; c < CW; ++c) {
      qs[c] = sh.col[buf][c].qscale;
      m[c] = 0.0f;
      l[c] = 0.0f;
    }
    uint32_t unseen = 0xffffffffu >> (32 - CW);  // columns that have seen no key yet
    // exponent of the least power of two not below the value scales of the piece's keys so far: with
    // weights p v_scale 2^(kLift - unit_e), O counts in units of 2^(unit_e - kLift)
    int unit_e = kLeastExp;
    for (int i = 0; i < take; ++i, ++n) {
      const int st = (int)(n % C::kStages);
      bad |= !kv_wait(&sh.abort, sh.sfull[n & 1], (uint32_t)(n >> 1) & 1u);
      bad |= !kv_wait(&sh.abort, sh.vfull[st], (uint32_t)(n / C::kStages) & 1u);
      tc::fence_after_sync();
      float u[CW];
      {
        const uint32_t at = lanes + C::kColS + (uint32_t)(n & 1) * C::NS;
        uint32_t d[CW];
        tmem_ld<CW>(at, d);
#pragma unroll
        for (int c = 0; c < CW; ++c) u[c] = __uint_as_float(d[c]);
        tmem_ld<CW>(at + C::NC, d);
#pragma unroll
        for (int c = 0; c < CW; ++c) u[c] = fmaf(__uint_as_float(d[c]), 0.0625f, u[c]);
        if constexpr (C::DQ == 3) {
          tmem_ld<CW>(at + 2 * C::NC, d);
#pragma unroll
          for (int c = 0; c < CW; ++c) u[c] = fmaf(__uint_as_float(d[c]), 0.00390625f, u[c]);
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.sfree[n & 1]));
      const int key0 = (tile + i) * kKeys, key = key0 + row;
      const float ks = sh.ks[st][row >> a.page_log2];
      float vs = sh.vs[st][row >> a.page_log2];
      const bool there = vs >= 0.0f && key >= lo && key < hi;
      vs = fmaxf(vs, kLeastScale);
      if constexpr (C::CAP) {
        float most = 0.0f;
#pragma unroll
        for (int c = 0; c < CW; ++c) {
          u[c] *= ks * qs[c];
          most = fmaxf(most, fabsf(u[c]));
        }
        if (__all_sync(0xffffffffu, most <= kTanhSmall)) {  // the same for the warp: scores well below the cap
#pragma unroll
          for (int c = 0; c < CW; ++c) u[c] = fmaf(cap2, tanh_small(u[c]), -m[c]);
        } else {
#pragma unroll
          for (int c = 0; c < CW; ++c) u[c] = fmaf(cap2, tanh_any(u[c]), -m[c]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < CW; ++c) u[c] = fmaf(u[c], ks * qs[c], -m[c]);  // the scales first: u * ks may leave fp32
      }
      if (!there) {
#pragma unroll
        for (int c = 0; c < CW; ++c) u[c] = -INFINITY;
      } else if (key0 + kKeys > all_hi || key0 < all_lo) {
#pragma unroll
        for (int c = 0; c < CW; ++c)
          if (key >= sh.col[buf][c].hi || key < sh.col[buf][c].lo) u[c] = -INFINITY;
      }
      bool exceed = there && vs > exp2i(unit_e);
#pragma unroll
      for (int c = 0; c < CW; ++c) exceed |= u[c] > kSlack;
      if (unseen) {
#pragma unroll
        for (int c = 0; c < CW; ++c) exceed |= ((unseen >> c) & 1u) && u[c] > -INFINITY;
      }
      if (tc::named_sync_or(1, 128, exceed || bad)) {
        if (tc::named_sync_or(1, 128, bad)) {
          bad = true;
          break;
        }
        float t[CW];
#pragma unroll
        for (int c = 0; c < CW; ++c) t[c] = u[c];
        const float top = warp_columns<CW, true>(t, lane);
        if (lane < CW) sh.red[wq][lane] = top;
        const uint32_t top_v = __reduce_max_sync(0xffffffffu, there ? __float_as_uint(vs) : 0u);
        if (lane == 0) sh.top_v[wq] = top_v;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        if (i > 0) bad |= !kv_wait(&sh.abort, sh.pvdone, (uint32_t)(n - 1) & 1u);
        tc::fence_after_sync();
        const uint32_t v01 = max(sh.top_v[0], sh.top_v[1]), v23 = max(sh.top_v[2], sh.top_v[3]);
        const int grown = max(unit_e, pow2_above_exp(__uint_as_float(max(v01, v23))));
        const float shrink = grown - unit_e > 126 ? 0.0f : exp2i(unit_e - grown);
        unit_e = grown;
        float f[CW];
#pragma unroll
        for (int c = 0; c < CW; ++c) {
          const float mx = fmaxf(fmaxf(sh.red[0][c], sh.red[1][c]), fmaxf(sh.red[2][c], sh.red[3][c]));
          const bool fresh = (unseen >> c) & 1u;
          const float up = mx == -INFINITY ? 0.0f : (fresh ? mx : (mx > kSlack ? mx : 0.0f));
          if (fresh && mx != -INFINITY) unseen &= ~(1u << c);
          f[c] = fresh ? 1.0f : exp2_approx(-up);
          m[c] += up;
          l[c] *= f[c];
          f[c] *= shrink;  // O counts in the new unit
          u[c] -= up;
        }
        if (i > 0) {  // the accumulated output under the new maxima
#pragma unroll
          for (int d = 0; d < kDigitsP; ++d) {
            uint32_t o[CW];
            tmem_ld<CW>(lanes + C::kColO + d * C::NC, o);
#pragma unroll
            for (int c = 0; c < CW; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * f[c]);
            tmem_st<CW>(lanes + C::kColO + d * C::NC, o);
          }
          tc::tmem_wait_st();
        }
        asm volatile("bar.sync 1, 128;" ::: "memory");  // red may be written again
      } else if (i > 0) {
        bad |= !kv_wait(&sh.abort, sh.pvdone, (uint32_t)(n - 1) & 1u);  // P may be written again
      }
      const float weigh = vs * exp2i(kLift - unit_e);  // at most 2^kLift
      uint32_t dig[kDigitsP][CW / 4];
#pragma unroll
      for (int c = 0; c < CW; c += 4) {
        uint32_t p[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float p0 = exp2_approx(u[c + 2 * k]), p1 = exp2_approx(u[c + 2 * k + 1]);
          l[c + 2 * k] += p0;
          l[c + 2 * k + 1] += p1;
          const __half2 ph = __floats2half2_rn(p0 * weigh, p1 * weigh);
          p[k] = *reinterpret_cast<const uint32_t*>(&ph);
        }
#pragma unroll
        for (int d = 0; d < kDigitsP; ++d) {
          dig[d][c / 4] = __byte_perm(p[0], p[1], 0x7531);
          if (d + 1 < kDigitsP) {
            p[0] = next_digit(p[0]);
            p[1] = next_digit(p[1]);
          }
        }
      }
#pragma unroll
      for (int d = 0; d < kDigitsP; ++d) {
        const int col = d * C::NC;
        const uint32_t at = smem + C::kOffP + (col / 16) * (16 * kKeys) + row * 16 + col % 16;
        if constexpr (CW == 8) {
          asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(dig[d][0]), "r"(dig[d][1]) : "memory");
        } else {
#pragma unroll
          for (int k = 0; k < CW / 16; ++k)
            tc::st_shared_v4(at + k * (16 * kKeys),
                             make_uint4(dig[d][4 * k], dig[d][4 * k + 1], dig[d][4 * k + 2], dig[d][4 * k + 3]));
        }
      }
      if (!there) {  // whatever lies there (NaN included) times a zero probability
#pragma unroll
        for (int k = 0; k < C::kHD / 16; ++k)
          tc::st_shared_v4(smem + C::kOffV + st * C::kTile + row * C::kHD + k * 16, make_uint4(0u, 0u, 0u, 0u));
      }
      tc::fence_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&sh.pfull));
    }
    if (!bad && left > take) bad = !prepare_queries<C, T>(a, s, sh, smem, piece + 1);
    if (!bad) bad = !kv_wait(&sh.abort, sh.pvdone, (uint32_t)(n - 1) & 1u);
    if (tc::named_sync_or(1, 128, bad)) break;
    tc::fence_after_sync();
    // sums over the keys: the warp's rows, then the four warps
    const float sum = warp_columns<CW, false>(l, lane);
    if (lane < CW) sh.red[wq][lane] = sum;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    const bool whole = w.whole != 0;
    const int slot = w.first ? 1 : 0;
    float* part = a.part + ((int64_t)blockIdx.x * 2 + slot) * (C::NC * (C::kHD + 2));
    if (row < CW) {
      const float tot = (sh.red[0][row] + sh.red[1][row]) + (sh.red[2][row] + sh.red[3][row]);
      float mm = 0.0f;
#pragma unroll
      for (int c = 0; c < CW; ++c) mm = row == c ? m[c] : mm;
      const int to = sh.col[buf][row].row;
      sh.linv[row] = tot != 0.0f ? __fdiv_rn(exp2i(unit_e - kLift), tot) : 0.0f;
      if (whole) {
        if (a.lse && to >= 0) a.lse[to] = tot != 0.0f ? (mm + log2f(tot)) * kLn2 : -INFINITY;
      } else {
        part[C::NC * C::kHD + 2 * (row)] = mm;
        part[C::NC * C::kHD + 2 * (row) + 1] = tot;
      }
    }
    asm volatile("bar.sync 1, 128;" ::: "memory");
    {
      float o[CW];  // digits of a column are CW columns apart, from the last to the first
#pragma unroll
      for (int c = 0; c < CW; ++c) o[c] = 0.0f;
#pragma unroll
      for (int x = C::NP - 16; x >= 0; x -= 16) {
        uint32_t d[16];
        tc::tmem_ld16(lanes + C::kColO + x, d);
#pragma unroll
        for (int k = 16 - CW; k >= 0; k -= CW)
#pragma unroll
          for (int c = 0; c < CW; ++c) o[c] = fmaf(o[c], kDigitP, __uint_as_float(d[k + c]));
      }
      if (row < C::kHD) {
        if (whole) {
          T* out = reinterpret_cast<T*>(a.out);
#pragma unroll
          for (int c = 0; c < CW; ++c) {
            const int to = sh.col[buf][c].row;
            if (to >= 0) out[(int64_t)to * C::kHD + row] = from_float<T>(o[c] * sh.linv[c]);
          }
        } else {
#pragma unroll
          for (int c = 0; c < CW; ++c) part[(c) * C::kHD + row] = o[c] * sh.linv[c];
        }
      }
    }
    tc::fence_before_sync();
    asm volatile("bar.sync 1, 128;" ::: "memory");  // every thread is done with red, linv and the columns
    if (tid == 0) tc::mbar_arrive(tc::smem_u32(&sh.qfree[buf]));
  }
}

template <class C, typename T>
__global__ void __launch_bounds__(C::kThreads, C::kCtas) kv8_attn_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                const __grid_constant__ CUtensorMap vmap,
                                                                const KvAttnArgs a) {
  extern __shared__ uint8_t raw[];
  __shared__ KvShared<C> sh;
  uint8_t* smem = tc::align_smem_1024(raw);
  const int tid = threadIdx.x, warp = uniform(tid >> 5);
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.kfull[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh.vfull[i]), 33);
      tc::mbar_init(tc::smem_u32(&sh.kempty[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh.vempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.sfull[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh.sfree[i]), 4);
      tc::mbar_init(tc::smem_u32(&sh.rows[i]), 33);
      tc::mbar_init(tc::smem_u32(&sh.qfull[i]), 4);
      tc::mbar_init(tc::smem_u32(&sh.qfree[i]), 1);
    }
    tc::mbar_init(tc::smem_u32(&sh.pfull), 4);
    tc::mbar_init(tc::smem_u32(&sh.pvdone), 1);
    tc::mbar_init(tc::smem_u32(&sh.drain), 1);
    sh.abort = 0;
  }
  // Tensor memory is taken only when the predecessor has returned its own, and the successor
  // may start only when this CTA has taken its: kernels that wait for one another through
  // the launch order never also wait for one another's tensor memory.
  chain_wait();
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&sh.tmem), C::kCols);
  const Shape s = shape_of<C::NC>(a);
  uint32_t bad = 0;
  find_share<C::kThreads>(a, s, sh.sums, &sh.share, &bad);
  if (bad && blockIdx.x == 0) flag(a.status, bad);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  chain_launch_dependents();
  const uint32_t tmem = uniform(sh.tmem);
  if (warp < C::kSoft / 32) {
    soften<C, T>(a, s, sh, smem, tmem);
  } else if (warp == C::kSoft / 32) {
    produce<C>(a, s, sh, tc::smem_u32(smem), &kmap, &vmap);
  } else {
    multiply<C>(sh, tc::smem_u32(smem), tmem);
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tmem, C::kCols);
  if (tid == 0 && sh.abort) flag(a.status, CSA2_DEV_TIMEOUT);
}

// ---- host --------------------------------------------------------------------------------
// Columns per tile: 8 or 16 that hold a request's queries times the heads of a group, so decode
// pays for no empty columns; beyond 16 the f16 kernel (0).  Both sides measured: at 16 columns the
// digits take 143 us and the f16 kernel 210 (16 sequences of 32K-64K tokens, groups of 16); 32 columns
// of digits took 295 us with groups of 32, and 78 us for 32 sequences of 1K-8K with two queries of 16
// heads, where the f16 kernel takes 212 and 49.
static int columns_of(int Hq, int Hk, int max_q) {
  const int64_t want = (int64_t)(Hq / Hk) * max_q;
  return want <= 8 ? 8 : want <= 16 ? 16 : 0;
}
// Rows per item of the f16 kernel.
static int rows_of(int Hq, int Hk, int max_q) { return (int64_t)(Hq / Hk) * max_q <= 128 ? 128 : 256; }
size_t kv8_attn_workspace_bytes(int Hq, int Hk, int hd, int max_q, int num_sms) {
  const int nc = columns_of(Hq, Hk, max_q), ctas = num_sms * kv8_ctas(nc, hd);
  if (nc == 0) return kv8_wide_workspace_bytes(hd, rows_of(Hq, Hk, max_q), num_sms);
  return (size_t)ctas * 2 * nc * (hd + 2) * sizeof(float) + (size_t)ctas * kMetaInts * sizeof(int32_t);
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                              const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// The cache as rows of hd bytes; a box is one head's rows of one page.
static bool encode_rows(CUtensorMap* m, const uint8_t* cache, int64_t rows, int hd, int page, bool swizzle) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[2] = {(cuuint64_t)hd, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)hd};
  const cuuint32_t box[2] = {(cuuint32_t)hd, (cuuint32_t)page}, one[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(cache), dims, strides, box, one,
            CU_TENSOR_MAP_INTERLEAVE_NONE,
            !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : hd == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C, typename T>
static cudaError_t launch_kv8_t(const CUtensorMap& km, const CUtensorMap& vm, KvAttnArgs a, void* ws, int num_sms,
                                cudaStream_t stream) {
  const int ctas = num_sms * C::kCtas;
  a.part = static_cast<float*>(ws);
  a.meta = reinterpret_cast<int32_t*>(a.part + (size_t)ctas * 2 * C::NC * (C::kHD + 2));
  cudaError_t e = cudaFuncSetAttribute(kv8_attn_kernel<C, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_chained(kv8_attn_kernel<C, T>, dim3(ctas), dim3(C::kThreads), C::kSmem, stream, 0, km, vm, a);
  if (e != cudaSuccess) return e;
  e = launch_chained(kv8_merge_kernel<C::NC, C::kHD, T>, dim3(ctas, C::NC / 8), dim3(kMergeThreads), 0, stream, 0, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int HD, int DQ, bool CAP, typename T>
static cudaError_t launch_kv8_nc(int nc, const CUtensorMap& km, const CUtensorMap& vm, const KvAttnArgs& a, void* ws,
                                 int num_sms, cudaStream_t stream) {
  if (nc == 8) return launch_kv8_t<KvCfg<HD, 8, DQ, CAP>, T>(km, vm, a, ws, num_sms, stream);
  return launch_kv8_t<KvCfg<HD, 16, DQ, CAP>, T>(km, vm, a, ws, num_sms, stream);
}

template <int HD, bool CAP>
static cudaError_t launch_kv8_type(int f16, int nc, const CUtensorMap& km, const CUtensorMap& vm, const KvAttnArgs& a,
                                   void* ws, int num_sms, cudaStream_t stream) {
  return f16 ? launch_kv8_nc<HD, 3, CAP, __half>(nc, km, vm, a, ws, num_sms, stream)
             : launch_kv8_nc<HD, 2, CAP, __nv_bfloat16>(nc, km, vm, a, ws, num_sms, stream);
}

cudaError_t launch_kv8_attn(const void* q, int64_t q_stride, int f16, int64_t T, int Hq, int Hk, int hd,
                            const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale, const float* v_scale,
                            int64_t n_pages, int page, const int32_t* table, int max_pages, const int32_t* q_start,
                            const int32_t* seq_len, int R, int max_q, float sm_scale, int window, float softcap,
                            void* out, float* lse, void* ws, uint32_t* status, cudaStream_t stream, int num_sms) {
  KvAttnArgs a = {};
  a.q = static_cast<const uint8_t*>(q);
  a.q_stride = q_stride * 2;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.table = table;
  a.q_start = q_start;
  a.seq_len = seq_len;
  a.R = R;
  a.Hq = Hq;
  a.Hk = Hk;
  a.max_pages = max_pages;
  a.page_log2 = log2_of(page);
  a.n_pages = n_pages;
  a.T = T;
  a.sm_scale = sm_scale;
  a.window = window;
  a.softcap = softcap;
  a.out = static_cast<uint8_t*>(out);
  a.lse = lse;
  a.status = status;
  CUtensorMap km, vm;
  const int64_t rows = n_pages * Hk * page;
  const int nc = columns_of(Hq, Hk, max_q);
  if (!encode_rows(&km, k_cache, rows, hd, page, nc > 0) || !encode_rows(&vm, v_cache, rows, hd, page, nc > 0))
    return cudaErrorInvalidValue;
  if (nc == 0) return launch_kv8_wide(a, f16, hd, rows_of(Hq, Hk, max_q), km, vm, ws, num_sms, stream);
  if (hd == 64)
    return softcap > 0.0f ? launch_kv8_type<64, true>(f16, nc, km, vm, a, ws, num_sms, stream)
                          : launch_kv8_type<64, false>(f16, nc, km, vm, a, ws, num_sms, stream);
  return softcap > 0.0f ? launch_kv8_type<128, true>(f16, nc, km, vm, a, ws, num_sms, stream)
                        : launch_kv8_type<128, false>(f16, nc, km, vm, a, ws, num_sms, stream);
}

}  // namespace csa2
