// Attention over the paged 8-bit KV cache for many query rows per key head (chunks of prompts,
// drafted tokens, large groups): csa2_kv8_attn's kernel beyond 16 rows (columns_of in kv8_attn.cu).  The list
// of key tiles, its even split over the CTAs and the joining of split items are kv8_list.cuh's.
//
// With many rows a key tile is used often enough to pay for turning its E4M3 codes into f16
// once: both products are then tcgen05.mma kind::f16 at one column per score, where the digit
// form of kv8_attn.cu needs two or three.  f16 holds every code exactly.  A query row enters as
// f16 after a power of two has brought its largest element into [2^14, 2^15): exact for bf16 and
// fp16 down to 2^-28 of that element.  Weights are rounded to f16 under a shift of 2^5.
//   S[128 rows x 128 keys] = Q . K_tile^T,   O[128 rows x hd] += P . V_tile  (P from tensor memory)
// A page's K scale times the row's scale multiplies the scores of its keys, and the logarithm of
// its weight w = v_scale over the largest v_scale of the piece so far (a power of two) is added: one
// fused multiply-add per score.  exp2 of that is the weight of the key's V codes, and over w its share
// of the softmax sum.  w counts as 2^kLeastWeight at least (f16 drops what is that small all the same):
// weights that fp32 cannot hold beside the maximum are then below 2^-60 of the sum as well, so no
// value scale, however large, takes a key out of it.
//
// Two slots of S, P and O keep the tensor cores busy while the other slot's softmax runs:
//   * more than 128 rows: slot g holds rows 128 g .. of the item, both use every key tile;
//   * up to 128 rows: both slots hold the same rows and take the key tiles in turn; their sums
//     are joined when the piece ends.
// A softmax thread owns one row, so its maximum, sum and rescaling need no exchange.
//
// 8 x 64 drafts of 64 heads over 8K-32K keys take 473 to 483 us (837 TFLOP/s; the 1000 W cap lowers the
// clock), chunks of 1024 rows 684 to 689 (889 TFLOP/s).  Of a slot's about 4000 cycles per key tile
// of 256 rows the softmax takes 2300 (maximum 750, exponentials 1000), its two products 1024, waits
// and issue the rest; the tensor cores are busy 2048 of them.  With few rows the copies in flight
// bound it (3.6 TB/s at 32 rows).
//
// Roles: warps 0-3 and 4-7 softmax of slot 0 and 1; warp 13 brings tiles from their pages by TMA
// in the order K0 K1 V0 K2 V1 K3 ...; warps 8-11 turn them into f16 in a ring of shared memory
// tiles; warp 12 issues the products.  Every wait is bounded: on expiry the CTA
// flags CSA2_DEV_TIMEOUT, drains its copies and products and returns.
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

// Weights are 2^(t - m + 5) with m raised only when a score exceeds it by more than 10, so they end at
// f16's 2^15; f16 holds them to half a step down to 2^-19 of the largest and drops what is below 2^-30.
// The accumulated output is rescaled on a raise; with a slack of 2 one tile in five did (a softmax
// warp's 561 of 3350 cycles per tile).  Six bits more at the low end for a slack of 4 cost 5%: 507
// against 483 us (drafts), 731 against 687 (chunks).
constexpr int kWideLift = 5, kLeastWeight = -56;
constexpr float kWideSlack = 10.0f;

// ROWS: the most rows of an item, 128 or 256.  With 128 one tile of queries is kept, and the shared
// memory saved holds more copies in flight, which few rows are bound by: 16 sequences of 32K-64K
// tokens with groups of 32 heads take 219 us against 260 with the 256-row shape, 8 of 16K-32K with
// 16 drafts of 8 heads 94 against 109.  Beyond 128 rows a key tile serves 256 at once.
template <int HD, int ROWS, bool CAP_>
struct KvWide {
  static constexpr int kHD = HD, NC = ROWS;
  static constexpr bool CAP = CAP_;
  static constexpr int kThreads = 512;
  static constexpr uint32_t kHalf = 128 * 128;         // 128 rows of 64 f16, 128-byte swizzle
  static constexpr uint32_t kTile = kHalf * (HD / 64);  // a K, V or Q tile
  static constexpr uint32_t kRaw = kKeys * HD;          // the same tile as E4M3
  static constexpr int kRing = HD == 128 ? 4 : 6, kStages = (HD == 128 ? 2 : 6) + (ROWS == 128 ? (HD == 128 ? 2 : 4) : 0);
  // per-tile scales kept: a tile's are written before its copy waits for a stage, so the tile whose
  // place they take must be done when the copies can be kStages + kRing items ahead (two per tile)
  static constexpr int kScales = HD == 64 ? 16 : 8;
  static_assert(kStages + kRing <= 2 * kScales - 4, "scales of a tile in use would be overwritten");
  static constexpr uint32_t kOffQ = 0, kOffRing = (ROWS / 128) * kTile, kOffRaw = kOffRing + kRing * kTile;
  static constexpr uint32_t kSmem = kOffRaw + kStages * kRaw + 1024;
  static constexpr uint32_t kColO = 256;  // S0, S1 (and P in their first 64 columns), O0, O1
  // registers per thread of the softmax, converting and loading / issuing warpgroups; the kernel is
  // launched with 128 (checked before the launch), which covers their sum
  static constexpr int kRegsSoft = 192, kRegsConv = 56, kRegsMma = 72;
};

template <class C>
struct WideShared {
  uint64_t rfull[C::kStages], rempty[C::kStages];  // tiles as E4M3
  uint64_t full[C::kRing], empty[C::kRing];        // tiles as f16
  uint64_t qfull[2], sfull[2], pfull[2][2], ofull[2], drain;  // pfull: by half of the keys
  uint32_t tmem;
  int abort;
  Share share;
  int take, one_slot;           // the piece the softmax warps are at: its tiles, whether its rows fit a slot
  int rows[C::kStages][2];      // first and last + 1 row of the tile that holds a key of the block
  uint32_t pages[C::kStages];   // bit p: its p-th page exists
  // per tile and page: k_scale, log2 of w 2^kWideLift, its reciprocal, the unit of w 2^kWideLift
  float4 sc[C::kScales][kMaxTilePages];
};

template <int N>
__device__ __forceinline__ void reg_inc() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void reg_dec() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Two fp32 operations per instruction on neighbouring registers, and a three-way maximum.
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// All 128 score columns of this thread's TMEM lane: four loads in flight, one wait.  The empty
// statements keep every use of the values behind the wait.
__device__ __forceinline__ void tmem_ld128(uint32_t addr, uint32_t (&r)[128]) {
#pragma unroll
  for (int c = 0; c < 128; c += 32)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[c]), "=r"(r[c + 1]), "=r"(r[c + 2]), "=r"(r[c + 3]), "=r"(r[c + 4]), "=r"(r[c + 5]),
          "=r"(r[c + 6]), "=r"(r[c + 7]), "=r"(r[c + 8]), "=r"(r[c + 9]), "=r"(r[c + 10]), "=r"(r[c + 11]),
          "=r"(r[c + 12]), "=r"(r[c + 13]), "=r"(r[c + 14]), "=r"(r[c + 15]), "=r"(r[c + 16]), "=r"(r[c + 17]),
          "=r"(r[c + 18]), "=r"(r[c + 19]), "=r"(r[c + 20]), "=r"(r[c + 21]), "=r"(r[c + 22]), "=r"(r[c + 23]),
          "=r"(r[c + 24]), "=r"(r[c + 25]), "=r"(r[c + 26]), "=r"(r[c + 27]), "=r"(r[c + 28]), "=r"(r[c + 29]),
          "=r"(r[c + 30]), "=r"(r[c + 31])
        : "r"(addr + c)
        : "memory");
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int c = 0; c < 128; ++c) asm volatile("" : "+r"(r[c]));
}

// Rows of the item that a piece works on; both slots share them when they fit one.
template <class C>
__device__ __forceinline__ bool one_slot_rows(const Shape& s, const Walk& w) {
  if constexpr (C::NC == 128) return true;
  const int i0 = w.qb * s.QB, i1 = i0 + s.QB < w.x.n ? i0 + s.QB : w.x.n;
  return (i1 - i0) * s.HB <= 128;
}

// ---- tiles from their pages (one warp) -----------------------------------------------------
template <class C>
__device__ void load_tiles(const KvAttnArgs& a, const Shape& s, WideShared<C>& sh, uint32_t smem,
                           const CUtensorMap* kmap, const CUtensorMap* vmap) {
  const int lane = threadIdx.x & 31;
  const int page = 1 << a.page_log2, ppt = kKeys >> a.page_log2;
  const uint32_t page_bytes = (uint32_t)page * C::kHD;
  uint32_t bad = 0, n = 0;  // n: tiles copied
  uint32_t tile_k = 0;      // K tiles copied
  bool ok = true;
  Walk w = {};
  for (w.start(a, s, sh.share); ok && w.left > 0; w.next(a, s)) {
    const int h = w.hh / s.nhb;
    const int32_t* row = a.table + (int64_t)w.r * a.max_pages;
    const int p_beg = w.g.lo >> a.page_log2, p_end = w.g.lo < w.g.hi ? (w.g.hi + page - 1) >> a.page_log2 : 0;
    // lane p: the id of the p-th page of a tile, -2 where the block sees nothing of it
    const auto id_of = [&](int i) {
      const int p = (w.g.tile + w.off + i) * ppt + lane;
      return i < w.take && lane < ppt && p >= p_beg && p < p_end ? row[p] : -2;
    };
    const auto there = [&](int32_t id) { return id >= 0 && id < a.n_pages; };
    const auto scale_of = [&](int32_t id) {
      const int64_t head = (int64_t)id * a.Hk + h;
      return there(id) ? make_float2(a.k_scale[head], a.v_scale[head]) : make_float2(0.0f, -1.0f);
    };
    const auto copy = [&](int32_t id, int i, const CUtensorMap* map) {
      const int st = (int)(n % C::kStages);
      ok = __all_sync(0xffffffffu, kv_wait(&sh.abort, sh.rempty[st], (n / C::kStages + 1) & 1u));
      if (!ok) return;
      const bool valid = there(id);
      const uint32_t mask = __ballot_sync(0xffffffffu, valid);
      const uint32_t bar = tc::smem_u32(&sh.rfull[st]);
      if (lane == 0) {
        const int key0 = (w.g.tile + w.off + i) * kKeys;
        sh.rows[st][0] = w.g.lo - key0;
        sh.rows[st][1] = w.g.hi - key0;
        sh.pages[st] = mask;
        tc::mbar_arrive_expect_tx(bar, __popc(mask) * page_bytes);
      }
      __syncwarp();
      if (valid)
        tma_rows(smem + C::kOffRaw + st * C::kRaw + lane * page_bytes, map, (int)(((int64_t)id * a.Hk + h) << a.page_log2), bar);
      ++n;
    };
    int unit_e = kLeastExp;  // exponent of the largest v_scale of the piece so far
    const auto scales = [&](float2 x) {
      const float vs = fmaxf(x.y, kLeastScale);
      unit_e = max(unit_e, __reduce_max_sync(0xffffffffu, x.y >= 0.0f ? pow2_above_exp(vs) : kLeastExp));
      const float w = fmaxf(vs * exp2i(kWideLift - unit_e), exp2i(kLeastWeight)), unit = exp2i(unit_e - kWideLift);
      if (lane < ppt)
        sh.sc[tile_k % C::kScales][lane] = x.y >= 0.0f ? make_float4(x.x, __log2f(w), __fdividef(1.0f, w), unit)
                                              : make_float4(0.0f, -INFINITY, 0.0f, unit);
      ++tile_k;
    };
    // ids two K tiles ahead, scales one
    int32_t id_v = id_of(0), id_k = id_v, id1 = id_of(1), id2;
    float2 sc = scale_of(id_k);
    for (int i = -1; ok && i < w.take; ++i) {  // K(i + 1), V(i)
      if (i + 1 < w.take) {
        if (id_k != -2 && !there(id_k)) bad = CSA2_DEV_BAD_INDEX;
        id2 = id_of(i + 3);
        const float2 next = scale_of(id1);
        scales(sc);
        copy(id_k, i + 1, kmap);
        sc = next;
      }
      if (ok && i >= 0) copy(id_v, i, vmap);
      id_v = id_k;
      id_k = id1;
      id1 = id2;
    }
  }
  if (!ok)  // given up: no copy may land after the CTA has gone
    for (uint32_t i = n > C::kStages ? n - C::kStages : 0; i < n; ++i)
      tc::mbar_wait(tc::smem_u32(&sh.rfull[i % C::kStages]), (i / C::kStages) & 1u, kKvPolls);
  if (bad) flag(a.status, bad);
}

// ---- E4M3 tiles to f16 tiles (128 threads) -------------------------------------------------
// A thread turns 8 codes into one 16-byte chunk at a time; its rows differ by multiples of 8, so
// the swizzle is the same for all of them.
template <class C, bool kAll>
__device__ __forceinline__ void convert_tile(uint32_t from, uint32_t to, int row0, int lo, int hi, uint32_t pages,
                                             int page_log2) {
  constexpr int kStep = 1024 / C::kHD;  // rows per 128 threads
  constexpr int kBatch = 8;  // loads in flight
#pragma unroll
  for (int b = 0; b < kKeys / kStep; b += kBatch) {
    uint32_t x[kBatch][2];
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(x[k][0]), "=r"(x[k][1]) : "r"(from + (b + k) * 1024) : "memory");
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if constexpr (!kAll) {
        // what no key of the block fills may be any bits: zeros, which zero probabilities keep
        const int row = row0 + (b + k) * kStep;
        if (row < lo || row >= hi || !((pages >> (row >> page_log2)) & 1u)) x[k][0] = x[k][1] = 0u;
      }
      tc::st_shared_v4(to + (b + k) * (kStep * 128),
                       make_uint4(f16x2_of_e4m3x2(x[k][0] & 0xFFFFu), f16x2_of_e4m3x2(x[k][0] >> 16),
                                  f16x2_of_e4m3x2(x[k][1] & 0xFFFFu), f16x2_of_e4m3x2(x[k][1] >> 16)));
    }
  }
}

template <class C>
__device__ void convert_tiles(const KvAttnArgs& a, WideShared<C>& sh, uint32_t smem) {
  constexpr int kChunks = C::kHD / 8;  // 8-code chunks per row
  const int tid = threadIdx.x & 127, row0 = tid / kChunks;
  const uint32_t chunk = tid % kChunks;
  const uint32_t from = smem + C::kOffRaw + tid * 8;
  const uint32_t to = smem + C::kOffRing + (chunk / 8) * C::kHalf + row0 * 128 + (((chunk ^ row0) & 7u) << 4);
  const uint32_t every = (1u << (kKeys >> a.page_log2)) - 1u;
  const int64_t items = 2 * sh.share.left;
  for (uint32_t n = 0; n < items; ++n) {
    const uint32_t st = n % C::kStages, slot = n % C::kRing;
    const bool ok = kv_wait(&sh.abort, sh.rfull[st], (n / C::kStages) & 1u) &&
                    kv_wait(&sh.abort, sh.empty[slot], (n / C::kRing + 1) & 1u);
    if (!__all_sync(0xffffffffu, ok)) return;
    const int lo = sh.rows[st][0], hi = sh.rows[st][1];
    const uint32_t pages = sh.pages[st];
    if (lo <= 0 && hi >= kKeys && pages == every)
      convert_tile<C, true>(from + st * C::kRaw, to + slot * C::kTile, row0, lo, hi, pages, a.page_log2);
    else
      convert_tile<C, false>(from + st * C::kRaw, to + slot * C::kTile, row0, lo, hi, pages, a.page_log2);
    tc::fence_async_smem();
    __syncwarp();
    if ((tid & 31) == 0) {  // one arrival per warp
      tc::mbar_arrive(tc::smem_u32(&sh.full[slot]));
      tc::mbar_arrive(tc::smem_u32(&sh.rempty[st]));
    }
  }
}

// ---- products (one warp) --------------------------------------------------------------------
template <class C>
__device__ void multiply_wide(WideShared<C>& sh, uint32_t smem, uint32_t tmem) {
  constexpr uint32_t kIdS = tc::idesc_f16(128, kKeys, false, false);
  constexpr uint32_t kIdO = tc::idesc_f16(128, C::kHD, false, true);
  const uint64_t dq0 = tc::smem_desc_sw128(smem + C::kOffQ, 16, 1024);
  const uint64_t dk0 = tc::smem_desc_sw128(smem + C::kOffRing, 16, 1024);
  const uint64_t dv0 = tc::smem_desc_sw128(smem + C::kOffRing, C::kHalf, 1024);
  uint32_t base = 0, piece = 0;  // ring items of the pieces before; pieces
  uint32_t np[2] = {0, 0};       // probabilities consumed per slot
  const bool on = (threadIdx.x & 31) == 0;
  bool ok = true;
  int take = 0;
  auto ring = [&](int i, bool v) {  // ring item of tile i of this piece
    return base + (v ? (i + 1 < take ? 2 * i + 2 : 2 * i + 1) : (i > 0 ? 2 * i - 1 : 0));
  };
  auto tile_there = [&](uint32_t item) {
    return kv_wait_all(sh, sh.full[item % C::kRing], (item / C::kRing) & 1u);
  };
  auto release = [&](uint32_t item) { commit_if(on, tc::smem_u32(&sh.empty[item % C::kRing])); };
  auto scores = [&](uint32_t item, int q, int g) {
    const uint64_t dk = tc::desc_add(dk0, (item % C::kRing) * C::kTile), dq = tc::desc_add(dq0, q * C::kTile);
#pragma unroll
    for (int k = 0; k < C::kHD / 16; ++k) {
      const uint32_t o = (k / 4) * C::kHalf + (k % 4) * 32;
      mma_ss(on, tmem + g * 128, tc::desc_add(dq, o), tc::desc_add(dk, o), kIdS, k > 0);
    }
    commit_if(on, tc::smem_u32(&sh.sfull[g]));
  };
  auto outputs = [&](uint32_t item, int g, bool fresh) {
    const uint64_t dv = tc::desc_add(dv0, (item % C::kRing) * C::kTile);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      ok = kv_wait_all(sh, sh.pfull[g][q], np[g] & 1u);
      if (!ok) return;
      tc::fence_after_sync();
#pragma unroll
      for (int k = 4 * q; k < 4 * q + 4; ++k)
        mma_ts(on, tmem + C::kColO + g * C::kHD, tmem + g * 128 + k * 8, tc::desc_add(dv, k * 2048), kIdO, !fresh || k > 0);
    }
    ++np[g];
  };
  for (int left = uniform((int)sh.share.left); ok && left > 0; left -= take, ++piece) {
    ok = kv_wait_all(sh, sh.qfull[0], piece & 1u) && kv_wait_all(sh, sh.qfull[1], piece & 1u);
    if (!ok) break;
    take = uniform(sh.take);
    const bool one_slot = C::NC == 128 || uniform(sh.one_slot) != 0;
    ok = tile_there(ring(0, false));
    if (!ok) break;
    tc::fence_after_sync();
    if (one_slot) {  // key tiles in turn
      scores(ring(0, false), 0, 0);
      release(ring(0, false));
      if (take > 1) {
        ok = tile_there(ring(1, false));
        if (!ok) break;
        scores(ring(1, false), 0, 1);
        release(ring(1, false));
      }
      for (int i = 0; ok && i < take; ++i) {
        ok = tile_there(ring(i, true)) && (i + 2 >= take || tile_there(ring(i + 2, false)));
        if (ok) outputs(ring(i, true), i & 1, i < 2);
        if (!ok) break;
        release(ring(i, true));
        if (i + 2 < take) {
          scores(ring(i + 2, false), 0, i & 1);
          release(ring(i + 2, false));
        }
      }
      if (ok) {
        commit_if(on, tc::smem_u32(&sh.ofull[0]));
        commit_if(on, tc::smem_u32(&sh.ofull[1]));
      }
    } else {
      scores(ring(0, false), 0, 0);
      scores(ring(0, false), 1, 1);
      release(ring(0, false));
      for (int i = 0; ok && i < take; ++i) {
        const bool last = i + 1 == take;
        ok = tile_there(ring(i, true)) && (last || tile_there(ring(i + 1, false)));
        if (ok) outputs(ring(i, true), 0, i == 0);
        if (!ok) break;
        if (last) commit_if(on, tc::smem_u32(&sh.ofull[0]));
        else scores(ring(i + 1, false), 0, 0);
        outputs(ring(i, true), 1, i == 0);
        if (!ok) break;
        release(ring(i, true));
        if (last) {
          commit_if(on, tc::smem_u32(&sh.ofull[1]));
        } else {
          scores(ring(i + 1, false), 1, 1);
          release(ring(i + 1, false));
        }
      }
    }
    base += 2 * take;
  }
  if (!ok) {  // given up: no product may run after the tensor memory is freed
    commit_if(on, tc::smem_u32(&sh.drain));
    tc::mbar_wait(tc::smem_u32(&sh.drain), 0, kKvPolls);
  }
}

// ---- softmax ---------------------------------------------------------------------------------
template <class C, typename T>
__device__ void soften_wide(const KvAttnArgs& a, const Shape& s, WideShared<C>& sh, uint8_t* smem_p, uint32_t tmem) {
  const uint32_t smem = tc::smem_u32(smem_p);
  const int tid = threadIdx.x, g = tid >> 7, row = tid & 127;
  const uint32_t lanes = tmem + ((uint32_t)((tid >> 5) & 3) << 21);
  const uint32_t s_at = lanes + g * 128, o_at = lanes + C::kColO + g * C::kHD;
  float4* joint = reinterpret_cast<float4*>(smem_p + C::kOffQ);  // every product with the queries is done by then
  const float cap2 = C::CAP ? a.softcap * kLog2e : 0.0f;
  if (tid == 0) a.meta[(int64_t)blockIdx.x * kMetaInts] = 0;
  bool bad = false;
  uint32_t n_s = 0, tile0 = 0, piece = 0;  // this slot's tiles; K tiles and pieces before this piece
  Walk w = {};
  for (w.start(a, s, sh.share); w.left > 0; w.next(a, s), ++piece) {
    const bool shared_rows = one_slot_rows<C>(s, w);
    const int c = shared_rows ? row : g * 128 + row;
    const int qi = c / s.HB, hd = c - qi * s.HB, i = w.qb * s.QB + qi;
    const int h = w.hh / s.nhb, hb = w.hh % s.nhb;
    const bool live = qi < s.QB && i < w.x.n && hd < s.G - hb * s.HB;
    const int64_t to = live ? (int64_t)(w.x.q0 + i) * a.Hq + h * s.G + hb * s.HB + hd : -1;
    const int64_t pos = (int64_t)w.x.pos0 + i;
    const int hi = !live || pos < 0 ? 0 : (pos + 1 < w.x.cap ? (int)pos + 1 : w.x.cap);
    const int lo = a.window > 0 && pos + 1 > a.window ? (int)(pos + 1 - a.window) : 0;
    // a warp without a query: its rows of Q are zero, so its scores are too, and their bits will do
    // for probabilities whose products nobody reads
    const bool idle = !__any_sync(0xffffffffu, live);
    float qs, m = 0.0f, l = 0.0f, unit = 1.0f;  // unit: what O's numbers count
    bool fresh = true;  // no key seen yet
    if (!bad) {  // the row as f16
      uint4 raw[C::kHD / 8];
#pragma unroll
      for (int k = 0; k < C::kHD / 8; ++k) raw[k] = make_uint4(0u, 0u, 0u, 0u);
      if (live) {
        const uint4* p = reinterpret_cast<const uint4*>(a.q + (int64_t)(w.x.q0 + i) * a.q_stride +
                                                        (int64_t)(h * s.G + hb * s.HB + hd) * (C::kHD * 2));
#pragma unroll
        for (int k = 0; k < C::kHD / 8; ++k) raw[k] = p[k];
      }
      float amax = 0.0f;
#pragma unroll
      for (int k = 0; k < C::kHD / 8; ++k) {
        float x[8];
        unpack8<T>(raw[k], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
      }
      int e = (int)(__float_as_uint(amax) >> 23) - 127;  // amax in [2^e, 2^(e+1))
      e = e < -112 ? -112 : e;  // both powers of two below are normal
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
      const float per = a.sm_scale * __uint_as_float((uint32_t)(127 + e - 14) << 23);
      // an infinite element leaves no digits of the others: the row's scores are NaN
      qs = isinf(amax) ? __int_as_float(0x7FFFFFFF) : C::CAP ? per / a.softcap : per * kLog2e;
      if (!shared_rows || g == 0) {
#pragma unroll
        for (int k = 0; k < C::kHD / 8; ++k) {
          float x[8];
          unpack8<T>(raw[k], x);
          uint32_t y[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const __half2 v = __floats2half2_rn(x[2 * j] * up, x[2 * j + 1] * up);
            y[j] = *reinterpret_cast<const uint32_t*>(&v);
          }
          tc::st_shared_v4(smem + C::kOffQ + g * C::kTile + (k / 8) * C::kHalf + tc::swz(row, (k % 8) * 16, 128),
                           make_uint4(y[0], y[1], y[2], y[3]));
        }
      }
      if (tid == 0) {
        sh.take = w.take;
        sh.one_slot = shared_rows;
      }
      tc::fence_async_smem();
      __syncwarp();
      if ((tid & 31) == 0) tc::mbar_arrive(tc::smem_u32(&sh.qfull[g]));
    }
    // keys that every row of the block sees: the first query ends soonest, the last starts latest
    const int last_q = (w.qb + 1) * s.QB < w.x.n ? (w.qb + 1) * s.QB - 1 : w.x.n - 1;
    const int64_t all_hi64 = (int64_t)w.x.pos0 + w.qb * s.QB + 1;
    const int all_hi = all_hi64 < 0 ? 0 : (all_hi64 < w.x.cap ? (int)all_hi64 : w.x.cap);
    const int64_t all_lo = a.window > 0 ? (int64_t)w.x.pos0 + last_q + 1 - a.window : 0;
    const int by = shared_rows ? 2 : 1, first_tile = shared_rows ? g : 0;
    for (int j = first_tile; !bad && j < w.take; j += by, ++n_s) {
      const float4* sc = sh.sc[(tile0 + j) % C::kScales];
      bad = !__all_sync(0xffffffffu, kv_wait(&sh.abort, sh.sfull[g], n_s & 1u));
      if (bad) break;
      if (idle) {
        if ((tid & 31) == 0) {
          tc::mbar_arrive(tc::smem_u32(&sh.pfull[g][0]));
          tc::mbar_arrive(tc::smem_u32(&sh.pfull[g][1]));
        }
        continue;
      }
      tc::fence_after_sync();
      union {
        uint32_t u[128];
        float f[128];
      } t;
      tmem_ld128(s_at, t.u);
      const int key0 = (w.g.tile + w.off + j) * kKeys;
      if constexpr (C::CAP) {
        float most = 0.0f;
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const float k2 = sc[(p * 16) >> a.page_log2].x * qs;
          const uint64_t kk = pack2(k2, k2);
#pragma unroll
          for (int k = p * 16; k < p * 16 + 16; k += 2) {
            unpack2(mul2(pack2(t.f[k], t.f[k + 1]), kk), t.f[k], t.f[k + 1]);
            most = fmaxf(most, fmaxf(fabsf(t.f[k]), fabsf(t.f[k + 1])));
          }
        }
        if (__all_sync(0xffffffffu, most <= kTanhSmall)) {  // the same for the warp: scores well below the cap
          const uint64_t c1 = pack2(kTanh1, kTanh1), c2 = pack2(kTanh2, kTanh2), c3 = pack2(kTanh3, kTanh3),
                         c4 = pack2(kTanh4, kTanh4), c5 = pack2(kTanh5, kTanh5), cap = pack2(cap2, cap2);
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const float o = sc[(p * 16) >> a.page_log2].y - m;
            const uint64_t off = pack2(o, o);
#pragma unroll
            for (int k = p * 16; k < p * 16 + 16; k += 2) {
              const uint64_t x = pack2(t.f[k], t.f[k + 1]), z = mul2(x, x);
              const uint64_t q = fma2(fma2(fma2(fma2(c5, z, c4), z, c3), z, c2), z, c1);
              unpack2(fma2(cap, fma2(mul2(x, z), q, x), off), t.f[k], t.f[k + 1]);
            }
          }
        } else {
#pragma unroll
          for (int p = 0; p < 8; ++p) {
            const float off = sc[(p * 16) >> a.page_log2].y - m;
#pragma unroll
            for (int k = p * 16; k < p * 16 + 16; ++k) t.f[k] = fmaf(cap2, tanh_any(t.f[k]), off);
          }
        }
      } else {
#pragma unroll
        for (int p = 0; p < 8; ++p) {
          const float4 x = sc[(p * 16) >> a.page_log2];
          const uint64_t k2 = pack2(x.x * qs, x.x * qs), off = pack2(x.y - m, x.y - m);
#pragma unroll
          for (int k = p * 16; k < p * 16 + 16; k += 2)
            unpack2(fma2(pack2(t.f[k], t.f[k + 1]), k2, off), t.f[k], t.f[k + 1]);
        }
      }
      if (key0 + kKeys > all_hi || key0 < all_lo) {
        const int nhi = hi - key0, nlo = lo - key0;
#pragma unroll
        for (int k = 0; k < 128; ++k)
          if (k >= nhi || k < nlo) t.f[k] = -INFINITY;
      }
      float mx[4] = {t.f[0], t.f[1], t.f[2], t.f[3]};
#pragma unroll
      for (int k = 4; k + 7 < 128; k += 8)
#pragma unroll
        for (int x = 0; x < 4; ++x) mx[x] = max3(mx[x], t.f[k + 2 * x], t.f[k + 2 * x + 1]);
#pragma unroll
      for (int x = 0; x < 4; ++x) mx[x] = fmaxf(mx[x], t.f[124 + x]);
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) - kWideLift;
      const bool raise = fresh ? top > -INFINITY : top > kWideSlack;
      const float unit_j = sc[0].w;
      if (__any_sync(0xffffffffu, raise || unit_j != unit)) {
        const float up = raise ? top : 0.0f, f = fresh ? 1.0f : exp2_approx(-up), f_o = f * (unit * pow2_inverse(unit_j));
        unit = unit_j;
        m += up;
        l *= f;
        fresh = fresh && !raise;
#pragma unroll
        for (int k = 0; k < 128; ++k) t.f[k] -= up;
        if (j != first_tile) {  // the products of the tiles before are complete: S was issued after them
#pragma unroll
          for (int k = 0; k < C::kHD; k += 16) {
            uint32_t o[16];
            tc::tmem_ld16(o_at + k, o);
#pragma unroll
            for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * f_o);
            tc::tmem_st16_nowait(o_at + k, o);
          }
        }
      }
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        uint32_t pk[32];
#pragma unroll
        for (int p = 4 * q; p < 4 * q + 4; ++p) {
          uint64_t sum = pack2(0.0f, 0.0f);
#pragma unroll
          for (int k = p * 16; k < p * 16 + 16; k += 2) {
            const float p0 = exp2_approx(t.f[k]), p1 = exp2_approx(t.f[k + 1]);
            sum = add2(sum, pack2(p0, p1));
            const __half2 v = __floats2half2_rn(p0, p1);
            pk[k / 2 - q * 32] = *reinterpret_cast<const uint32_t*>(&v);
          }
          float even, odd;
          unpack2(sum, even, odd);
          l = fmaf(even + odd, sc[(p * 16) >> a.page_log2].z, l);
        }
        tc::tmem_st32_nowait(s_at + q * 32, pk);
        tc::tmem_wait_st();
        tc::fence_before_sync();
        __syncwarp();
        if ((tid & 31) == 0) tc::mbar_arrive(tc::smem_u32(&sh.pfull[g][q]));  // the products of these 64 keys may start
      }
    }
    tile0 += w.take;
    if (!bad) bad = !__all_sync(0xffffffffu, kv_wait(&sh.abort, sh.ofull[g], piece & 1u));
    float f0 = unit, f1 = 0.0f;
    if (shared_rows) {  // slot 1's maximum, sum and unit to slot 0, which joins them
      if (g == 1) joint[row] = make_float4(m, l, unit, 0.0f);
      bad = tc::named_sync_or(1, 256, bad);
      if (g == 0) {
        const float4 o = joint[row];
        const float both = l == 0.0f ? o.x : (o.y == 0.0f ? m : fmaxf(m, o.x));
        f0 = l == 0.0f ? 0.0f : exp2f(m - both);
        f1 = o.y == 0.0f ? 0.0f : exp2f(o.x - both);
        l = (l == 0.0f ? 0.0f : l * f0) + (o.y == 0.0f ? 0.0f : o.y * f1);
        f0 *= unit;
        f1 *= o.z;
        m = both;
      }
    }
    tc::fence_after_sync();
    if (!bad && !(shared_rows && g == 1)) {
      const bool whole = w.first && w.last, join = shared_rows && w.take > 1;
      float* part = a.part + ((int64_t)blockIdx.x * 2 + (w.first ? 1 : 0)) * (C::NC * (C::kHD + 2));
      const float inv = l != 0.0f ? __fdiv_rn(1.0f, l) : 0.0f;
      f0 *= inv;
      f1 *= inv;
      if (whole) {
        if (a.lse && to >= 0) a.lse[to] = l != 0.0f ? (m + log2f(l)) * kLn2 : -INFINITY;
      } else if (live) {
        *reinterpret_cast<float2*>(part + C::NC * C::kHD + 2 * c) = make_float2(m, l);
      }
#pragma unroll
      for (int k = 0; k < C::kHD; k += 16) {
        uint32_t o[16];
        float x[16];
        tc::tmem_ld16(o_at + k, o);
#pragma unroll
        for (int y = 0; y < 16; ++y) x[y] = __uint_as_float(o[y]) * f0;
        if (join) {
          tc::tmem_ld16(o_at + C::kHD + k, o);
#pragma unroll
          for (int y = 0; y < 16; ++y) x[y] = fmaf(__uint_as_float(o[y]), f1, x[y]);
        }
        if (!live) continue;
        if (whole) {
          uint32_t y[8];
#pragma unroll
          for (int z = 0; z < 8; ++z) {
            const T lo16 = from_float<T>(x[2 * z]), hi16 = from_float<T>(x[2 * z + 1]);
            y[z] = (uint32_t)*reinterpret_cast<const uint16_t*>(&lo16) |
                   ((uint32_t)*reinterpret_cast<const uint16_t*>(&hi16) << 16);
          }
          uint4* out = reinterpret_cast<uint4*>(a.out + (to * C::kHD + k) * 2);
          out[0] = make_uint4(y[0], y[1], y[2], y[3]);
          out[1] = make_uint4(y[4], y[5], y[6], y[7]);
        } else {
          float4* out = reinterpret_cast<float4*>(part + c * C::kHD + k);
#pragma unroll
          for (int z = 0; z < 4; ++z) out[z] = make_float4(x[4 * z], x[4 * z + 1], x[4 * z + 2], x[4 * z + 3]);
        }
      }
      if (!whole && w.first && tid == 0) note_item(a, sh.share, w);
    }
    tc::fence_before_sync();
    if (shared_rows)  // slot 1's output has been read, the next piece may overwrite it
      bad = tc::named_sync_or(1, 256, bad);
  }
}

template <class C, typename T>
__global__ void __launch_bounds__(C::kThreads, 1) kv8_wide_kernel(const __grid_constant__ CUtensorMap kmap,
                                                                   const __grid_constant__ CUtensorMap vmap,
                                                                   const KvAttnArgs a) {
  extern __shared__ uint8_t raw[];
  __shared__ WideShared<C> sh;
  uint8_t* smem = tc::align_smem_1024(raw);
  const int tid = threadIdx.x, warp = uniform(tid >> 5);
  if (tid == 0) {
    for (int i = 0; i < C::kStages; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.rfull[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh.rempty[i]), 4);
    }
    for (int i = 0; i < C::kRing; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.full[i]), 4);
      tc::mbar_init(tc::smem_u32(&sh.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_u32(&sh.qfull[i]), 4);
      tc::mbar_init(tc::smem_u32(&sh.sfull[i]), 1);
      tc::mbar_init(tc::smem_u32(&sh.pfull[i][0]), 4);
      tc::mbar_init(tc::smem_u32(&sh.pfull[i][1]), 4);
      tc::mbar_init(tc::smem_u32(&sh.ofull[i]), 1);
    }
    tc::mbar_init(tc::smem_u32(&sh.drain), 1);
    sh.abort = 0;
  }
  // tensor memory in launch order, as in kv8_attn_kernel
  chain_wait();
  if (warp == 0) tc::tmem_alloc(tc::smem_u32(&sh.tmem), 512);
  const Shape s = shape_of<C::NC>(a);
  uint32_t bad = 0;
  find_share<C::kThreads>(a, s, reinterpret_cast<int64_t*>(smem), &sh.share, &bad);
  if (bad && blockIdx.x == 0) flag(a.status, bad);
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  chain_launch_dependents();
  const uint32_t tmem = uniform(sh.tmem);
  if (warp < 8) {
    reg_inc<C::kRegsSoft>();
    soften_wide<C, T>(a, s, sh, smem, tmem);
  } else if (warp < 12) {
    reg_dec<C::kRegsConv>();
    convert_tiles<C>(a, sh, tc::smem_u32(smem));
  } else {
    reg_dec<C::kRegsMma>();
    if (warp == 12) multiply_wide<C>(sh, tc::smem_u32(smem), tmem);
    else if (warp == 13) load_tiles<C>(a, s, sh, tc::smem_u32(smem), &kmap, &vmap);
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
  if (tid == 0 && sh.abort) flag(a.status, CSA2_DEV_TIMEOUT);
}

// ---- host ------------------------------------------------------------------------------------
size_t kv8_wide_workspace_bytes(int hd, int rows, int num_sms) {
  return (size_t)num_sms * 2 * rows * (hd + 2) * sizeof(float) + (size_t)num_sms * kMetaInts * sizeof(int32_t);
}

template <class C, typename T>
static cudaError_t launch_wide_t(KvAttnArgs a, const CUtensorMap& km, const CUtensorMap& vm, void* ws, int num_sms,
                                 cudaStream_t stream) {
  cudaFuncAttributes f;
  cudaError_t e = cudaFuncGetAttributes(&f, kv8_wide_kernel<C, T>);
  if (e != cudaSuccess) return e;
  // the warpgroups' register shares come out of what the launch gives
  if (f.numRegs * C::kThreads < 256 * C::kRegsSoft + 128 * (C::kRegsConv + C::kRegsMma)) return cudaErrorInvalidConfiguration;
  a.part = static_cast<float*>(ws);
  a.meta = reinterpret_cast<int32_t*>(a.part + (size_t)num_sms * 2 * C::NC * (C::kHD + 2));
  e = cudaFuncSetAttribute(kv8_wide_kernel<C, T>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  e = launch_chained(kv8_wide_kernel<C, T>, dim3(num_sms), dim3(C::kThreads), C::kSmem, stream, 0, km, vm, a);
  if (e != cudaSuccess) return e;
  e = launch_chained(kv8_merge_kernel<C::NC, C::kHD, T>, dim3(num_sms, C::NC / 8), dim3(kMergeThreads), 0,
                     stream, 0, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int HD, int ROWS, bool CAP>
static cudaError_t launch_wide_type(int f16, const KvAttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, void* ws,
                                    int num_sms, cudaStream_t stream) {
  return f16 ? launch_wide_t<KvWide<HD, ROWS, CAP>, __half>(a, km, vm, ws, num_sms, stream)
             : launch_wide_t<KvWide<HD, ROWS, CAP>, __nv_bfloat16>(a, km, vm, ws, num_sms, stream);
}
template <int HD, int ROWS>
static cudaError_t launch_wide_cap(int f16, const KvAttnArgs& a, const CUtensorMap& km, const CUtensorMap& vm, void* ws,
                                   int num_sms, cudaStream_t stream) {
  return a.softcap > 0.0f ? launch_wide_type<HD, ROWS, true>(f16, a, km, vm, ws, num_sms, stream)
                          : launch_wide_type<HD, ROWS, false>(f16, a, km, vm, ws, num_sms, stream);
}

cudaError_t launch_kv8_wide(const KvAttnArgs& a, int f16, int hd, int rows, const CUtensorMap& km, const CUtensorMap& vm,
                            void* ws, int num_sms, cudaStream_t stream) {
  if (hd == 64)
    return rows == 128 ? launch_wide_cap<64, 128>(f16, a, km, vm, ws, num_sms, stream)
                       : launch_wide_cap<64, 256>(f16, a, km, vm, ws, num_sms, stream);
  return rows == 128 ? launch_wide_cap<128, 128>(f16, a, km, vm, ws, num_sms, stream)
                     : launch_wide_cap<128, 256>(f16, a, km, vm, ws, num_sms, stream);
}

}  // namespace csa2
