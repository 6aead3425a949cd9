// kernel_wide_sm103.cu -- the decode for trees with many rows, on clusters of two CTAs whose tensor
// cores work on one product together (cta_group::2).
//
// A unit is up to 128 packed rows (row = token * H + head) of one request against a page-aligned key
// range, in tiles of 128 keys = two pages. CTA r of the pair holds 64 of the rows:
//
//   S[row, key]  = Q[row, 0:576] . K[key, 0:576]^T      (M = 128 rows, N = 128 keys, 36 or 18 K-steps)
//   O[row, dv]  += P[row, key] . V[key, dv]              (M = 128, N = 256 values, twice; K = 128 keys)
//
// Of a product's two operands a CTA holds its own rows of the left one and half of the right one: page
// r of a tile for S, and its 256 of the 512 value columns of both pages for O. What the two SMs read
// from shared memory for a row and a page is 1.9 KB, where the 48-row tiles of one CTA read 4.5 KB
// (kernel_sm103.cu; that pipe is what bounds them), and a product of 128 rows runs at the tensor
// cores' full rate, where those run at half of it (M = 64 keys) for S. The price is that a CTA's page
// comes twice for its half of the value columns: 136 KB a tile (bf16) and SM, mostly from L2.
//
// The accumulators of M = 128 in a pair: rows of CTA r in lanes 0-63 and, for the upper half of N,
// again in lanes 64-127 of its tensor memory. So a softmax thread has one row and one page of it.
//
// Tensor memory (columns): O at 0-127 (values 0-255) and 128-255 (values 256-511), S in two buffers
// at 256 and 320. Shared memory: Q, the page ring (bf16: one page in three pieces of three 64-column
// chunks, so that a piece is refilled while the product goes on; e4m3: two pages), the value columns
// of a tile's two pages, P of the two pages. O takes the pages one after the other, so that P and the
// values of one are replaced while the other's product runs.
//
// Warps: 0 copies of pages, 3 of value columns. 1: in CTA 0 issues S, in CTA 1 tells CTA 0 that its
// pieces have landed; 2 the same for O. 4-11 softmax: warp (lane quadrant, group) has 32 of the 64 keys
// of its lanes' page. A row's reference moves only when a score passes it by some octaves, as in
// the narrow kernel; the rows of the two CTAs need not agree on that.
// Measured: 4 x 64 nodes, 16 heads, 32768 bf16 keys 187 us (1.57 PFLOP/s, 0.83 of the measured peak; in
// 48-row tiles 512): products and page copies share the shared memory. 32 trees of 5 to 16 nodes, 48
// heads, 8k to 16k keys over block scales 366 us, where the softmax warps' work on P's two 8-bit parts
// and the moves of references bound it.
// Every wait is bounded; a CTA whose wait gave up stops, and the other one's waits end likewise.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <stdint.h>

#include <mutex>

#include "decode_common.cuh"
#include "mla_decode.h"
#include "plan_format.h"
#include "ptx.cuh"
#include "softmax_parts.cuh"
#include "status.h"

namespace mla {
namespace wide {

constexpr int kRows = 128, kHalfRows = 64;
constexpr int kTileKeys = 128;  // two pages
constexpr int kChunks = 9;
constexpr int kThreads = 384;
// Octaves that a score may pass its row's reference by before that moves (bf16 P). P and the sums are
// floating-point numbers, so a late reference costs no bits, only range: P up to 2^32. With the 8
// octaves of the narrow kernel most tiles had one of 128 rows move (4 x 64 nodes, 16 heads, 32768
// keys: 325 us; with 32 314, and most of what else was then won).
constexpr float kRefSlackWide = 32.0f;
constexpr uint32_t kTmemO = 0, kTmemS = 256, kTmemCols = 512;

template <bool kFp8>
struct Geo {
  static constexpr int kRowBytes = kFp8 ? 64 : 128;         // a key's 64 columns of a chunk
  static constexpr int kChunkBytes = kPage * kRowBytes;
  static constexpr int kQChunkBytes = kHalfRows * 128;      // bf16, or e4m3 in two parts of 4096
  static constexpr int kPieces = kFp8 ? 1 : 3;              // of a page
  static constexpr int kPieceChunks = kChunks / kPieces;
  static constexpr int kSlots = kFp8 ? 2 : 3;             // of the page ring, a piece each
  static constexpr int kSlotBytes = kPieceChunks * kChunkBytes;
  static constexpr int kVPage = 4 * kChunkBytes;            // a page's 64 keys x 128 values of either half
  static constexpr int kPBytes = 2 * kHalfRows * 128;       // 64 rows x 128 keys, bf16 or two 8-bit parts
  static constexpr int kOffK = kChunks * kQChunkBytes;
  static constexpr int kOffV = kOffK + kSlots * kSlotBytes;
  static constexpr int kOffP = kOffV + 2 * kVPage;
  static constexpr int kOffScales = kOffP + kPBytes;        // e4m3: block scales of two tiles
  static constexpr int kScaleBytes = kTileKeys / 2 * 24;    // of a tile, by pairs of keys
  static constexpr int kOffMisc = kOffScales + (kFp8 ? 2 * kScaleBytes : 0);
  static constexpr int kMiscBytes = 2816;
  static constexpr int kSmem = kOffMisc + kMiscBytes;
  static_assert(kSmem <= 232448, "exceeds the 227 KB per-CTA shared memory");
  static_assert(kOffK % 1024 == 0 && kOffV % 1024 == 0 && kOffP % 1024 == 0, "swizzle atoms");
};

// Scales of an e4m3 cache: one for all; a thread's 32 keys in one block, so that they come with one load;
// smaller blocks, with a load for each pair of keys.
enum : int { kOneScale = 0, kLargeBlocks = 1, kSmallBlocks = 2 };

struct Misc {
  uint64_t q_full;
  uint64_t k_full[3], k_empty[3], k_peer[3];  // pieces: landed here; read by S; landed in CTA 1
  uint64_t v_full[2], v_empty[2], v_peer[2];  // by page of the tile
  uint64_t s_full[2], s_empty[2];
  uint64_t p_ready[2][2], o_done[2][2];       // by page of the tile, the tile's parity
  uint64_t sc_full[2], sc_free[2];            // a tile's scales
  uint64_t drained[2];
  uint32_t tmem_base;
  int abort;
  int unit[12];
  float red[4][kHalfRows];                    // by (page of the tile, group): maxima, then sums
  float colscale[kHalfRows];                  // e4m3: score scale of a row
};
static_assert(sizeof(Misc) <= Geo<false>::kMiscBytes, "misc block too small");

// ---------------------------------------------------------------- cta_group::2
__device__ __forceinline__ void tmem_alloc2(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(ptx::smem_addr(dst)), "r"(cols) : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() { asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_dealloc2(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
template <bool kFp8>
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if constexpr (kFp8)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrive on `bar` of both CTAs once every product that this thread issued has completed.
__device__ __forceinline__ void commit_both(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(ptx::smem_addr(bar)),
      "h"((uint16_t)3)
      : "memory");
}
__device__ __forceinline__ void commit_here(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(ptx::smem_addr(bar)) : "memory");
}
// 32 lanes x 32 columns: thread i of the warp gets lane (base lane + i).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
               "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])), "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15])),
               "r"(__float_as_uint(v[16])), "r"(__float_as_uint(v[17])), "r"(__float_as_uint(v[18])), "r"(__float_as_uint(v[19])), "r"(__float_as_uint(v[20])), "r"(__float_as_uint(v[21])), "r"(__float_as_uint(v[22])), "r"(__float_as_uint(v[23])),
               "r"(__float_as_uint(v[24])), "r"(__float_as_uint(v[25])), "r"(__float_as_uint(v[26])), "r"(__float_as_uint(v[27])), "r"(__float_as_uint(v[28])), "r"(__float_as_uint(v[29])), "r"(__float_as_uint(v[30])), "r"(__float_as_uint(v[31]))
               : "memory");
}

// Arrive on a barrier of CTA 0. What it announces (P, copies that have landed, scores that have been
// read) lies in this CTA's own shared and tensor memory and is only touched there, by its own SM's tensor
// core, to which fence.proxy.async or tcgen05.fence has handed it over before; so the arrival releases
// at CTA scope, also from CTA 1. (A release at cluster scope waits for all of a warp's stores to be
// seen by the other SM: 4 x 64 nodes over 32768 bf16 keys 314 us, 247 so.)
__device__ __forceinline__ void arrive_first(uint64_t* bar, uint32_t rank) {
  if (rank == 0)
    ptx::mbar_arrive(bar);
  else
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(ptx::mapa(ptx::smem_addr(bar), 0)) : "memory");
}

// The dither of split_p for keys j and j + 1 in the upper bytes of two halves: multiples of the golden
// ratio, modulo 1, in 16 bits (an even j's half may carry into its neighbour's, which is as good).
constexpr uint32_t kDither16 = 0x9E37u, kDither2Step = (2u * kDither16 & 0xFFFFu) * 0x10001u;
__device__ __forceinline__ uint32_t dither2_of(int j) {
  const uint32_t a = kDither16 * (uint32_t)j;
  return (a & 0xFFFFu) | (a + kDither16) << 16;
}

template <bool kFp8, int kScales>
__device__ __forceinline__ void softmax_role(uint8_t* smem, Misc* ms, const Params& p, uint32_t tmem, uint32_t rank, int qd,
                                             int grp, int lane, int sidx) {
  using G = Geo<kFp8>;
  constexpr bool kScaled = kScales != kOneScale;
  constexpr float kPShift = kFp8 ? kPShiftFp8 : 0.f;
  constexpr float kMoveAbove = (kFp8 ? kRefSlackFp8 : kRefSlackWide) + kPShift;
  volatile int* abort = &ms->abort;
  const int b = ms->unit[0], qrow0 = ms->unit[1] + kHalfRows * (int)rank;
  const int nrows = max(0, min(kHalfRows, ms->unit[2] - kHalfRows * (int)rank));
  const int kv_begin = ms->unit[3], kv_end = ms->unit[4], ctx = ms->unit[8], qlen = ms->unit[9], tok0 = ms->unit[10];
  const int part_row0 = ms->unit[5] < 0 ? -1 : ms->unit[5] + kHalfRows * (int)rank;
  const int ntiles = (kv_end - kv_begin + kTileKeys - 1) / kTileKeys;
  const int row = (qd & 1) * 32 + lane, pg = qd >> 1;  // this thread's row, its page of a tile
  const int w8 = sidx >> 5;
  const uint32_t lanes = (uint32_t)(qd * 32) << 16;
  const int n0 = ctx - qlen;  // keys before the request's verify tokens
  const bool live = row < nrows;
  const int tok = live ? (qrow0 + row) / p.H : 0;
  const int lim = live ? (p.tree_masks ? n0 : n0 + tok - tok0 + 1) : 0;
  const uint32_t* words = p.tree_masks ? p.tree_masks + (size_t)tok * p.mask_words : nullptr;
  // the keys that every row of the unit sees: those before the verify tokens, for a chain one more
  const int all_see = min(kv_end, n0);
  if (sidx == 0 && (p.seq_lens[b] != ctx || p.q_lens[b] != qlen)) {
    report(p.status, MLA_DEVICE_PLAN_MISMATCH);
    *abort = 1;
  }
  float cs = p.score_scale_log2;
  if constexpr (kFp8) {
    // Q rows -> e4m3 hi and lo rows, as in the narrow kernel; rows w8, w8 + 8, ..
#pragma unroll 1
    for (int k0 = 0; k0 < 8; k0 += 4) {
      uint32_t raw[4][9];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int grow = qrow0 + w8 + 8 * (k0 + k);
        const uint32_t* src = reinterpret_cast<const uint32_t*>(p.q + (size_t)grow * kDqk + 18 * lane);
#pragma unroll
        for (int j = 0; j < 9; ++j) raw[k][j] = grow < p.q_rows ? src[j] : 0u;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = w8 + 8 * (k0 + k);
        float v[18];
        float mx = 0.f;
#pragma unroll
        for (int j = 0; j < 9; ++j) {
          const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&raw[k][j]));
          v[2 * j] = f.x;
          v[2 * j + 1] = f.y;
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        int e = 0;
        if (mx > 0.f && mx < INFINITY) e = max(-100, min(100, 7 - ((int)((__float_as_uint(mx) >> 23) & 0xFF) - 127)));
        const float sc = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
        for (int j = 0; j < 18; j += 2) {
          const float w0 = v[j] * sc, w1 = v[j + 1] * sc;
          const float h0 = round_to_e4m3_precision(w0), h1 = round_to_e4m3_precision(w1);
          const int col = 18 * lane + j;
          uint8_t* chunk = smem + (col >> 6) * G::kQChunkBytes;
          *reinterpret_cast<uint16_t*>(chunk + sw64_offset(r, col & 63)) = (uint16_t)e4m3x2(h0, h1);
          *reinterpret_cast<uint16_t*>(chunk + kHalfRows * 64 + sw64_offset(r, col & 63)) = (uint16_t)e4m3x2(w0 - h0, w1 - h1);
        }
        if (lane == 0) ms->colscale[r] = p.score_scale_log2 * __uint_as_float((uint32_t)(127 - e) << 23);
      }
    }
    ptx::fence_async_smem();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&ms->q_full);
  }
  bool stop = softmax_any(*abort != 0), fail = false;
  if (kFp8) cs = ms->colscale[row];
  float4 one = make_float4(0.f, 0.f, 0.f, 0.f);  // kLargeBlocks: the scale of this thread's keys, times cs; its logarithm in .z
  // x (v cs) + log2 v of keys i and i + 1
  auto in_octaves = [&](float2 v, const float4* scales, int i) {
    if constexpr (kScales == kOneScale) return ptx::mul2(v, make_float2(cs, cs));
    if constexpr (kScales == kLargeBlocks) return ptx::fma2(v, make_float2(one.x, one.x), make_float2(one.z, one.z));
    const float4 a = scales[i / 2];
    return ptx::fma2(ptx::mul2(v, make_float2(cs, cs)), make_float2(a.x, a.y), make_float2(a.z, a.w));
  };
  auto o_done = [&](int k, int u) { return warp_wait(&ms->o_done[k][u & 1], (u >> 1) & 1, abort, p); };  // O of page k of tile u
  float ref = -INFINITY, l = 0.f;
  for (int t = 0; !stop && t < ntiles; ++t) {
    const int sb = t & 1;
    const int key0 = kv_begin + t * kTileKeys + kPage * pg + 32 * grp;  // this thread's 32 keys
    uint32_t sees = 0xffffffffu;
    if (__builtin_expect(kv_begin + (t + 1) * kTileKeys > all_see, 0)) {
      // up to 32 bits: keys before the verify tokens, then the mask's or the chain's
      const int d = key0 - n0;
      const int left = kv_end - key0;
      if (words) {
        uint32_t bits;
        if (d >= 0) {
          const int w = d >> 5, wn = (qlen + 31) >> 5;
          const uint32_t lo = w < wn ? __ldg(words + w) : 0u, hi = w + 1 < wn ? __ldg(words + w + 1) : 0u;
          bits = __funnelshift_r(lo, hi, d & 31);
        } else if (d <= -32) {
          bits = 0xffffffffu;
        } else {
          bits = (__ldg(words) << -d) | ((1u << -d) - 1u);
        }
        sees = bits;
      } else {
        const int n = lim - key0;
        sees = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
      }
      // (bits from the last token on are not looked at: those keys lie behind kv_end, or the range's end)
      if (left < 32) sees &= left <= 0 ? 0u : (1u << left) - 1u;
      if (!live) sees = 0u;
    }
    float x[32], top = -INFINITY;
    bool need = false;
    if (!fail) fail = !warp_wait(&ms->s_full[sb], (t >> 1) & 1, abort, p);
    if (kScaled && !fail) fail = !warp_wait(&ms->sc_full[sb], (t >> 1) & 1, abort, p);
    // block scales of this thread's pairs of keys: (v, v', log2 v, log2 v'), and (1 / v, 1 / v')
    const uint8_t* table = smem + G::kOffScales + sb * G::kScaleBytes;
    const float4* scales = reinterpret_cast<const float4*>(table) + (kPage * pg + 32 * grp) / 2;
    const float2* inverse = reinterpret_cast<const float2*>(table + kTileKeys / 2 * 16) + (kPage * pg + 32 * grp) / 2;
    if (!fail) {
      ptx::tc_fence_after();
      tmem_ld32(tmem + kTmemS + 64 * sb + 32 * grp + lanes, x);
      ptx::tmem_ld_wait();
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive_first(&ms->s_empty[sb], rank);
      if constexpr (kScales == kLargeBlocks) {
        one = scales[0];
        one.x *= cs;
      }
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 v = in_octaves(make_float2(x[i], x[i + 1]), scales, i);
        x[i] = v.x;
        x[i + 1] = v.y;
      }
      if (__builtin_expect(sees != 0xffffffffu, 0)) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = (sees >> i) & 1u ? x[i] : -INFINITY;
      }
      top = x[0];
#pragma unroll
      for (int i = 1; i < 32; ++i) top = fmaxf(top, x[i]);
      need = top > ref + kMoveAbove;
    }
    const bool moved = softmax_any(need || fail);
    float alpha = 1.f;
    if (moved) {
      if constexpr (kFp8) {
        // With little room above a reference (P is 8 bits wide) moves are frequent: look at the next
        // tile's scores too, where all rows see all of it; it would move many of the same rows (29 nodes,
        // 12 heads, 2^18 keys 157 -> 150 us).
        if (!fail && kv_begin + (t + 2) * kTileKeys <= all_see) {
          const int nb = (t + 1) & 1;
          fail = !warp_wait(&ms->s_full[nb], ((t + 1) >> 1) & 1, abort, p);
          if (kScaled && !fail) fail = !warp_wait(&ms->sc_full[nb], ((t + 1) >> 1) & 1, abort, p);
          if (!fail) {
            float y[32];
            const float4* next = reinterpret_cast<const float4*>(smem + G::kOffScales + nb * G::kScaleBytes) + (kPage * pg + 32 * grp) / 2;
            ptx::tc_fence_after();
            tmem_ld32(tmem + kTmemS + 64 * nb + 32 * grp + lanes, y);
            ptx::tmem_ld_wait();
            ptx::tc_fence_before();
            if constexpr (kScales == kLargeBlocks) {
              one = next[0];
              one.x *= cs;
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const float2 v = in_octaves(make_float2(y[i], y[i + 1]), next, i);
              top = fmaxf(top, fmaxf(v.x, v.y));
            }
          }
        }
      }
      ms->red[2 * pg + grp][row] = top;
      if (softmax_any(fail || *abort != 0)) {
        stop = true;
        break;
      }
      const float m = fmaxf(fmaxf(ms->red[0][row], ms->red[1][row]), fmaxf(ms->red[2][row], ms->red[3][row]));
      const float nw = fmaxf(ref, m - kPShift);
      alpha = nw == ref ? 1.f : ex2(ref - nw);
      ref = nw;
      l *= alpha;
    }
    // O of the rows that move, between O(t - 1) and O(t); all warps' before any P(t) is handed on
    auto rescale = [&]() {
      if (t >= 1 && !fail) {
        for (int k = 0; k < 2 && !fail; ++k) fail = !o_done(k, t - 1);
        if (!fail && __any_sync(0xffffffffu, alpha != 1.f)) {
          ptx::tc_fence_after();
          // this thread's row in half `grp` of the values
#pragma unroll 1
          for (int c = 0; c < 128; c += 64) {
            float o[64];
            const uint32_t at = tmem + kTmemO + 128 * grp + c + lanes;
            tmem_ld32(at, o);
            tmem_ld32(at + 32, o + 32);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 64; ++i) o[i] *= alpha;
#pragma unroll
            for (int i = 0; i < 64; i += 32) tmem_st32(at + i, o + i);
          }
          ptx::tmem_st_wait();
          ptx::tc_fence_before();
        }
      }
      softmax_any(false);  // (`red` too is read before the next tile writes it)
    };
    if (!fail) {
      float2 s = make_float2(0.f, 0.f);
      uint32_t w[kFp8 ? 8 : 16], wl[kFp8 ? 8 : 1];
      const float nref = ref == -INFINITY ? 0.f : -ref;  // (a row that has seen no key yet: all scores are -inf)
      uint32_t dither = dither2_of(key0);
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float2 v = ptx::add2(make_float2(x[i], x[i + 1]), make_float2(nref, nref));
        const float2 pv = make_float2(ex2(v.x), ex2(v.y));
        if constexpr (kScales == kSmallBlocks)
          s = ptx::fma2(pv, inverse[i / 2], s);
        else
          s = ptx::add2(s, pv);
        if constexpr (kFp8) {
          uint32_t hi, lo;
          split_p(pv.x, pv.y, __byte_perm(dither, 0u, 0x4341), hi, lo);
          dither += kDither2Step;
          w[i / 4] = i % 4 ? __byte_perm(w[i / 4], hi, 0x5410) : hi;
          wl[i / 4] = i % 4 ? __byte_perm(wl[i / 4], lo, 0x5410) : lo;
        } else {
          w[i / 2] = pack_bf16(pv.x, pv.y);
        }
      }
      l += kScales == kLargeBlocks ? (s.x + s.y) * inverse[0].x : s.x + s.y;
      if (kScaled) {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ms->sc_free[sb]);
      }
      if (moved) rescale();
      const bool any = kv_begin + t * kTileKeys + kPage * pg < kv_end;  // (a unit's last tile may have one page)
      if (t >= 1 && any) fail = !o_done(pg, t - 1);  // (P and the values of the page are single: the next ones follow O)
      if (!fail && any) {
        if constexpr (kFp8) {
          uint8_t* hi = smem + G::kOffP + pg * (kHalfRows * 64);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int off = sw64_offset(row, 32 * grp + 16 * j);
            *reinterpret_cast<uint4*>(hi + off) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
            *reinterpret_cast<uint4*>(hi + kHalfRows * 128 + off) = make_uint4(wl[4 * j], wl[4 * j + 1], wl[4 * j + 2], wl[4 * j + 3]);
          }
        } else {
          uint8_t* line = smem + G::kOffP + pg * (kHalfRows * 128) + row * 128;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint4*>(line + (((4 * grp + j) ^ (row & 7)) << 4)) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        }
        if (__builtin_expect(kv_begin + t * kTileKeys + kPage * (pg + 1) > kv_end, 0)) {
          // values behind the key range: zero, so that P = 0 meets V = 0 (a key and a half to a thread)
          fail = !warp_wait(&ms->v_full[pg], t & 1, abort, p);
          if (!fail && kv_begin + t * kTileKeys + kPage * pg + row >= kv_end) {
            uint8_t* at = smem + G::kOffV + pg * G::kVPage + grp * (2 * G::kChunkBytes) + row * G::kRowBytes;
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int j = 0; j < G::kRowBytes / 16; ++j) *reinterpret_cast<uint4*>(at + c * G::kChunkBytes + 16 * j) = make_uint4(0, 0, 0, 0);
          }
          __syncwarp();
        }
        ptx::fence_async_smem();
        ptx::tc_fence_before();
        __syncwarp();
        if (!fail && lane == 0) arrive_first(&ms->p_ready[pg][sb], rank);
      }
    }
  }
  // ---- row sums, LSE, O / l
  if (!stop) {
    stop = softmax_any(fail || *abort != 0);
    if (!stop) {
      ms->red[2 * pg + grp][row] = l;
      softmax_sync();
      l = (ms->red[0][row] + ms->red[1][row]) + (ms->red[2][row] + ms->red[3][row]);
      const int npages = (kv_end - kv_begin + kPage - 1) / kPage;
      fail = !o_done(0, ntiles - 1);
      if (!fail && npages >= 2) fail = !o_done(1, npages / 2 - 1);
      stop = softmax_any(fail || *abort != 0);
    }
  }
  if (stop) return;
  ptx::tc_fence_after();
  if (pg == 0 && grp == 0 && live) {
    const float lse = l > 0.f ? (ref + lg2(l)) * 0.69314718055994531f : -INFINITY;
    if (part_row0 >= 0)
      p.part_lse[part_row0 + row] = lse;
    else if (p.lse)
      p.lse[qrow0 + row] = lse;
  }
  const float os = l > 0.f ? p.out_scale / l : 0.f;
  const int dv = 256 * grp + 128 * pg;
  __nv_bfloat16* dst = p.out + (size_t)(qrow0 + row) * kDv + dv;
  float* part = (float*)p.part_o + (size_t)(part_row0 + row) * kDv + dv;
#pragma unroll 1
  for (int c = 0; c < 128; c += 32) {
    float o[32];
    tmem_ld32(tmem + kTmemO + 128 * grp + c + lanes, o);
    ptx::tmem_ld_wait();
    if (!live) continue;
#pragma unroll
    for (int i = 0; i < 32; ++i) o[i] *= os;
    if (part_row0 < 0) {
#pragma unroll
      for (int i = 0; i < 32; i += 8)
        *reinterpret_cast<uint4*>(dst + c + i) = make_uint4(pack_bf16(o[i], o[i + 1]), pack_bf16(o[i + 2], o[i + 3]),
                                                            pack_bf16(o[i + 4], o[i + 5]), pack_bf16(o[i + 6], o[i + 7]));
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 4) *reinterpret_cast<float4*>(part + c + i) = make_float4(o[i], o[i + 1], o[i + 2], o[i + 3]);
    }
  }
}

template <bool kFp8, int kScales>
__global__ void __launch_bounds__(kThreads, 1)
    wide_decode_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_k,
                       const __grid_constant__ CUtensorMap tmap_v, Params p) {
  using G = Geo<kFp8>;
  constexpr bool kScaled = kScales != kOneScale;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc* ms = (Misc*)(smem + G::kOffMisc);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const uint32_t rank = ptx::cluster_ctarank();
  volatile int* abort = &ms->abort;
  ptx::pdl_launch_dependents();
  if (warp == 0) {
    if (lane == 0) {
      // the swizzles are laid out from 1024-byte boundaries; shared memory starts at one
      ms->abort = (ptx::smem_addr(smem) & 1023u) != 0 ? 1 : 0;
      if (ms->abort) report(p.status, MLA_DEVICE_WAIT_TIMEOUT);
      ptx::mbar_init(&ms->q_full, kFp8 ? 8 : 1);
      for (int i = 0; i < 3; ++i) {
        ptx::mbar_init(&ms->k_full[i], 1);
        ptx::mbar_init(&ms->k_empty[i], 1);
        ptx::mbar_init(&ms->k_peer[i], 1);
      }
      for (int i = 0; i < 2; ++i) {
        ptx::mbar_init(&ms->v_full[i], 1);
        ptx::mbar_init(&ms->v_empty[i], 1);
        ptx::mbar_init(&ms->v_peer[i], 1);
        ptx::mbar_init(&ms->s_full[i], 1);
        ptx::mbar_init(&ms->s_empty[i], 16);
        ptx::mbar_init(&ms->sc_full[i], 1);
        ptx::mbar_init(&ms->sc_free[i], 8);
        for (int k = 0; k < 2; ++k) {
          ptx::mbar_init(&ms->p_ready[i][k], 8);
          ptx::mbar_init(&ms->o_done[i][k], 1);
        }
        ptx::mbar_init(&ms->drained[i], 1);
      }
      ptx::fence_mbar_init();
    }
    if (lane < 12) ms->unit[lane] = reinterpret_cast<const int32_t*>(p.units + (blockIdx.x >> 1))[lane];
  } else if (warp == 1) {
    tmem_alloc2(&ms->tmem_base, kTmemCols);
    tmem_relinquish2();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_arrive();
  ptx::cluster_wait();
  ptx::tc_fence_after();
  const uint32_t tmem = ms->tmem_base;
  const int kv_begin = ms->unit[3], kv_end = ms->unit[4];
  const int ntiles = (kv_end - kv_begin + kTileKeys - 1) / kTileKeys;
  const int npages = (kv_end - kv_begin + kPage - 1) / kPage;
  const int32_t* table = p.page_table + (size_t)ms->unit[0] * p.pt_stride + kv_begin / kPage;
  const uint32_t s0 = ptx::smem_addr(smem);
  // page i of the unit (a tile's missing second page: the first one again). An id is checked where it is
  // used, so that its load is not waited for before.
  auto page_id = [&](int i) { return table[i < npages ? i : npages - 1]; };
  auto checked = [&](int page) {
    if (page >= 0 && page < p.num_pages) return page;
    report(p.status, MLA_DEVICE_BAD_PAGE);
    return 0;
  };

  if (warp == 0) {
    // ------------------------------------------------------------ copies of Q and of this CTA's pages
    const bool first_unit = (blockIdx.x >> 1) == 0;
    int issued = 0;
    bool ok = !*abort;
    if (!kFp8 && ok && lane == 0) {
      ptx::mbar_arrive_expect_tx(&ms->q_full, kChunks * G::kQChunkBytes);
      ptx::tma_load_3d(smem, &tmap_q, &ms->q_full, 0, ms->unit[1] + kHalfRows * (int)rank, 0);
    }
    // lanes 0-15 hold the ids of the tiles' first pages, lanes 16-31 of the second ones, two tiles ahead
    int id = checked(page_id(lane >> 4)), id1 = ntiles > 1 ? page_id(2 + (lane >> 4)) : 0;
    float sc[4];
    auto load_scales = [&](int t, int page) {  // of four keys of the tile
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int key = 4 * lane + k;
        const bool in = kv_begin + t * kTileKeys + key < kv_end;
        sc[k] = in ? p.kv_scales[((size_t)page * kPage + (key & 63)) >> p.block_log2] : 1.f;
      }
    };
    if (kScaled && ok) load_scales(0, id);
    for (int t = 0; ok && t < ntiles; ++t) {
      const int page = __shfl_sync(0xffffffffu, id, 16 * (int)rank);
      if (t + 1 < ntiles) id1 = checked(id1);
      const int next = __shfl_sync(0xffffffffu, id1, 16 * (int)rank);
      for (int g = 0; ok && g < G::kPieces; ++g) {
        const int n = t * G::kPieces + g, slot = n % G::kSlots;
        if (n >= G::kSlots) ok = warp_wait(&ms->k_empty[slot], ((n / G::kSlots) - 1) & 1, abort, p);
        if (!ok) break;
        if (lane == 0 && !(first_unit && 2 * t + (int)rank == p.skip_copy)) {  // (left out to test the waits' limits)
          ptx::mbar_arrive_expect_tx(&ms->k_full[slot], G::kSlotBytes);
          ptx::tma_load_3d(smem + G::kOffK + slot * G::kSlotBytes, &tmap_k, &ms->k_full[slot], 0, page * kPage, g * G::kPieceChunks);
          if (t + 1 < ntiles) ptx::tma_prefetch_l2_3d(&tmap_k, 0, next * kPage, g * G::kPieceChunks);
        }
        __syncwarp();
        issued = n + 1;
      }
      const int id2 = t + 2 < ntiles ? page_id(2 * (t + 2) + (lane >> 4)) : 0;
      if constexpr (kScaled) {
        if (ok && t >= 2) ok = warp_wait(&ms->sc_free[t & 1], ((t - 2) >> 1) & 1, abort, p);
        if (!ok) break;
        uint8_t* tables = smem + G::kOffScales + (t & 1) * G::kScaleBytes;
#pragma unroll
        for (int k = 0; k < 4; k += 2) {
          const float v0 = fmaxf(sc[k], 0x1p-60f), v1 = fmaxf(sc[k + 1], 0x1p-60f);
          reinterpret_cast<float4*>(tables)[2 * lane + k / 2] = make_float4(sc[k], sc[k + 1], lg2(v0), lg2(v1));
          reinterpret_cast<float2*>(tables + kTileKeys / 2 * 16)[2 * lane + k / 2] = make_float2(1.f / v0, 1.f / v1);
        }
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ms->sc_full[t & 1]);
        if (t + 1 < ntiles) load_scales(t + 1, id1);
      }
      id = id1;
      id1 = id2;
    }
    // every copy lands before the CTA may exit
    if (lane == 0) {
      for (int n = max(0, issued - G::kSlots); n < issued; ++n) {
        if (first_unit && 2 * (n / G::kPieces) + (int)rank == p.skip_copy) continue;
        const long long t0 = clock64();
        while (!ptx::mbar_try_wait(&ms->k_full[n % G::kSlots], (n / G::kSlots) & 1) && clock64() - t0 < p.wait_budget) {
        }
      }
      if (!kFp8 && !*abort) {
        const long long t0 = clock64();
        while (!ptx::mbar_try_wait(&ms->q_full, 0) && clock64() - t0 < p.wait_budget) {
        }
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------ copies of this CTA's value columns
    bool ok = !*abort;
    int issued = 0, page = page_id(0);
    for (; ok && issued < npages; ++issued) {
      const int pg = issued & 1, t = issued >> 1;
      page = checked(page);
      if (t >= 1) ok = warp_wait(&ms->v_empty[pg], (t - 1) & 1, abort, p);
      if (!ok) break;
      if (lane == 0) {
        uint8_t* dst = smem + G::kOffV + pg * G::kVPage;
        ptx::mbar_arrive_expect_tx(&ms->v_full[pg], G::kVPage);
        ptx::tma_load_3d(dst, &tmap_v, &ms->v_full[pg], 0, page * kPage, 2 * (int)rank);
        ptx::tma_load_3d(dst + 2 * G::kChunkBytes, &tmap_v, &ms->v_full[pg], 0, page * kPage, 4 + 2 * (int)rank);
      }
      __syncwarp();
      page = page_id(issued + 1);
    }
    if (lane == 0) {
      for (int n = max(0, issued - 2); n < issued; ++n) {
        const long long t0 = clock64();
        while (!ptx::mbar_try_wait(&ms->v_full[n & 1], (n >> 1) & 1) && clock64() - t0 < p.wait_budget) {
        }
      }
    }
    __syncwarp();
  } else if (warp <= 2) {
    // One thread of the warp does all of the role's waiting and issuing (a whole warp that polls takes
    // ~100 cycles a barrier: 4 x 64 nodes over 32768 bf16 keys 247 us, with one thread 187).
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (ptx::mbar_try_wait(bar, parity)) return true;
      const long long t0 = clock64();
      while (!*abort) {
        if (ptx::mbar_try_wait(bar, parity)) return true;
        if (clock64() - t0 > p.wait_budget) {
          *abort = 1;
          report(p.status, MLA_DEVICE_WAIT_TIMEOUT);
        }
      }
      return false;
    };
    if (ptx::elect_one()) {
      bool ok = !*abort, issued = false;
      if (warp == 1 && rank == 1) {
        // ---------------------------------------------------------- CTA 1: tell CTA 0 what has landed
        ok = ok && wait(&ms->q_full, 0);
        for (int n = 0; ok && n < ntiles * G::kPieces; ++n) {
          ok = wait(&ms->k_full[n % G::kSlots], (n / G::kSlots) & 1);
          if (ok) arrive_first(&ms->k_peer[n % G::kSlots], rank);
        }
      } else if (rank == 1) {
        for (int n = 0; ok && n < npages; ++n) {
          ok = wait(&ms->v_full[n & 1], (n >> 1) & 1);
          if (ok) arrive_first(&ms->v_peer[n & 1], rank);
        }
      } else if (warp == 1) {
        // ---------------------------------------------------------- S(t) = Q . K^T into buffer t % 2
        ok = ok && wait(&ms->q_full, 0);
        const uint32_t idesc = kFp8 ? ptx::idesc_e4m3(kRows, kTileKeys, 0, 0) : ptx::idesc_bf16(kRows, kTileKeys, 0, 0);
        for (int t = 0; ok && t < ntiles; ++t) {
          if (t >= 2) ok = wait(&ms->s_empty[t & 1], ((t - 2) >> 1) & 1);
          const uint32_t d = tmem + kTmemS + 64 * (t & 1);
          for (int g = 0; ok && g < G::kPieces; ++g) {
            const int n = t * G::kPieces + g, slot = n % G::kSlots;
            ok = wait(&ms->k_full[slot], (n / G::kSlots) & 1) && wait(&ms->k_peer[slot], (n / G::kSlots) & 1);
            if (!ok) break;
            ptx::tc_fence_after();
            const uint32_t k0 = s0 + G::kOffK + slot * G::kSlotBytes, q0 = s0 + g * G::kPieceChunks * G::kQChunkBytes;
            if constexpr (kFp8) {
#pragma unroll 1
              for (int c = 0; c < G::kPieceChunks; ++c)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                  for (int part = 0; part < 2; ++part)
                    mma2<true>(d, ptx::smem_desc(q0 + c * G::kQChunkBytes + part * (kHalfRows * 64) + 32 * k, 16, 512, ptx::kSwizzle64B),
                               ptx::smem_desc(k0 + c * G::kChunkBytes + 32 * k, 16, 512, ptx::kSwizzle64B), idesc, (c | k | part) != 0 ? 1u : 0u);
            } else {
#pragma unroll 1
              for (int c = 0; c < G::kPieceChunks; ++c)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma2<false>(d, ptx::smem_desc(q0 + c * G::kQChunkBytes + 32 * k, 16, 1024, ptx::kSwizzle128B),
                              ptx::smem_desc(k0 + c * G::kChunkBytes + 32 * k, 16, 1024, ptx::kSwizzle128B), idesc, (g | c | k) != 0 ? 1u : 0u);
            }
            commit_both(&ms->k_empty[slot]);
            if (g == G::kPieces - 1) commit_both(&ms->s_full[t & 1]);
            issued = true;
          }
        }
      } else {
        // ---------------------------------------------------------- O += P(t) . V(t), a page at a time
        const uint32_t idesc = kFp8 ? ptx::idesc_e4m3(kRows, 256, 0, 1) : ptx::idesc_bf16(kRows, 256, 0, 1);
        for (int n = 0; ok && n < npages; ++n) {
          const int pg = n & 1, t = n >> 1;
          ok = wait(&ms->v_full[pg], t & 1) && wait(&ms->v_peer[pg], t & 1) && wait(&ms->p_ready[pg][t & 1], (t >> 1) & 1);
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t v0 = s0 + G::kOffV + pg * G::kVPage, p0 = s0 + G::kOffP;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t d = tmem + kTmemO + 128 * h, vh = v0 + h * (2 * G::kChunkBytes);
            if constexpr (kFp8) {
#pragma unroll
              for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int part = 0; part < 2; ++part)
                  mma2<true>(d, ptx::smem_desc(p0 + part * (kHalfRows * 128) + pg * (kHalfRows * 64) + 32 * k, 16, 512, ptx::kSwizzle64B),
                             ptx::smem_desc(vh + 2048 * k, G::kChunkBytes, 512, ptx::kSwizzle64B), idesc | (part ? ptx::kA_E5M2 : 0u),
                             (n | k | part) != 0 ? 1u : 0u);
            } else {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma2<false>(d, ptx::smem_desc(p0 + pg * (kHalfRows * 128) + 32 * k, 16, 1024, ptx::kSwizzle128B),
                            ptx::smem_desc(vh + 2048 * k, G::kChunkBytes, 1024, ptx::kSwizzle128B), idesc, (n | k) != 0 ? 1u : 0u);
            }
          }
          commit_both(&ms->v_empty[pg]);
          commit_both(&ms->o_done[pg][t & 1]);
          issued = true;
        }
      }
      if (issued) {  // every product retires before tensor memory is released
        commit_here(&ms->drained[warp - 1]);
        const long long t0 = clock64();
        while (!ptx::mbar_try_wait(&ms->drained[warp - 1], 0) && clock64() - t0 < p.wait_budget) {
        }
      }
    }
    __syncwarp();
  } else {
    softmax_role<kFp8, kScales>(smem, ms, p, tmem, rank, warp & 3, (warp - 4) >> 2, lane, tid - 128);
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  // neither CTA leaves while the other's products or arrivals may reach it
  ptx::cluster_arrive();
  ptx::cluster_wait();
  if (warp == 1) {
    ptx::tc_fence_after();
    tmem_dealloc2(tmem, kTmemCols);
  }
}

}  // namespace wide

int wide_rows_cap() { return wide::kRows; }

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();  // defined next to the single-CTA kernel

// [rows, 576] as (64 columns, rows, 9 chunks), boxes of box_rows rows and box_chunks chunks.
static CUresult encode_wide(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const void* base, bool fp8, uint64_t rows,
                            uint32_t box_rows, uint32_t box_chunks) {
  const uint64_t esz = fp8 ? 1 : 2;
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, 9};
  cuuint64_t strides[2] = {(cuuint64_t)(kDqk * esz), (cuuint64_t)(64 * esz)};
  cuuint32_t box[3] = {64, box_rows, box_chunks};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides,
             box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, fp8 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

cudaError_t set_wide_kernel_attributes() {
  cudaError_t e = cudaFuncSetAttribute(wide::wide_decode_kernel<false, wide::kOneScale>, cudaFuncAttributeMaxDynamicSharedMemorySize, wide::Geo<false>::kSmem);
  for (auto fn : {wide::wide_decode_kernel<true, wide::kOneScale>, wide::wide_decode_kernel<true, wide::kLargeBlocks>, wide::wide_decode_kernel<true, wide::kSmallBlocks>})
    if (e == cudaSuccess) e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, wide::Geo<true>::kSmem);
  return e;
}

int launch_wide_kernel(const PlanHeader* h, const void* q, const void* kv_cache, int num_pages, const Params& prm, cudaStream_t st) {
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return set_error(MLA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  const bool fp8 = h->kv_dtype == MLA_KV_FP8_E4M3;
  alignas(64) CUtensorMap tq, tk, tv;
  const uint64_t kv_rows = (uint64_t)num_pages * kPage;
  CUresult r = encode_wide(enc, &tq, q, false, (uint64_t)h->total_q * (uint64_t)h->num_heads, wide::kHalfRows, 9);
  if (r == CUDA_SUCCESS) r = encode_wide(enc, &tk, kv_cache, fp8, kv_rows, kPage, fp8 ? 9 : 3);
  if (r == CUDA_SUCCESS) r = encode_wide(enc, &tv, kv_cache, fp8, kv_rows, kPage, 2);
  if (r != CUDA_SUCCESS) return set_error(MLA_ERR_CUDA, "tensor maps for the wide kernel failed (CUresult %d)", (int)r);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)(2 * h->n_units), 1, 1);
  cfg.blockDim = dim3(wide::kThreads, 1, 1);
  cfg.dynamicSmemBytes = fp8 ? wide::Geo<true>::kSmem : wide::Geo<false>::kSmem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {2, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto fn = !fp8             ? wide::wide_decode_kernel<false, wide::kOneScale>
            : !prm.kv_scales ? wide::wide_decode_kernel<true, wide::kOneScale>
            : prm.block_log2 >= 5 ? wide::wide_decode_kernel<true, wide::kLargeBlocks>
                                  : wide::wide_decode_kernel<true, wide::kSmallBlocks>;
  const cudaError_t ce = cudaLaunchKernelEx(&cfg, fn, tq, tk, tv, prm);
  if (ce != cudaSuccess) return set_error(MLA_ERR_CUDA, "wide kernel launch: %s", cudaGetErrorString(ce));
  return MLA_OK;
}

}  // namespace mla
