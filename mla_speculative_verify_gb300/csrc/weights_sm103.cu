// weights_sm103.cu -- mla_key_weights: the attention weight that every cached key received
// from a verify call, added to a running sum (what an eviction goes by):
//
//   w[b, j] = decay * w[b, j] + sum over counted rows (i, h) of exp(s_ijh - lse_ih)
//
// with the scores s and the log-sum-exp of the decode. No value product and no running
// maximum are needed, since lse is known, so one pass over the cache does it:
//
//   S^T[key, row] = K[key, 0:576] . Q[row, 0:576]^T      (M = 128 keys, N = up to 128 rows)
//
// on the tcgen05 tensor cores. In this orientation a key is one lane of tensor memory: a
// thread reads its key's scores of all rows and adds their exponentials in registers; no sum
// crosses threads and no order depends on timing, so results repeat bit for bit.
//
// Rows. The q * H rows of a request are cut into G groups of at most 128. Keys go through
// shared memory in tiles of 128 (two pages), 64 of the 576 columns at a time, so that the Q
// group stays resident (up to 144 KB) beside a ring of K pieces. With G > 1 a CTA takes a few
// tiles (sub_tiles, which fit L2 over all CTAs) through all groups before it goes on, so the
// cache leaves HBM once; the sums of those keys wait in shared memory.
//
// An e4m3 cache is multiplied as stored (kind::f8f6f4). q_split_kernel first writes each Q row,
// times the power of two that brings its largest entry to [128, 256), as an e4m3 part and the
// remainder in e5m2. A bf16 entry has 8 significant bits: the first part takes 4 and leaves at
// most 8 units of the last of them, which e5m2's 3 bits hold, so entries down to 2^-13 of the
// row's largest are exact; below that the error is at most 2^-20 of the largest (with both parts
// in e4m3 it was 2^-18 from 2^-9 on: 3.7e-6 in weights that fp32 has to 1.2e-6).
// Both parts' products go into one accumulator: side by side in 2 x rows
// columns they took half the products, but left two accumulators and twice the columns to read
// (170 against 134 us for 32 requests of 8k-16k keys, 128 heads).
//
// The tensor cores cut the bits below an accumulator's last one at every step, always towards
// zero, so a score of 36 steps in one accumulator is off by ~2^-20 of itself: 1.9e-5 in the
// weights of a million keys with scores of 20 and more. Each tile's columns are therefore summed
// in parts (bf16: nine of 64 columns, e4m3: three of 192), each in an accumulator that starts at
// zero, and the parts are added in fp32 registers, rounded. The accumulators are taken in turns,
// so one part is read while the next are computed.
//
// Warp roles (one CTA per SM): warp 0 loads (TMA), warps 1-3 issue the products, warps 4-7 and
// 8-11 take the scores out, a tile each in turns. All of them walk the same work list
// (Walk). Waits are bounded as in the decode kernel.
//
// Measured: 96 rows over 1M bf16 keys 188 us, 6.4 TB/s, 0.95 of the measured copy rate: bound by
// HBM. 128 to 512 rows over 32 x 8k-16k e4m3 keys 130 us: bound by the products' operand reads
// (128 rows x 128 keys read shared memory as long as they compute, and the keys' arrival and the
// rows' tables want it too; without the keys' copies it is 109); HBM would need 38 us and the
// products 86.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "mla_decode.h"
#include "plan_format.h"
#include "decode_common.cuh"
#include "ptx.cuh"
#include "status.h"

namespace mla {

int current_device_ready(DeviceKernels* out);               // defined next to the decode kernel
PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder();     // defined next to the decode kernel
int block_log2_of(int block_tokens);                        // defined with the plan
int check_plan(const void* plan_host, size_t plan_bytes, const PlanHeader** out);

namespace {

constexpr int kKeys = 128;          // keys per tile (two pages)
constexpr int kPieces = 9;          // 576 = 9 x 64 columns
constexpr int kMaxRows = 128;       // rows of a group
constexpr int kMaxStages = 16;
constexpr int kMaxSlots = 6;        // accumulators, taken in turns by the parts

// The parts of a tile; a part is a stage of the ring. One thread issues a product only every ~125
// cycles and loses ~300 to a stage's waits and commits, more than the products themselves take,
// so several warps issue parts in turns. An issuer waits for a stage's or an accumulator's next
// phase, which says nothing while the phase before it is open; so each of them belongs to one
// issuer: their numbers are multiples of the issuers'. At 128 rows beside Q there is room for four
// bf16 stages and 512 columns are four accumulators, so two issuers use all of both (768 rows over
// 131k keys: one issuer 150 us, two 131, three 145). e4m3 pieces are half as large, so three make
// a part, and a tile's three parts are the three stages of three issuers (batch of 128 heads
// against parts of one piece: 207 -> 179 us); bf16 parts of three would leave two stages (a
// million keys 202 -> 208 us).
constexpr int kMaxIssuers = 3;  // of warps 1-3; warp 0 loads
template <bool kFp8>
struct Parts {
  static constexpr int kCount = kFp8 ? 3 : 9;     // parts of a score's 576 columns
  static constexpr int kPer = kPieces / kCount;   // pieces of a part
  static constexpr int kIssuers = kFp8 ? 3 : 2;
  static constexpr bool kFixed = kCount % kIssuers == 0;  // a piece is always multiplied by the same issuer
  static_assert(kFixed || (kPer == 1 && kIssuers == 2), "the pieces' barriers expect one of these");
};
constexpr int kMaxSub = 32;         // tiles of one sub-range: a loading warp holds a page id in each lane
constexpr int kMaxSubSums = 8;      // of those when sums wait in shared memory (G > 1)
constexpr int kThreads = 384;
constexpr int kSmemCap = 232448;    // 227 KB per CTA

// Registers of a thread at the launch, and after the warpgroup of warps 0-3 has given some to the
// other two, whose threads hold 128 sums and two reads of 32 columns (with 208 for those some of
// them go through memory: batch of 128 heads, e4m3, 131 -> 143 us).
constexpr int kRegsLaunch = 168, kRegsWork = 56, kRegsWeights = 224;
static_assert(128 * kRegsWork + 256 * kRegsWeights <= kThreads * kRegsLaunch, "the launch's registers must cover the split");

struct WeightsMisc {
  uint64_t kv_full[kMaxStages], kv_empty[kMaxStages];
  uint64_t q_full[kPieces], q_empty[kPieces];
  uint64_t d_full[2][kMaxSlots], d_empty[kMaxSlots], mma_done[kMaxIssuers];
  uint32_t tmem_base;
  int abort;
  alignas(16) float nlse[2][kMaxRows];    // of each warpgroup's current group: -lse of the rows
  alignas(16) float rscale[2][kMaxRows];  // e4m3: each row's part of its scores' scale
  alignas(16) int lim[2][kMaxRows];       // keys that each row sees
  alignas(16) float sums[kMaxSubSums][kKeys];
};
constexpr int kMiscBytes = (sizeof(WeightsMisc) + 1023) / 1024 * 1024;

struct WeightsParams {
  const PlanRequest* reqs;
  PlanRequest first;       // reqs[0], so that a call with one request need not read it
  int batch, H, pt_stride, num_pages, block_log2;
  const int32_t* page_table;
  const float* kv_scales;  // NULL without block scales
  const float* lse;
  const int32_t* counted;  // NULL: every row counts
  const float* q_scale;    // e4m3: per row, undoes its power of two
  float* weights;
  long long w_stride;
  float decay, sm_scale, kv_scale;
  int rows_n;              // MMA rows of every group (multiple of 32)
  int total_rows;
  int stages, slots, sub_tiles;
  long long total_work;    // sum over requests of tiles * groups
  int32_t* status;
  long long wait_budget;  // cycles a bounded wait may take (kWaitBudget; kWaitBudgetTest in a timeout test)
  int skip_copy;          // part of the first CTA that is never copied (timeout test), or -1
};

// This CTA's share of the work list, as every role's warps walk it. The list is request by
// request, a request's tiles each weighing its groups; CTA i of n takes the tiles whose
// place in the list lies in [W i / n, W (i + 1) / n). 32 requests are looked at together.
struct Walk {
  long long lo, hi, base;  // base: place of request b0
  int b0;
  PlanRequest r;           // this lane's request
  long long at;            // its place
  uint32_t todo;           // lanes of the current 32 requests that hold work of this CTA

  __device__ __forceinline__ void start(const WeightsParams& p) {
    lo = p.total_work * blockIdx.x / gridDim.x;
    hi = p.total_work * (blockIdx.x + 1) / gridDim.x;
    base = 0;
    b0 = -32;
    todo = 0;
  }
  static __device__ __forceinline__ int groups(const WeightsParams& p, int q) {
    return (q * p.H + p.rows_n - 1) / p.rows_n;
  }
  // The next request with tiles [t0, t1) for this CTA; false at the end.
  __device__ __forceinline__ bool next(const WeightsParams& p, int& b, PlanRequest& req, int& t0, int& t1) {
    const int lane = threadIdx.x & 31;
    while (todo == 0) {
      b0 += 32;
      if (b0 >= p.batch || base >= hi) return false;
      const bool live = b0 + lane < p.batch;
      r = !live ? PlanRequest{0, 0, 0, 1} : p.batch == 1 ? p.first : p.reqs[b0 + lane];
      const long long mine = (long long)((r.ctx + kKeys - 1) / kKeys) * groups(p, r.q);
      long long incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      at = base + incl - mine;
      todo = __ballot_sync(0xffffffffu, mine > 0 && at < hi && at + mine > lo);
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    const int l = __ffs(todo) - 1;
    todo &= todo - 1;
    b = b0 + l;
    req.ctx = __shfl_sync(0xffffffffu, r.ctx, l);
    req.q = __shfl_sync(0xffffffffu, r.q, l);
    req.tok0 = __shfl_sync(0xffffffffu, r.tok0, l);
    req.fold = 1;
    const long long a = __shfl_sync(0xffffffffu, at, l);
    const int g = groups(p, req.q), tiles = (req.ctx + kKeys - 1) / kKeys;
    auto first_tile = [&](long long place) {  // the first tile at or after a place of the list
      const long long d = place - a;
      return d <= 0 ? 0 : (int)min((long long)tiles, (d + g - 1) / g);
    };
    t0 = first_tile(lo);
    t1 = first_tile(hi);
    return true;
  }
};

// A place in a ring of n barriers and how often it has come round.
struct Ring {
  uint32_t n, at, phase;
  __device__ __forceinline__ explicit Ring(uint32_t n_) : n(n_), at(0), phase(0) {}
  __device__ __forceinline__ void step(uint32_t by = 1) {  // (a divisor of n, from a place below it)
    at += by;
    if (at >= n) {
      at -= n;
      ++phase;
    }
  }
};

// A value that all lanes of the warp hold, as one the compiler knows to be such. Whatever a branch,
// an address or a descriptor of the loading and issuing warps depends on comes through here or
// through a vote: their loops are chains of single instructions, and kept in per-lane registers
// such values slowed those warps by a tenth (768 rows over 131k bf16 keys 147 against 131 us).
template <typename T>
__device__ __forceinline__ T uniform(T v) {
  return __shfl_sync(0xffffffffu, v, 0);
}

// Rows of request b that count (its first counted[b] tokens).
__device__ __forceinline__ int counted_rows(const WeightsParams& p, int b, int q) {
  const int c = p.counted ? uniform(max(0, min(q, p.counted[b]))) : q;
  return c * p.H;
}

// The epilogue warpgroups (wg 0 and 1, warps of quadrant qd) take a sub-range's tiles in turns:
// while one adds the parts of its tile, the other's exponentials are computed. A thread owns the
// key of its tensor-memory lane and all N = 32 NC rows of the group. (With half of a tile's rows
// each, the two were at the same work at the same time and met at a barrier after every tile:
// 768 rows over 131k e4m3 keys 85 us, in turns 76.)
template <int NC, bool kFp8>
__device__ __forceinline__ void weights_role(const WeightsParams& p, WeightsMisc* ms, Walk& walk, uint32_t tmem, int wg,
                                             int qd, int lane) {
  constexpr int n = 32 * NC;
  const int key_in = 32 * qd + lane;
  const uint32_t acc0 = tmem + ((uint32_t)(32 * qd) << 16);
  const float* nlse = ms->nlse[wg];
  const float* rscale = ms->rscale[wg];
  const int* lim = ms->lim[wg];
  volatile int* abort = &ms->abort;
  Ring slots(p.slots);
  uint32_t parity = 0;  // bit i: of this warpgroup's next wait for accumulator i
  bool ok = true;
  int b, t0, t1;
  PlanRequest req;
  while (walk.next(p, b, req, t0, t1)) {
    const int rows = counted_rows(p, b, req.q), groups = (rows + n - 1) / n;
    const int32_t* ids = p.page_table + (size_t)b * p.pt_stride;
    float* wrow = p.weights + (size_t)b * p.w_stride;
    if (groups == 0) {  // no row counts: the sums only decay
      for (int t = t0 + wg; t < t1; t += 2) {
        const int key = t * kKeys + key_in;
        if (key < req.ctx) wrow[key] = p.decay == 0.f ? 0.f : wrow[key] * p.decay;
      }
      continue;
    }
    const int sub = groups > 1 ? p.sub_tiles : kMaxSub;
    for (int s0 = t0; s0 < t1; s0 += sub) {
      const int s1 = min(t1, s0 + sub);
      for (int g = 0; g < groups; ++g) {
        const int mine = min(n, rows - g * n);  // rows of the group that are there
        if (groups > 1 || s0 == t0) {
          const int row0 = req.tok0 * p.H + g * n;
          ptx::bar_sync(1 + wg, 128);  // this warpgroup is done with the old table
          if (key_in < n) {
            const bool live = key_in < mine;
            const float l = live ? p.lse[row0 + key_in] : INFINITY;
            ms->nlse[wg][key_in] = l == -INFINITY ? -INFINITY : -l;  // a row that saw nothing adds nothing
            if (kFp8) ms->rscale[wg][key_in] = live ? p.sm_scale * p.q_scale[row0 + key_in] : 0.f;
            ms->lim[wg][key_in] = live ? req.ctx - req.q + (g * n + key_in) / p.H + 1 : 0;
          }
          ptx::bar_sync(1 + wg, 128);
        }
        const int lim_min = req.ctx - req.q + g * n / p.H + 1;  // what the group's first row sees
        for (int t = s0; t < s1; ++t) {
          if (((t - s0) & 1) != wg) {  // the other warpgroup's tile
            for (int u = 0; u < Parts<kFp8>::kCount; ++u) slots.step();
            continue;
          }
          const int key = t * kKeys + key_in;
          const bool live = key < req.ctx;
          float old = 0.f, ks = kFp8 ? p.kv_scale : p.sm_scale;  // the key's part of its scores' scale
          if (g == groups - 1 && live && p.decay != 0.f) old = wrow[key] * p.decay;
          if (kFp8 && p.kv_scales && live) {
            int id = ids[key / kPage];
            id = id >= 0 && id < p.num_pages ? id : 0;
            ks = p.kv_scales[((size_t)id * kPage + key % kPage) >> p.block_log2];
          }
          float x[n], y[2][32];  // the parts' sums; 32 columns are added while the next are read
          auto load = [&](uint32_t acc, float* to) {
            ptx::tmem_ld16(acc, to);
            ptx::tmem_ld16(acc + 16, to + 16);
          };
          auto add = [&](int c) {
#pragma unroll
            for (int j = 0; j < 32; j += 2) {
              const float2 v = ptx::add2(make_float2(x[32 * c + j], x[32 * c + j + 1]),
                                         make_float2(y[c & 1][j], y[c & 1][j + 1]));
              x[32 * c + j] = v.x;
              x[32 * c + j + 1] = v.y;
            }
          };
          auto wait = [&]() {
            if (ok) ok = warp_wait(&ms->d_full[wg][slots.at], parity >> slots.at & 1, abort, p);
            parity ^= 1u << slots.at;
            ptx::tc_fence_after();
            return acc0 + slots.at * n;
          };
          auto done = [&]() {
            ptx::tc_fence_before();
            __syncwarp();
            if (ok && lane == 0) ptx::mbar_arrive(&ms->d_empty[slots.at]);
            slots.step();
          };
          {
            const uint32_t acc = wait();
#pragma unroll
            for (int c = 0; c < NC; ++c) load(acc + 32 * c, x + 32 * c);
            ptx::tmem_ld_wait();
            done();
          }
#pragma unroll 1
          for (int u = 1; u < Parts<kFp8>::kCount; ++u) {
            const uint32_t acc = wait();
            load(acc, y[0]);
            ptx::tmem_ld_wait();
#pragma unroll
            for (int c = 1; c < NC; ++c) {
              load(acc + 32 * c, y[c & 1]);
              add(c - 1);
              ptx::tmem_ld_wait();
            }
            done();
            add(NC - 1);
          }
          float2 s[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          if (ok) {
            const float2 ks2 = make_float2(ks, ks);
            // exp(score - lse) of rows j, j + 1; score - lse is rounded once, at its own size, before
            // it goes to base 2: a score and an lse of 40 rounded apart would each put 2e-6 into it
            auto weight2 = [&](int j, float2 r, float2 l) {
              float2 v = make_float2(x[j], x[j + 1]);
              if (kFp8) v = ptx::mul2(v, r);
              v = ptx::fma2(v, ks2, l);
              v = ptx::mul2(v, make_float2(1.4426950408889634f, 1.4426950408889634f));
              return make_float2(ex2(v.x), ex2(v.y));
            };
            if ((t + 1) * kKeys <= lim_min && mine == n) {  // every row sees every key of the tile
#pragma unroll
              for (int j = 0; j < n; j += 4) {
                const float4 r = kFp8 ? *reinterpret_cast<const float4*>(rscale + j) : make_float4(0.f, 0.f, 0.f, 0.f);
                const float4 l = *reinterpret_cast<const float4*>(nlse + j);
                s[0] = ptx::add2(s[0], weight2(j, make_float2(r.x, r.y), make_float2(l.x, l.y)));
                s[1] = ptx::add2(s[1], weight2(j + 2, make_float2(r.z, r.w), make_float2(l.z, l.w)));
              }
            } else {
              // a row past the group, or one that does not see this key, holds anything
#pragma unroll
              for (int c = 0; c < 2 * NC; ++c) {
                if (16 * c >= mine) break;
#pragma unroll
                for (int j = 16 * c; j < 16 * c + 16; j += 2) {
                  float2 e = weight2(j, kFp8 ? *reinterpret_cast<const float2*>(rscale + j) : make_float2(0.f, 0.f),
                                     *reinterpret_cast<const float2*>(nlse + j));
                  e.x = key < lim[j] ? e.x : 0.f;
                  e.y = key < lim[j + 1] ? e.y : 0.f;
                  s[(j >> 1) & 1] = ptx::add2(s[(j >> 1) & 1], e);
                }
              }
            }
          }
          float w = (s[0].x + s[1].x) + (s[0].y + s[1].y);
          if (groups > 1) {
            float* slot = &ms->sums[t - s0][key_in];  // this thread's own, through all groups
            if (g > 0) w += *slot;
            *slot = w;
          }
          if (ok && g == groups - 1 && live) wrow[key] = old + w;
        }
      }
    }
  }
}

template <bool kFp8>
__global__ void __launch_bounds__(kThreads, 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmap_q, const __grid_constant__ CUtensorMap tmap_kv,
                       const __grid_constant__ CUtensorMap tmap_page, WeightsParams p) {
  constexpr int kRowBytes = kFp8 ? 64 : 128;             // a row's bytes in one 64-column piece
  constexpr int kPieceBytes = kKeys * kRowBytes;
  using R = Parts<kFp8>;
  constexpr int kPer = R::kPer;
  constexpr int kStageBytes = kPer * kPieceBytes;
  constexpr int kHalf = kPage * kRowBytes;               // one page of a piece
  constexpr uint32_t kSwizzle = kFp8 ? ptx::kSwizzle64B : ptx::kSwizzle128B;
  constexpr uint32_t kSbo = 8 * kRowBytes;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (ptx::smem_addr(smem_raw) & 1023u)) & 1023u);
  WeightsMisc* ms = (WeightsMisc*)smem;
  uint8_t* sQ = smem + kMiscBytes;
  const int n = p.rows_n;
  const int q_piece = n * 128;                           // bytes of a Q piece (e4m3: n hi rows, then n lo rows)
  uint8_t* sK = sQ + kPieces * q_piece;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  volatile int* abort = &ms->abort;

  if (warp == 0 && lane == 0) {
    ms->abort = 0;
    for (int i = 0; i < p.stages; ++i) {
      ptx::mbar_init(&ms->kv_full[i], 1);
      ptx::mbar_init(&ms->kv_empty[i], 1);
    }
    for (int i = 0; i < kPieces; ++i) {
      ptx::mbar_init(&ms->q_full[i], 1);
      ptx::mbar_init(&ms->q_empty[i], Parts<kFp8>::kFixed ? 1 : Parts<kFp8>::kIssuers);
    }
    for (int i = 0; i < p.slots; ++i) {
      ptx::mbar_init(&ms->d_full[0][i], 1);
      ptx::mbar_init(&ms->d_full[1][i], 1);
      ptx::mbar_init(&ms->d_empty[i], 4);
    }
    for (int i = 0; i < kMaxIssuers; ++i) ptx::mbar_init(&ms->mma_done[i], 1);
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&tmap_q);
    ptx::prefetch_tmap(&tmap_kv);
  } else if (warp == 1) {
    ptx::tmem_alloc(&ms->tmem_base, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = uniform(ms->tmem_base);
  Walk walk;
  walk.start(p);
  int b, t0, t1;
  PlanRequest req;
  auto load_q = [&](int c, int row) {  // piece c of the group that begins at `row` (one lane)
    ptx::mbar_arrive_expect_tx(&ms->q_full[c], q_piece);
    ptx::tma_load_3d(sQ + c * q_piece, &tmap_q, &ms->q_full[c], 0, row, c);
    if (kFp8) ptx::tma_load_3d(sQ + c * q_piece + n * 64, &tmap_q, &ms->q_full[c], 0, p.total_rows + row, c);
  };

  if (warp < 4) {
    ptx::regs_down<kRegsWork>();
  } else {
    ptx::regs_up<kRegsWeights>();
  }
  if (warp == 0) {
    // ------------------------------------------------------------ loads
    if (kFp8) ptx::pdl_wait_primary();  // Q's parts come from the kernel before
    Ring ring(p.stages);
    uint32_t qfill = 0;  // Q groups loaded so far (the first by the issuers)
    int fill = 0;        // parts copied so far
    bool ok = true;
    while (ok && walk.next(p, b, req, t0, t1)) {
      const int rows = counted_rows(p, b, req.q), groups = (rows + n - 1) / n;
      if (groups == 0 || t0 >= t1) continue;
      const int sub = groups > 1 ? p.sub_tiles : kMaxSub;
      const int npages = (req.ctx + kPage - 1) / kPage;
      const int32_t* ids = p.page_table + (size_t)b * p.pt_stride;
      auto load_ids = [&](int tile, int which) {  // lane l: page `which` (0, 1) of tile `tile` + l
        const int pg = 2 * (tile + lane) + which;
        int id = lane < sub && tile + lane < t1 && pg < npages ? ids[pg] : 0;
        if (id < 0 || id >= p.num_pages) {
          report(p.status, MLA_DEVICE_BAD_PAGE);
          id = 0;
        }
        return id;
      };
      int cur0 = load_ids(t0, 0), cur1 = load_ids(t0, 1);
      for (int s0 = t0; ok && s0 < t1; s0 += sub) {
        const int s1 = min(t1, s0 + sub);
        const int nxt0 = s1 < t1 ? load_ids(s1, 0) : 0, nxt1 = s1 < t1 ? load_ids(s1, 1) : 0;
        for (int g = 0; ok && g < groups; ++g) {
          const bool new_q = groups > 1 || s0 == t0;
          for (int t = s0; ok && t < s1; ++t) {
            const bool two = 2 * t + 1 < npages;  // (the last tile may have one page)
            const int id0 = __shfl_sync(0xffffffffu, cur0, t - s0), id1 = __shfl_sync(0xffffffffu, cur1, t - s0);
            // A ring of one e4m3 tile: ask L2 for the whole pages of the next tile that HBM has to
            // deliver. 512k keys, 96 rows: 61 us, without 66; where the ring holds two tiles (64
            // rows) the requests only stand in the copies' way, 59 against 56; with bf16 parts
            // they do at any size (96 rows 110 against 101, 128 rows 117 against 106).
            if (kFp8 && p.stages == R::kIssuers) {
              const bool in = t + 1 < s1;
              const int tn = g == 0 && in ? t + 1 : g == groups - 1 && !in ? s1 : t1;
              const int next0 = __shfl_sync(0xffffffffu, in ? cur0 : nxt0, in ? t + 1 - s0 : 0);
              const int next1 = __shfl_sync(0xffffffffu, in ? cur1 : nxt1, in ? t + 1 - s0 : 0);
              if (tn < t1 && ptx::elect_one()) {
                ptx::tma_prefetch_l2_3d(&tmap_page, 0, next0 * kPage, 0);
                if (2 * tn + 1 < npages) ptx::tma_prefetch_l2_3d(&tmap_page, 0, next1 * kPage, 0);
              }
            }
            for (int c0 = 0; ok && c0 < kPieces; c0 += kPer) {
              for (int c = c0; new_q && qfill > 0 && t == s0 && c < c0 + kPer; ++c) {
                ok = warp_wait(&ms->q_empty[c], (qfill - 1) & 1, abort, p);
                if (!ok) break;
                if (ptx::elect_one()) load_q(c, req.tok0 * p.H + g * n);
                __syncwarp();
              }
              if (ok && ring.phase > 0) ok = warp_wait(&ms->kv_empty[ring.at], (ring.phase - 1) & 1, abort, p);
              if (!ok) break;
              if (!(blockIdx.x == 0 && fill == p.skip_copy) && ptx::elect_one()) {
                uint8_t* dst = sK + ring.at * kStageBytes;
                ptx::mbar_arrive_expect_tx(&ms->kv_full[ring.at], (two ? 2 : 1) * kPer * kHalf);
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
                  ptx::tma_load_3d(dst + j * kPieceBytes, &tmap_kv, &ms->kv_full[ring.at], 0, id0 * kPage, c0 + j);
                  if (two)
                    ptx::tma_load_3d(dst + j * kPieceBytes + kHalf, &tmap_kv, &ms->kv_full[ring.at], 0, id1 * kPage, c0 + j);
                }
              }
              __syncwarp();
              ring.step();
              ++fill;
            }
          }
          if (new_q) ++qfill;
        }
        cur0 = nxt0;
        cur1 = nxt1;
      }
    }
    // After an abort every copy must have landed before the CTA may exit: the ring's last ones
    // and the Q pieces'. (Of a barrier's two phases one is always over; where no copy is under
    // way the other ends by the short limit.)
    if (*abort && lane == 0) {
      for (int i = 0; i < p.stages + kPieces; ++i)
        for (uint32_t par = 0; par < 2; ++par) {
          uint64_t* bar = i < p.stages ? &ms->kv_full[i] : &ms->q_full[i - p.stages];
          const long long t0c = clock64();
          while (!ptx::mbar_try_wait(bar, par) && clock64() - t0c < kWaitBudgetTest) {
          }
        }
    }
    __syncwarp();
  } else if (warp <= R::kIssuers) {
    // ------------------------------------------------------------ products
    // The issuers take the parts in turns. Each accumulator is written by one thread in order, so
    // the sums repeat. Where a piece of Q is not always the same issuer's, each of them waits for
    // all new pieces, and says of each when its products with it are over.
    const uint32_t sq = ptx::smem_addr(sQ), sk = ptx::smem_addr(sK);
    const uint32_t idesc = kFp8 ? ptx::idesc_e4m3(kKeys, n, 0, 0) : ptx::idesc_bf16(kKeys, n, 0, 0);
    const int u0 = warp - 1;
    Ring ring(p.stages), slots(p.slots);
    ring.at = slots.at = u0;
    int first = u0;  // this issuer's first part of the tile
    uint32_t qphase = 0;
    bool ok = true, issued = false, loaded = false;
    if (kFp8) ptx::pdl_wait_primary();  // Q's parts come from the kernel before
    while (ok && walk.next(p, b, req, t0, t1)) {
      const int rows = counted_rows(p, b, req.q), groups = (rows + n - 1) / n;
      if (groups == 0 || t0 >= t1) continue;
      // the first group's Q: each issuer its own pieces, while warp 0 asks for the keys
      if (!loaded && ptx::elect_one())
        for (int u = u0; u < R::kCount; u += R::kIssuers)
          for (int c = kPer * u; c < kPer * (u + 1); ++c) load_q(c, req.tok0 * p.H);
      __syncwarp();
      loaded = true;
      const int sub = groups > 1 ? p.sub_tiles : kMaxSub;
      for (int s0 = t0; ok && s0 < t1; s0 += sub) {
        const int s1 = min(t1, s0 + sub);
        for (int g = 0; ok && g < groups; ++g) {
          const bool new_q = groups > 1 || s0 == t0, last_q = groups > 1 || s1 == t1;
          for (int t = s0; ok && t < s1; ++t) {
            const bool last = last_q && t == s1 - 1;  // the group's last products
            const bool fresh = new_q && t == s0;      // and its first
            int u = first;
            for (; ok && u < R::kCount; u += R::kIssuers) {
              const int c0 = kPer * u;
              if (fresh) {
                for (int c = R::kFixed || u == 0 ? c0 : c0 - 1; ok && c < c0 + kPer; ++c)
                  ok = warp_wait(&ms->q_full[c], qphase & 1, abort, p);
              }
              // what the accumulator held has been read
              if (ok && slots.phase > 0) ok = warp_wait(&ms->d_empty[slots.at], (slots.phase - 1) & 1, abort, p);
              if (ok) ok = warp_wait(&ms->kv_full[ring.at], ring.phase & 1, abort, p);
              if (!ok) break;
              ptx::tc_fence_after();
              const uint32_t d = tmem + slots.at * n;
              const uint64_t ad = ptx::smem_desc(sk + ring.at * kStageBytes, 16, kSbo, kSwizzle);
              const uint64_t bd = ptx::smem_desc(sq + c0 * q_piece, 16, kSbo, kSwizzle);
              if (ptx::elect_one()) {
#pragma unroll
                for (int j = 0; j < kPer; ++j) {
#pragma unroll
                  for (int k = 0; k < kRowBytes / 32; ++k) {  // the address field counts 16 bytes
                    const uint64_t a = ad + j * (kPieceBytes / 16) + 2 * k, q = bd + j * (q_piece / 16) + 2 * k;
                    const uint32_t add = (j | k) == 0 ? 0u : 1u;
                    if constexpr (kFp8) {
                      ptx::mma_e4m3_ss(d, a, q, idesc, add);
                      ptx::mma_e4m3_ss(d, a, q + n * 64 / 16, idesc | ptx::kB_E5M2, 1u);
                    } else {
                      ptx::mma_bf16_ss(d, a, q, idesc, add);
                    }
                  }
                }
                ptx::mma_commit(&ms->kv_empty[ring.at]);
                if (last) {
                  for (int j = 0; j < kPer; ++j) ptx::mma_commit(&ms->q_empty[c0 + j]);
                  if (!R::kFixed && u > 0) ptx::mma_commit(&ms->q_empty[c0 - 1]);
                }
                ptx::mma_commit(&ms->d_full[(t - s0) & 1][slots.at]);
              }
              __syncwarp();
              issued = true;
              ring.step(R::kIssuers);
              slots.step(R::kIssuers);
            }
            first = u - R::kCount;
            if (!R::kFixed && first == 0) {  // another issuer had the last piece
              if (ok && fresh) ok = warp_wait(&ms->q_full[kPieces - 1], qphase & 1, abort, p);
              if (ok && last && ptx::elect_one()) ptx::mma_commit(&ms->q_empty[kPieces - 1]);
              __syncwarp();
            }
          }
          if (new_q) ++qphase;
        }
      }
    }
    // every product must retire before tensor memory is released (the same lane issued them all)
    if (issued && ptx::elect_one()) drain_mmas(&ms->mma_done[warp - 1], p.wait_budget);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ weights
    const int wg = (warp - 4) >> 2, qd = warp & 3;
    if (kFp8) ptx::pdl_wait_primary();  // q_scale comes from the kernel before
    if (n == 32)
      weights_role<1, kFp8>(p, ms, walk, tmem, wg, qd, lane);
    else if (n == 64)
      weights_role<2, kFp8>(p, ms, walk, tmem, wg, qd, lane);
    else if (n == 96)
      weights_role<3, kFp8>(p, ms, walk, tmem, wg, qd, lane);
    else
      weights_role<4, kFp8>(p, ms, walk, tmem, wg, qd, lane);
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 512);
  }
}

// Q [rows, 576] bf16 -> its e4m3 and its e5m2 part [2][rows][576] and the factor that undoes each row's power
// of two. One warp per row: 72 pieces of 8 entries, lane l holds pieces l, l + 32 and (l < 8) 64 + l.
constexpr int kSplitWarps = 8;
__global__ void __launch_bounds__(32 * kSplitWarps) q_split_kernel(const uint4* q, int rows, uint8_t* parts,
                                                                   float* q_scale) {
  ptx::pdl_launch_dependents();
  const int row = blockIdx.x * kSplitWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (row >= rows) return;
  uint4 v[3];
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 3; ++i) v[i] = 32 * i + lane < 72 ? q[(size_t)row * 72 + 32 * i + lane] : make_uint4(0u, 0u, 0u, 0u);
  auto entry = [&](int i, int k) {
    const uint32_t w = k < 2 ? v[i].x : k < 4 ? v[i].y : k < 6 ? v[i].z : v[i].w;
    return __uint_as_float((k & 1) ? (w & 0xFFFF0000u) : (w << 16));
  };
#pragma unroll
  for (int i = 0; i < 3; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(entry(i, k)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  int e = 0;
  if (mx > 0.f && mx < INFINITY) e = max(-100, min(100, 7 - ((int)(__float_as_uint(mx) >> 23) - 127)));
  const float sc = __uint_as_float((uint32_t)(e + 127) << 23);
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    if (32 * i + lane >= 72) continue;
    uint32_t hi[2] = {0u, 0u}, lo[2] = {0u, 0u};
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      const float a = entry(i, k) * sc, c = entry(i, k + 1) * sc;
      const __nv_fp8x2_storage_t h = __nv_cvt_float2_to_fp8x2(make_float2(a, c), __NV_SATFINITE, __NV_E4M3);
      const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3);
      const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&hr));
      const __nv_fp8x2_storage_t r = __nv_cvt_float2_to_fp8x2(make_float2(a - back.x, c - back.y), __NV_SATFINITE, __NV_E5M2);
      hi[k >> 2] |= (uint32_t)h << (8 * (k & 3));
      lo[k >> 2] |= (uint32_t)r << (8 * (k & 3));
    }
    const size_t at = (size_t)row * 576 + 8 * (32 * i + lane);
    *reinterpret_cast<uint2*>(parts + at) = make_uint2(hi[0], hi[1]);
    *reinterpret_cast<uint2*>(parts + (size_t)rows * 576 + at) = make_uint2(lo[0], lo[1]);
  }
  if (lane == 0) q_scale[row] = __uint_as_float((uint32_t)(127 - e) << 23);
}

size_t weights_workspace(const PlanHeader* h) {
  if (h->kv_dtype != MLA_KV_FP8_E4M3) return 0;
  const size_t rows = (size_t)h->total_q * h->num_heads;
  return (rows * 1152 + 255) / 256 * 256 + (rows * sizeof(float) + 255) / 256 * 256;
}

// [rows, 576] as (64 columns, rows, 9 pieces), boxes of box_rows rows and box_pieces pieces.
CUresult encode(PFN_cuTensorMapEncodeTiled_v12000 enc, CUtensorMap* map, const void* base, bool fp8, uint64_t rows,
                uint32_t box_rows, uint32_t box_pieces) {
  const uint64_t esz = fp8 ? 1 : 2;
  cuuint64_t dims[3] = {64, (cuuint64_t)rows, (cuuint64_t)kPieces};
  cuuint64_t strides[2] = {(cuuint64_t)(kDqk * esz), (cuuint64_t)(64 * esz)};
  cuuint32_t box[3] = {64, box_rows, box_pieces};
  cuuint32_t es[3] = {1, 1, 1};
  return enc(map, fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base),
             dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE,
             fp8 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
}

}  // namespace

cudaError_t set_weights_kernel_attributes(int* regs) {
  *regs = 255;
  for (const void* fn : {(const void*)key_weights_kernel<false>, (const void*)key_weights_kernel<true>}) {
    cudaFuncAttributes a;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemCap);
    if (e == cudaSuccess) e = cudaFuncGetAttributes(&a, fn);
    if (e != cudaSuccess) return e;
    *regs = std::min(*regs, a.numRegs);
  }
  return cudaSuccess;
}

}  // namespace mla

using namespace mla;

extern "C" int mla_key_weights_workspace(const void* plan_host, size_t plan_bytes, size_t* workspace_bytes_out) {
  clear_error();
  const PlanHeader* h = nullptr;
  const int rc = check_plan(plan_host, plan_bytes, &h);
  if (rc != MLA_OK) return rc;
  if (!workspace_bytes_out) return set_error(MLA_ERR_INVALID_ARG, "workspace_bytes_out must not be NULL");
  *workspace_bytes_out = weights_workspace(h);
  return MLA_OK;
}

extern "C" int mla_key_weights(const void* plan_dev, const void* plan_host, size_t plan_bytes, const void* q,
                               const void* kv_cache, const float* kv_scales, int block_tokens,
                               const int32_t* page_table, int page_table_stride, int num_pages, const float* lse,
                               const int32_t* counted, float sm_scale, float kv_scale, float decay, float* weights,
                               long long weights_stride, void* workspace, size_t workspace_bytes, int32_t* status_dev,
                               void* stream) {
  clear_error();
  const PlanHeader* h = nullptr;
  int rc = check_plan(plan_host, plan_bytes, &h);
  if (rc != MLA_OK) return rc;
  if (!plan_dev || !q || !kv_cache || !page_table || !lse || !weights)
    return set_error(MLA_ERR_INVALID_ARG, "plan_dev, q, kv_cache, page_table, lse and weights must not be NULL");
  if (((uintptr_t)plan_dev & 15u) || ((uintptr_t)q & 15u) || ((uintptr_t)kv_cache & 15u))
    return set_error(MLA_ERR_INVALID_ARG, "plan_dev, q and kv_cache must be 16-byte aligned");
  for (const void* ptr : {(const void*)page_table, (const void*)lse, (const void*)weights, (const void*)counted,
                          (const void*)kv_scales, (const void*)status_dev})
    if ((uintptr_t)ptr & 3u)
      return set_error(MLA_ERR_INVALID_ARG, "page_table, lse, weights, counted, kv_scales and status_dev must be 4-byte aligned");
  const bool fp8 = h->kv_dtype == MLA_KV_FP8_E4M3;
  if (kv_scales && !fp8) return set_error(MLA_ERR_INVALID_ARG, "block scales belong to an fp8 e4m3 cache");
  const int bl = kv_scales ? block_log2_of(block_tokens) : 0;
  if (bl < 0) return set_error(MLA_ERR_UNSUPPORTED, "block_tokens must be 1, 2, 4, .. 64 (got %d)", block_tokens);
  if (num_pages < 1 || (long long)num_pages * kPage > 0xFFFFFFFFLL)
    return set_error(MLA_ERR_INVALID_ARG, "num_pages out of range (got %d)", num_pages);
  if (page_table_stride < h->max_pages)
    return set_error(MLA_ERR_INVALID_ARG, "page_table_stride %d is smaller than the %d pages of the longest request",
                     page_table_stride, h->max_pages);
  if (!(sm_scale > 0.f) || !isfinite(sm_scale) || !(kv_scale > 0.f) || !isfinite(kv_scale))
    return set_error(MLA_ERR_INVALID_ARG, "sm_scale and kv_scale must be finite and > 0");
  if (!isfinite(decay)) return set_error(MLA_ERR_INVALID_ARG, "decay must be finite");
  // the lengths that the plan was built for
  const PlanRequest* reqs = (const PlanRequest*)((const uint8_t*)plan_host + h->req_off);
  int max_ctx = 0, most_rows = 0;
  for (int i = 0; i < h->batch; ++i) {
    max_ctx = std::max(max_ctx, reqs[i].ctx);
    const int r = reqs[i].q * h->num_heads, g = (r + kMaxRows - 1) / kMaxRows;
    most_rows = std::max(most_rows, ((r + g - 1) / g + 31) / 32 * 32);
  }
  if (weights_stride < max_ctx)
    return set_error(MLA_ERR_INVALID_ARG, "weights_stride %lld is smaller than the longest request's %d keys",
                     weights_stride, max_ctx);
  const size_t need = weights_workspace(h);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return set_error(MLA_ERR_BUFFER, "workspace needs %zu bytes (got %zu)", need, workspace ? workspace_bytes : (size_t)0);
  if (need > 0 && ((uintptr_t)workspace & 255u)) return set_error(MLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");

  DeviceKernels device;
  rc = current_device_ready(&device);
  if (rc != MLA_OK) return rc;
  if (device.weights != cudaSuccess)
    return set_error(MLA_ERR_CUDA, "key weights kernel attributes: %s", cudaGetErrorString(device.weights));
  // launched with fewer registers than its warpgroups share out, the kernel would wait for them forever
  if (device.weights_regs < kRegsLaunch)
    return set_error(MLA_ERR_UNSUPPORTED, "the key weights kernel was compiled to %d registers a thread and needs %d",
                     device.weights_regs, kRegsLaunch);
  const int piece = fp8 ? 8192 : 16384, tile_bytes = kPieces * piece;
  const int fixed = 1024 + kMiscBytes + kPieces * most_rows * 128;
  const int per = fp8 ? Parts<true>::kPer : Parts<false>::kPer;
  const int issuers = fp8 ? Parts<true>::kIssuers : Parts<false>::kIssuers;
  const int stages = std::min(kMaxStages, (kSmemCap - fixed) / (per * piece)) / issuers * issuers;
  const int smem = fixed + stages * per * piece;
  auto fn = fp8 ? key_weights_kernel<true> : key_weights_kernel<false>;
  PFN_cuTensorMapEncodeTiled_v12000 enc = tensor_map_encoder();
  if (!enc) return set_error(MLA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");

  WeightsParams prm{};
  prm.total_rows = h->total_q * h->num_heads;
  long long tiles = 0;
  for (int i = 0; i < h->batch; ++i) {
    const long long t = (reqs[i].ctx + kKeys - 1) / kKeys;
    tiles += t;
    prm.total_work += t * ((reqs[i].q * h->num_heads + most_rows - 1) / most_rows);
  }
  const unsigned grid = (unsigned)std::min<long long>(tiles, device.sms);
  prm.reqs = (const PlanRequest*)((const uint8_t*)plan_dev + h->req_off);
  prm.first = reqs[0];
  prm.batch = h->batch;
  prm.H = h->num_heads;
  prm.pt_stride = page_table_stride;
  prm.num_pages = num_pages;
  prm.block_log2 = bl;
  prm.page_table = page_table;
  prm.kv_scales = kv_scales;
  prm.lse = lse;
  prm.counted = counted;
  prm.weights = weights;
  prm.w_stride = weights_stride;
  prm.decay = decay;
  prm.sm_scale = sm_scale;
  prm.kv_scale = kv_scale;
  prm.rows_n = most_rows;
  prm.stages = stages;
  prm.slots = std::min(kMaxSlots, 512 / most_rows) / issuers * issuers;
  // Tiles that all CTAs together keep in L2 while the groups pass over them, an even number as two
  // warpgroups take turns. Where HBM refills L2 meanwhile, less than half of it: 32 requests of 16k
  // keys, 512 rows, bf16 325 us at 90 MB, 312 at 50 (e4m3 223, 213). Keys that all fit stay there
  // anyhow, and longer passes load Q less often (768 rows over 131k e4m3 keys 72 us, 79 at 50 MB).
  const long long room = tiles * tile_bytes <= (80LL << 20) ? 90LL << 20 : 50LL << 20;
  prm.sub_tiles = std::max(2, std::min<int>(kMaxSubSums, (int)(room / ((long long)tile_bytes * grid))) / 2 * 2);
  prm.status = status_dev;
  prm.wait_budget = h->debug_skip_copy > 0 ? kWaitBudgetTest : kWaitBudget;
  prm.skip_copy = h->debug_skip_copy - 1;
  const void* q_src = q;
  if (fp8) {
    prm.q_scale = (const float*)((uint8_t*)workspace + ((size_t)prm.total_rows * 1152 + 255) / 256 * 256);
    q_src = workspace;
  }
  alignas(64) CUtensorMap tq, tkv, tpage;
  CUresult r = encode(enc, &tq, q_src, fp8, (uint64_t)prm.total_rows * (fp8 ? 2 : 1), (uint32_t)most_rows, 1);
  if (r == CUDA_SUCCESS) r = encode(enc, &tkv, kv_cache, fp8, (uint64_t)num_pages * kPage, kPage, 1);
  if (r == CUDA_SUCCESS) r = encode(enc, &tpage, kv_cache, fp8, (uint64_t)num_pages * kPage, kPage, kPieces);
  if (r != CUDA_SUCCESS) return set_error(MLA_ERR_CUDA, "tensor map for q or kv_cache failed (CUresult %d)", (int)r);
  cudaStream_t st = (cudaStream_t)stream;
  if (fp8) {
    q_split_kernel<<<(prm.total_rows + kSplitWarps - 1) / kSplitWarps, 32 * kSplitWarps, 0, st>>>(
        (const uint4*)q, prm.total_rows, (uint8_t*)workspace, const_cast<float*>(prm.q_scale));
    const cudaError_t ce = cudaGetLastError();
    if (ce != cudaSuccess) return set_error(MLA_ERR_CUDA, "Q split kernel launch: %s", cudaGetErrorString(ce));
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = st;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = fp8 ? 1 : 0;
  const cudaError_t ce = cudaLaunchKernelEx(&cfg, fn, tq, tkv, tpage, prm);
  if (ce != cudaSuccess) return set_error(MLA_ERR_CUDA, "key weights kernel launch: %s", cudaGetErrorString(ce));
  return MLA_OK;
}
