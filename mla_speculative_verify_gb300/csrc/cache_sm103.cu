// cache_sm103.cu -- the paged latent cache's own operators: mla_cache_append writes new rows
// into an e4m3 cache with a scale for each block of tokens, mla_cache_evict keeps the keys
// with the largest accumulated attention weight and moves them to new pages.
//
// Block scales. A block is block_tokens consecutive tokens of a page (1, 2, 4, .. 64); the
// value of a stored code c is c * scale(block). An append gives a block the least power of
// two 2^e, e in [-60, 60], with amax <= 448 * 2^e (448 is the largest e4m3 value), so that
// x / scale and a later change of scale are exact but for e4m3's own rounding. A block that
// already holds earlier tokens keeps the larger of its old and the new scale, and where that
// grows its old codes are rounded to the new one.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "decode_common.cuh"
#include "mla_decode.h"
#include "plan_format.h"
#include "ptx.cuh"
#include "status.h"

namespace mla {

int current_device_ready(DeviceKernels* out);  // defined next to the decode kernel
int block_log2_of(int block_tokens);           // defined with the plan

namespace {

constexpr int kScaleExpMin = -60, kScaleExpMax = 60;

// The least 2^e, e in [-60, 60], with amax <= 448 * 2^e, from amax's bits: 448 = 1.75 * 2^8, so
// e is amax's own exponent - 8, one more if its mantissa is above 1.75.
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(kScaleExpMin, min(kScaleExpMax, e));
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// A change of scale: codes are multiplied by `ratio` and rounded to e4m3 again. down = k where
// the ratio is 2^-k, k in [1, 14]: the exponent field of a code whose result is a normal number
// just drops by k.
struct Rescale {
  float ratio;
  int down;
  __device__ __forceinline__ explicit Rescale(float r) : ratio(r), down(0) {
    const uint32_t u = __float_as_uint(r);
    const int k = 127 - (int)(u >> 23);
    if ((u & 0x7FFFFFu) == 0 && k >= 1 && k <= 14) down = k;
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t codes) const {
    if (down > 0) {
      // bit 7 of each byte of `fits`: magnitude >= 8 (k + 1), and of `nan`: magnitude 0x7F
      const uint32_t mag = codes & 0x7F7F7F7Fu;
      const uint32_t fits = mag + 0x01010101u * (0x80 - 8 * (down + 1)), nan = mag + 0x01010101u;
      if ((fits & ~nan & 0x80808080u) == 0x80808080u) return codes - 0x08080808u * down;
    }
    float f[4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(codes >> (16 * k)), __NV_E4M3);
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
      f[2 * k] = v.x * ratio;
      f[2 * k + 1] = v.y * ratio;
    }
    return e4m3x4(f[0], f[1], f[2], f[3]);
  }
};

// ------------------------------------------------------------------ append
struct AppendArgs {
  const uint4* rows;  // [total, 576] bf16 as 72 16-byte pieces a row
  int total;
  const int32_t* page_table;
  int pt_stride, num_pages, max_new, block_log2;
  const int32_t* ends;
  const int32_t* cu;
  uint8_t* codes;
  float* scales;
  int32_t* status;
};

// One CTA per page that a request's new rows reach (blockIdx = page within those, request).
// Eight lanes hold a row (nine 16-byte pieces each, 128 contiguous bytes of a row per load),
// so the page's rows are read once, all loads in flight together, and stay in registers
// between the maximum and the rounding. The rows' loads do not wait for the page's id. Bound by
// HBM: 131072 rows in 37 us, 6.1 TB/s (0.90 of the measured copy rate), 262144 rows in 66 us,
// 6.9 TB/s (some of the codes stay in L2). With 256 threads, two rows to eight lanes and the page
// id first it was 43 us.
constexpr int kAppendThreads = 512;

__global__ void __launch_bounds__(kAppendThreads, 2) append_kernel(AppendArgs a) {
  __shared__ float row_max[kPage], scale[kPage], ratio[kPage], half_max[2];
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int r0 = a.cu[b], n = a.cu[b + 1] - r0, end = a.ends[b];
  if (n == 0) return;
  if (r0 < 0 || n < 0 || n > a.max_new || r0 > a.total - n || end < n || (end - 1) / kPage >= a.pt_stride) {
    if (tid == 0 && blockIdx.x == 0) report(a.status, MLA_DEVICE_PLAN_MISMATCH);
    return;
  }
  const int start = end - n;
  const int pg = start / kPage + blockIdx.x;
  if ((long long)pg * kPage >= end) return;
  const int page = a.page_table[(size_t)b * a.pt_stride + pg];
  const int lo = max(start - pg * kPage, 0), hi = min(end - pg * kPage, kPage);  // new rows of the page
  const int sub = lane & 7, r = tid >> 3;
  const bool live = r >= lo && r < hi;
  uint4 v[9];
  const uint4* src = a.rows + (size_t)(live ? r0 + (pg * kPage + r - start) : 0) * 72 + sub;
#pragma unroll
  for (int j = 0; j < 9; ++j) v[j] = live ? __ldcs(src + 8 * j) : make_uint4(0u, 0u, 0u, 0u);
  if (page < 0 || page >= a.num_pages) {
    if (tid == 0) report(a.status, MLA_DEVICE_BAD_PAGE);
    return;
  }
  float* page_scales = a.scales + ((size_t)page << (6 - a.block_log2));
  // a block whose first row is older than the new ones keeps what it holds
  const int blk = tid >> a.block_log2, blk_row0 = blk << a.block_log2;
  float s_old = 0.f;
  if (tid < kPage && blk_row0 < lo) s_old = page_scales[blk];
  // the largest magnitude from the bits (bf16 magnitudes order as integers); infinities and
  // NaN are left out, in a second pass that only rows which hold some take
  uint32_t m2 = 0;
#pragma unroll
  for (int j = 0; j < 9; ++j) {
    m2 = __vmaxu2(m2, __vmaxu2(v[j].x & 0x7FFF7FFFu, v[j].y & 0x7FFF7FFFu));
    m2 = __vmaxu2(m2, __vmaxu2(v[j].z & 0x7FFF7FFFu, v[j].w & 0x7FFF7FFFu));
  }
  uint32_t top = max(m2 & 0xFFFFu, m2 >> 16);
  if (top >= 0x7F80u) {
    top = 0;
#pragma unroll
    for (int j = 0; j < 9; ++j) {
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t x = w[k] & 0x7FFFu, y = (w[k] >> 16) & 0x7FFFu;
        if (x < 0x7F80u) top = max(top, x);
        if (y < 0x7F80u) top = max(top, y);
      }
    }
  }
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (sub == 0) row_max[r] = __uint_as_float(top << 16);
  __syncthreads();
  if (tid < kPage) {
    float m = row_max[tid];
    for (int o = 1; o < min(1 << a.block_log2, 32); o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if (a.block_log2 == 6) {
      if (lane == 0) half_max[warp] = m;
      ptx::bar_sync(1, kPage);
      m = fmaxf(half_max[0], half_max[1]);
    }
    const float s = fmaxf(scale_for(m), s_old);
    scale[tid] = s;
    ratio[tid] = s_old / s;
    // the block's first row writes its scale, if the block has new rows at all
    if (tid == blk_row0 && blk_row0 < hi && blk_row0 + (1 << a.block_log2) > lo) page_scales[blk] = s;
  }
  __syncthreads();
  uint2* dst = reinterpret_cast<uint2*>(a.codes + ((size_t)page * kPage + r) * kDqk) + sub;
  if (live) {
    const float s = scale[r];
    // a power of two divides exactly through its reciprocal; a block that kept another
    // writer's scale divides
    const bool two = (__float_as_uint(s) & 0x7FFFFFu) == 0 && s >= 0x1p-120f && s <= 0x1p120f;
    const float inv = two ? 1.f / s : 0.f;
#pragma unroll
    for (int j = 0; j < 9; ++j) {
      const uint32_t w[4] = {v[j].x, v[j].y, v[j].z, v[j].w};
      float f[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
      }
      if (two) {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] *= inv;
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __fdiv_rn(f[k], s);
      }
      dst[8 * j] = make_uint2(e4m3x4(f[0], f[1], f[2], f[3]), e4m3x4(f[4], f[5], f[6], f[7]));
    }
  } else if (r < lo && (r >> a.block_log2) == (lo >> a.block_log2) && ratio[r] != 1.f) {
    const Rescale to(ratio[r]);
#pragma unroll
    for (int j = 0; j < 9; ++j) {
      const uint2 c = dst[8 * j];
      dst[8 * j] = make_uint2(to(c.x), to(c.y));
    }
  }
}

// ------------------------------------------------------------------ eviction: which keys stay
struct SelectArgs {
  const float* weights;
  long long w_stride;
  const int32_t* lens;
  int max_seq, budget, n_first, n_last;
  int32_t* kept;
  float* weights_dst;
  long long wd_stride;
  int32_t* lens_dst;
  int32_t* status;
};

constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kSelStep = 128;    // keys a warp takes at once; a warp's share is a multiple
constexpr int kSelCopies = 4;    // copies of a CTA's histogram: equal weights hit one bin
constexpr int kSelKeys = 8192;   // keys of a CTA, at most
constexpr int kSelMaxCtas = 8;   // CTAs of a cluster, at most
constexpr int kSelWarpKeys = kSelKeys / kSelWarps;
constexpr int kSelCacheBytes = 4 * kSelWarps * (kSelWarpKeys + 4);

// A weight as an unsigned key of the same order; -0 counts as 0, NaN as the lowest.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ float weight_of(uint32_t key) {
  return key == 0u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// One cluster of CTAs per request (blockIdx.y). The k-th largest key of the middle is found
// from its bits, 11, 11 and 10 at a time: every CTA counts its keys by the next bits among
// those that match the bits found so far, the cluster adds the counts (each CTA reads its
// peers' through distributed shared memory), and each finds the same bin. Then the kept keys
// are numbered in order: those above the threshold, and of those equal to it the first ones.
// A warp owns a contiguous piece of the keys in every pass; the weights are read once and kept
// in shared memory. Places behind the last key hold the lowest key: they come after every real
// one, so none is ever taken. What bounds it is the chain of passes: 4 requests of 4k keys 9 us,
// 32 of 32k 15 us.
template <bool kOne>  // one CTA per request
__global__ void __launch_bounds__(kSelThreads, 1) evict_select_kernel(SelectArgs a) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  extern __shared__ __align__(16) uint32_t cache[];  // per warp its keys, and 4 places more
  __shared__ uint64_t loaded[kSelWarps];
  __shared__ __align__(16) uint32_t copies[kSelCopies][kBins], hist[2][kBins];
  __shared__ uint32_t coarse[2][kSelWarps];  // this CTA's counts of 64 bins each
  __shared__ uint32_t part[2][kSelThreads];  // words read from the peers
  __shared__ uint32_t gt_of[kSelWarps], eq_of[kSelWarps], totals[2];
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = kOne ? 0 : (int)cluster.block_rank(), ctas = kOne ? 1 : (int)cluster.num_blocks();
  auto sync_all = [&] {
    if (kOne)
      __syncthreads();
    else
      cluster.sync();
  };
  const int n = a.lens[b];
  const float* w = a.weights + (size_t)b * a.w_stride;
  int32_t* kept = a.kept + (size_t)b * a.budget;
  float* wd = a.weights_dst ? a.weights_dst + (size_t)b * a.wd_stride : nullptr;
  const int gtid = rank * kSelThreads + tid, gthreads = ctas * kSelThreads;
  const bool bad = n < 0 || n > a.max_seq;
  const int out = bad ? 0 : min(n, a.budget);
  // lens_dst may be lens: the new length is written behind a barrier that the whole cluster reaches
  // with the old one
  auto write_length = [&] {
    if (gtid != 0) return;
    a.lens_dst[b] = out;
    if (bad) report(a.status, MLA_DEVICE_PLAN_MISMATCH);
  };
  if (out < a.budget || n == a.budget) {  // everything stays (the whole cluster leaves here)
    sync_all();
    write_length();
    for (int r = gtid; r < a.budget; r += gthreads) {
      kept[r] = r < out ? r : -1;
      if (wd && r < out) wd[r] = w[r];
    }
    return;
  }
  const int lo = a.n_first, m = n - a.n_first - a.n_last, k = a.budget - a.n_first - a.n_last;
  for (int r = gtid; r < a.n_first; r += gthreads) {
    kept[r] = r;
    if (wd) wd[r] = w[r];
  }
  for (int r = gtid; r < a.n_last; r += gthreads) {
    kept[a.budget - a.n_last + r] = n - a.n_last + r;
    if (wd) wd[a.budget - a.n_last + r] = w[n - a.n_last + r];
  }
  if (k == 0) {  // the whole cluster again
    sync_all();
    write_length();
    return;
  }
  const int per = ((m + ctas * kSelWarps - 1) / (ctas * kSelWarps) + kSelStep - 1) / kSelStep * kSelStep;
  const long long i0 = ((long long)rank * kSelWarps + warp) * per;  // this warp's first key
  const float* wm = w + lo;
  // The warp's weights come in by a bulk copy, which wants 16-byte boundaries: they lie in shared
  // memory as they do in their 16 bytes of global memory, and up to three before the first
  // boundary and after the last come in by themselves.
  const int count = (int)max(0ll, min((long long)per, m - i0));
  const int off = (int)(((uintptr_t)(wm + i0) >> 2) & 3);
  uint32_t* cw = cache + warp * (kSelWarpKeys + 4) + off;
  uint32_t* cl = cw + lane;
  const int head = min(count, (4 - off) & 3), body_words = (count - head) & ~3, rest = count - head - body_words;
  if (lane == 0) {
    ptx::mbar_init(&loaded[warp], 1);
    ptx::fence_mbar_init();
    if (body_words > 0) {
      ptx::mbar_arrive_expect_tx(&loaded[warp], 4 * body_words);
      ptx::bulk_load(cw + head, wm + i0 + head, 4 * body_words, &loaded[warp]);
    }
  }
  if (lane < head) cw[lane] = __float_as_uint(wm[i0 + lane]);
  if (lane < rest) cw[head + body_words + lane] = __float_as_uint(wm[i0 + head + body_words + lane]);
  for (int i = tid; i < kSelCopies * kBins; i += kSelThreads) (&copies[0][0])[i] = 0u;
  __syncthreads();
  if (body_words > 0) {
    const long long t0 = clock64();
    while (!ptx::mbar_try_wait(&loaded[warp], 0)) {
      if (clock64() - t0 > kWaitBudget) {
        report(a.status, MLA_DEVICE_WAIT_TIMEOUT);
        break;
      }
    }
  }
  __syncwarp();
  for (int i = 0; i < per; i += 32) cl[i] = i + lane < count ? order_key(__uint_as_float(cl[i])) : 0u;
  // body(keys i + lane, i + lane + 32, .., i) for every step of the warp's keys
  auto sweep = [&](auto body) {
#pragma unroll 2
    for (int i = 0; i < per; i += kSelStep) {
      uint32_t key[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) key[u] = cl[i + 32 * u];
      body(key, i);
    }
  };

  uint32_t prefix = 0, want = (uint32_t)k;  // bits found so far; rank within the keys that match them
  uint32_t* mine = copies[lane % kSelCopies];
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int above = pass == 1 ? 21 : 10;  // the bits from this one up are found (pass 0: none)
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    sweep([&](const uint32_t (&key)[4], int) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (pass == 0 || (key[u] >> above) == prefix) atomicAdd(&mine[(key[u] >> shift) & mask], 1u);
    });
    __syncthreads();
    {
      uint2 sum = make_uint2(0u, 0u);
#pragma unroll
      for (int c = 0; c < kSelCopies; ++c) {
        uint2* h = reinterpret_cast<uint2*>(&copies[c][2 * tid]);
        sum.x += h->x;
        sum.y += h->y;
        *h = make_uint2(0u, 0u);
      }
      // (two buffers: a peer may still read the last pass's)
      *reinterpret_cast<uint2*>(&hist[pass & 1][2 * tid]) = sum;
      uint32_t s64 = sum.x + sum.y;  // a warp holds 64 bins
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s64 += __shfl_xor_sync(0xffffffffu, s64, o);
      if (lane == 0) coarse[pass & 1][warp] = s64;
    }
    sync_all();
    if (pass == 0) write_length();
    // Coarse to fine, so that few words cross the cluster: first the 64 bins that hold the
    // wanted rank, by the counts of 64 bins each, then the one among them. Warp r reads CTA r's;
    // then every warp finds the same.
    if (!kOne) {
      part[0][tid] = warp < ctas ? cluster.map_shared_rank(&coarse[pass & 1][0], warp)[lane] : 0u;
      __syncthreads();
    }
    uint32_t n0 = 0, n1 = 0;  // lane l: the counts of bins 64 (31 - l) ..
    if (kOne)
      n0 = coarse[pass & 1][kSelWarps - 1 - lane];
    else
      for (int r = 0; r < ctas; ++r) n0 += part[0][32 * r + kSelWarps - 1 - lane];
    uint32_t incl = n0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    int at = __ffs(__ballot_sync(0xffffffffu, incl >= want)) - 1;  // (there is one: want is a rank)
    want -= __shfl_sync(0xffffffffu, incl - n0, at);
    const uint32_t base = 64 * (kSelWarps - 1 - at);
    if (!kOne) {
      part[1][tid] = (tid >> 6) < ctas ? cluster.map_shared_rank(&hist[pass & 1][0], tid >> 6)[base + (tid & 63)] : 0u;
      __syncthreads();
    }
    n0 = n1 = 0;  // lane l: bins 63 - 2 l and 62 - 2 l of those
    for (int r = 0; r < ctas; ++r) {
      const uint2 c = *reinterpret_cast<const uint2*>(kOne ? &hist[pass & 1][base + 62 - 2 * lane] : &part[1][64 * r + 62 - 2 * lane]);
      n0 += c.y;
      n1 += c.x;
    }
    incl = n0 + n1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    at = __ffs(__ballot_sync(0xffffffffu, incl >= want)) - 1;
    const uint32_t before = __shfl_sync(0xffffffffu, incl - n0 - n1, at), upper = __shfl_sync(0xffffffffu, n0, at);
    const bool second = before + upper < want;
    const uint32_t bin = base + 63 - 2 * at - (second ? 1 : 0);
    prefix = pass == 0 ? bin : (prefix << (pass == 1 ? 11 : 10)) | bin;
    want -= before + (second ? upper : 0u);
  }
  // prefix is the threshold's key; `want` of the keys equal to it stay. One more sweep notes
  // which keys are above it and which equal it, a bit each (in the histograms' place). Bits are
  // then counted a word to a lane: a word to a warp, at four counts a clock, bounded this sweep.
  const int words = per / 32;
  uint2* marks = reinterpret_cast<uint2*>(&copies[0][0]) + warp * words;
  sweep([&](const uint32_t (&key)[4], int i) {
    uint32_t above[4], equal[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int u = 0; u < 4; ++u) above[u] = __ballot_sync(0xffffffffu, key[u] > prefix);
    if (__any_sync(0xffffffffu, key[0] == prefix || key[1] == prefix || key[2] == prefix || key[3] == prefix)) {
#pragma unroll
      for (int u = 0; u < 4; ++u) equal[u] = __ballot_sync(0xffffffffu, key[u] == prefix);
    }
    if (lane == 0) {
      uint4* m = reinterpret_cast<uint4*>(marks + i / 32);
      m[0] = make_uint4(above[0], equal[0], above[1], equal[1]);
      m[1] = make_uint4(above[2], equal[2], above[3], equal[3]);
    }
  });
  __syncwarp();
  uint32_t gt = 0, eq = 0;
  for (int j = lane; j < words; j += 32) {
    gt += __popc(marks[j].x);
    eq += __popc(marks[j].y);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
  }
  if (lane == 0) {
    gt_of[warp] = gt;
    eq_of[warp] = eq;
  }
  __syncthreads();
  // what the warps before this one hold, and (for the peers) what the CTA holds
  gt = gt_of[lane];
  eq = eq_of[lane];
  uint32_t gt_before = lane < warp ? gt : 0u, eq_before = lane < warp ? eq : 0u;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    gt += __shfl_xor_sync(0xffffffffu, gt, o);
    eq += __shfl_xor_sync(0xffffffffu, eq, o);
    gt_before += __shfl_xor_sync(0xffffffffu, gt_before, o);
    eq_before += __shfl_xor_sync(0xffffffffu, eq_before, o);
  }
  if (!kOne) {
    if (tid == 0) {
      totals[0] = gt;
      totals[1] = eq;
    }
    cluster.sync();
    gt = lane < rank ? cluster.map_shared_rank(&totals[0], lane)[0] : 0u;
    eq = lane < rank ? cluster.map_shared_rank(&totals[0], lane)[1] : 0u;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      gt += __shfl_xor_sync(0xffffffffu, gt, o);
      eq += __shfl_xor_sync(0xffffffffu, eq, o);
    }
    ptx::cluster_arrive();  // this CTA has read its peers' counts
    gt_before += gt;
    eq_before += eq;
  }
  gt = gt_before;
  eq = eq_before;
  // lane's words: which keys stay, and how many stay before them
  gt += (uint32_t)a.n_first + min(eq, want);  // (kept keys before this warp's)
  for (int j0 = 0; j0 < words; j0 += 32) {
    const int j = j0 + lane;
    uint2 mark = j < words ? marks[j] : make_uint2(0u, 0u);
    const uint32_t ties = __popc(mark.y);
    uint32_t incl = ties;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    const uint32_t before = eq + incl - ties;
    uint32_t room = want > before ? want - before : 0u;  // ties that still stay
    if (room < ties) {  // the lowest `room` of them
      uint32_t rest = mark.y;
      for (; room > 0; --room) rest &= rest - 1;
      mark.y &= ~rest;
    }
    eq += __shfl_sync(0xffffffffu, incl, 31);
    const uint32_t stay = mark.x | mark.y, n_stay = __popc(stay);
    incl = n_stay;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (j < words) marks[j] = make_uint2(stay, gt + incl - n_stay);
    gt += __shfl_sync(0xffffffffu, incl, 31);
  }
  __syncwarp();
  const uint32_t below = (1u << lane) - 1u;
  const int first = lo + (int)i0 + lane;
  for (int j = 0; j < words; j += 4) {  // (a multiple of four words)
    uint2 mark[4];
    uint32_t pos[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      mark[u] = marks[j + u];
      pos[u] = mark[u].y + __popc(mark[u].x & below);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if (!((mark[u].x >> lane) & 1u)) continue;
      kept[pos[u]] = first + 32 * (j + u);
      if (wd) wd[pos[u]] = weight_of(cl[32 * (j + u)]);
    }
  }
  if (!kOne) ptx::cluster_wait();  // no CTA leaves while a peer may still read its counts
}

// ------------------------------------------------------------------ eviction: long requests
// The same selection spread over the whole GPU, for requests of more keys than a cluster's 8 CTAs
// hold in shared memory (wide_selection below has both sides' times). A CTA takes 4096
// keys, eight to a thread, and every pass is a launch of its own, which sees the counts of the
// one before:
//   step 0..2  counts of the next 11, 11, 10 bits among the keys that match the bits found so far
//   step 3     how many keys of each CTA's are above the threshold, and equal to it
//   step 4     the kept keys, numbered from those counts
constexpr int kWideThreads = 512, kWideWarps = kWideThreads / 32;
constexpr int kWidePer = 8, kWideKeys = kWideThreads * kWidePer;
constexpr int kWideFrom = kSelMaxCtas * kSelKeys;  // keys of the longest request above which these are launched
constexpr int kSelMaxKeys = 1 << 21;               // the longest request that can be asked for
constexpr int kWideMaxChunks = kSelMaxKeys / kWideKeys;

struct alignas(256) WideState {  // per request, in the workspace; zero before step 0
  uint32_t hist[3][kBins];
  uint2 found[3];  // bits found by step s + 1, rank among the keys that match them
  int len;         // the old length, from step 3 for step 4, which writes the new one, perhaps over it
  uint2 counts[kWideMaxChunks];
};

template <int kStep>
__global__ void __launch_bounds__(kWideThreads) evict_wide_kernel(SelectArgs a, WideState* states) {
  __shared__ __align__(16) uint32_t copies[kStep < 3 ? kSelCopies : 1][kStep < 3 ? kBins : 1];
  __shared__ uint32_t sums[2][kWideWarps];
  __shared__ uint2 hit;
  ptx::pdl_wait_primary();
  if (kStep < 4) ptx::pdl_launch_dependents();  // the next step's CTAs come up and wait for this grid
  // (the warp's index as a value known to be the same in all lanes: 2^20 keys 127.7 -> 124.2 us)
  const int b = blockIdx.y, chunk = blockIdx.x, tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  WideState& st = states[b];
  const int n = kStep == 4 ? st.len : a.lens[b];
  if (kStep == 3 && chunk == 0 && tid == 0) st.len = n;
  const float* w = a.weights + (size_t)b * a.w_stride;
  const bool bad = n < 0 || n > a.max_seq;
  const int out = bad ? 0 : min(n, a.budget);
  const int m = n - a.n_first - a.n_last, k = a.budget - a.n_first - a.n_last;
  const bool all = out < a.budget || n == a.budget;  // everything stays
  if constexpr (kStep == 4) {
    int32_t* kept = a.kept + (size_t)b * a.budget;
    float* wd = a.weights_dst ? a.weights_dst + (size_t)b * a.wd_stride : nullptr;
    if (chunk == 0 && tid == 0) {
      a.lens_dst[b] = out;
      if (bad) report(a.status, MLA_DEVICE_PLAN_MISMATCH);
    }
    const int g0 = chunk * kWideThreads + tid, gs = gridDim.x * kWideThreads;
    if (all) {
      for (int r = g0; r < a.budget; r += gs) {
        kept[r] = r < out ? r : -1;
        if (wd && r < out) wd[r] = w[r];
      }
      return;
    }
    for (int r = g0; r < a.n_first; r += gs) {
      kept[r] = r;
      if (wd) wd[r] = w[r];
    }
    for (int r = g0; r < a.n_last; r += gs) {
      kept[a.budget - a.n_last + r] = n - a.n_last + r;
      if (wd) wd[a.budget - a.n_last + r] = w[n - a.n_last + r];
    }
  }
  if (all || k == 0) return;
  const int i0 = chunk * kWideKeys + warp * 32 * kWidePer + lane;  // this lane's keys: i0, i0 + 32, ..
  if (chunk * kWideKeys >= m && kStep != 3) return;
  const float* wm = w + a.n_first;
  float x[kWidePer];
  uint32_t key[kWidePer];
#pragma unroll
  for (int u = 0; u < kWidePer; ++u) x[u] = i0 + 32 * u < m ? wm[i0 + 32 * u] : 0.f;
#pragma unroll
  for (int u = 0; u < kWidePer; ++u) key[u] = i0 + 32 * u < m ? order_key(x[u]) : 0u;  // (behind the last: the lowest)
  if (kStep < 3) {
    for (int i = tid; i < kSelCopies * kBins; i += kWideThreads) (&copies[0][0])[i] = 0u;
  }
  uint2 known = make_uint2(0u, (uint32_t)k);  // bits found so far, rank among the keys that match them
  if (kStep >= 1 && kStep <= 3) {
    // the bin of the last step's counts that holds the rank: bins from the top, four to a thread
    if (kStep >= 2) known = st.found[kStep - 2];
    const uint4 c = *reinterpret_cast<const uint4*>(&st.hist[kStep - 1][kBins - 4 - 4 * tid]);
    const uint32_t own = c.x + c.y + c.z + c.w;
    uint32_t incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += t;
    }
    if (lane == 31) sums[0][warp] = incl;
    __syncthreads();
    uint32_t before = incl - own;
    for (int i = 0; i < warp; ++i) before += sums[0][i];
    if (before < known.y && before + own >= known.y) {
      const uint32_t bins[4] = {c.w, c.z, c.y, c.x};
      uint32_t rank = known.y - before;
      int at = 0;
      while (at < 3 && rank > bins[at]) rank -= bins[at++];
      const uint32_t bin = (uint32_t)(kBins - 1 - 4 * tid - at);
      hit = make_uint2(kStep == 1 ? bin : (known.x << (kStep == 2 ? 11 : 10)) | bin, rank);
    }
    __syncthreads();
    known = hit;
    if (chunk == 0 && tid == 0) st.found[kStep - 1] = known;
  } else if (kStep == 4) {
    known = st.found[2];
  } else {
    __syncthreads();
  }
  if constexpr (kStep < 3) {
    constexpr int shift = kStep == 0 ? 21 : kStep == 1 ? 10 : 0;
    constexpr int above = kStep == 1 ? 21 : 10;
    constexpr uint32_t mask = kStep == 2 ? 1023u : 2047u;
    uint32_t* mine = copies[lane % kSelCopies];
#pragma unroll
    for (int u = 0; u < kWidePer; ++u)
      if (i0 + 32 * u < m && (kStep == 0 || (key[u] >> above) == known.x)) atomicAdd(&mine[(key[u] >> shift) & mask], 1u);
    __syncthreads();
    for (int i = tid; i < kBins; i += kWideThreads) {
      uint32_t c = 0;
#pragma unroll
      for (int j = 0; j < kSelCopies; ++j) c += copies[j][i];
      if (c) atomicAdd(&st.hist[kStep][i], c);  // (whole numbers: the order of CTAs changes nothing)
    }
  } else {
    uint32_t above[kWidePer], equal[kWidePer], gt = 0, eq = 0;
#pragma unroll
    for (int u = 0; u < kWidePer; ++u) {
      above[u] = __ballot_sync(0xffffffffu, key[u] > known.x);
      equal[u] = __ballot_sync(0xffffffffu, key[u] == known.x && i0 + 32 * u < m);
      gt += __popc(above[u]);
      eq += __popc(equal[u]);
    }
    if (lane == 0) {
      sums[0][warp] = gt;
      sums[1][warp] = eq;
    }
    if constexpr (kStep == 4) {
      // what the CTAs before this one hold
      uint2 c = make_uint2(0u, 0u);
      for (int i = tid; i < chunk; i += kWideThreads) {
        c.x += st.counts[i].x;
        c.y += st.counts[i].y;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        c.x += __shfl_xor_sync(0xffffffffu, c.x, o);
        c.y += __shfl_xor_sync(0xffffffffu, c.y, o);
      }
      __shared__ uint2 part[kWideWarps];
      if (lane == 0) part[warp] = c;
      __syncthreads();
      gt = eq = 0;
      for (int i = 0; i < kWideWarps; ++i) {
        gt += part[i].x;
        eq += part[i].y;
      }
      for (int i = 0; i < warp; ++i) {
        gt += sums[0][i];
        eq += sums[1][i];
      }
      int32_t* kept = a.kept + (size_t)b * a.budget;
      float* wd = a.weights_dst ? a.weights_dst + (size_t)b * a.wd_stride : nullptr;
      const uint32_t below = (1u << lane) - 1u;
#pragma unroll
      for (int u = 0; u < kWidePer; ++u) {
        const uint32_t e = eq + __popc(equal[u] & below);
        if (((above[u] >> lane) & 1u) || (((equal[u] >> lane) & 1u) && e < known.y)) {
          const uint32_t pos = (uint32_t)a.n_first + gt + __popc(above[u] & below) + min(e, known.y);
          kept[pos] = a.n_first + i0 + 32 * u;
          if (wd) wd[pos] = x[u];
        }
        gt += __popc(above[u]);
        eq += __popc(equal[u]);
      }
    } else {
      __syncthreads();
      if (tid == 0) {
        uint2 c = make_uint2(0u, 0u);
        for (int i = 0; i < kWideWarps; ++i) {
          c.x += sums[0][i];
          c.y += sums[1][i];
        }
        st.counts[chunk] = c;
      }
    }
  }
}

// ------------------------------------------------------------------ eviction: moving the rows
struct GatherArgs {
  const int32_t* kept;
  const int32_t* lens_dst;
  int budget;
  const uint4* src;
  uint4* dst;
  const float* scales_src;
  float* scales_dst;
  int block_log2;
  const int32_t* pt_src;
  const int32_t* pt_dst;
  int pt_src_stride, pt_dst_stride, pages_src, pages_dst;
  int pages, batch;  // pages of the longest result, requests
  int32_t* status;
};

// CTAs that take new pages in turn (page i of the list: request i / pages, its page i % pages).
// P = 16-byte pieces of a row (72: bf16, 36: e4m3), held by P / 9 lanes with nine pieces each.
// To find a row takes five loads one after the other (new length, new page, index, old page,
// scale: ~3 us), so two warps of their own look up the next page's rows while the other eight
// move this one's. For a block-scaled cache the new block takes the largest scale of its rows and
// codes from a block with a smaller one are rounded to it. Bound by HBM: 262144 bf16 rows in 97 us
// (604 MB, 0.92 of the measured copy rate); 262144 e4m3 rows, 576 scattered bytes each, most of
// them to another scale, in 55 us (302 MB, 0.81); converted one by one instead of by the exponent
// they took 62 us.
constexpr int kMoveThreads = 256, kGatherThreads = kMoveThreads + kPage;

template <int P, bool kScaled>
__global__ void __launch_bounds__(kGatherThreads, 3) evict_gather_kernel(GatherArgs a) {
  constexpr int kLanes = P / 9;                           // 8 or 4 lanes to a row
  constexpr int kRowsPass = kMoveThreads / kLanes;        // 32 or 64 rows at a time
  __shared__ long long src_row[2][kPage];                 // per row of a page: its old row, or -1
  __shared__ float ratio[2][kPage], half_max[2];
  __shared__ int dst_page[2], dst_rows[2];
  ptx::pdl_wait_primary();
  const int tid = threadIdx.x, lane = tid & 31;
  const long long items = (long long)a.pages * a.batch;

  // the index warps: page `item` of the list into buffer `k`
  auto look_up = [&](long long item, int k) {
    const int i = tid - kMoveThreads;  // row of the page
    const int b = (int)(item / a.pages), pg = (int)(item % a.pages);
    int rows = min(kPage, a.lens_dst[b] - pg * kPage);
    int page = -1;
    if (rows > 0) {
      page = a.pt_dst[(size_t)b * a.pt_dst_stride + pg];
      if (page < 0 || page >= a.pages_dst) {
        if (i == 0) report(a.status, MLA_DEVICE_BAD_PAGE);
        rows = 0;
      }
    }
    long long row = -1;
    float s = 0.f;
    if (i < rows) {
      const int j = a.kept[(size_t)b * a.budget + pg * kPage + i];
      const int p = a.pt_src[(size_t)b * a.pt_src_stride + j / kPage];
      if (p >= 0 && p < a.pages_src) {
        row = (long long)p * kPage + j % kPage;
        if (kScaled) s = a.scales_src[row >> a.block_log2];
      } else {
        report(a.status, MLA_DEVICE_BAD_PAGE);
      }
    }
    src_row[k][i] = row;
    if (i == 0) {
      dst_page[k] = page;
      dst_rows[k] = rows;
    }
    if constexpr (kScaled) {
      float m = s;
      for (int o = 1; o < min(1 << a.block_log2, 32); o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (a.block_log2 == 6) {
        if (lane == 0) half_max[i >> 5] = m;
        ptx::bar_sync(1, kPage);
        m = fmaxf(half_max[0], half_max[1]);
        ptx::bar_sync(1, kPage);
      }
      ratio[k][i] = m > 0.f ? s / m : 1.f;
      const int blk = i >> a.block_log2;
      if (i == blk << a.block_log2 && i < rows) a.scales_dst[((size_t)page << (6 - a.block_log2)) + blk] = m;
    }
  };

  if (tid >= kMoveThreads && blockIdx.x < items) look_up(blockIdx.x, 0);
  __syncthreads();
  int k = 0;
  for (long long item = blockIdx.x; item < items; item += gridDim.x, k ^= 1) {
    if (tid >= kMoveThreads) {
      if (item + gridDim.x < items) look_up(item + gridDim.x, k ^ 1);
    } else {
      const int rows = dst_rows[k], page = dst_page[k];
      const int sub = tid % kLanes;
#pragma unroll
      for (int r = tid / kLanes; r < kPage; r += kRowsPass) {
        const long long row = r < rows ? src_row[k][r] : -1;
        if (row < 0) continue;
        const uint4* src = a.src + row * P + sub;
        uint4* dst = a.dst + ((size_t)page * kPage + r) * P + sub;
        uint4 v[9];
#pragma unroll
        for (int j = 0; j < 9; ++j) v[j] = __ldcs(src + kLanes * j);
        if (kScaled && ratio[k][r] != 1.f) {
          const Rescale to(ratio[k][r]);
#pragma unroll
          for (int j = 0; j < 9; ++j) v[j] = make_uint4(to(v[j].x), to(v[j].y), to(v[j].z), to(v[j].w));
        }
#pragma unroll
        for (int j = 0; j < 9; ++j) dst[kLanes * j] = v[j];
      }
    }
    __syncthreads();
  }
}

// Whether a row of [batch, a_stride] (of which a_row entries are used) overlaps one of [batch,
// b_stride]. Rows of both are in order, so one walk over the two lists finds it.
bool rows_overlap(const float* a, long long a_stride, int a_row, const float* b, long long b_stride, int b_row, int batch) {
  auto at = [](const float* p, long long stride, int i) { return (uintptr_t)p + 4ull * (uintptr_t)stride * (uintptr_t)i; };
  const uintptr_t a_bytes = 4ull * (uintptr_t)a_row, b_bytes = 4ull * (uintptr_t)b_row;
  if (a_bytes == 0 || b_bytes == 0) return false;
  if (at(a, a_stride, batch - 1) + a_bytes <= (uintptr_t)b || at(b, b_stride, batch - 1) + b_bytes <= (uintptr_t)a) return false;
  for (int i = 0, j = 0; i < batch && j < batch;) {
    const uintptr_t x = at(a, a_stride, i), y = at(b, b_stride, j);
    if (x + a_bytes <= y)
      ++i;
    else if (y + b_bytes <= x)
      ++j;
    else
      return true;
  }
  return false;
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

}  // namespace

cudaError_t set_select_kernel_attributes() {
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCacheBytes);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(evict_select_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSelCacheBytes);
  return e;
}

}  // namespace mla

using namespace mla;

extern "C" int mla_cache_append(const void* rows, int total_rows, const int32_t* cu_new, const int32_t* seq_lens,
                                int batch, int max_new, void* kv_cache, float* kv_scales, int block_tokens,
                                const int32_t* page_table, int page_table_stride, int num_pages, int32_t* status_dev,
                                void* stream) {
  clear_error();
  if (batch < 1 || batch > 65535) return set_error(MLA_ERR_INVALID_ARG, "batch must be in [1, 65535] (got %d)", batch);
  if (total_rows < 0 || max_new < 0 || max_new > total_rows)
    return set_error(MLA_ERR_INVALID_ARG, "need 0 <= max_new <= total_rows (got %d and %d)", max_new, total_rows);
  const int bl = block_log2_of(block_tokens);
  if (bl < 0) return set_error(MLA_ERR_UNSUPPORTED, "block_tokens must be 1, 2, 4, .. 64 (got %d)", block_tokens);
  if (num_pages < 1 || page_table_stride < 1)
    return set_error(MLA_ERR_INVALID_ARG, "num_pages and page_table_stride must be >= 1 (got %d and %d)", num_pages,
                     page_table_stride);
  if (max_new == 0) return MLA_OK;
  if (!rows || !cu_new || !seq_lens || !kv_cache || !kv_scales || !page_table)
    return set_error(MLA_ERR_INVALID_ARG, "rows, cu_new, seq_lens, kv_cache, kv_scales and page_table must not be NULL");
  if (!aligned16(rows) || !aligned16(kv_cache))
    return set_error(MLA_ERR_INVALID_ARG, "rows and kv_cache must be 16-byte aligned");
  if (!aligned4(cu_new) || !aligned4(seq_lens) || !aligned4(kv_scales) || !aligned4(page_table) || !aligned4(status_dev))
    return set_error(MLA_ERR_INVALID_ARG, "cu_new, seq_lens, kv_scales, page_table and status_dev must be 4-byte aligned");
  DeviceKernels device;
  const int rc = current_device_ready(&device);
  if (rc != MLA_OK) return rc;
  const AppendArgs a{(const uint4*)rows, total_rows, page_table, page_table_stride, num_pages, max_new, bl,
                     seq_lens, cu_new, (uint8_t*)kv_cache, kv_scales, status_dev};
  // max_new rows touch at most this many pages, wherever in a page they start
  const unsigned pages = (unsigned)(((long long)max_new + kPage - 2) / kPage + 1);
  append_kernel<<<dim3(pages, (unsigned)batch), kAppendThreads, 0, (cudaStream_t)stream>>>(a);
  const cudaError_t ce = cudaGetLastError();
  if (ce != cudaSuccess) return set_error(MLA_ERR_CUDA, "append kernel launch: %s", cudaGetErrorString(ce));
  return MLA_OK;
}

namespace mla {
// Long requests are selected by the five launches, others by clusters. Whole calls that keep 64
// keys, clusters against launches: 1 x 64k keys 19 against 19 us, 8 x 64k 19 against 25, 1 x 128k
// 23 against 19, 4 x 128k 23 against 23, 8 x 128k 37 against 27, 1 x 1M 42 against 27 (the
// longer ones then in clusters of 16, of which eight do not run at once; kSelMaxCtas is 8).
static bool wide_selection(int max_seq) { return max_seq > kWideFrom; }
}  // namespace mla

extern "C" int mla_cache_evict_workspace(int batch, int max_seq, size_t* workspace_bytes_out) {
  clear_error();
  if (batch < 1 || max_seq < 0 || !workspace_bytes_out)
    return set_error(MLA_ERR_INVALID_ARG, "need batch >= 1, max_seq >= 0 and workspace_bytes_out");
  *workspace_bytes_out = wide_selection(max_seq) ? (size_t)batch * sizeof(WideState) : 0;
  return MLA_OK;
}

extern "C" int mla_cache_evict(const float* weights, long long weights_stride, const int32_t* seq_lens, int batch,
                               int max_seq, int budget, int n_first, int n_last, int kv_dtype, const void* kv_cache,
                               const float* kv_scales, int block_tokens, const int32_t* page_table,
                               int page_table_stride, int num_pages, void* kv_cache_dst, float* kv_scales_dst,
                               const int32_t* page_table_dst, int page_table_dst_stride, int num_pages_dst,
                               int32_t* kept, int32_t* seq_lens_dst, float* weights_dst, long long weights_dst_stride,
                               void* workspace, size_t workspace_bytes, int32_t* status_dev, void* stream) {
  clear_error();
  if (batch < 1 || batch > 65535) return set_error(MLA_ERR_INVALID_ARG, "batch must be in [1, 65535] (got %d)", batch);
  if (max_seq < 0) return set_error(MLA_ERR_INVALID_ARG, "max_seq must be >= 0 (got %d)", max_seq);
  if (max_seq > kSelMaxKeys)
    return set_error(MLA_ERR_UNSUPPORTED, "max_seq must be at most %d (got %d)", kSelMaxKeys, max_seq);
  if (budget < 1 || n_first < 0 || n_last < 0 || (long long)n_first + n_last > budget)
    return set_error(MLA_ERR_INVALID_ARG, "need budget >= 1 and n_first + n_last <= budget (got %d, %d and %d)", budget,
                     n_first, n_last);
  if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3)
    return set_error(MLA_ERR_INVALID_ARG, "kv_dtype must be MLA_KV_BF16 or MLA_KV_FP8_E4M3 (got %d)", kv_dtype);
  if ((kv_scales == nullptr) != (kv_scales_dst == nullptr))
    return set_error(MLA_ERR_INVALID_ARG, "kv_scales and kv_scales_dst must both be given, or neither");
  if (kv_scales && kv_dtype != MLA_KV_FP8_E4M3)
    return set_error(MLA_ERR_INVALID_ARG, "block scales belong to an fp8 e4m3 cache");
  const int bl = kv_scales ? block_log2_of(block_tokens) : 0;
  if (bl < 0) return set_error(MLA_ERR_UNSUPPORTED, "block_tokens must be 1, 2, 4, .. 64 (got %d)", block_tokens);
  if (!weights || !seq_lens || !kv_cache || !page_table || !kv_cache_dst || !page_table_dst || !kept || !seq_lens_dst)
    return set_error(MLA_ERR_INVALID_ARG, "weights, seq_lens, the caches, their page tables, kept and seq_lens_dst must not be NULL");
  if (!aligned16(kv_cache) || !aligned16(kv_cache_dst))
    return set_error(MLA_ERR_INVALID_ARG, "kv_cache and kv_cache_dst must be 16-byte aligned");
  if (!aligned4(weights) || !aligned4(seq_lens) || !aligned4(kv_scales) || !aligned4(kv_scales_dst) ||
      !aligned4(page_table) || !aligned4(page_table_dst) || !aligned4(kept) || !aligned4(seq_lens_dst) ||
      !aligned4(weights_dst) || !aligned4(status_dev))
    return set_error(MLA_ERR_INVALID_ARG, "every pointer must be aligned to its element");
  const int most = std::min(budget, max_seq);  // rows of the longest result
  const long long pages_src = ((long long)max_seq + kPage - 1) / kPage, pages_dst = ((long long)most + kPage - 1) / kPage;
  if (num_pages < 1 || num_pages_dst < 1 || page_table_stride < pages_src || page_table_dst_stride < pages_dst)
    return set_error(MLA_ERR_INVALID_ARG, "the page tables have %d and %d entries a row, %lld and %lld are needed",
                     page_table_stride, page_table_dst_stride, pages_src, pages_dst);
  if (weights_stride < max_seq || (weights_dst && weights_dst_stride < most))
    return set_error(MLA_ERR_INVALID_ARG, "weights_stride %lld or weights_dst_stride %lld is smaller than a row",
                     weights_stride, weights_dst_stride);
  const bool wide = wide_selection(max_seq);
  const size_t need = wide ? (size_t)batch * sizeof(WideState) : 0;
  if (need > 0 && (!workspace || workspace_bytes < need))
    return set_error(MLA_ERR_BUFFER, "workspace needs %zu bytes (got %zu)", need, workspace ? workspace_bytes : (size_t)0);
  if (need > 0 && ((uintptr_t)workspace & 255u)) return set_error(MLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  // what the kernels read must not be what other CTAs of theirs write
  if (weights_dst && rows_overlap(weights, weights_stride, max_seq, weights_dst, weights_dst_stride, most, batch))
    return set_error(MLA_ERR_INVALID_ARG, "weights_dst must not overlap weights");
  if (seq_lens_dst != seq_lens && seq_lens_dst < seq_lens + batch && seq_lens < seq_lens_dst + batch)
    return set_error(MLA_ERR_INVALID_ARG, "seq_lens_dst must be seq_lens itself, or not overlap it");
  if (kv_cache == kv_cache_dst && page_table == page_table_dst)
    return set_error(MLA_ERR_INVALID_ARG, "the new pages must not be the old ones: page_table_dst is page_table");
  DeviceKernels device;
  const int rc = current_device_ready(&device);
  if (rc != MLA_OK) return rc;
  if (device.select != cudaSuccess)
    return set_error(MLA_ERR_CUDA, "selection kernel attributes: %s", cudaGetErrorString(device.select));

  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.stream = (cudaStream_t)stream;
  cfg.attrs = attr;
  cudaError_t ce;
  const SelectArgs s{weights, weights_stride, seq_lens, max_seq, budget, n_first, n_last,
                     kept, weights_dst, weights_dst_stride, seq_lens_dst, status_dev};
  if (wide) {
    ce = cudaMemsetAsync(workspace, 0, need, cfg.stream);
    cfg.gridDim = dim3((unsigned)((max_seq + kWideKeys - 1) / kWideKeys), (unsigned)batch, 1);
    cfg.blockDim = dim3(kWideThreads, 1, 1);
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    int step = 0;
    for (auto fn : {evict_wide_kernel<0>, evict_wide_kernel<1>, evict_wide_kernel<2>, evict_wide_kernel<3>, evict_wide_kernel<4>}) {
      cfg.numAttrs = step++ > 0 ? 1 : 0;
      if (ce == cudaSuccess) ce = cudaLaunchKernelEx(&cfg, fn, s, (WideState*)workspace);
    }
  } else {
    // a cluster of CTAs per request, one for every 8192 keys
    int ctas = 1;
    while (ctas * kSelKeys < max_seq) ctas *= 2;
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)batch, 1);
    cfg.blockDim = dim3(kSelThreads, 1, 1);
    cfg.dynamicSmemBytes = kSelCacheBytes;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.numAttrs = 1;
    ce = cudaLaunchKernelEx(&cfg, ctas == 1 ? evict_select_kernel<true> : evict_select_kernel<false>, s);
  }
  if (ce != cudaSuccess) return set_error(MLA_ERR_CUDA, "eviction selection launch: %s", cudaGetErrorString(ce));
  if (pages_dst == 0) return MLA_OK;

  const GatherArgs g{kept, seq_lens_dst, budget, (const uint4*)kv_cache, (uint4*)kv_cache_dst, kv_scales,
                     kv_scales_dst, bl, page_table, page_table_dst, page_table_stride, page_table_dst_stride, num_pages,
                     num_pages_dst, (int)pages_dst, batch, status_dev};
  cfg.gridDim = dim3((unsigned)std::min<long long>(pages_dst * batch, 3LL * device.sms), 1, 1);
  cfg.blockDim = dim3(kGatherThreads, 1, 1);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  auto fn = kv_dtype == MLA_KV_BF16 ? evict_gather_kernel<72, false>
            : kv_scales             ? evict_gather_kernel<36, true>
                                    : evict_gather_kernel<36, false>;
  ce = cudaLaunchKernelEx(&cfg, fn, g);
  if (ce != cudaSuccess) return set_error(MLA_ERR_CUDA, "eviction gather kernel launch: %s", cudaGetErrorString(ce));
  return MLA_OK;
}
