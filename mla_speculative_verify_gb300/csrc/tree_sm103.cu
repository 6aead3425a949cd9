// tree_sm103.cu -- trees of drafted tokens: mla_tree_masks turns parents into the visibility words
// that the decode reads, mla_tree_verify walks a tree down as far as the target's distribution
// accepts its tokens and draws the next one.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "decode_common.cuh"
#include "mla_decode.h"
#include "ptx.cuh"
#include "status.h"

namespace mla {

int current_device_ready(DeviceKernels* out);  // defined next to the decode kernel

namespace {

namespace cg = cooperative_groups;

// A request's nodes cu[b] .. cu[b + 1] - 1, or an empty range and `bad` where they do not fit.
__device__ __forceinline__ int request_nodes(const int32_t* cu, int b, int total, int max_nodes, int* first, bool* bad) {
  const int a = cu[b], e = cu[b + 1];
  *bad = a < 0 || e < a || e > total || e - a > max_nodes;
  *first = a;
  return *bad ? 0 : e - a;
}

// ------------------------------------------------------------------ masks
// One thread per node climbs from it to the root; as parents have lower indices, the words fill from
// the last one down. Parents come from shared memory: a step of the climb is one load there. The launch
// bounds it: 512 trees of 20 to 64 nodes in 3.9 us, one of 12 nodes in 3.4.
constexpr int kMaskThreads = 64;

struct MaskArgs {
  const int32_t* parents;
  const int32_t* cu;
  int total, max_nodes, words;
  uint32_t* masks;
  int32_t* depths;
  int32_t* status;
};

__global__ void __launch_bounds__(kMaskThreads) tree_masks_kernel(MaskArgs a) {
  extern __shared__ int32_t up[];
  int first;
  bool bad;
  const int q = request_nodes(a.cu, blockIdx.x, a.total, a.max_nodes, &first, &bad);
  if (bad && threadIdx.x == 0 && blockIdx.y == 0) report(a.status, MLA_DEVICE_PLAN_MISMATCH);
  const int lo = blockIdx.y * kMaskThreads;
  if (lo >= q) return;
  const int hi = min(q, lo + kMaskThreads);
  for (int i = threadIdx.x; i < hi; i += kMaskThreads) {
    int p = a.parents[first + i];
    if (p >= i) {
      if (i >= lo) report(a.status, MLA_DEVICE_BAD_TREE);
      p = -1;
    }
    up[i] = p < 0 ? -1 : p;
  }
  __syncthreads();
  const int i = lo + threadIdx.x;
  if (i >= hi) return;
  uint32_t* row = a.masks + (size_t)(first + i) * a.words;
  int at = i, seen = 0;
  for (int w = a.words - 1; w >= 0; --w) {
    uint32_t bits = 0;
    while (at >= 0 && (at >> 5) == w) {
      bits |= 1u << (at & 31);
      at = up[at];
      ++seen;
    }
    row[w] = bits;
  }
  if (a.depths) a.depths[first + i] = seen - 1;
}

// ------------------------------------------------------------------ verify
// A cluster of CTAs walks one request's tree; each CTA reads its part of the vocabulary. At node u,
// with p = softmax(target logits[u] / T) over the vocabulary:
//   one pass over the row gives every thread a running maximum and sum (and over the draft's row),
//   CTAs send one another their pairs, and every CTA joins the pairs in the same order, so all take
//   the same decisions without asking one another.
//   The children are tried in order. Without draft logits the draft is taken as certain: child token
//   x is accepted if c * R < r(x), where r is p without the tokens tried before and R its sum. With
//   draft logits (q the softmax of row u) it is accepted if c * R * q(x) < r(x), where after a
//   rejection r = max(p - S q, 0), S the sum of the R so far: max(max(p - a q, 0) - b q, 0) is
//   max(p - (a + b) q, 0), so a rejected child costs one sum over the vocabulary and no stored r.
// At the node where none is accepted the next token is argmax r(x) / E(x), E the caller's
// exponentially distributed numbers: a draw from r whose result hardly depends on rounding, unlike a
// search in r's running sum, where a border is nearer than fp32's sums are exact.
//   What bounds it: few requests, the ~3 us that a node takes from its row's first load to the cluster's
// decision, one node after the other (32 trees of up to 32 nodes over 131072 bf16 logits 27 us); many,
// the issue of the pass's instructions, 64 % of the slots, at 3.9 TB/s of the rows that are visited (256
// chains of 5 with both distributions over 131072 tokens 145 us, where HBM would take 83).
constexpr int kVerThreads = 256;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerMaxCluster = 16;
constexpr float kLargest = 3.402823466e38f, kLeast = 1.175494351e-38f;  // fp32's largest and least normal numbers

struct VerifyArgs {
  const void* target;
  const void* draft;
  long long t_stride, d_stride, n_stride;
  int vocab, total, max_nodes, path_stride;
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* cu;
  const float* temperature;
  const float* uniforms;
  const float* noise;
  int32_t* path;
  int32_t* out_tokens;
  int32_t* accepted;
  int32_t* status;
};

// Eight logits as they lie in memory.
template <typename T>
struct Raw {
  alignas(16) uint32_t w[2 * sizeof(T)];
};

// NaN logits count as -inf, infinite ones as their type's largest number.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), kLargest); }
__device__ __forceinline__ float clean(__nv_bfloat16 x) {
  return fminf(fmaxf(__bfloat162float(x), -INFINITY), __uint_as_float(0x7F7F0000u));
}
template <typename T>
__device__ __forceinline__ void clean(Raw<T>& r) {
#pragma unroll
  for (int j = 0; j < (int)(2 * sizeof(T)); ++j) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t lowest = 0xFF80FF80u, largest = 0x7F7F7F7Fu;
      __nv_bfloat162 v = *reinterpret_cast<__nv_bfloat162*>(&r.w[j]);
      v = __hmin2(__hmax2(v, *reinterpret_cast<const __nv_bfloat162*>(&lowest)), *reinterpret_cast<const __nv_bfloat162*>(&largest));
      r.w[j] = *reinterpret_cast<uint32_t*>(&v);
    } else {
      r.w[j] = __float_as_uint(clean(__uint_as_float(r.w[j])));
    }
  }
}
// The largest of n groups; NaN if there is one among them.
template <typename T>
__device__ __forceinline__ float largest_of(const Raw<T>* r, int n) {
  if constexpr (sizeof(T) == 2) {
    __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&r[0].w[0]);
#pragma unroll
    for (int j = 1; j < 4 * n; ++j) m = __hmax2_nan(m, *reinterpret_cast<const __nv_bfloat162*>(&r[j / 4].w[j % 4]));
    const __nv_bfloat16 h = __hmax_nan(__low2bfloat16(m), __high2bfloat16(m));
    return __bfloat162float(h);
  } else {
    float m = __uint_as_float(r[0].w[0]);
#pragma unroll
    for (int j = 1; j < 8 * n; ++j) asm("max.NaN.f32 %0, %0, %1;" : "+f"(m) : "f"(__uint_as_float(r[j / 8].w[j % 8])));
    return m;
  }
}
// The same with NaN and infinite ones as they count. (They are rare: only then the groups are cleaned.)
template <typename T>
__device__ __forceinline__ float settle(Raw<T>* r, int n) {
  float m = largest_of(r, n);
  if (__builtin_expect(!(m < INFINITY), 0)) {
#pragma unroll
    for (int k = 0; k < n; ++k) clean(r[k]);
    m = largest_of(r, n);
  }
  return m;
}
// Elements 2 j and 2 j + 1.
template <typename T>
__device__ __forceinline__ float2 pair_of(const Raw<T>& r, int j) {
  if constexpr (sizeof(T) == 2)
    return make_float2(__uint_as_float(r.w[j] << 16), __uint_as_float(r.w[j] & 0xFFFF0000u));
  else
    return make_float2(__uint_as_float(r.w[2 * j]), __uint_as_float(r.w[2 * j + 1]));
}

// The eight logits from element e0 of a row on, which may begin before it or end behind it (-inf
// there). Called for a row's ends, and for a draft's row that starts elsewhere between 16-byte
// boundaries than the target's.
template <typename T>
__device__ __noinline__ Raw<T> load8(const T* row, int e0, int vocab) {
  Raw<T> r;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const bool in = e0 + j >= 0 && e0 + j < vocab;
    if constexpr (sizeof(T) == 2) {
      const uint32_t x = in ? (uint32_t)__ldg(reinterpret_cast<const unsigned short*>(row) + e0 + j) : 0xFF80u;
      r.w[j / 2] = j % 2 ? r.w[j / 2] | x << 16 : x;
    } else {
      r.w[j] = in ? __float_as_uint(__ldg(row + e0 + j)) : 0xFF800000u;
    }
  }
  return r;
}
// Group g of a row that starts at a 16-byte boundary.
template <typename T>
__device__ __forceinline__ Raw<T> whole8(const T* row, int g) {
  Raw<T> r;
#pragma unroll
  for (int h = 0; h < (int)sizeof(T) / 2; ++h)
    *reinterpret_cast<uint4*>(&r.w[4 * h]) = __ldg(reinterpret_cast<const uint4*>(row) + (ptrdiff_t)g * (int)(sizeof(T) / 2) + h);
  return r;
}
template <typename T>
__device__ __forceinline__ Raw<T> nothing() {  // eight times -inf
  Raw<T> r;
#pragma unroll
  for (int j = 0; j < (int)(2 * sizeof(T)); ++j) r.w[j] = sizeof(T) == 2 ? 0xFF80FF80u : 0xFF800000u;
  return r;
}
// Eight numbers of a row of noise, 1 outside it; those at a 16-byte boundary as such.
struct Noise {
  alignas(16) float v[8];
};
__device__ __noinline__ Noise load_noise8(const float* row, int e0, int vocab) {
  Noise n;
#pragma unroll
  for (int j = 0; j < 8; ++j) n.v[j] = e0 + j >= 0 && e0 + j < vocab ? __ldg(row + e0 + j) : 1.f;
  return n;
}
__device__ __forceinline__ Noise whole_noise8(const float* at) {
  Noise n;
#pragma unroll
  for (int h = 0; h < 2; ++h) *reinterpret_cast<float4*>(&n.v[4 * h]) = __ldg(reinterpret_cast<const float4*>(at) + h);
  return n;
}
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Logits are taken in octaves, x c with c = log2(e) / T, relative to a reference k that is the largest
// x c of those before it, rounded: x c - k is then one rounding of a small number, and references
// differ by exact numbers. (c is off by 2^-24 of itself, for all logits of a row alike.) Where x c
// may pass fp32's range, it is cut to +-2^126.
constexpr float kFarOctaves = 0x1p60f;
__device__ __forceinline__ float cut_octaves(float x, float c) { return fminf(fmaxf(x * c, -0x1p126f), 0x1p126f); }
// Of 2^(x c - k) over what a thread, a warp, a CTA has seen; k = -inf and s = 0 if nothing.
struct Pair {
  float k, s;
};
__device__ __forceinline__ float minus(float k) { return k == -INFINITY ? 0.f : -k; }  // -inf - (-inf) is never asked
// x c - k, given -k.
__device__ __forceinline__ float octaves(float x, float c, float nk) {
  if (x == -INFINITY) return -INFINITY;
  return fabsf(nk) < kFarOctaves ? fmaf(x, c, nk) : cut_octaves(x, c) + nk;
}
// The eight of a group as 2^(x c - k).
template <typename T>
__device__ __forceinline__ void weights8(const Raw<T>& r, float c, float nk, float* v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = pair_of(r, j);
    float2 z = ptx::fma2(x, make_float2(c, c), make_float2(nk, nk));
    if (__builtin_expect(!(fabsf(nk) < kFarOctaves), 0)) z = make_float2(octaves(x.x, c, nk), octaves(x.y, c, nk));
    v[2 * j] = ex2(z.x);
    v[2 * j + 1] = ex2(z.y);
  }
}

// A warp's largest value; the sum of a power of two of lanes. In one order, the same in every lane.
__device__ __forceinline__ float warp_max(float x) {
  const int i = __float_as_int(x);  // as an integer that is ordered as the numbers are
  const int k = __reduce_max_sync(0xffffffffu, i ^ ((i >> 31) & 0x7FFFFFFF));
  return __int_as_float(k ^ ((k >> 31) & 0x7FFFFFFF));
}
template <int kLanes>
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = kLanes / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <int kLanes>
__device__ __forceinline__ Pair warp_join(Pair p) {
  const float k = warp_max(p.k);
  return {k, warp_sum<kLanes>(p.s * ex2(p.k + minus(k)))};
}

struct Best {  // the largest value, of equal ones the lowest index
  float v;
  int i;
};
__device__ __forceinline__ Best warp_best(Best b) {
  const float m = warp_max(b.v);
  const unsigned i = __reduce_min_sync(0xffffffffu, b.v == m ? (unsigned)b.i : (unsigned)INT_MAX);
  return {m, (int)i};
}

struct VerifyShared {
  uint64_t bar[2];
  alignas(16) float4 slot[2][kVerMaxCluster];  // by the exchange's parity, the sending CTA
  Pair warp_pair[kVerWarps][2];
  Best warp_best[kVerWarps];
  float warp_sum[kVerWarps];
  int kids[32];  // up to 32 of the node's children
  int go;        // the accepted child, -1: none is left, -2: rejected, the residual's sum is wanted, -3: go on
  int kid_at;    // the next one of `kids`
  int n_tried;
  float taken;   // S
};

// CTAs to a cluster are few, so each sends what it has to all: one 16-byte store into every CTA's
// slot, counted on that CTA's barrier. Two sets of slots and barriers in turns are enough: nobody can
// send for the exchange after next before this one has been read everywhere. The waits are bounded:
// CTAs that see different inputs (written while the call runs) end with MLA_DEVICE_WAIT_TIMEOUT.
struct Exchange {
  VerifyShared* sh;
  int ctas, rank, count;
  int32_t* status;
  bool failed;
  // Called by all threads; lanes 0 .. ctas - 1 of warp 0 hold the CTA's value. Returns the slots.
  __device__ __forceinline__ const float4* operator()(float4 v, int warp, int lane) {
    const int k = count & 1;
    const uint32_t parity = (count >> 1) & 1;
    ++count;
    if (warp == 0 && lane < ctas)
      ptx::st_async_v4f(ptx::mapa(ptx::smem_addr(&sh->slot[k][rank]), lane), v.x, v.y, v.z, v.w,
                        ptx::mapa(ptx::smem_addr(&sh->bar[k]), lane));
    bool ok = ptx::mbar_try_wait_cluster(&sh->bar[k], parity);
    if (!ok) {
      const long long t0 = clock64();
      while (!(ok = ptx::mbar_try_wait_cluster(&sh->bar[k], parity)) && clock64() - t0 < kWaitBudget) {
      }
    }
    if (__syncthreads_or(!ok)) {
      if (!failed && threadIdx.x == 0) report(status, MLA_DEVICE_WAIT_TIMEOUT);
      failed = true;
    } else if (threadIdx.x == 0) {
      // armed for the exchange after next, whose first message follows this CTA's next one
      ptx::mbar_arrive_expect_tx(&sh->bar[k], 16u * (uint32_t)ctas);
    }
    return sh->slot[k];
  }
};

template <typename T, bool kDraft>
__global__ void __launch_bounds__(kVerThreads, 1024 / kVerThreads) tree_verify_kernel(VerifyArgs a) {
  __shared__ VerifyShared sh;
  extern __shared__ int32_t nodes[];  // of the request: parents, tokens, uniforms, tokens tried at a node
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  int first;
  bool bad;
  const int q = request_nodes(a.cu, b, a.total, a.max_nodes, &first, &bad);
  int32_t* path = a.path + (size_t)b * a.path_stride;
  int32_t* out = a.out_tokens + (size_t)b * a.path_stride;
  if (q == 0) {  // (the whole cluster leaves)
    if (rank == 0) {
      if (tid == 0) {
        if (bad) report(a.status, MLA_DEVICE_PLAN_MISMATCH);
        a.accepted[b] = 0;
      }
      for (int i = tid; i < a.path_stride; i += kVerThreads) path[i] = out[i] = -1;
    }
    return;
  }
  if (tid == 0) {
    for (int k = 0; k < 2; ++k) {
      ptx::mbar_init(&sh.bar[k], 1);
      ptx::mbar_arrive_expect_tx(&sh.bar[k], 16u * (uint32_t)C);
    }
    ptx::fence_mbar_init();
  }
  __syncwarp();
  ptx::cluster_arrive();  // (others write here only once the barriers are there)
  const float temp = a.temperature ? a.temperature[b] : 1.f;
  const bool greedy = !a.uniforms || !(temp >= 0x1p-20f);
  int32_t *up = nodes, *tokens = nodes + a.max_nodes, *tried_tokens = nodes + 3 * a.max_nodes;
  float* uniforms = reinterpret_cast<float*>(nodes + 2 * a.max_nodes);
  for (int i = tid; i < q; i += kVerThreads) {
    int p = i == 0 ? -1 : a.parents[first + i];
    if (p >= i) {
      if (rank == 0) report(a.status, MLA_DEVICE_BAD_TREE);
      p = -1;
    }
    up[i] = p;
    tokens[i] = a.tokens[first + i];
    if (!greedy) uniforms[i] = a.uniforms[first + i];
  }
  const float c = greedy ? 0.f : 1.44269504f / fminf(temp, 0x1p20f);
  const T* target0 = static_cast<const T*>(a.target);
  const T* draft0 = static_cast<const T*>(a.draft);
  const float* noise = greedy ? nullptr : a.noise + (size_t)b * a.n_stride;
  Exchange exchange{&sh, C, rank, 0, a.status, false};
  __syncwarp();
  ptx::cluster_wait();
  __syncthreads();

  int u = 0, len = 0;
  while (true) {
    const T* trow = target0 + (size_t)(first + u) * a.t_stride;
    const T* drow = kDraft ? draft0 + (size_t)(first + u) * a.d_stride : nullptr;
    // groups of eight elements that start at a 16-byte boundary of the target's row
    const int head = (int)(((uintptr_t)trow & 15u) / sizeof(T));
    const int groups = (a.vocab + head + 7) / 8;
    const int per = (groups + C - 1) / C, g0 = rank * per, g1 = min(groups, g0 + per);
    // whole groups of this CTA; a draft's row that starts elsewhere between 16-byte boundaries has none
    const bool alike = !kDraft || ((uintptr_t)(drow - head) & 15u) == 0;
    const int f0 = max(g0, head > 0 ? 1 : 0), f1 = alike ? max(f0, min(g1, (a.vocab + head) / 8)) : f0;
    const T *tbase = trow - head, *dbase = kDraft ? drow - head : nullptr;
    auto target8 = [&](int g) { return __builtin_expect(g >= f0 && g < f1, 1) ? whole8(tbase, g) : load8(trow, 8 * g - head, a.vocab); };
    auto draft8 = [&](int g) { return __builtin_expect(g >= f0 && g < f1, 1) ? whole8(dbase, g) : load8(drow, 8 * g - head, a.vocab); };
    const bool full = len + 1 >= a.path_stride;  // no room for another node: the walk ends here

    // the best over the cluster; i = INT_MAX where nobody has one
    auto best_of_all = [&](Best mine) {
      mine = warp_best(mine);
      if (lane == 0) sh.warp_best[warp] = mine;
      __syncthreads();
      if (warp == 0) mine = warp_best(sh.warp_best[lane % kVerWarps]);
      const float4 s = exchange(make_float4(mine.v, __int_as_float(mine.i), 0.f, 0.f), warp, lane)[lane % C];
      return warp_best(Best{s.x, __float_as_int(s.y)});
    };

    // the node's children from index `from` on, up to 32 of them, into sh.kids (warp 0); where to go on
    auto find_kids = [&](int from, int* n) {
      *n = 0;
      int i0 = from;
      for (; i0 < q && *n < 32; i0 += 32) {
        const int i = i0 + lane;
        const unsigned m = __ballot_sync(0xffffffffu, i < q && up[i] == u);
        const int at = *n + __popc(m & ((1u << lane) - 1u));
        if ((m >> lane & 1u) && at < 32) sh.kids[at] = i;
        *n += __popc(m);
      }
      *n = min(*n, 32);
      __syncwarp();
      return *n == 32 ? sh.kids[31] + 1 : q;
    };

    if (greedy) {
      Best mine{-INFINITY, INT_MAX};
      for (int g = g0 + tid; g < g1; g += 4 * kVerThreads) {
        Raw<T> r[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = g + k * kVerThreads < g1 ? target8(g + k * kVerThreads) : nothing<T>();
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float m = settle(&r[k], 1);
          if (m > mine.v) {
#pragma unroll
            for (int j = 3; j >= 0; --j) {
              const float2 v = pair_of(r[k], j);
              if (v.y == m) mine.i = 8 * (g + k * kVerThreads) - head + 2 * j + 1;
              if (v.x == m) mine.i = 8 * (g + k * kVerThreads) - head + 2 * j;
            }
            mine.v = m;
          }
        }
      }
      const Best all = best_of_all(mine);
      const int word = all.i == INT_MAX ? -1 : all.i;
      if (warp == 0) {
        int go = -1;
        for (int i0 = u + 1; !full && !exchange.failed && go < 0 && i0 < q; i0 += 32) {
          const int i = i0 + lane;
          const unsigned m = __ballot_sync(0xffffffffu, i < q && up[i] == u && word >= 0 && tokens[i] == word);
          if (m) go = i0 + __ffs(m) - 1;
        }
        if (lane == 0) {
          sh.go = go;
          if (rank == 0) {
            path[len] = u;
            out[len] = word;
          }
        }
      }
      __syncthreads();
      ++len;
      if (sh.go < 0) break;
      u = sh.go;
      __syncthreads();
      continue;
    }

    // ---- the first groups, and while they are on their way the children and their logits
    constexpr int kDeep = (kDraft ? 2 : 4) * 2 / (int)sizeof(T);
    Raw<T> r[kDeep], w[kDraft ? kDeep : 1];
    auto fetch = [&](int g) {
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int at = g + k * kVerThreads;
        r[k] = at < g1 ? target8(at) : nothing<T>();
        if (kDraft) w[kDraft ? k : 0] = at < g1 ? draft8(at) : nothing<T>();
      }
    };
    fetch(g0 + tid);
    int n_kids = 0, kids_end = q, kid_i = -1, kid_x = -1;
    T kid_t{}, kid_d{};
    float coin = 1.f;
    auto read_kids = [&]() {
      kid_i = lane < n_kids ? sh.kids[lane] : -1;
      kid_x = kid_i >= 0 ? tokens[kid_i] : -1;
      coin = kid_i >= 0 ? uniforms[kid_i] : 1.f;
      if (kid_x >= a.vocab) kid_x = -1;
      if (kid_x >= 0) {
        kid_t = __ldg(trow + kid_x);
        if (kDraft) kid_d = __ldg(drow + kid_x);
      }
    };
    if (warp == 0) {
      if (!full) kids_end = find_kids(u + 1, &n_kids);
      read_kids();
    }

    // ---- maximum and sum of the row(s)
    Pair pt{-INFINITY, 0.f}, pd{-INFINITY, 0.f};
    auto add = [&](Pair& p, Raw<T>* r, int n) {
      const float m = settle(r, n), k = m == -INFINITY ? m : cut_octaves(m, c);
      if (k > p.k) {
        p.s *= ex2(p.k - k);
        p.k = k;
      }
      const float nk = minus(p.k);
      float2 s = make_float2(0.f, 0.f);
      if (__builtin_expect(fabsf(nk) < kFarOctaves, 1)) {
#pragma unroll
        for (int i = 0; i < n; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 z = ptx::fma2(pair_of(r[i], j), make_float2(c, c), make_float2(nk, nk));
            s = ptx::add2(s, make_float2(ex2(z.x), ex2(z.y)));
          }
      } else {
#pragma unroll
        for (int i = 0; i < n; ++i) {
          float v[8];
          weights8(r[i], c, nk, v);
#pragma unroll
          for (int j = 0; j < 8; ++j) s.x += v[j];
        }
      }
      p.s += s.x + s.y;
    };
    for (int g = g0 + tid; g < g1; g += kDeep * kVerThreads) {  // the next groups are on their way while these are added
      Raw<T> r1[kDeep], w1[kDraft ? kDeep : 1];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        r1[k] = r[k];
        if (kDraft) w1[kDraft ? k : 0] = w[kDraft ? k : 0];
      }
      if (g + kDeep * kVerThreads < g1) fetch(g + kDeep * kVerThreads);
      add(pt, r1, kDeep);
      if (kDraft) add(pd, w1, kDeep);
    }
    pt = warp_join<32>(pt);
    if (kDraft) pd = warp_join<32>(pd);
    if (lane == 0) {
      sh.warp_pair[warp][0] = pt;
      sh.warp_pair[warp][1] = pd;
    }
    __syncthreads();
    if (warp == 0) {
      pt = warp_join<kVerWarps>(sh.warp_pair[lane % kVerWarps][0]);
      if (kDraft) pd = warp_join<kVerWarps>(sh.warp_pair[lane % kVerWarps][1]);
    }
    const float4 slot = exchange(make_float4(pt.k, pt.s, pd.k, pd.s), warp, lane)[lane % C];
    // (lanes beyond the cluster's size hold nothing)
    const Pair P = warp_join<16>(lane < C ? Pair{slot.x, slot.y} : Pair{-INFINITY, 0.f});
    const Pair Q = kDraft ? warp_join<16>(lane < C ? Pair{slot.z, slot.w} : Pair{-INFINITY, 0.f}) : Pair{0.f, 1.f};
    const float p_s = __shfl_sync(0xffffffffu, P.s, 0), q_s = __shfl_sync(0xffffffffu, Q.s, 0);
    const float np = minus(P.k), nq = minus(Q.k);
    const float inv_p = p_s > 0.f ? reciprocal(p_s) : 0.f, inv_q = q_s > 0.f ? reciprocal(q_s) : 0.f;

    // ---- the children, in order
    float left = 1.f;      // R
    float taken = 0.f;     // S
    int tried = 0, go;
    if (tid == 0) {
      sh.kid_at = 0;
      sh.n_tried = 0;
    }
    while (true) {
      if (warp == 0) {
        __syncwarp();
        // c R < p: px = p, compared with c R; c R q < p - S q: px = p / q, compared with c R + S, so that
        // numbers below fp32's range count too
        float px = -1.f;
        const float xt = kid_x >= 0 ? clean(kid_t) : -INFINITY, xd = kDraft && kid_x >= 0 ? clean(kid_d) : -INFINITY;
        if (xt > -INFINITY) {
          // (a row of the largest numbers: no more than all of it)
          const float zt = fminf(octaves(xt, c, np), 0.f);
          if (kDraft)
            px = xd > -INFINITY ? ex2(zt - fminf(octaves(xd, c, nq), 0.f)) * inv_p * q_s : INFINITY;
          else
            px = fmaxf(ex2(zt) * inv_p, 1e-45f);
        }
        int decision = -1, k = sh.kid_at;
        for (; k < n_kids && decision == -1; ++k) {
          const int x = __shfl_sync(0xffffffffu, kid_x, k);
          const float pk = __shfl_sync(0xffffffffu, px, k), ck = __shfl_sync(0xffffffffu, coin, k);
          if (x < 0) continue;
          if (!kDraft) {  // a token that a sibling had before has nothing left
            bool again = false;
            for (int t = lane; t < tried; t += 32) again |= tried_tokens[t] == x;
            if (__any_sync(0xffffffffu, again)) continue;
          }
          if (ck * left + taken < pk) {
            decision = __shfl_sync(0xffffffffu, kid_i, k);
          } else if (kDraft) {
            decision = -2;
          } else {
            if (lane == 0) tried_tokens[tried] = x;
            ++tried;
            left -= fmaxf(pk, 0.f);
            __syncwarp();
          }
        }
        if (decision < 0 && k == n_kids && kids_end < q) {  // more than 32 children
          kids_end = find_kids(kids_end, &n_kids);
          read_kids();
          k = 0;
          if (decision == -1 && n_kids > 0) decision = -3;
        }
        if (kDraft && decision == -2 && k == n_kids) {
          taken += left;
          decision = -1;  // no other child asks for the residual's sum
        }
        if (lane == 0) {
          sh.go = exchange.failed && decision < -1 ? -1 : decision;
          sh.kid_at = k;
          sh.n_tried = tried;
          sh.taken = taken;
        }
      }
      __syncthreads();
      go = sh.go;
      if (go == -3) {
        __syncthreads();
        continue;
      }
      if (!kDraft || go != -2) break;
      // a rejected child of a drawn draft, and another one to be tried: R of the residual
      taken += left;
      float s = 0.f;
      for (int g = g0 + tid; g < g1; g += kVerThreads) {
        Raw<T> r = target8(g), w = draft8(g);
        float v[8], d[8], t = 0.f;
        settle(&r, 1);
        settle(&w, 1);
        weights8(r, c, np, v);
        weights8(w, c, nq, d);
#pragma unroll
        for (int j = 0; j < 8; ++j) t += fmaxf(fmaf(-taken, d[j] * inv_q, v[j] * inv_p), 0.f);
        s += t;
      }
      s = warp_sum<32>(s);
      if (lane == 0) sh.warp_sum[warp] = s;
      __syncthreads();
      if (warp == 0) s = warp_sum<kVerWarps>(sh.warp_sum[lane % kVerWarps]);
      const float part = exchange(make_float4(s, 0.f, 0.f, 0.f), warp, lane)[lane % C].x;
      left = __shfl_sync(0xffffffffu, warp_sum<16>(lane < C ? part : 0.f), 0);
    }
    if (rank == 0 && tid == 0) path[len] = u;
    if (go >= 0 && !exchange.failed) {
      if (rank == 0 && tid == 0) out[len] = tokens[go];
      ++len;
      u = go;
      __syncthreads();
      continue;
    }
    // ---- none is accepted: the next token, from the residual; from p where that has nothing left
    tried = kDraft ? 0 : sh.n_tried;
    taken = kDraft ? sh.taken : 0.f;
    int word = -1;
    for (int turn = 0; turn < 2; ++turn) {
      Best mine{0.f, INT_MAX};
      const bool less = kDraft && turn == 0 && taken > 0.f;
      // all loads of the next group are on their way while this one is scored
      const bool noise_alike = ((uintptr_t)(noise - head) & 15u) == 0;
      Raw<T> r, w = nothing<T>();
      Noise e;
      auto fetch = [&](int g) {
        r = target8(g);
        if (less) w = draft8(g);
        e = __builtin_expect(noise_alike && g >= f0 && g < f1, 1) ? whole_noise8(noise - head + 8 * (ptrdiff_t)g)
                                                                  : load_noise8(noise, 8 * g - head, a.vocab);
      };
      if (g0 + tid < g1) fetch(g0 + tid);
      for (int g = g0 + tid; g < g1; g += kVerThreads) {  // (rising: of equal ones a thread keeps the lowest)
        Raw<T> r1 = r, w1 = w;
        const Noise e1 = e;
        if (g + kVerThreads < g1) fetch(g + kVerThreads);
        const int e0 = 8 * g - head;
        float v[8];
        settle(&r1, 1);
        weights8(r1, c, np, v);
        if (less) {
          float d[8];
          settle(&w1, 1);
          weights8(w1, c, nq, d);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = fmaf(-taken, d[j] * inv_q, v[j] * inv_p);
        }
        if (!kDraft && turn == 0) {
          for (int t = 0; t < tried; ++t) {
            const int at = tried_tokens[t] - e0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (at == j) v[j] = 0.f;
          }
        }
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {  // noise of 0, negative numbers and NaN: the least normal number
          v[j] *= reciprocal(fmaxf(e1.v[j], kLeast));
          top = fmaxf(top, v[j]);
        }
        if (top > mine.v) {
          mine.v = top;
#pragma unroll
          for (int j = 7; j >= 0; --j)
            if (v[j] == top) mine.i = e0 + j;
        }
      }
      const Best all = best_of_all(mine);
      if (all.i != INT_MAX) {
        word = all.i;
        break;
      }
    }
    if (rank == 0 && tid == 0) out[len] = word;
    ++len;
    break;
  }
  if (rank == 0) {
    if (tid == 0) a.accepted[b] = len;
    for (int i = len + tid; i < a.path_stride; i += kVerThreads) path[i] = out[i] = -1;
  }
  // no CTA leaves while another's message to it is under way
  __syncwarp();
  ptx::cluster_arrive();
  ptx::cluster_wait();
}

template <typename T>
const void* verify_kernel_of(bool draft) {
  return draft ? (const void*)tree_verify_kernel<T, true> : (const void*)tree_verify_kernel<T, false>;
}

// Whether [a, a + na) and [b, b + nb) bytes meet.
bool meet(const void* a, size_t na, const void* b, size_t nb) {
  return a && b && (uintptr_t)a < (uintptr_t)b + nb && (uintptr_t)b < (uintptr_t)a + na;
}

}  // namespace

cudaError_t set_verify_kernel_attributes() {
  for (const void* fn : {verify_kernel_of<__nv_bfloat16>(false), verify_kernel_of<__nv_bfloat16>(true),
                         verify_kernel_of<float>(false), verify_kernel_of<float>(true)}) {
    const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace mla

using namespace mla;

extern "C" int mla_tree_masks(const int32_t* parents, const int32_t* cu_nodes, int batch, int total_nodes, int max_nodes,
                              uint32_t* masks, int mask_words, int32_t* depths, int32_t* status_dev, void* stream) {
  clear_error();
  if (batch < 1) return set_error(MLA_ERR_INVALID_ARG, "batch must be >= 1 (got %d)", batch);
  if (total_nodes < 0) return set_error(MLA_ERR_INVALID_ARG, "total_nodes must be >= 0 (got %d)", total_nodes);
  if (max_nodes < 0 || max_nodes > MLA_TREE_MAX_NODES)
    return set_error(MLA_ERR_INVALID_ARG, "max_nodes must be in [0, %d] (got %d)", MLA_TREE_MAX_NODES, max_nodes);
  if (max_nodes == 0 || total_nodes == 0) return MLA_OK;
  if (!parents || !cu_nodes || !masks) return set_error(MLA_ERR_INVALID_ARG, "parents, cu_nodes and masks must not be NULL");
  for (const void* p : {(const void*)parents, (const void*)cu_nodes, (const void*)masks, (const void*)depths, (const void*)status_dev})
    if ((uintptr_t)p & 3u)
      return set_error(MLA_ERR_INVALID_ARG, "parents, cu_nodes, masks, depths and status_dev must be 4-byte aligned");
  if (mask_words < (max_nodes + 31) / 32)
    return set_error(MLA_ERR_INVALID_ARG, "mask_words %d is too few for %d nodes", mask_words, max_nodes);
  const size_t nodes = 4 * (size_t)total_nodes, cu = 4 * ((size_t)batch + 1), words = nodes * (size_t)mask_words;
  if (meet(masks, words, parents, nodes) || meet(masks, words, cu_nodes, cu) || meet(depths, nodes, parents, nodes) ||
      meet(depths, nodes, cu_nodes, cu) || meet(masks, words, depths, nodes))
    return set_error(MLA_ERR_INVALID_ARG, "masks and depths must not overlap the other arrays");
  DeviceKernels device;
  const int rc = current_device_ready(&device);
  if (rc != MLA_OK) return rc;
  MaskArgs a{parents, cu_nodes, total_nodes, max_nodes, mask_words, masks, depths, status_dev};
  const dim3 grid((unsigned)batch, (unsigned)((max_nodes + kMaskThreads - 1) / kMaskThreads));
  tree_masks_kernel<<<grid, kMaskThreads, sizeof(int32_t) * (size_t)max_nodes, (cudaStream_t)stream>>>(a);
  const cudaError_t ce = cudaGetLastError();
  if (ce != cudaSuccess) return set_error(MLA_ERR_CUDA, "tree masks kernel launch: %s", cudaGetErrorString(ce));
  return MLA_OK;
}

extern "C" int mla_tree_verify(int logits_dtype, const void* target_logits, long long target_stride,
                               const void* draft_logits, long long draft_stride, int vocab, const int32_t* tokens,
                               const int32_t* parents, const int32_t* cu_nodes, int batch, int total_nodes, int max_nodes,
                               const float* temperature, const float* uniforms, const float* noise, long long noise_stride,
                               int32_t* path, int32_t* out_tokens, int path_stride, int32_t* accepted,
                               int32_t* status_dev, void* stream) {
  clear_error();
  if (logits_dtype != MLA_LOGITS_BF16 && logits_dtype != MLA_LOGITS_FP32)
    return set_error(MLA_ERR_INVALID_ARG, "logits_dtype must be MLA_LOGITS_BF16 or MLA_LOGITS_FP32 (got %d)", logits_dtype);
  if (batch < 1 || batch > 1 << 20) return set_error(MLA_ERR_INVALID_ARG, "batch must be in [1, 2^20] (got %d)", batch);
  if (total_nodes < 0) return set_error(MLA_ERR_INVALID_ARG, "total_nodes must be >= 0 (got %d)", total_nodes);
  if (max_nodes < 0 || max_nodes > MLA_TREE_MAX_NODES)
    return set_error(MLA_ERR_INVALID_ARG, "max_nodes must be in [0, %d] (got %d)", MLA_TREE_MAX_NODES, max_nodes);
  if (vocab < 1 || vocab > 1 << 30) return set_error(MLA_ERR_INVALID_ARG, "vocab must be in [1, 2^30] (got %d)", vocab);
  if (path_stride < 1) return set_error(MLA_ERR_INVALID_ARG, "path_stride must be >= 1 (got %d)", path_stride);
  if (!cu_nodes || !path || !out_tokens || !accepted)
    return set_error(MLA_ERR_INVALID_ARG, "cu_nodes, path, out_tokens and accepted must not be NULL");
  if (total_nodes > 0 && (!target_logits || !tokens || !parents))
    return set_error(MLA_ERR_INVALID_ARG, "target_logits, tokens and parents must not be NULL");
  if (total_nodes > 0 && !uniforms != !noise)
    return set_error(MLA_ERR_INVALID_ARG, "uniforms and noise must both be given, or (all requests greedy) neither");
  if (target_stride < vocab) return set_error(MLA_ERR_INVALID_ARG, "target_stride %lld is smaller than vocab %d", target_stride, vocab);
  if (draft_logits && draft_stride < vocab)
    return set_error(MLA_ERR_INVALID_ARG, "draft_stride %lld is smaller than vocab %d", draft_stride, vocab);
  if (noise && noise_stride < vocab)
    return set_error(MLA_ERR_INVALID_ARG, "noise_stride %lld is smaller than vocab %d", noise_stride, vocab);
  const size_t esz = logits_dtype == MLA_LOGITS_BF16 ? 2 : 4;
  if (((uintptr_t)target_logits | (uintptr_t)draft_logits) & (esz - 1))
    return set_error(MLA_ERR_INVALID_ARG, "logits must be aligned to their elements");
  const size_t nodes = 4 * (size_t)total_nodes, cu = 4 * ((size_t)batch + 1), rows = 4 * (size_t)batch;
  const size_t paths = rows * (size_t)path_stride;
  const struct { const void* p; size_t n; } in[] = {{tokens, nodes}, {parents, nodes}, {cu_nodes, cu}, {temperature, rows},
                                                    {uniforms, nodes},
                                                    {noise, noise ? 4 * ((size_t)noise_stride * (batch - 1) + vocab) : 0}},
               outs[] = {{path, paths}, {out_tokens, paths}, {accepted, rows}};
  for (const auto& i : in)
    if ((uintptr_t)i.p & 3u)
      return set_error(MLA_ERR_INVALID_ARG, "tokens, parents, cu_nodes, temperature, uniforms and noise must be 4-byte aligned");
  for (const auto& o : outs) {
    if ((uintptr_t)o.p & 3u) return set_error(MLA_ERR_INVALID_ARG, "path, out_tokens and accepted must be 4-byte aligned");
    for (const auto& i : in)
      if (meet(o.p, o.n, i.p, i.n)) return set_error(MLA_ERR_INVALID_ARG, "path, out_tokens and accepted must not overlap the inputs");
    for (const auto& i : outs)
      if (&i != &o && meet(o.p, o.n, i.p, i.n)) return set_error(MLA_ERR_INVALID_ARG, "path, out_tokens and accepted must not overlap");
    if (total_nodes > 0 && (meet(o.p, o.n, target_logits, esz * ((size_t)target_stride * (total_nodes - 1) + vocab)) ||
                            meet(o.p, o.n, draft_logits, esz * ((size_t)draft_stride * (total_nodes - 1) + vocab))))
      return set_error(MLA_ERR_INVALID_ARG, "path, out_tokens and accepted must not overlap the logits");
  }
  if ((uintptr_t)status_dev & 3u) return set_error(MLA_ERR_INVALID_ARG, "status_dev must be 4-byte aligned");
  DeviceKernels device;
  const int rc = current_device_ready(&device);
  if (rc != MLA_OK) return rc;
  if (device.verify != cudaSuccess)
    return set_error(MLA_ERR_CUDA, "tree verification kernel attributes: %s", cudaGetErrorString(device.verify));
  VerifyArgs a{target_logits, draft_logits, target_stride, draft_stride, noise_stride, vocab, total_nodes, max_nodes,
               path_stride, tokens, parents, cu_nodes, temperature, uniforms, noise, path, out_tokens, accepted, status_dev};
  const bool draft = draft_logits != nullptr;
  // CTAs to a request, a power of two up to 16: as many as four to an SM, with three groups of eight to
  // two threads at least; more where each then still has six to a thread. (us with 2, 4, 8, 16 CTAs, the
  // rule's choice in brackets; bf16. Drafts, 131072 tokens: 64 requests 104, 66, [50], 60; 256 requests 155,
  // 143, [142], 190; 32000 tokens, 256 requests [54], 58, 75, 141. Without drafts, 131072 tokens: 32 requests
  // 51, 33, 26, [25]; 64 requests 53, 37, [29], 39; 32000 tokens, 32 requests 21, 17, [17], 18.)
  int c = 1;
  while (c < kVerMaxCluster) {
    const long long each = vocab / (8LL * 2 * c);  // groups
    if (2 * each < 3 * kVerThreads || ((long long)batch * c * 2 > 4LL * device.sms && each < 6 * kVerThreads)) break;
    c *= 2;
  }
  const void* fn = esz == 2 ? verify_kernel_of<__nv_bfloat16>(draft) : verify_kernel_of<float>(draft);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)(batch * c), 1, 1);
  cfg.blockDim = dim3(kVerThreads, 1, 1);
  cfg.dynamicSmemBytes = 4 * sizeof(int32_t) * (size_t)std::max(1, max_nodes);
  cfg.stream = (cudaStream_t)stream;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)c, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void* args[] = {&a};
  const cudaError_t ce = cudaLaunchKernelExC(&cfg, fn, args);
  if (ce != cudaSuccess) return set_error(MLA_ERR_CUDA, "tree verification kernel launch: %s", cudaGetErrorString(ce));
  return MLA_OK;
}
