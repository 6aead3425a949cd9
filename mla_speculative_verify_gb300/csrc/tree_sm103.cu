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
// the last one down. Parents come from shared memory: a step of the climb is one load there.
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
//   CTAs pass on their pairs through shared memory of the cluster, and every CTA joins the pairs in
//   the same order, so all take the same decisions without asking one another.
//   The children are tried in order. Without draft logits the draft is taken as certain: child token
//   x is accepted if c * R < r(x), where r is p without the tokens tried before and R its sum. With
//   draft logits (q the softmax of row u) it is accepted if c * R * q(x) < r(x), where after a
//   rejection r = max(p - S q, 0), S the sum of the R so far: max(max(p - a q, 0) - b q, 0) is
//   max(p - (a + b) q, 0), so a rejected child costs one sum over the vocabulary and no stored r.
// At the node where none is accepted the next token is argmax r(x) / E(x), E the caller's
// exponentially distributed numbers: a draw from r whose result hardly depends on rounding, unlike a
// search in r's running sum, where a border is nearer than fp32's sums are exact.
constexpr int kVerThreads = 512;
constexpr int kVerWarps = kVerThreads / 32;
constexpr int kVerMaxCluster = 16;
constexpr int kMaxTried = 1024;  // nodes of a request: children tried at one node

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

struct Pair {  // sum of exp(x - m), or the best (value, index)
  float m, s;
};

// NaN logits count as -inf, infinite ones as the largest number.
__device__ __forceinline__ float clean(float x) { return x == x ? fminf(x, 3.402823466e38f) : -INFINITY; }

template <typename T>
__device__ __forceinline__ float logit(const T* row, int i) {
  if constexpr (sizeof(T) == 2)
    return clean(__bfloat162float(row[i]));
  else
    return clean(row[i]);
}

// Eight logits from element e0 of a row (which may lie before it or reach behind its end: -inf there).
// Whole groups at 16-byte boundaries are read as such.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int e0, int vocab, float* v) {
  if (e0 >= 0 && e0 + 8 <= vocab && ((uintptr_t)(row + e0) & 15u) == 0) {
    if constexpr (sizeof(T) == 2) {
      const uint4 w = __ldg(reinterpret_cast<const uint4*>(row + e0));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[2 * j] = clean(__uint_as_float(u[j] << 16));
        v[2 * j + 1] = clean(__uint_as_float(u[j] & 0xFFFF0000u));
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(row + e0) + h);
        v[4 * h] = clean(w.x); v[4 * h + 1] = clean(w.y); v[4 * h + 2] = clean(w.z); v[4 * h + 3] = clean(w.w);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e0 + j >= 0 && e0 + j < vocab ? logit(row, e0 + j) : -INFINITY;
  }
}
__device__ __forceinline__ void load_noise8(const float* row, int e0, int vocab, float* v) {
  if (e0 >= 0 && e0 + 8 <= vocab && ((uintptr_t)(row + e0) & 15u) == 0) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 w = __ldg(reinterpret_cast<const float4*>(row + e0) + h);
      v[4 * h] = w.x; v[4 * h + 1] = w.y; v[4 * h + 2] = w.z; v[4 * h + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = e0 + j >= 0 && e0 + j < vocab ? __ldg(row + e0 + j) : 1.f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = fmaxf(v[j], 1.175494351e-38f);  // 0, negative or NaN: the least normal number
}

// exp((x - m) / T) as 2^((x - m) c) with c = log2(e) / T held in two parts; 0 where x or m is -inf.
struct Scale {
  float hi, lo;
  __device__ __forceinline__ float octaves(float d) const { return fmaf(d, hi, d * lo); }
  __device__ __forceinline__ float operator()(float x, float m) const {
    const float d = x - m;
    return d >= -3.402823466e38f ? ex2(octaves(d)) : 0.f;
  }
};

__device__ __forceinline__ Pair join(Pair a, Pair b, Scale c) {  // of two sums
  const float m = fmaxf(a.m, b.m);
  if (m == -INFINITY) return {m, 0.f};
  return {m, a.s * c(a.m, m) + b.s * c(b.m, m)};
}

struct Best {  // the largest value, of equal ones the lowest index
  float v;
  int i;
  __device__ __forceinline__ void take(float x, int at) {
    if (x > v || (x == v && at < i)) {
      v = x;
      i = at;
    }
  }
};

struct VerifyShared {
  Pair part[2][kVerMaxCluster][2];   // by the step's parity, CTA: target, draft
  Best best[2][kVerMaxCluster];
  float sums[2][kVerMaxCluster];
  Pair warp_pair[kVerWarps][2];
  Best warp_best[kVerWarps];
  float warp_sum[kVerWarps];
  int go;        // the accepted child, -1: none is left, -2: rejected, the residual's sum is wanted
  int next_kid;  // where the search for children goes on
  int n_tried;
  float taken;   // S
  int tried[kMaxTried];
};

template <typename T, bool kDraft>
__global__ void __launch_bounds__(kVerThreads, 2) tree_verify_kernel(VerifyArgs a) {
  __shared__ VerifyShared sh;
  extern __shared__ int32_t up[];  // parents of the request's nodes
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
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
  ptx::cluster_arrive();  // (a CTA's shared memory is written by others only once it runs)
  for (int i = tid; i < q; i += kVerThreads) {
    int p = i == 0 ? -1 : a.parents[first + i];
    if (p >= i) {
      if (rank == 0) report(a.status, MLA_DEVICE_BAD_TREE);
      p = -1;
    }
    up[i] = p;
  }
  const float temp = a.temperature ? a.temperature[b] : 1.f;
  const bool greedy = !a.uniforms || !(temp >= 0x1p-20f);
  Scale scale{0.f, 0.f};
  if (!greedy) {
    const float t = fminf(temp, 0x1p20f);
    const double c = 1.4426950408889634 / (double)t;
    scale.hi = (float)c;
    scale.lo = (float)(c - (double)scale.hi);
  }
  const T* target0 = static_cast<const T*>(a.target);
  const T* draft0 = static_cast<const T*>(a.draft);
  const float* noise = greedy ? nullptr : a.noise + (size_t)b * a.n_stride;
  int parity = 0;  // of the exchanges
  ptx::cluster_wait();

  int u = 0, len = 0;
  while (true) {
    const T* trow = target0 + (size_t)(first + u) * a.t_stride;
    const T* drow = kDraft ? draft0 + (size_t)(first + u) * a.d_stride : nullptr;
    // groups of eight elements that start at a 16-byte boundary of the target's row
    const int head = (int)(((uintptr_t)trow & 15u) / sizeof(T));
    const int groups = (a.vocab + head + 7) / 8;
    const int per = (groups + C - 1) / C, g0 = rank * per, g1 = min(groups, g0 + per);

    // the largest over the cluster of `mine`
    auto best_of_all = [&](Best mine) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mine.take(__shfl_xor_sync(0xffffffffu, mine.v, o), __shfl_xor_sync(0xffffffffu, mine.i, o));
      if (lane == 0) sh.warp_best[warp] = mine;
      __syncthreads();
      if (warp == 0) {
        mine = sh.warp_best[lane % kVerWarps];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mine.take(__shfl_xor_sync(0xffffffffu, mine.v, o), __shfl_xor_sync(0xffffffffu, mine.i, o));
        if (lane < C) cluster.map_shared_rank(&sh, lane)->best[parity][rank] = mine;
      }
      cluster.sync();
      Best all = sh.best[parity][0];
      for (int r = 1; r < C; ++r) all.take(sh.best[parity][r].v, sh.best[parity][r].i);
      parity ^= 1;
      return all;
    };

    const bool full = len + 1 >= a.path_stride;  // no room for another node: the walk ends here
    if (greedy) {
      Best mine{-INFINITY, INT_MAX};
      for (int g = g0 + tid; g < g1; g += kVerThreads) {
        float v[8];
        load8(trow, 8 * g - head, a.vocab, v);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (v[j] > mine.v) mine = {v[j], 8 * g - head + j};
      }
      const Best all = best_of_all(mine);
      const int word = all.i == INT_MAX ? -1 : all.i;
      if (warp == 0) {
        int go = -1;
        for (int i0 = u + 1; !full && go < 0 && i0 < q; i0 += 32) {
          const int i = i0 + lane;
          const bool hit = i < q && up[i] == u && word >= 0 && a.tokens[first + i] == word;
          const unsigned m = __ballot_sync(0xffffffffu, hit);
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

    // ---- maximum and sum of the row(s)
    Pair pt{-INFINITY, 0.f}, pd{-INFINITY, 0.f};
    auto add8 = [&](Pair& p, const float* v) {
      float m = p.m;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, v[j]);
      if (m == -INFINITY) return;
      if (m > p.m) {
        p.s *= scale(p.m, m);
        p.m = m;
      }
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s += scale(v[j], m);
      p.s += s;
    };
    for (int g = g0 + tid; g < g1; g += kVerThreads) {
      float v[8], w[8];
      load8(trow, 8 * g - head, a.vocab, v);
      if (kDraft) load8(drow, 8 * g - head, a.vocab, w);
      add8(pt, v);
      if (kDraft) add8(pd, w);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      pt = join(pt, {__shfl_xor_sync(0xffffffffu, pt.m, o), __shfl_xor_sync(0xffffffffu, pt.s, o)}, scale);
      if (kDraft) pd = join(pd, {__shfl_xor_sync(0xffffffffu, pd.m, o), __shfl_xor_sync(0xffffffffu, pd.s, o)}, scale);
    }
    if (lane == 0) {
      sh.warp_pair[warp][0] = pt;
      sh.warp_pair[warp][1] = pd;
    }
    __syncthreads();
    if (warp == 0 && lane < C) {
      Pair x = sh.warp_pair[0][0], y = sh.warp_pair[0][1];
      for (int i = 1; i < kVerWarps; ++i) {
        x = join(x, sh.warp_pair[i][0], scale);
        if (kDraft) y = join(y, sh.warp_pair[i][1], scale);
      }
      VerifyShared* to = cluster.map_shared_rank(&sh, lane);
      to->part[parity][rank][0] = x;
      to->part[parity][rank][1] = y;
    }
    cluster.sync();
    Pair P = sh.part[parity][0][0], Q = sh.part[parity][0][1];
    for (int r = 1; r < C; ++r) {
      P = join(P, sh.part[parity][r][0], scale);
      if (kDraft) Q = join(Q, sh.part[parity][r][1], scale);
    }
    parity ^= 1;
    const float inv_p = P.s > 0.f ? 1.f / P.s : 0.f, inv_q = kDraft && Q.s > 0.f ? 1.f / Q.s : 0.f;

    // ---- the children, in order
    if (tid == 0) {
      sh.next_kid = full ? q : u + 1;
      sh.n_tried = 0;
      sh.taken = 0.f;
    }
    float left = 1.f;  // R
    int go;
    while (true) {
      __syncthreads();
      if (warp == 0) {
        int decision = -1, tried = sh.n_tried;
        const float taken = sh.taken;
        float sum = left;  // (no draft: R goes down child by child)
        int i0 = sh.next_kid;
        for (; decision == -1 && i0 < q; i0 += 32) {
          const int i = i0 + lane;
          const bool kid = i < q && up[i] == u;
          // c R < p: bar = c, px = p; c R q < p - S q: bar = c, px = p / q, compared with c R + S, so that
          // numbers below fp32's range count too
          int x = -1;
          float px = -1.f, bar = 0.f;
          if (kid) {
            x = a.tokens[first + i];
            if (x >= 0 && x < a.vocab) {
              bar = a.uniforms[first + i];
              const float lt = logit(trow, x);
              if (lt > -INFINITY) {
                if (kDraft) {
                  const float lq = logit(drow, x);
                  px = lq > -INFINITY ? ex2(scale.octaves(lt - P.m) - scale.octaves(lq - Q.m)) * inv_p * Q.s : INFINITY;
                } else {
                  px = fmaxf(scale(lt, P.m) * inv_p, 1e-45f);
                }
              }
            }
          }
          unsigned kids = __ballot_sync(0xffffffffu, kid);
          while (kids && decision == -1) {
            const int k = __ffs(kids) - 1;
            kids &= kids - 1;
            const int xk = __shfl_sync(0xffffffffu, x, k);
            const float pk = __shfl_sync(0xffffffffu, px, k);
            const float bk = __shfl_sync(0xffffffffu, bar, k);
            if (xk < 0 || xk >= a.vocab) continue;
            if (!kDraft) {  // a token that a sibling had before has nothing left
              bool again = false;
              for (int t = lane; t < tried; t += 32) again |= sh.tried[t] == xk;
              if (__any_sync(0xffffffffu, again)) continue;
            }
            if (bk * sum + (kDraft ? taken : 0.f) < pk) {
              decision = i0 + k;
            } else if (kDraft) {
              decision = -2;
              i0 += k + 1 - 32;  // go on behind this child
            } else {
              if (lane == 0) sh.tried[tried] = xk;
              ++tried;
              sum -= fmaxf(pk, 0.f);
              __syncwarp();
            }
          }
        }
        if (lane == 0) {
          sh.go = decision;
          sh.next_kid = i0;
          sh.n_tried = tried;
          if (decision == -2) sh.taken = taken + left;
        }
      }
      __syncthreads();
      go = sh.go;
      if (!kDraft || go != -2) break;
      // a rejected child of a drawn draft: R of the residual, if another child may ask for it
      bool more = false;
      for (int i = sh.next_kid + tid; i < q; i += kVerThreads) more |= up[i] == u;
      if (!__syncthreads_or(more)) {
        go = -1;
        break;
      }
      const float taken = sh.taken;
      float s = 0.f;
      for (int g = g0 + tid; g < g1; g += kVerThreads) {
        float v[8], w[8], t = 0.f;
        load8(trow, 8 * g - head, a.vocab, v);
        load8(drow, 8 * g - head, a.vocab, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) t += fmaxf(fmaf(-taken, scale(w[j], Q.m) * inv_q, scale(v[j], P.m) * inv_p), 0.f);
        s += t;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) sh.warp_sum[warp] = s;
      __syncthreads();
      if (warp == 0 && lane < C) {
        float t = 0.f;
        for (int i = 0; i < kVerWarps; ++i) t += sh.warp_sum[i];
        cluster.map_shared_rank(&sh, lane)->sums[parity][rank] = t;
      }
      cluster.sync();
      left = 0.f;
      for (int r = 0; r < C; ++r) left += sh.sums[parity][r];
      parity ^= 1;
    }
    if (rank == 0 && tid == 0) path[len] = u;
    if (go >= 0) {
      if (rank == 0 && tid == 0) out[len] = a.tokens[first + go];
      ++len;
      u = go;
      __syncthreads();
      continue;
    }
    // ---- none is accepted: the next token, from the residual; from p where that has nothing left
    const int tried = kDraft ? 0 : sh.n_tried;
    const float taken = kDraft ? sh.taken : 0.f;
    int word = -1;
    for (int turn = 0; turn < 2; ++turn) {
      Best mine{0.f, INT_MAX};
      for (int g = g0 + tid; g < g1; g += kVerThreads) {
        const int e0 = 8 * g - head;
        float v[8], e[8];
        load8(trow, e0, a.vocab, v);
        load_noise8(noise, e0, a.vocab, e);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = scale(v[j], P.m);
        if (turn == 0) {
          if constexpr (kDraft) {
            if (taken > 0.f) {
              float w[8];
              load8(drow, e0, a.vocab, w);
#pragma unroll
              for (int j = 0; j < 8; ++j) v[j] = fmaxf(fmaf(-taken, scale(w[j], Q.m) * inv_q, v[j] * inv_p), 0.f);
            }
          } else {
            for (int t = 0; t < tried; ++t) {
              const int at = sh.tried[t] - e0;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                if (at == j) v[j] = 0.f;
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float r = v[j] / e[j];
          if (r > mine.v) mine = {r, e0 + j};
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
    if ((uintptr_t)p & 3u) return set_error(MLA_ERR_INVALID_ARG, "parents, cu_nodes, masks, depths and status_dev must be 4-byte aligned");
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
    if ((uintptr_t)i.p & 3u) return set_error(MLA_ERR_INVALID_ARG, "tokens, parents, cu_nodes, temperature, uniforms and noise must be 4-byte aligned");
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
  // CTAs to a request: up to 16, while the batch leaves SMs for them and each has some work
  int c = 1;
  while (c < kVerMaxCluster && (long long)batch * c * 2 <= 2 * device.sms && (long long)vocab > 2048LL * c) c *= 2;
  const bool draft = draft_logits != nullptr;
  const void* fn = esz == 2 ? verify_kernel_of<__nv_bfloat16>(draft) : verify_kernel_of<float>(draft);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3((unsigned)(batch * c), 1, 1);
  cfg.blockDim = dim3(kVerThreads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(int32_t) * (size_t)std::max(1, max_nodes);
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
