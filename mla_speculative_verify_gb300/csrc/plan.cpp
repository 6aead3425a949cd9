// plan.cpp -- host-only split-KV work partition for MLA verify decode.
//
// The planner works from host-known scalars only (seq_lens, q_lens, H, the SM
// count), as the host plan of flashinfer PR #5588 ("What was measured" table,
// host-plan row) does. Steps:
//   1. fold_sq (sglang PR #33650, "Why" paragraph): F = largest divisor of q with
//      H * F <= 128; the q tokens form q / F groups of F * H packed rows
//      (row = token * H + head, contiguous in Q and in the output).
//   2. A group's packed rows are cut into CTA row tiles of at most rows_cap rows
//      (the shared-memory budget of one CTA, see kernel_sm103.cu). The tiles of
//      one group are adjacent in the unit list, so they stream the same pages at
//      the same time and the second read is served by L2.
//   3. Each group's key range [0, ctx) is cut into page-aligned splits of about the
//      per-SM share of the work; split units write partial (O, LSE) rows that the
//      merge kernel combines.
#include <algorithm>
#include <cmath>
#include <exception>
#include <functional>
#include <queue>
#include <cstdio>
#include <cstring>
#include <string>
#include <vector>

#include "mla_decode.h"
#include "plan_format.h"
#include "status.h"

namespace mla {

int rows_cap_for(int kv_dtype);  // defined next to the kernel
int max_splits_for_merge();       // defined next to the merge kernel
int pair_rows_cap();              // defined next to the two-CTA kernel
int wide_rows_cap();              // defined next to the wide kernel

static int fold_factor(int q, int H) {
  int best = 1;
  for (int f = 1; f <= q; ++f)
    if (q % f == 0 && (long long)H * f <= 128) best = f;
  return best;
}

static size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// log2 of a block's tokens (1, 2, 4, .. 64, so that a block never leaves its page), or -1.
int block_log2_of(int block_tokens) {
  for (int l = 0; (1 << l) <= kPage; ++l)
    if (block_tokens == 1 << l) return l;
  return -1;
}

size_t workspace_bytes_for(int n_part_rows, bool tree) {
  if (n_part_rows <= 0) return 0;
  return align_up((size_t)n_part_rows * kDv * (tree ? kTreePartOElemBytes : kPartOElemBytes), 256) + align_up((size_t)n_part_rows * sizeof(float), 256);
}

namespace {

constexpr int kMaxKeys = 1 << 30;  // of a request

struct RowTile { int b, qrow0, nrows, pages; };
// tiles [t0, t1) of one fold group: consecutive, same request, qrow0 contiguous
struct Group { size_t t0, t1; int b, pages, n_split, cap; };  // cap: piece length in pages (0: equal pieces)

int piece_pages(const Group& g, int s) {
  if (g.cap > 0) return std::min(g.pages, (s + 1) * g.cap) - s * g.cap;
  return (int)((long long)g.pages * (s + 1) / g.n_split - (long long)g.pages * s / g.n_split);
}

// What a partition is made of: the kernel's tiles, and what the model of their time knows.
struct Geometry {
  bool wide, whole_requests;
  int cap;            // rows of a tile
  int slots;          // units that run at once
  int min_pages;      // of a piece
  double start_cost;  // of a unit, in page-times
  double page_us;     // a page-time (only compared between geometries)
};

struct Partition {
  std::vector<RowTile> tiles;
  std::vector<PlanRequest> reqs;
  std::vector<Group> groups;
  double end_us;  // when the model's last unit ends (known where the pieces are searched for, or if `compared`)
};

Partition cut_batch(const int32_t* seq_lens_h, const int32_t* q_lens_h, int batch, int num_heads, bool fp8,
                    const mla_plan_options& o, const Geometry& geo, bool compared) {
  Partition out;
  std::vector<RowTile>& tiles = out.tiles;
  std::vector<PlanRequest>& reqs = out.reqs;
  std::vector<Group>& groups = out.groups;
  reqs.resize(batch);
  const int cap = geo.cap, slots = geo.slots, min_pages = geo.min_pages;
  const double start_cost = geo.start_cost;
  // --- row tiles ----------------------------------------------------------------------
  int tok0 = 0;
  for (int b = 0; b < batch; ++b) {
    int ctx = seq_lens_h[b], q = q_lens_h[b];
    int F = geo.whole_requests ? q : o.force_fold > 0 ? o.force_fold : fold_factor(q, num_heads);
    reqs[b] = PlanRequest{ctx, q, tok0, F};
    int R = F * num_heads;                       // packed rows per fold group
    int n_rt = (R + cap - 1) / cap;
    int T = ((R + n_rt - 1) / n_rt + 15) / 16 * 16;
    if (T > cap) T = cap;
    int pages = (ctx + kPage - 1) / kPage;
    for (int g = 0; g < q / F; ++g) {
      int grow0 = (tok0 + g * F) * num_heads;
      for (int r0 = 0; r0 < R; r0 += T) {
        tiles.push_back(RowTile{b, grow0 + r0, std::min(T, R - r0), pages});
      }
    }
    tok0 += q;
  }

  // --- fold groups ------------------------------------------------------------------
  for (size_t i = 0; i < tiles.size();) {
    size_t j = i;
    int grp_rows = 0;
    const int b = tiles[i].b;
    const int R = reqs[b].fold * num_heads;
    while (j < tiles.size() && tiles[j].b == b && grp_rows < R) { grp_rows += tiles[j].nrows; ++j; }
    groups.push_back(Group{i, j, b, tiles[i].pages, 1, 1});
    i = j;
  }

  // --- splits ----------------------------------------------------------------------
  // Each group is cut into pieces of T pages (the last one shorter); all row tiles of the
  // group are cut at the same boundaries. The units are ordered longest first (below), so
  // the full-length units fill the SMs and the short tails run back to back on the SMs
  // left over. T is the per-SM share of the tile-pages divided by k, for the k whose
  // schedule ends first in a model of the hardware's in-order CTA dispatch: a unit costs
  // a start-up of kStart page-times (its prologue, first copies and Q preparation, the
  // epilogue and its split partial) plus its pages, each weighted by its row tile's cost
  // (a tile of <= 32 rows of an e4m3 cache takes less than a 48-row tile). The model's
  // constants were fitted to measured call times over forced piece lengths on GB300
  // (bf16: a unit start ~ 6 page-times; e4m3: ~ 16). It sees each request's q, so a batch
  // of ragged query lengths, whose fold groups differ in tile count, gets other piece
  // lengths than a uniform one of the same total work. A split keeps at least min_pages
  // pages.
  const int max_splits = max_splits_for_merge();
  auto row_cost = [&](int nrows) { return (!geo.wide && fp8 && nrows <= 32) ? 0.9 : 1.0; };
  long long tile_pages = 0;
  for (const Group& g : groups) tile_pages += (long long)(g.t1 - g.t0) * g.pages;
  auto assign = [&](long long T) {
    for (auto& g : groups) {
      long long n = o.force_splits > 0 ? o.force_splits : (g.pages + T - 1) / T;
      g.n_split = (int)std::max<long long>(1, std::min<long long>(std::min<long long>(n, g.pages), max_splits));
      // pieces of T pages, unless the split count was capped or forced: then equal pieces
      g.cap = (o.force_splits <= 0 && (long long)g.n_split == (g.pages + T - 1) / T) ? (int)T : 0;
    }
  };
  // the end of the schedule with pieces of T pages
  std::vector<std::pair<int, double>> lens;  // (pages, per-page cost) of every unit
  auto end_of = [&](long long T) {
    assign(T);
    lens.clear();
    for (const Group& g : groups)
      for (int s = 0; s < g.n_split; ++s)
        for (size_t t = g.t0; t < g.t1; ++t) lens.emplace_back(piece_pages(g, s), row_cost(tiles[t].nrows));
    std::stable_sort(lens.begin(), lens.end(),
                     [](const std::pair<int, double>& a, const std::pair<int, double>& b) { return a.first > b.first; });
    std::priority_queue<double, std::vector<double>, std::greater<double>> sm;
    for (int i = 0; i < slots; ++i) sm.push(0.0);
    double end = 0;
    for (const auto& L : lens) {
      const double t = sm.top() + start_cost + L.first * L.second;
      sm.pop();
      sm.push(t);
      end = std::max(end, t);
    }
    return end;
  };
  long long best_T = std::max<long long>(min_pages, (tile_pages + slots - 1) / slots);
  if (o.unit_pages > 0) best_T = o.unit_pages;
  double best_end = -1;
  if (o.force_splits > 0 || o.unit_pages > 0) {
    if (compared) best_end = end_of(best_T);
  } else {
    // candidates: the per-SM share divided by 1, 1.25, ... 8, and the longest group's
    // pages divided into 1 .. 64 equal pieces
    std::vector<long long> cands;
    for (int k4 : {4, 5, 6, 8, 10, 12, 16, 20, 24, 32})
      cands.push_back((4 * tile_pages + (long long)slots * k4 - 1) / ((long long)slots * k4));
    int longest = 0;
    for (const Group& g : groups) longest = std::max(longest, g.pages);
    for (int n = 1; n <= 64; ++n) cands.push_back((longest + n - 1) / n);
    std::sort(cands.begin(), cands.end());
    cands.erase(std::unique(cands.begin(), cands.end()), cands.end());
    for (long long c : cands) {
      const long long T = std::max<long long>(min_pages, c);
      // more than 16 waves of units (beyond one unit per row tile) never pays for its
      // start-up costs; skipping those keeps the search cheap for very long batches
      long long n_units = 0;
      for (const Group& g : groups) n_units += (long long)(g.t1 - g.t0) * ((g.pages + T - 1) / T);
      if (n_units > std::max<long long>(16LL * slots, (long long)tiles.size()) && !cands.empty() && c != cands.back())
        continue;
      const double end = end_of(T);
      if (best_end < 0 || end < best_end - 1e-9) {
        best_end = end;
        best_T = T;
      }
    }
  }
  assign(best_T);
  out.end_us = best_end * geo.page_us;
  return out;
}

}  // namespace

}  // namespace mla

using namespace mla;

// mla_decode_plan_ex, and with whole_requests mla_decode_plan_tree: a fold group is all of a request's tokens.
static int plan_batch(const int32_t* seq_lens_h, const int32_t* q_lens_h, int batch, int num_heads, int page_size,
                      int kv_dtype, int num_sms, const mla_plan_options* opts, bool whole_requests, void* plan_buf,
                      size_t plan_buf_bytes, size_t* plan_bytes_out, size_t* workspace_bytes_out) {
  if (!seq_lens_h || !q_lens_h) return set_error(MLA_ERR_INVALID_ARG, "seq_lens_h and q_lens_h must not be NULL");
  if (batch < 1) return set_error(MLA_ERR_INVALID_ARG, "batch must be >= 1 (got %d)", batch);
  if (num_heads < 1 || num_heads > MLA_MAX_HEADS)
    return set_error(MLA_ERR_UNSUPPORTED, "num_heads must be in [1, %d] (got %d)", MLA_MAX_HEADS, num_heads);
  if (page_size != kPage) return set_error(MLA_ERR_UNSUPPORTED, "only page_size 64 is supported (got %d)", page_size);
  if (kv_dtype != MLA_KV_BF16 && kv_dtype != MLA_KV_FP8_E4M3)
    return set_error(MLA_ERR_INVALID_ARG, "kv_dtype must be MLA_KV_BF16 or MLA_KV_FP8_E4M3 (got %d)", kv_dtype);
  if (num_sms < 1) return set_error(MLA_ERR_INVALID_ARG, "num_sms must be >= 1 (got %d)", num_sms);
  mla_plan_options o{};
  if (opts) o = *opts;
  int cap = rows_cap_for(kv_dtype);
  const bool force_wide = whole_requests && o.max_rows_per_cta == wide_rows_cap();
  if (o.max_rows_per_cta > 0 && !force_wide) {
    if (o.max_rows_per_cta % 16 != 0 || o.max_rows_per_cta > cap)
      return set_error(MLA_ERR_INVALID_ARG, "max_rows_per_cta must be a multiple of 16 and <= %d (got %d)", cap,
                       o.max_rows_per_cta);
    cap = o.max_rows_per_cta;
  }
  if (o.force_splits < 0 || o.min_pages_per_split < 0 || o.force_fold < 0 || o.unit_pages < 0 || o.cta_pair < 0 ||
      o.pair_slots < 0 || o.debug_skip_copy < 0)
    return set_error(MLA_ERR_INVALID_ARG, "plan options must be >= 0");
  if (o.force_splits > 0 && o.unit_pages > 0)
    return set_error(MLA_ERR_INVALID_ARG, "force_splits and unit_pages exclude each other");
  if (whole_requests && (o.force_fold > 0 || o.cta_pair > 0))
    return set_error(MLA_ERR_INVALID_ARG, "a plan for trees takes neither force_fold nor cta_pair");

  long long total_q = 0;
  int max_pages = 0;
  for (int b = 0; b < batch; ++b) {
    int ctx = seq_lens_h[b], q = q_lens_h[b];
    if (q < 1) return set_error(MLA_ERR_INVALID_ARG, "q_lens[%d] = %d must be >= 1", b, q);
    if (ctx < q) return set_error(MLA_ERR_INVALID_ARG, "seq_lens[%d] = %d is smaller than q_lens[%d] = %d", b, ctx, b, q);
    // (the kernels count keys in 32 bits, some tiles ahead)
    if (ctx > kMaxKeys) return set_error(MLA_ERR_INVALID_ARG, "seq_lens[%d] = %d must be <= %d", b, ctx, kMaxKeys);
    if (o.force_fold > 0 && q % o.force_fold != 0)
      return set_error(MLA_ERR_INVALID_ARG, "force_fold %d does not divide q_lens[%d] = %d", o.force_fold, b, q);
    total_q += q;
    max_pages = std::max(max_pages, (ctx + kPage - 1) / kPage);
  }
  if (total_q * num_heads > (1LL << 30)) return set_error(MLA_ERR_INVALID_ARG, "too many query rows");

  // On request (cta_pair), a bf16 cache whose every fold group has 49..96 packed rows runs
  // on clusters of two CTAs, one unit per fold group and key piece: each CTA streams half
  // of every page's columns, so the page enters the pair once instead of once per 48-row
  // tile. (Off by default: on GB300 the 48-row single-CTA tiles are faster.)
  bool pair = kv_dtype == MLA_KV_BF16 && o.cta_pair > 0 && o.max_rows_per_cta == 0;
  for (int b = 0; pair && b < batch; ++b) {
    const int F = o.force_fold > 0 ? o.force_fold : fold_factor(q_lens_h[b], num_heads);
    const int R = F * num_heads;
    pair = R > cap && R <= pair_rows_cap();
  }
  if (pair) cap = pair_rows_cap();
  const bool fp8 = kv_dtype == MLA_KV_FP8_E4M3;
  const int pair_slots = o.pair_slots > 0 ? o.pair_slots : std::max(1, num_sms / 2);
  const int asked = o.min_pages_per_split;
  Geometry geo{false, whole_requests, cap, pair ? pair_slots : num_sms, asked > 0 ? asked : 4, fp8 ? 16.0 : 6.0, 1.0};
  Partition part;
  bool wide = force_wide;
  if (whole_requests) {
    // Trees run in tiles of 48 rows, or in tiles of 128 on clusters of two CTAs where the model's schedule
    // of those ends first. Fitted to forced piece lengths over six short and ten long batches: a unit
    // starts in 9 us (bf16) or 12 (e4m3) and takes 1.6 or 1.2 us a page in narrow tiles; 15 or 17 us and
    // 0.65 or 0.72 in wide ones. (8 nodes, 12 heads: 12 us narrow, 16 wide over 4096 keys, 60 and 40 over
    // 131072; 32 trees of 48 heads over block scales 584 and 393; pieces of a page instead of four, 4096 keys:
    // 15.8 -> 10.9; 24 page-times to start a wide unit instead of 10, the 32 trees: 418 -> 393.)
    Geometry narrow = geo, broad = geo;
    narrow.min_pages = asked > 0 ? asked : 1;
    narrow.start_cost = fp8 ? 10.0 : 6.0;
    narrow.page_us = fp8 ? 1.2 : 1.6;
    broad.wide = true;
    broad.cap = wide_rows_cap();
    broad.slots = pair_slots;
    broad.min_pages = asked > 0 ? asked : 2;
    broad.start_cost = 24.0;
    broad.page_us = fp8 ? 0.72 : 0.65;
    const bool compared = o.max_rows_per_cta == 0;  // of both tiles, not the one that is asked for
    if (force_wide || compared) part = cut_batch(seq_lens_h, q_lens_h, batch, num_heads, fp8, o, geo = broad, compared);
    if (!force_wide) {
      Partition other = cut_batch(seq_lens_h, q_lens_h, batch, num_heads, fp8, o, narrow, compared);
      wide = compared && part.end_us < other.end_us;
      if (!wide) {
        part = std::move(other);
        geo = narrow;
      }
    }
  } else {
    part = cut_batch(seq_lens_h, q_lens_h, batch, num_heads, fp8, o, geo, false);
  }
  const std::vector<RowTile>& tiles = part.tiles;
  const std::vector<PlanRequest>& reqs = part.reqs;
  const std::vector<Group>& groups = part.groups;
  const int slots = geo.slots;

  long long all_part_rows = 0;
  for (const Group& g : groups)
    if (g.n_split > 1)
      for (size_t t = g.t0; t < g.t1; ++t) all_part_rows += (long long)g.n_split * tiles[t].nrows;
  if (all_part_rows > INT32_MAX) return set_error(MLA_ERR_INVALID_ARG, "too many partial rows: fewer splits are needed");

  std::vector<PlanUnit> units;
  std::vector<PlanMerge> merges;
  int part_rows = 0;
  for (const Group& g : groups) {
    const int b = g.b, n_split = g.n_split, pages = g.pages;
    std::vector<int> part0(g.t1 - g.t0, -1);
    if (n_split > 1) {
      for (size_t t = g.t0; t < g.t1; ++t) {
        part0[t - g.t0] = part_rows;
        merges.push_back(PlanMerge{tiles[t].qrow0, tiles[t].nrows, part_rows, n_split});
        part_rows += n_split * tiles[t].nrows;
      }
    }
    for (int s = 0; s < n_split; ++s) {
      int p_begin, p_end;
      if (g.cap > 0) {  // pieces of T = g.cap pages, the last one shorter
        p_begin = s * g.cap;
        p_end = std::min(pages, (s + 1) * g.cap);
      } else {
        p_begin = (int)((long long)pages * s / n_split);
        p_end = (int)((long long)pages * (s + 1) / n_split);
      }
      int kb = p_begin * kPage, ke = std::min(reqs[b].ctx, p_end * kPage);
      for (size_t t = g.t0; t < g.t1; ++t) {
        PlanUnit u;
        u.b = b; u.qrow0 = tiles[t].qrow0; u.nrows = tiles[t].nrows;
        u.kv_begin = kb; u.kv_end = ke;
        u.part_row0 = n_split > 1 ? part0[t - g.t0] + s * tiles[t].nrows : -1;
        u.split = s; u.n_splits = n_split;
        u.ctx = reqs[b].ctx; u.q = reqs[b].q; u.tok0 = reqs[b].tok0;
        // pages read by one row tile only: the request is a single fold group of one tile
        u.flags = (reqs[b].q / reqs[b].fold == 1 && g.t1 - g.t0 == 1) ? kUnitKvReadOnce : 0;
        units.push_back(u);
      }
    }
  }
  // Longest units first: when the grid needs more than one wave, the SMs that finish
  // early pick up the short units. (Stable, so the tiles of a group stay adjacent.)
  if ((long long)units.size() > slots)
    std::stable_sort(units.begin(), units.end(), [](const PlanUnit& a, const PlanUnit& c) {
      return a.kv_end - a.kv_begin > c.kv_end - c.kv_begin;
    });

  size_t req_off = sizeof(PlanHeader);
  size_t units_off = align_up(req_off + sizeof(PlanRequest) * batch, 32);
  size_t merge_off = align_up(units_off + sizeof(PlanUnit) * units.size(), 32);
  size_t total = align_up(merge_off + sizeof(PlanMerge) * merges.size(), 64);
  if (total > (size_t)INT32_MAX) return set_error(MLA_ERR_INVALID_ARG, "plan too large");
  if (plan_bytes_out) *plan_bytes_out = total;
  if (workspace_bytes_out) *workspace_bytes_out = workspace_bytes_for(part_rows, whole_requests);
  if (!plan_buf || plan_buf_bytes < total)
    return set_error(MLA_ERR_BUFFER, "plan buffer needs %zu bytes (got %zu)", total, plan_buf ? plan_buf_bytes : (size_t)0);

  uint8_t* base = (uint8_t*)plan_buf;
  memset(base, 0, total);
  PlanHeader h{};
  h.magic = kPlanMagic; h.version = kPlanVersion;
  h.batch = batch; h.num_heads = num_heads; h.kv_dtype = kv_dtype; h.total_q = (int32_t)total_q;
  h.n_units = (int32_t)units.size(); h.n_merge = (int32_t)merges.size();
  int used_cap = 0;
  for (auto& u : units) used_cap = std::max(used_cap, u.nrows);
  h.rows_cap = used_cap; h.n_part_rows = part_rows; h.max_pages = max_pages;
  h.req_off = (int32_t)req_off; h.units_off = (int32_t)units_off; h.merge_off = (int32_t)merge_off;
  h.total_bytes = (int32_t)total;
  h.debug_skip_copy = o.debug_skip_copy;
  h.cta_pair = pair ? 1 : 0;
  h.wide = wide ? 1 : 0;
  h.tree = whole_requests ? 1 : 0;
  memcpy(base, &h, sizeof h);
  memcpy(base + req_off, reqs.data(), sizeof(PlanRequest) * batch);
  if (!units.empty()) memcpy(base + units_off, units.data(), sizeof(PlanUnit) * units.size());
  if (!merges.empty()) memcpy(base + merge_off, merges.data(), sizeof(PlanMerge) * merges.size());
  return MLA_OK;
}

// No exception leaves a C entry: the planner's vectors throw where the host has no memory for them.
template <typename... Args>
static int make_plan(Args... args) {
  clear_error();
  try {
    return plan_batch(args...);
  } catch (const std::exception& e) {
    return set_error(MLA_ERR_MEMORY, "no host memory for the plan (%s)", e.what());
  }
}

extern "C" int mla_decode_plan_ex(const int32_t* seq_lens_h, const int32_t* q_lens_h, int batch, int num_heads,
                                  int page_size, int kv_dtype, int num_sms, const mla_plan_options* opts,
                                  void* plan_buf, size_t plan_buf_bytes, size_t* plan_bytes_out,
                                  size_t* workspace_bytes_out) {
  return make_plan(seq_lens_h, q_lens_h, batch, num_heads, page_size, kv_dtype, num_sms, opts, false, plan_buf,
                   plan_buf_bytes, plan_bytes_out, workspace_bytes_out);
}

// A tree's size has any divisors: folded by the largest one a tree of 29 tokens would run as 29 tiles
// of one token each. A row's mask is its own, so the tiles are cut from all of a request's rows.
extern "C" int mla_decode_plan_tree(const int32_t* seq_lens_h, const int32_t* q_lens_h, int batch, int num_heads,
                                    int page_size, int kv_dtype, int num_sms, const mla_plan_options* opts,
                                    void* plan_buf, size_t plan_buf_bytes, size_t* plan_bytes_out,
                                    size_t* workspace_bytes_out) {
  return make_plan(seq_lens_h, q_lens_h, batch, num_heads, page_size, kv_dtype, num_sms, opts, true, plan_buf,
                   plan_buf_bytes, plan_bytes_out, workspace_bytes_out);
}

extern "C" int mla_decode_plan(const int32_t* seq_lens_h, const int32_t* q_lens_h, int batch, int num_heads,
                               int page_size, int kv_dtype, int num_sms, void* plan_buf, size_t plan_buf_bytes,
                               size_t* plan_bytes_out, size_t* workspace_bytes_out) {
  return mla_decode_plan_ex(seq_lens_h, q_lens_h, batch, num_heads, page_size, kv_dtype, num_sms, nullptr, plan_buf,
                            plan_buf_bytes, plan_bytes_out, workspace_bytes_out);
}

namespace mla {

int check_plan(const void* plan_host, size_t plan_bytes, const PlanHeader** out) {
  if (!plan_host) return set_error(MLA_ERR_INVALID_ARG, "plan_host must not be NULL");
  if (plan_bytes < sizeof(PlanHeader)) return set_error(MLA_ERR_PLAN, "plan is %zu bytes, smaller than its header", plan_bytes);
  const PlanHeader* h = (const PlanHeader*)plan_host;
  if (h->magic != kPlanMagic || h->version != kPlanVersion)
    return set_error(MLA_ERR_PLAN, "plan bytes were not written by this library version");
  if ((size_t)h->total_bytes != plan_bytes)
    return set_error(MLA_ERR_PLAN, "plan_bytes %zu differs from the plan's size %d", plan_bytes, h->total_bytes);
  // what chooses the kernel and its tiles
  const auto flag = [](int32_t v) { return v == 0 || v == 1; };
  const int cap = h->wide ? wide_rows_cap() : h->cta_pair ? pair_rows_cap() : rows_cap_for(h->kv_dtype);
  if (!flag(h->wide) || !flag(h->tree) || !flag(h->cta_pair) || (h->wide && !h->tree) || (h->cta_pair && h->tree) ||
      (h->cta_pair && h->kv_dtype != MLA_KV_BF16) || h->rows_cap < 1 || h->rows_cap > cap)
    return set_error(MLA_ERR_PLAN, "the plan's header contradicts itself (wide %d, tree %d, cta_pair %d, kv_dtype %d, row tiles of %d)",
                     h->wide, h->tree, h->cta_pair, h->kv_dtype, h->rows_cap);
  *out = h;
  return MLA_OK;
}

}  // namespace mla

extern "C" int mla_decode_plan_info(const void* plan_host, size_t plan_bytes, int* n_units, int* n_merge,
                                    int* total_q, int* num_heads, int* kv_dtype) {
  clear_error();
  const PlanHeader* h = nullptr;
  int rc = check_plan(plan_host, plan_bytes, &h);
  if (rc != MLA_OK) return rc;
  if (n_units) *n_units = h->n_units;
  if (n_merge) *n_merge = h->n_merge;
  if (total_q) *total_q = h->total_q;
  if (num_heads) *num_heads = h->num_heads;
  if (kv_dtype) *kv_dtype = h->kv_dtype;
  return MLA_OK;
}
