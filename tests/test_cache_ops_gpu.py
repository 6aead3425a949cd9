"""The cache operators on the GPU against plain 64-bit forms: append to a block-scaled e4m3
cache, the decode over it, the accumulated key weights and the eviction, through the public
entry points."""
import numpy as np
import pytest
import torch

from mla_speculative_verify_gb300 import binding, cache, inputs
from mla_speculative_verify_gb300.decoder import VerifyDecoder
from tests import cache_reference as ref

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
PAGE, D = 64, 576


def dev(a):
    return (torch.from_numpy(np.ascontiguousarray(a)) if isinstance(a, np.ndarray) else a).cuda()


def same(got: torch.Tensor, want: np.ndarray):
    assert np.array_equal(got.cpu().double().numpy(), want, equal_nan=True)


# ------------------------------------------------------------------------------- append
def append_case(lens_new, pasts, block, seed=0, magnitude=1.0):
    """Host tensors of an append: filled cache, scales (powers of two), table, rows."""
    g = torch.Generator().manual_seed(seed)
    ends = np.asarray(lens_new) + np.asarray(pasts)
    batch = ref.Batch(1, np.maximum(ends, 1), np.ones(len(ends)), "bf16", seed=seed, extra_pages=3, poison=False)
    codes = (torch.randn((batch.pages, PAGE, D), generator=g) * 60).clamp(-448, 448).to(F8).view(torch.uint8)
    scales = torch.exp2(torch.randint(-9, -3, (batch.pages, PAGE // block), generator=g).float())
    rows = torch.randn((int(sum(lens_new)), D), generator=g) * magnitude
    rows *= torch.exp2(torch.randint(-6, 6, (rows.shape[0], 1), generator=g).float())
    return batch, codes, scales, rows.to(torch.bfloat16), ends.astype(np.int32), np.concatenate(
        [[0], np.cumsum(lens_new)]).astype(np.int32)


def run_append(batch, codes, scales, rows, ends, cu, max_new=None, stream=None):
    c, s = codes.clone().cuda(), scales.clone().cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.append(rows.cuda(), c, s, dev(batch.table), dev(ends), dev(cu),
                 int(np.diff(cu).max()) if max_new is None else max_new, status, stream)
    torch.cuda.synchronize()
    return c, s, int(status.item())


@pytest.mark.parametrize("block", [1, 2, 4, 8, 16, 32, 64])
@pytest.mark.parametrize("lens_new,pasts", [([1], [0]), ([1], [63]), ([4, 1, 0, 7], [61, 64, 30, 5]),
                                            ([130, 64, 1, 200], [0, 64, 127, 33]), ([63, 65], [1, 62])])
def test_append(block, lens_new, pasts):
    batch, codes, scales, rows, ends, cu = append_case(lens_new, pasts, block, seed=block)
    values, want_s = ref.code_values(codes), scales.double().numpy()
    ref.append(rows, values, want_s, batch.table, ends, cu, block)
    c, s, status = run_append(batch, codes, scales, rows, ends, cu)
    assert status == 0
    same(c.view(F8), values)
    same(s, want_s)


def test_append_many_requests():
    g = np.random.default_rng(6)
    batch, codes, scales, rows, ends, cu = append_case(g.integers(0, 90, size=90), g.integers(0, 200, size=90), 8, seed=6)
    values, want_s = ref.code_values(codes), scales.double().numpy()
    ref.append(rows, values, want_s, batch.table, ends, cu, 8)
    c, s, status = run_append(batch, codes, scales, rows, ends, cu)
    assert status == 0
    same(c.view(F8), values)
    same(s, want_s)


def test_append_special_values():
    """Zero rows, infinities, NaN, bf16's largest and least values, another writer's scale."""
    batch, codes, scales, rows, ends, cu = append_case([40, 24], [10, 64], 16, seed=3)
    rows[0:6] = 0
    rows[7, 3], rows[8, 4], rows[9, 5] = float("inf"), float("-inf"), float("nan")
    rows[30, :8] = torch.tensor([3.0e38, -3.0e38, 1e-40, 0.0, -0.0, 1.0, -1.0, 2e-38])
    scales[batch.table[0, 0], 0] = 0.37  # not a power of two, and larger than the new rows ask for
    values, want_s = ref.code_values(codes), scales.double().numpy()
    ref.append(rows, values, want_s, batch.table, ends, cu, 16)
    c, s, status = run_append(batch, codes, scales, rows, ends, cu)
    assert status == 0
    same(c.view(F8), values)
    same(s, want_s)


def test_append_twice_is_once():
    """Appending the same rows again changes nothing (a replayed step)."""
    batch, codes, scales, rows, ends, cu = append_case([5, 9], [60, 3], 32, seed=4)
    c, s, _ = run_append(batch, codes, scales, rows, ends, cu)
    c2, s2, _ = run_append(batch, c.cpu(), s.cpu(), rows, ends, cu)
    assert torch.equal(c, c2) and torch.equal(s, s2)


def test_append_bad_requests_write_nothing():
    batch, codes, scales, rows, ends, cu = append_case([5, 9, 3], [60, 3, 0], 16, seed=5)
    for bad, bit in (("page", binding.MLA_DEVICE_BAD_PAGE), ("more than max_new", binding.MLA_DEVICE_PLAN_MISMATCH),
                     ("shorter than its rows", binding.MLA_DEVICE_PLAN_MISMATCH)):
        table, e, most = batch.table.copy(), ends.copy(), 9
        b2 = type("B", (), {"table": table})
        if bad == "page":
            table[1, 0] = batch.pages
        elif bad == "more than max_new":
            most = 8
        else:
            e[1] = 8
        values, want_s = ref.code_values(codes), scales.double().numpy()
        only = np.array([cu[0], cu[1], cu[1], cu[2]], np.int32)  # request 1 left out
        ref.append(torch.cat([rows[:5], rows[14:]]), values, want_s, batch.table, np.array([ends[0], 0, ends[2]]),
                   np.array([0, 5, 5, 8]), 16)
        c, s, status = run_append(b2, codes, scales, rows, e, cu, max_new=most)
        assert status == bit, bad
        same(c.view(F8), values)
        same(s, want_s)


# ------------------------------------------------------------------------------- decode
def decode(batch, options=None):
    d = VerifyDecoder(batch.seq_lens, batch.q_lens, batch.H, "bf16" if batch.kind == "bf16" else "fp8", options=options)
    out = torch.full((batch.q.shape[0], batch.H, 512), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((batch.q.shape[0], batch.H), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    t = {"q": batch.q.cuda(), "kv": batch.kv.cuda(), "table": dev(batch.table),
         "scales": None if batch.scales is None else batch.scales.cuda()}
    d.run(t["q"], t["kv"], t["table"], out, lse, kv_scale=batch.kv_scale, status=status, kv_scales=t["scales"])
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return d, t, out, lse


SHAPES = [(12, [1], [1]), (12, [64], [3]), (1, [65], [2]), (12, [700], [8]), (33, [129, 64, 300], [1, 3, 2]),
          (128, [200, 7], [2, 5]), (48, [513], [4]), (96, [260], [1])]


@pytest.mark.parametrize("heads,seq,q", SHAPES)
@pytest.mark.parametrize("block", [1, 16, 64])
def test_decode_scaled(heads, seq, q, block):
    batch = ref.Batch(heads, seq, q, "e4m3", block, seed=heads + block)
    want, bound, lse, lse_bound = ref.attend(batch)
    _, _, out, got_lse = decode(batch)
    assert (np.abs(got_lse.cpu().double().numpy() - lse) <= lse_bound).all()
    assert (np.abs(out.cpu().double().numpy() - want) <= bound).all()


@pytest.mark.parametrize("splits", [1, 5, 20])
@pytest.mark.parametrize("spread", [0.0, 8.0])
def test_decode_scaled_splits_and_spread(splits, spread):
    """Split over the keys, and scales that lie up to 2^16 apart: blocks with a small scale hold
    small values, and keys with a large one win the softmax of many rows."""
    batch = ref.Batch(12, [64 * 20 + 5], [4], "e4m3", 32, spread=spread, seed=7)
    want, bound, lse, lse_bound = ref.attend(batch)
    _, _, out, got_lse = decode(batch, binding.PlanOptions(force_splits=splits))
    assert (np.abs(got_lse.cpu().double().numpy() - lse) <= lse_bound).all()
    assert (np.abs(out.cpu().double().numpy() - want) <= bound).all()


def test_decode_scaled_zero_blocks_and_far_scales():
    """Blocks with the scale 0 (values 0, weight as any score of 0) beside scales of 2^-40 and 2^-9."""
    batch = ref.Batch(12, [640], [2], "e4m3", 64, spread=0.0, seed=8, poison=False)
    page = batch.table[0]
    batch.scales[page[1], 0] = 0.0
    batch.scales[page[2], 0] = 2.0 ** -40
    batch.scales[page[3], 0] = 2.0 ** -9
    want, bound, lse, lse_bound = ref.attend(batch)
    _, _, out, got_lse = decode(batch)
    assert (np.abs(got_lse.cpu().double().numpy() - lse) <= lse_bound).all()
    assert (np.abs(out.cpu().double().numpy() - want) <= bound).all()


def test_decode_scaled_equal_scales_match_one_scale():
    """A cache whose blocks all have one scale gives what the per-tensor scale gives, within both bounds."""
    one = ref.Batch(12, [1000], [4], "e4m3", 0, seed=9, poison=False)
    many = ref.Batch(12, [1000], [4], "e4m3", 0, seed=9, poison=False)
    many.block, many.scales = 16, torch.full((many.pages, 4), many.kv_scale)
    want, bound, _, _ = ref.attend(one)
    _, _, a, la = decode(one)
    _, _, b, lb = decode(many)
    assert (np.abs(a.cpu().double().numpy() - want) <= bound).all()
    assert (np.abs(b.cpu().double().numpy() - want) <= bound).all()
    assert (la - lb).abs().max().item() <= 1e-5


# ------------------------------------------------------------------------------- key weights
def run_weights(batch, decay, old, counted=None, lse=None, d=None, t=None, stream=None):
    if d is None:
        d, t, _, lse = decode(batch)
    w = torch.from_numpy(old.astype(np.float32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d.key_weights(t["q"], t["kv"], t["table"], lse, w, decay, None if counted is None else dev(np.asarray(counted, np.int32)),
                  kv_scale=batch.kv_scale, kv_scales=t["scales"], status=status, stream=stream)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    return w, lse


KINDS = [("bf16", 0), ("e4m3", 0), ("e4m3", 1), ("e4m3", 64)]


@pytest.mark.parametrize("kind,block", KINDS)
@pytest.mark.parametrize("heads,seq,q", SHAPES)
def test_key_weights(heads, seq, q, kind, block):
    batch = ref.Batch(heads, seq, q, kind, block, seed=heads + block)
    old = np.random.default_rng(1).random((len(seq), max(seq) + 3)).astype(np.float32)
    w, lse = run_weights(batch, 0.75, old)
    want, bound = ref.weights(batch, lse.cpu().double().numpy(), 0.75, old)
    got = w.cpu().double().numpy()
    assert (np.abs(got - want) <= bound + 1e-30).all()
    for b, n in enumerate(seq):  # behind the last key nothing is touched
        assert np.array_equal(got[b, n:], old[b, n:].astype(np.float64))


@pytest.mark.parametrize("kind,block", KINDS)
def test_key_weights_many_rows(kind, block):
    """Several groups of rows (up to 128 each) over several tiles, one of them short."""
    batch = ref.Batch(96, [64 * 11 + 9, 300], [6, 3], kind, block, seed=21)
    old = np.zeros((2, 713))
    w, lse = run_weights(batch, 1.0, old)
    want, bound = ref.weights(batch, lse.cpu().double().numpy(), 1.0, old)
    assert (np.abs(w.cpu().double().numpy() - want) <= bound + 1e-30).all()


@pytest.mark.parametrize("kind,block", KINDS)
def test_key_weights_counted_and_no_decay(kind, block):
    """Only accepted tokens count; decay 0 does not read the old sums (NaN here)."""
    batch = ref.Batch(40, [500, 90, 130], [5, 4, 3], kind, block, seed=22)
    counted = [2, 0, 9]
    old = np.full((3, 500), np.nan)
    w, lse = run_weights(batch, 0.0, old, counted)
    want, bound = ref.weights(batch, lse.cpu().double().numpy(), 0.0, old, counted)
    got = w.cpu().double().numpy()
    for b, n in enumerate(batch.seq_lens):
        assert (np.abs(got[b, :n] - want[b, :n]) <= bound[b, :n] + 1e-30).all()
        assert np.isnan(got[b, n:]).all()


def test_key_weights_of_hidden_rows():
    """lse = -inf (a row that saw nothing) adds nothing; rows beside a request's, of another
    request with NaN in its queries, do not reach it; equal calls give equal bits."""
    batch = ref.Batch(12, [300, 200], [2, 2], "bf16", 0, seed=23)
    d, t, _, lse = decode(batch)
    t["q"][2:] = float("nan")
    lse[0, :] = float("-inf")
    old = np.zeros((2, 300))
    w, _ = run_weights(batch, 1.0, old, lse=lse, d=d, t=t)
    w2, _ = run_weights(batch, 1.0, old, lse=lse, d=d, t=t)
    l = lse.cpu().double().numpy()
    l[0, :] = np.inf
    batch.seq_lens, batch.q_lens = batch.seq_lens[:1], batch.q_lens[:1]
    want, bound = ref.weights(batch, l, 1.0, old)
    assert (np.abs(w.cpu().double().numpy() - want)[0] <= bound[0] + 1e-30).all()
    assert torch.equal(w[0], w2[0])


def test_key_weights_sum_to_the_rows():
    """Every row's weights sum to one, so a request's sums add up to its rows (a long context)."""
    batch = ref.Batch(12, [20000, 9000], [4, 2], "bf16", 0, seed=24)
    w, _ = run_weights(batch, 0.0, np.zeros((2, 20000)))
    total = w.double().sum(1).cpu().numpy()
    assert np.abs(total / [48, 24] - 1).max() < 1e-4


@pytest.mark.parametrize("kind,block", [("bf16", 0), ("e4m3", 16)])
def test_timeouts_are_reported_not_hung(kind, block):
    """A plan whose test-only option keeps one copy from being issued and shortens every bounded
    wait to ~2 ms: the decode and the key weights give up, report it, and the next calls are exact."""
    batch = ref.Batch(12, [64 * 40 + 7], [4], kind, block, seed=27)
    _, t, _, lse = decode(batch)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = VerifyDecoder(batch.seq_lens, batch.q_lens, 12, "bf16" if kind == "bf16" else "fp8",
                        options=binding.PlanOptions(force_splits=4, debug_skip_copy=3))
    if block:
        bad.run(t["q"], t["kv"], t["table"], torch.empty((4, 12, 512), dtype=torch.bfloat16, device="cuda"),
                status=status, kv_scales=t["scales"])
        torch.cuda.synchronize()
        assert int(status.item()) & binding.MLA_DEVICE_WAIT_TIMEOUT
        status.zero_()
    bad.key_weights(t["q"], t["kv"], t["table"], lse, torch.zeros((1, 2567), device="cuda"), kv_scales=t["scales"],
                    status=status)
    torch.cuda.synchronize()
    assert int(status.item()) & binding.MLA_DEVICE_WAIT_TIMEOUT
    old = np.zeros((1, 2567))
    w, lse = run_weights(batch, 1.0, old)
    want, bound = ref.weights(batch, lse.cpu().double().numpy(), 1.0, old)
    assert (np.abs(w.cpu().double().numpy() - want) <= bound + 1e-30).all()


@pytest.mark.parametrize("kind,block", [("bf16", 0), ("e4m3", 0), ("e4m3", 64)])
def test_bad_pages_are_reported(kind, block):
    """A page id outside the cache is reported and touches nothing else: the other request's sums
    and rows stay exact."""
    batch = ref.Batch(12, [300, 200], [2, 1], kind, block, seed=28, extra_pages=20, poison=False)
    d, t, _, lse = decode(batch)
    table = batch.table.copy()
    table[0, 2] = batch.pages
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    w = torch.zeros((2, 300), device="cuda")
    d.key_weights(t["q"], t["kv"], dev(table), lse, w, kv_scale=batch.kv_scale, kv_scales=t["scales"], status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == binding.MLA_DEVICE_BAD_PAGE
    want, bound = ref.weights(batch, lse.cpu().double().numpy(), 1.0, np.zeros((2, 300)))
    assert (np.abs(w.cpu().double().numpy() - want)[1] <= bound[1]).all()
    if block:
        status.zero_()
        out = torch.empty((3, 12, 512), dtype=torch.bfloat16, device="cuda")
        d.run(t["q"], t["kv"], dev(table), out, status=status, kv_scales=t["scales"])
        torch.cuda.synchronize()
        assert int(status.item()) == binding.MLA_DEVICE_BAD_PAGE
        want_out, out_bound, _, _ = ref.attend(batch)
        assert (np.abs(out[2].cpu().double().numpy() - want_out[2]) <= out_bound[2]).all()
    # eviction: an old page of request 0 and a new page of request 1 out of range
    table_dst = batch.free[:4].reshape(2, 2).copy()
    bad_dst = table_dst.copy()
    bad_dst[1, 1] = -1
    weights = np.random.default_rng(1).random((2, 300)).astype(np.float32)
    kept, lens = torch.empty((2, 100), dtype=torch.int32, device="cuda"), torch.empty(2, dtype=torch.int32, device="cuda")
    status.zero_()
    cache.evict(dev(weights), dev(batch.seq_lens), 100, 0, 0, t["kv"], dev(table), t["kv"], dev(bad_dst), kept, lens,
                scales=t["scales"], scales_dst=t["scales"], status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == binding.MLA_DEVICE_BAD_PAGE
    assert lens.tolist() == [100, 100]
    as_values = (lambda x: x.double().numpy()) if kind == "bf16" else ref.code_values
    values, values_dst = as_values(batch.kv), as_values(batch.kv)
    s = None if block == 0 else batch.scales.double().numpy()
    want = ref.evict(weights[1:], batch.seq_lens[1:], 100, 0, 0, values, s, batch.table[1:], values_dst,
                     None if s is None else s.copy(), table_dst[1:], block)
    assert kept[1].cpu().tolist() == want[0].tolist()
    got = as_values(t["kv"].cpu())
    assert np.array_equal(got[table_dst[1, 0]], values_dst[table_dst[1, 0]])
    assert np.array_equal(got[table_dst[1, 1]], values[table_dst[1, 1]])  # (named by nobody: as it was)


def test_key_weights_with_a_plan_for_cta_pairs():
    batch = ref.Batch(12, [700], [8], "bf16", seed=29)
    d, t, _, lse = decode(batch, binding.PlanOptions(cta_pair=1))
    assert d.cta_pair
    w, _ = run_weights(batch, 1.0, np.zeros((1, 700)), lse=lse, d=d, t=t)
    want, bound = ref.weights(batch, lse.cpu().double().numpy(), 1.0, np.zeros((1, 700)))
    assert (np.abs(w.cpu().double().numpy() - want) <= bound + 1e-30).all()


def test_offsets_beyond_32_bits():
    """A pool of 2.9 GB of codes whose pages in use lie at its end, as uint8 and as float8, gives
    what a small pool gives: append, decode, key weights and eviction."""
    big, n, q, H = 80000, 500, 3, 12
    gen = torch.Generator().manual_seed(30)
    rows = torch.randn((n, D), generator=gen).to(torch.bfloat16).cuda()
    queries = torch.randn((q, H, D), generator=gen).to(torch.bfloat16).cuda()
    weights = torch.rand((1, n), generator=gen).cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    d = VerifyDecoder([n], [q], H, "fp8")
    results = []
    for pages in (12, big):
        base = pages - 12
        codes = torch.zeros((pages, PAGE, D), dtype=torch.uint8, device="cuda")
        scales = torch.ones((pages, 4), device="cuda")
        table = (base + torch.arange(8, device="cuda")).int().view(1, 8)
        dst = (base + 8 + torch.arange(4, device="cuda")).int().view(1, 4)
        out, lse = torch.empty((q, H, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((q, H), device="cuda")
        w, kept, lens = torch.zeros((1, n), device="cuda"), torch.empty((1, 200), dtype=torch.int32, device="cuda"), i32([0])
        status = i32([0])
        view = codes.view(F8) if pages == big else codes
        cache.append(rows, view, scales, table, i32([n]), i32([0, n]), n, status)
        d.run(queries, view, table, out, lse, status=status, kv_scales=scales)
        d.key_weights(queries, view, table, lse, w, kv_scales=scales, status=status)
        cache.evict(weights, i32([n]), 200, 4, 8, view, table, view, dst, kept, lens, scales=scales, scales_dst=scales,
                    status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        results.append([x.clone() for x in (out, lse, w, kept, lens, codes[base:], scales[base:])])
        assert not codes[:base].any() if pages == 12 else not codes[:1000].any()
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_refused_tensors():
    """Wrong types, shapes and layouts on the GPU are refused before anything is launched."""
    z = lambda *s, t=torch.int32: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    rows, codes, scales = z(4, D, t=torch.bfloat16), z(3, PAGE, D, t=torch.uint8), z(3, 4, t=torch.float32)
    good = dict(rows=rows, codes=codes, scales=scales, page_table=z(1, 2), seq_lens=z(1), cu_new=z(2), max_new=4)
    for name, t in (("rows", rows.float()), ("rows", z(D, 4, t=torch.bfloat16).t()), ("rows", rows[0]), ("codes", codes[:, :32]),
                    ("codes", codes.float()), ("scales", z(3, 3, t=torch.float32)), ("scales", z(2, 4, t=torch.float32)),
                    ("scales", z(3, 128, t=torch.float32)), ("page_table", z(2)), ("page_table", z(2, 2, t=torch.int64)),
                    ("seq_lens", z(2)), ("cu_new", z(1)), ("seq_lens", z(1).cpu())):
        with pytest.raises(ValueError):
            cache.append(**dict(good, **{name: t}))
    with pytest.raises(binding.MlaError):
        cache.append(**dict(good, max_new=5))
    f32 = torch.float32
    good = dict(weights=z(1, 64, t=f32), seq_lens=z(1), budget=8, n_first=0, n_last=0, kv=codes, page_table=z(1, 1),
                kv_dst=codes, page_table_dst=z(1, 1), kept=z(1, 8), seq_lens_dst=z(1), scales=scales, scales_dst=scales)
    for name, t in (("weights", z(64, t=f32)), ("weights", z(64, 2, t=f32).t()[:1]), ("seq_lens", z(2)), ("kv", codes.float()),
                    ("kv_dst", codes.to(torch.bfloat16)), ("scales", None), ("scales_dst", z(3, 2, t=f32)), ("kept", z(1, 7)),
                    ("page_table_dst", z(2, 1)), ("seq_lens_dst", z(1, t=torch.int64))):
        with pytest.raises(ValueError):
            cache.evict(**dict(good, **{name: t}))
    with pytest.raises(binding.MlaError):
        cache.evict(**dict(good, n_first=9))
    d = VerifyDecoder([64], [1], 12, "fp8")
    good = dict(q=z(1, 12, D, t=torch.bfloat16), kv_cache=codes, page_table=z(1, 1), lse=z(1, 12, t=f32), weights=z(1, 64, t=f32))
    for name, t in (("q", z(1, 11, D, t=torch.bfloat16)), ("kv_cache", codes.to(torch.bfloat16)), ("kv_cache", codes[0, :32]),
                    ("lse", z(12, 2, t=f32).t()[:1]), ("weights", z(64, t=f32)), ("page_table", z(1)), ("kv_scales", z(2, 1, t=f32)),
                    ("counted", z(2))):
        with pytest.raises(ValueError):
            d.key_weights(**dict(good, **{name: t}))
    with pytest.raises(binding.MlaError):
        d.key_weights(**dict(good, weights=z(1, 63, t=f32)))
    out = z(1, 12, 512, t=torch.bfloat16)
    with pytest.raises(ValueError):
        d.run(good["q"], codes, z(1, 1), out, kv_scales=z(3, 5, t=f32))
    with pytest.raises(ValueError):
        VerifyDecoder([64], [1], 12, "bf16").run(good["q"], codes.to(torch.bfloat16), z(1, 1), out, kv_scales=scales)


@pytest.mark.parametrize("kind,block", [("bf16", 0), ("e4m3", 32)])
def test_key_weights_of_many_requests(kind, block):
    """More requests than a warp looks at together, several of them in one CTA's share and some
    over several CTAs."""
    g = np.random.default_rng(25)
    seq, q = g.integers(1, 400, size=75), g.integers(1, 4, size=75)
    q = np.minimum(seq, q)
    batch = ref.Batch(20, seq, q, kind, block, seed=25)
    old = g.random((75, 400)).astype(np.float32)
    w, lse = run_weights(batch, 0.5, old)
    want, bound = ref.weights(batch, lse.cpu().double().numpy(), 0.5, old)
    assert (np.abs(w.cpu().double().numpy() - want) <= bound + 1e-30).all()


@pytest.mark.parametrize("kind", ["bf16", "scaled"])
@pytest.mark.parametrize("heads,q", [(4, 2), (96, 3)])
def test_key_weights_long(kind, heads, q):
    """330k keys: more tiles to a CTA than one look-up of page ids holds, one and three groups of
    rows, against 64-bit torch on the GPU."""
    n = 330001
    pages = (n + 63) // 64
    gen = torch.Generator(device="cuda").manual_seed(q)
    x = torch.randn((pages, 64, D), generator=gen, device="cuda")
    table = torch.randperm(pages, generator=gen, device="cuda").int().view(1, -1)
    scales = None
    if kind == "bf16":
        kv = x.to(torch.bfloat16)
        k = kv.double()
    else:
        scales = torch.exp2(torch.randint(-9, -6, (pages, 4), generator=gen, device="cuda").float())
        kv = (x * 100).clamp(-448, 448).to(F8).view(torch.uint8)
        k = kv.view(F8).double() * scales.double().repeat_interleave(16, 1)[:, :, None]
    k = k[table[0].long()].view(-1, D)[:n]
    queries = torch.randn((q, heads, D), generator=gen, device="cuda").to(torch.bfloat16)
    d = VerifyDecoder([n], [q], heads, "bf16" if kind == "bf16" else "fp8")
    lse, w = torch.empty((q, heads), device="cuda"), torch.zeros((1, n), device="cuda")
    bound = torch.zeros(n, dtype=torch.float64, device="cuda")
    want = torch.zeros(n, dtype=torch.float64, device="cuda")
    for i in range(q):
        rows = queries[i].double()
        s = rows @ k[:n - q + i + 1].T * inputs.SM_SCALE
        lse[i] = torch.logsumexp(s, 1)
        p = torch.exp(s - lse[i].double()[:, None])
        err = 576 * 2.0 ** -23 * (rows.abs() @ k[:n - q + i + 1].abs().T)
        if kind != "bf16":
            err += 2.0 ** -17 * rows.abs().amax(1, keepdim=True) * k[:n - q + i + 1].abs().sum(1)
        want[:n - q + i + 1] += p.sum(0)
        bound[:n - q + i + 1] += (p * (inputs.SM_SCALE * err + 2.0 ** -16)).sum(0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    d.key_weights(queries, kv, table, lse, w, kv_scales=scales, status=status)
    assert int(status.item()) == 0
    assert ((w[0].double() - want).abs() <= bound).all()


@pytest.mark.parametrize("n", [20000, 70000])
def test_two_graphs_at_once(n):
    """Graphs of one decoder, captured one after the other and replayed on two streams at the same
    time, share no scratch: the key weights of an e4m3 cache, and an eviction of a request that a
    cluster, or the whole GPU, selects from."""
    batch = ref.Batch(24, [3000, 900], [4, 2], "e4m3", 16, seed=26)
    d, t, _, lse = decode(batch)
    wide = torch.rand((1, n), device="cuda")
    pages = (n + 63) // 64
    kv = torch.zeros((pages + 20, 64, D), dtype=torch.uint8, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").view(1, -1)
    outs, graphs = [], []
    for k in range(2):
        w = torch.zeros((2, 3000), device="cuda")
        kept, lens = torch.zeros((1, 640), dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
        dst = torch.arange(pages + 10 * k, pages + 10 * (k + 1), dtype=torch.int32, device="cuda").view(1, -1)
        q = t["q"] if k == 0 else t["q"].flip(0).contiguous()
        weights = wide if k == 0 else wide.flip(1).contiguous()
        keep = (w, kept, lens, dst, q, weights, torch.full((1,), n, dtype=torch.int32, device="cuda"))

        def step(w=w, kept=kept, lens=lens, dst=dst, q=q, weights=weights, n_dev=keep[-1]):
            d.key_weights(q, t["kv"], t["table"], lse, w, 0.0, kv_scales=t["scales"])
            cache.evict(weights, n_dev, 640, 1, 2, kv, table, kv, dst, kept, lens)

        step()
        torch.cuda.synchronize()
        outs.append((keep, w.clone(), kept.clone()))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for keep, _, _ in outs:
        keep[0].zero_()
        keep[1].zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for keep, w, kept in outs:
        assert torch.equal(keep[0], w) and torch.equal(keep[1], kept)


# ------------------------------------------------------------------------------- evict
def run_evict(batch, weights, budget, first, last, seed=0, max_seq=None, same_cache=True):
    """Evicts into free pages of the batch's own cache (or another one); compares everything."""
    lens = batch.seq_lens
    kept_n = np.minimum(lens, budget)
    per = (kept_n + PAGE - 1) // PAGE
    table_dst = np.zeros((len(lens), max(1, int(per.max(initial=1)))), np.int32)
    pool = list(batch.free) if same_cache else list(np.random.default_rng(seed).permutation(int(per.sum()) + 2))
    for b, k in enumerate(per):
        table_dst[b, :k] = [pool.pop() for _ in range(k)]
    kv = batch.kv.cuda()
    scales = None if batch.scales is None else batch.scales.cuda()
    if same_cache:
        kv_dst, scales_dst = kv, scales
    else:
        kv_dst = torch.zeros((int(per.sum()) + 2, PAGE, D), dtype=kv.dtype, device="cuda")
        scales_dst = None if scales is None else torch.ones((kv_dst.shape[0], scales.shape[1]), device="cuda")
    before = kv_dst.cpu(), None if scales is None else scales_dst.cpu()
    kept = torch.full((len(lens), budget), -7, dtype=torch.int32, device="cuda")
    lens_dst = torch.full((len(lens),), -7, dtype=torch.int32, device="cuda")
    w_dst = torch.full((len(lens), budget + 1), -7.0, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache.evict(dev(weights), dev(lens), budget, first, last, kv, dev(batch.table), kv_dst, dev(table_dst), kept,
                lens_dst, w_dst, scales, scales_dst, max_seq, status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    as_values = (lambda x: x.double().numpy()) if batch.kind == "bf16" else ref.code_values
    values, values_dst = as_values(batch.kv), as_values(before[0])
    s_dst = None if scales is None else before[1].double().numpy()
    want = ref.evict(weights, lens, budget, first, last, values, None if scales is None else batch.scales.double().numpy(),
                     batch.table, values_dst, s_dst, table_dst, batch.block)
    for b, k in enumerate(want):
        row = np.full(budget, -1)
        row[:len(k)] = k
        assert np.array_equal(kept[b].cpu().numpy(), row), b
        assert int(lens_dst[b]) == len(k)
        got_w = w_dst[b].cpu().numpy()
        assert np.array_equal(got_w[:len(k)], weights[b, k], equal_nan=True) and (got_w[len(k):] == -7).all()
    same(kv_dst if batch.kind == "bf16" else kv_dst.view(F8), values_dst)
    if scales is not None:
        same(scales_dst, s_dst)


def evict_batch(seq, kind, block, seed):
    """Free pages for twice the batch; weights heavy-tailed with many zeros and ties."""
    pages = int(((np.asarray(seq) + PAGE - 1) // PAGE).sum())
    batch = ref.Batch(1, seq, np.ones(len(seq)), kind, block, seed=seed, extra_pages=pages, poison=False)
    g = np.random.default_rng(seed)
    w = np.exp(2 * g.standard_normal((len(seq), max(seq) + 5))).astype(np.float32)
    w[g.random(w.shape) < 0.2] = 0.0
    w[g.random(w.shape) < 0.2] = 0.5
    return batch, w


@pytest.mark.parametrize("kind,block", [("bf16", 0), ("e4m3", 0), ("e4m3", 1), ("e4m3", 8), ("e4m3", 64)])
@pytest.mark.parametrize("seq,budget,first,last", [([1], 1, 0, 0), ([500, 64, 65, 333], 64, 4, 8),
                                                   ([300, 1, 100], 100, 0, 100), ([200, 201], 200, 3, 5),
                                                   ([777], 33, 33, 0), ([130], 129, 0, 0)])
def test_evict(seq, budget, first, last, kind, block):
    batch, w = evict_batch(seq, kind, block, seed=budget + block)
    run_evict(batch, w, budget, first, last)
    run_evict(batch, w, budget, first, last, same_cache=False)


@pytest.mark.parametrize("budget", [100, 9000, 39999])
def test_evict_long(budget):
    """Requests that several CTAs select over, beside short ones."""
    batch, w = evict_batch([40000, 900, 17000], "e4m3", 16, seed=budget)
    run_evict(batch, w, budget, 4, 50)


@pytest.mark.parametrize("budget,first,last", [(1, 0, 0), (5000, 7, 100), (90000, 0, 0), (70000, 35000, 35000)])
def test_evict_few_long_requests(budget, first, last):
    """Selection spread over the whole GPU: long requests, one that keeps all, an empty one."""
    batch, w = evict_batch([100001, 3, 70000], "e4m3", 64, seed=budget)
    run_evict(batch, w, budget, first, last)
    w[:] = 0.5  # ties decide everything
    w[:, 1::2] = np.nan
    run_evict(batch, w, budget, first, last)


def test_evict_many_requests():
    g = np.random.default_rng(8)
    batch, w = evict_batch(g.integers(1, 500, size=90), "e4m3", 16, seed=33)
    run_evict(batch, w, 130, 3, 30, same_cache=False)


def test_evict_special_weights():
    """Ties decided by index, negative weights, infinities, NaN as the lowest, -0 as 0."""
    batch, w = evict_batch([600, 600, 600, 600, 600], "bf16", 0, seed=31)
    w[0] = 0.25
    w[1] = -w[1] - 1
    w[2, ::3], w[2, 1::3], w[2, 2::3] = np.inf, -np.inf, np.nan
    w[3] = np.nan
    w[4, ::2], w[4, 1::2] = 0.0, -0.0
    run_evict(batch, w, 350, 5, 20)
    run_evict(batch, w, 150, 0, 0)


def test_evict_empty_and_unfit_lengths():
    """A request without keys, and lengths outside [0, max_seq]."""
    batch, w = evict_batch([300, 200, 100], "e4m3", 64, seed=32)
    kept = torch.full((3, 64), -7, dtype=torch.int32, device="cuda")
    lens_dst = torch.full((3,), -7, dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    kv, scales = batch.kv.cuda(), batch.scales.cuda()
    table_dst = dev(batch.free[:3].reshape(3, 1))
    cache.evict(dev(w), dev(np.array([0, 306, -1], np.int32)), 64, 0, 0, kv, dev(batch.table), kv, table_dst, kept,
                lens_dst, scales=scales, scales_dst=scales, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == binding.MLA_DEVICE_PLAN_MISMATCH
    assert (kept == -1).all() and (lens_dst == 0).all()
    assert torch.equal(kv.cpu(), batch.kv)


# ------------------------------------------------------------------------------- together
@pytest.mark.parametrize("block", [16, 64])
def test_a_server_step(block):
    """Append verify tokens, decode over them, add up the weights, evict, append again and decode
    the shortened cache, as one program runs them, on a stream of its own and then from a graph."""
    heads, q = 12, 4
    past = np.array([250, 64, 131], np.int32)
    seq = past + q
    g = torch.Generator().manual_seed(block)
    budget, first, last = 128, 4, 16
    pages = 5 + 2 + 3
    perm = torch.randperm(pages + 9, generator=g).int()
    table = torch.zeros((3, 5), dtype=torch.int32)
    table[0, :], table[1, :2], table[2, :3] = perm[:5], perm[5:7], perm[7:10]
    table_dst = perm[10:19].view(3, 3)
    codes = torch.zeros((pages + 9, PAGE, D), dtype=torch.uint8, device="cuda")
    scales = torch.ones((pages + 9, PAGE // block), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    prompt = torch.randn((int(past.sum()), D), generator=g).to(torch.bfloat16)
    new = torch.randn((3 * q, D), generator=g).to(torch.bfloat16)
    queries = torch.randn((3 * q, heads, D), generator=g).to(torch.bfloat16)
    new2 = torch.randn((3 * q, D), generator=g).to(torch.bfloat16)
    cu = lambda n: dev(np.concatenate([[0], np.cumsum(n)]).astype(np.int32))  # noqa: E731
    i32 = lambda n: dev(np.asarray(n, np.int32))  # noqa: E731
    seq2 = np.minimum(seq, budget) + q
    d1, d2 = VerifyDecoder(seq, [q] * 3, heads, "fp8"), VerifyDecoder(seq2, [q] * 3, heads, "fp8")
    t = dict(table=table.cuda(), dst=table_dst.cuda(), prompt=prompt.cuda(), new=new.cuda(), new2=new2.cuda(),
             q=queries.cuda(), past=i32(past), seq=i32(seq), seq2=i32(seq2), cu0=cu(past), cu=cu([q] * 3))
    out, lse = torch.empty((3 * q, heads, 512), dtype=torch.bfloat16, device="cuda"), torch.empty((3 * q, heads), device="cuda")
    out2, w = torch.empty_like(out), torch.zeros((3, 260), device="cuda")
    kept, lens_dst = torch.empty((3, budget), dtype=torch.int32, device="cuda"), torch.empty(3, dtype=torch.int32, device="cuda")

    def step(stream=None):
        cache.append(t["prompt"], codes, scales, t["table"], t["past"], t["cu0"], int(past.max()), status, stream)
        cache.append(t["new"], codes, scales, t["table"], t["seq"], t["cu"], q, status, stream)
        d1.run(t["q"], codes, t["table"], out, lse, status=status, stream=stream, kv_scales=scales)
        d1.key_weights(t["q"], codes, t["table"], lse, w, decay=0.0, kv_scales=scales, status=status, stream=stream)
        cache.evict(w, t["seq"], budget, first, last, codes, t["table"], codes, t["dst"], kept, lens_dst, None, scales,
                    scales, max_seq=int(seq.max()), status=status, stream=stream)
        cache.append(t["new2"], codes, scales, t["dst"], t["seq2"], t["cu"], q, status, stream)
        d2.run(t["q"], codes, t["dst"], out2, lse, status=status, stream=stream, kv_scales=scales)

    own = torch.cuda.Stream()
    own.wait_stream(torch.cuda.current_stream())
    step(own)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = [x.clone() for x in (out, out2, w, kept, lens_dst, codes, scales)]
    # against the plain forms: the cache as it now stands, its rows' order from `kept`
    batch = ref.Batch(heads, seq, [q] * 3, "e4m3", block, poison=False)
    batch.q, batch.kv, batch.scales, batch.table = queries, codes.cpu(), scales.cpu(), table.numpy()
    want, bound, _, _ = ref.attend(batch)
    assert (np.abs(out.cpu().double().numpy() - want) <= bound).all()
    for b, n in enumerate(seq):
        assert kept[b].cpu().tolist() == list(ref.keep(w[b].cpu().numpy(), n, budget, first, last)) + [-1] * max(0, budget - n)
    batch.seq_lens, batch.table = seq2, table_dst.numpy()
    want, bound, _, _ = ref.attend(batch)
    assert (np.abs(out2.cpu().double().numpy() - want) <= bound).all()
    # captured, and replayed twice
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(2):
        for x in (out, out2, w, kept, lens_dst):
            x.zero_()
        codes.zero_()
        scales.fill_(1.0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, (out, out2, w, kept, lens_dst, codes, scales)):
            assert torch.equal(a, b)


# ------------------------------------------------------------------------------- passes and turns
@pytest.mark.parametrize("splits", [1, 3])
def test_decode_scaled_scores_that_keep_rising(splits):
    """Every page's scores exceed all before it by octaves, so every tile moves the references."""
    batch = ref.Batch(12, [64 * 30 + 5], [8], "e4m3", 64, spread=0.0, seed=41)
    for t in range(30):
        batch.scales[batch.table[0][t], 0] = 0.04 * (t + 1)
    want, bound, lse, lse_bound = ref.attend(batch)
    _, _, out, got_lse = decode(batch, binding.PlanOptions(force_splits=splits))
    assert (np.abs(got_lse.cpu().double().numpy() - lse) <= lse_bound).all()
    assert (np.abs(out.cpu().double().numpy() - want) <= bound).all()


@pytest.mark.parametrize("kind,block", [("bf16", 0), ("e4m3", 16)])
@pytest.mark.parametrize("heads,q", [(16, 2), (24, 2), (80, 1), (128, 1), (128, 3), (100, 7)])
def test_key_weights_every_group_size(heads, q, kind, block):
    """32, 64, 96 and 128 rows to a group, one group or several, over one to eight tiles a request."""
    seq = [7, 128, 129, 400, 520, 769, 1000, 300]
    batch = ref.Batch(heads, seq, [q] * len(seq), kind, block, seed=heads + q)
    old = np.random.default_rng(2).random((len(seq), max(seq)))
    counted = [q, q, 1, q, 0, q, max(1, q - 1), q]
    w, lse = run_weights(batch, 0.5, old, counted)
    want, bound = ref.weights(batch, lse.cpu().double().numpy(), 0.5, old, counted)
    got = w.cpu().double().numpy()
    for b, n in enumerate(seq):
        assert (np.abs(got[b, :n] - want[b, :n]) <= bound[b, :n] + 1e-30).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("total", [20000, 170000])
def test_key_weights_of_a_batch_are_those_of_its_requests(kind, total):
    """A key's sum is taken in the same order whatever the batch around it: requests alone, in few
    and in many tiles at a time, give the batch's bits. (Caches that fit L2, and that do not.)"""
    n = [total // 8 + 37 * i for i in range(8)]
    heads, q = 48, 8  # three groups of rows
    per = [-(-k // 64) for k in n]
    g = torch.Generator(device="cuda").manual_seed(43)
    kv = torch.randn((sum(per), 64, 576), generator=g, device="cuda").to(torch.bfloat16)
    if kind == "fp8":
        kv = kv.to(torch.float8_e4m3fn)
    pages = torch.randperm(sum(per), generator=g, device="cuda").int()
    table = torch.zeros((8, max(per)), dtype=torch.int32, device="cuda")
    for b in range(8):
        table[b, :per[b]] = pages[sum(per[:b]):sum(per[:b + 1])]
    queries = torch.randn((8 * q, heads, 576), generator=g, device="cuda").to(torch.bfloat16)
    out = torch.empty((8 * q, heads, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((8 * q, heads), device="cuda")
    d = VerifyDecoder(n, [q] * 8, heads, kind)
    d.run(queries, kv, table, out, lse)
    w = torch.zeros((8, max(n)), device="cuda")
    d.key_weights(queries, kv, table, lse, w)
    again = torch.zeros((8, max(n)), device="cuda")
    d.key_weights(queries, kv, table, lse, again)
    assert torch.equal(w, again)
    for b in range(8):
        rows = slice(b * q, b * q + q)
        one = VerifyDecoder([n[b]], [q], heads, kind)
        alone = torch.zeros((1, n[b]), device="cuda")
        one.key_weights(queries[rows], kv, table[b:b + 1], lse[rows], alone)
        assert torch.equal(alone[0], w[b, :n[b]])
        assert abs(w[b].double().sum().item() / (heads * q) - 1) < 1e-4
        assert (w[b, n[b]:] == 0).all()


@pytest.mark.parametrize("kind,block,q", [("bf16", 0, 4), ("e4m3", 16, 4)])
def test_timeouts_with_several_groups_of_rows(kind, block, q):
    """As above with three groups of rows, where pieces of Q pass between the issuing warps."""
    batch = ref.Batch(96, [64 * 20 + 7], [q], kind, block, seed=44)
    _, t, _, lse = decode(batch)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    bad = VerifyDecoder(batch.seq_lens, batch.q_lens, 96, "bf16" if kind == "bf16" else "fp8",
                        options=binding.PlanOptions(force_splits=4, debug_skip_copy=8))
    bad.key_weights(t["q"], t["kv"], t["table"], lse, torch.zeros((1, 1287), device="cuda"), kv_scales=t["scales"],
                    status=status)
    torch.cuda.synchronize()
    assert int(status.item()) & binding.MLA_DEVICE_WAIT_TIMEOUT
    old = np.zeros((1, 1287))
    w, lse = run_weights(batch, 1.0, old)
    want, bound = ref.weights(batch, lse.cpu().double().numpy(), 1.0, old)
    assert (np.abs(w.cpu().double().numpy() - want) <= bound + 1e-30).all()
