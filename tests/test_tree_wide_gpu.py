"""The decode of trees in tiles of 128 rows on clusters of two CTAs, forced with max_rows_per_cta = 128,
against the plain 64-bit forms: rows and pages that do not fill a tile, all caches, splits, masks that leave
rows empty, references that move late, the waits' limits."""
import numpy as np
import pytest
import torch

from mla_speculative_verify_gb300 import binding
from mla_speculative_verify_gb300.decoder import VerifyDecoder
from tests import cache_reference as ref
from tests import tree_reference as tref
from tests.test_tree_ops_gpu import KINDS, check, decode, dev, i32, tref_rows

pytestmark = pytest.mark.gpu


def wide(**kw):
    return binding.PlanOptions(max_rows_per_cta=128, **kw)


SHAPES = [(12, [1], [1]), (1, [64], [3]), (12, [65], [8]), (12, [128], [8]), (12, [129], [11]), (1, [200], [64]), (1, [300], [65]),
          (12, [700], [29]), (33, [129, 64, 300], [1, 33, 20]), (128, [200, 7], [13, 5]), (16, [513, 96], [64, 96])]


@pytest.mark.parametrize("kind,block", KINDS)
@pytest.mark.parametrize("heads,seq,q", SHAPES)
def test_wide_tiles(heads, seq, q, kind, block):
    g = np.random.default_rng(heads + sum(seq))
    batch = ref.Batch(heads, seq, q, kind, block, seed=heads + block)
    masks, _ = tref.words([tref.random_tree(g, n) for n in q], (max(q) + 31) // 32)
    check(batch, masks, *decode(batch, masks, wide()))


@pytest.mark.parametrize("kind,block", KINDS[:4])
@pytest.mark.parametrize("options", [dict(force_splits=3), dict(unit_pages=1), dict(unit_pages=3), dict(force_splits=40)])
def test_wide_splits(kind, block, options):
    """Pieces of odd numbers of pages; pieces in which some rows see nothing."""
    g = np.random.default_rng(7)
    batch = ref.Batch(12, [2700, 90], [40, 70], kind, block, seed=9)
    masks, _ = tref.words([tref.random_tree(g, n) for n in (40, 70)], 3)
    check(batch, masks, *decode(batch, masks, wide(**options)))


@pytest.mark.parametrize("kind,block", KINDS[:4])
@pytest.mark.parametrize("splits", [0, 3])
def test_wide_rows_that_see_nothing(kind, block, splits):
    g = np.random.default_rng(3)
    batch = ref.Batch(12, [1200, 90], [1200, 20], kind, block, seed=4)
    masks = g.integers(-2 ** 31, 2 ** 31, size=(1220, 38), dtype=np.int64).astype(np.int32)
    masks[[0, 1, 63, 64, 700, 1199]] = 0
    masks[5], masks[5, 37] = 0, 1 << 15
    masks[1200:1205] = 0
    out, lse = decode(batch, masks, wide(force_splits=splits))
    pick = np.array([0, 1, 2, 5, 63, 64, 65, 640, 700, 1198, 1199] + list(range(1200, 1220)))
    for t, (o, l, bound, l_bound) in zip(pick, tref_rows(batch, masks, pick)):
        got, got_l = out[t].double().cpu().numpy(), lse[t].double().cpu().numpy()
        assert (np.abs(got - o) <= bound).all(), t
        if np.isneginf(l).all():
            assert np.isneginf(got_l).all() and (got == 0).all(), t
        else:
            assert (np.abs(got_l - l) <= l_bound).all(), t


@pytest.mark.parametrize("kind,block", KINDS[:4])
def test_wide_chain(kind, block):
    """Without masks the tokens are a chain; with a chain's masks every bit is the same; and equal calls
    give equal bits."""
    batch = ref.Batch(12, [700, 64, 3000], [8, 5, 33], kind, block, seed=21)
    masks, _ = tref.words([list(range(-1, n - 1)) for n in (8, 5, 33)], 2)
    a, b, c = decode(batch, masks, wide()), decode(batch, None, wide()), decode(batch, None, wide())
    check(batch, masks, *b)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(c[0], b[0]) and torch.equal(c[1], b[1])


@pytest.mark.parametrize("kind,block", KINDS[:4])
def test_wide_references_that_move(kind, block):
    """Scores that grow along the keys, for some rows only, so that references move in most tiles."""
    batch = ref.Batch(12, [1500], [16], kind, block, seed=31, poison=False)
    grow = torch.linspace(0.05, 4.0, 24 * 64).view(24, 64, 1)
    order = torch.from_numpy(batch.table[0].astype(np.int64))
    if kind == "bf16":
        batch.kv[order] = (batch.kv[order].float() * grow).to(torch.bfloat16)
    else:
        v = batch.kv[order].view(torch.float8_e4m3fn).float() * (grow / 4.0)
        batch.kv[order] = v.to(torch.float8_e4m3fn).view(torch.uint8)
    batch.q[3::4] *= 3.0
    masks, _ = tref.words([tref.random_tree(np.random.default_rng(5), 16)], 1)
    check(batch, masks, *decode(batch, masks, wide()))


def test_wide_is_chosen_for_many_rows():
    for kind in ("bf16", "fp8"):
        assert int(VerifyDecoder([4096], [64], 16, kind, tree=True).plan_host[68:72].view(np.int32)[0]) == 1
        assert int(VerifyDecoder([4096], [2], 12, kind, tree=True).plan_host[68:72].view(np.int32)[0]) == 0
        assert int(VerifyDecoder([4096], [64], 16, kind).plan_host[68:72].view(np.int32)[0]) == 0


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page", [1, 2, 4])
def test_wide_timeout_is_reported(kind, page):
    """A page whose copy is left out: the waits run out, the call ends, the next one is right."""
    batch = ref.Batch(12, [1000], [16], kind, 0, seed=41)
    masks, _ = tref.words([tref.random_tree(np.random.default_rng(6), 16)], 1)
    d = VerifyDecoder([1000], [16], 12, "bf16" if kind == "bf16" else "fp8", tree=True,
                      options=wide(force_splits=1, debug_skip_copy=page))
    out, lse = torch.zeros((16, 12, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((16, 12), device="cuda")
    status = i32([0])
    d.run(batch.q.cuda(), batch.kv.cuda(), dev(batch.table), out, lse, kv_scale=batch.kv_scale, status=status, tree_masks=dev(masks))
    torch.cuda.synchronize()
    assert int(status.item()) == binding.MLA_DEVICE_WAIT_TIMEOUT
    check(batch, masks, *decode(batch, masks, wide()))


def test_wide_bad_page_and_lengths():
    batch = ref.Batch(12, [1000], [16], "bf16", 0, seed=42)
    masks = dev(tref.words([tref.random_tree(np.random.default_rng(6), 16)], 1)[0])
    d = VerifyDecoder([1000], [16], 12, "bf16", tree=True, options=wide())
    out, lse, q, kv = torch.zeros((16, 12, 512), dtype=torch.bfloat16, device="cuda"), torch.zeros((16, 12), device="cuda"), batch.q.cuda(), batch.kv.cuda()
    table = batch.table.copy()
    table[0, 7] = batch.pages
    status = i32([0])
    d.run(q, kv, dev(table), out, lse, status=status, tree_masks=masks)
    torch.cuda.synchronize()
    assert int(status.item()) == binding.MLA_DEVICE_BAD_PAGE
    status.zero_()
    d.run(q, kv, dev(batch.table), out, lse, status=status, tree_masks=masks, seq_lens_dev=i32([999]))
    torch.cuda.synchronize()
    assert int(status.item()) & binding.MLA_DEVICE_PLAN_MISMATCH


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_other_entry_points_take_a_tree_plan(kind):
    """The decode in the library's own scratch, and the key weights: as with a chain's plan."""
    batch = ref.Batch(12, [700, 300], [16, 9], kind, 0, seed=51)
    kv_name = "bf16" if kind == "bf16" else "fp8"
    q, kv, table = batch.q.cuda(), batch.kv.cuda(), dev(batch.table)
    chain, _ = tref.words([list(range(-1, n - 1)) for n in (16, 9)], 1)
    out, lse = decode(batch, chain, wide())
    d = VerifyDecoder(batch.seq_lens, batch.q_lens, 12, kv_name, tree=True, options=wide())
    assert d.workspace_bytes > 0
    o, e, status = torch.zeros_like(out), torch.zeros_like(lse), i32([0])
    binding.run_static_ws(d.plan_dev.data_ptr(), d.plan_host, q.data_ptr(), kv.data_ptr(), table.data_ptr(), table.shape[1],
                          batch.pages, d.seq_lens_dev.data_ptr(), d.q_lens_dev.data_ptr(), 1.0 / 192.0 ** 0.5, batch.kv_scale,
                          o.data_ptr(), e.data_ptr(), status.data_ptr(), torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert int(status.item()) == 0 and torch.equal(o, out) and torch.equal(e, lse)
    plain = VerifyDecoder(batch.seq_lens, batch.q_lens, 12, kv_name)
    w, w2 = torch.zeros((2, 704), device="cuda"), torch.zeros((2, 704), device="cuda")
    d.key_weights(q, kv, table, lse, w, kv_scale=batch.kv_scale)
    plain.key_weights(q, kv, table, lse, w2, kv_scale=batch.kv_scale)
    torch.cuda.synchronize()
    assert torch.equal(w, w2)


def test_a_workspace_too_small_is_refused():
    d = VerifyDecoder([5000], [16], 12, "bf16", tree=True, options=wide())
    d.workspace_bytes -= 256
    with pytest.raises(binding.MlaError) as e:
        d.run(torch.zeros((16, 12, 576), dtype=torch.bfloat16, device="cuda"), torch.zeros((79, 64, 576), dtype=torch.bfloat16, device="cuda"),
              torch.zeros((1, 79), dtype=torch.int32, device="cuda"), torch.zeros((16, 12, 512), dtype=torch.bfloat16, device="cuda"),
              tree_masks=torch.zeros((16, 1), dtype=torch.int32, device="cuda"))
    assert e.value.code == binding.MLA_ERR_BUFFER


def test_wide_offsets_beyond_32_bits():
    """Pages whose bytes lie behind 2^32, in either kernel; the results of the same pages at the front."""
    pages = 62_000  # 4.6 GB
    big = torch.zeros((pages, 64, 576), dtype=torch.bfloat16, device="cuda")
    batch = ref.Batch(12, [400], [16], "bf16", 0, seed=52, poison=False)
    masks, _ = tref.words([tref.random_tree(np.random.default_rng(2), 16)], 1)
    far = np.array([[pages - 1 - int(p) for p in batch.table[0]]], np.int32)
    big[dev(far[0]).long()] = batch.kv.cuda()[dev(batch.table[0]).long()]
    for options in (wide(), None):
        want = decode(batch, masks, options)
        d = VerifyDecoder([400], [16], 12, "bf16", tree=True, options=options)
        out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        d.run(batch.q.cuda(), big, dev(far), out, lse, tree_masks=dev(masks))
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
