"""The tree operators without a GPU: refusals (every argument is checked on the host before the CUDA
runtime is touched), the plans for trees, and the plain forms against one another."""
import numpy as np
import pytest
import torch

from mla_speculative_verify_gb300 import binding, cache, tree
from tests import tree_reference as tref
from tests.plan_reader import read_plan

P, Q = 1 << 20, 1 << 34  # device pointers in all their alignments; nothing is read through them
INVALID, UNSUPPORTED, BUFFER, PLAN = (binding.MLA_ERR_INVALID_ARG, binding.MLA_ERR_UNSUPPORTED, binding.MLA_ERR_BUFFER,
                                      binding.MLA_ERR_PLAN)


def call(name, good, change):
    args = dict(good, **change)
    return getattr(binding.load(), name)(*args.values())


MASKS = dict(parents=P, cu_nodes=P, batch=4, total_nodes=100, max_nodes=40, masks=Q, mask_words=2, depths=2 * Q,
             status_dev=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(parents=None), dict(cu_nodes=None), dict(masks=None), dict(parents=P + 2), dict(masks=Q + 1), dict(depths=Q + 2),
    dict(status_dev=P + 3), dict(batch=0), dict(total_nodes=-1), dict(max_nodes=-1), dict(max_nodes=1025, mask_words=33),
    dict(mask_words=1), dict(mask_words=0), dict(masks=P), dict(masks=P - 799), dict(masks=P + 396), dict(depths=P),
    dict(depths=Q + 400)])
def test_masks_refusals(change):
    assert call("mla_tree_masks", MASKS, change) == INVALID
    assert binding.last_error()


def test_masks_of_nothing_is_no_call():
    assert call("mla_tree_masks", MASKS, dict(total_nodes=0, masks=None, parents=None)) == binding.MLA_OK
    assert call("mla_tree_masks", MASKS, dict(max_nodes=0, mask_words=0)) == binding.MLA_OK


VERIFY = dict(logits_dtype=0, target_logits=P, target_stride=1000, draft_logits=2 * Q, draft_stride=1000, vocab=1000,
              tokens=P, parents=P, cu_nodes=P, batch=4, total_nodes=100, max_nodes=40, temperature=P, uniforms=P, noise=P,
              noise_stride=1000, path=3 * Q, out_tokens=4 * Q, path_stride=9, accepted=5 * Q, status_dev=None, stream=None)


@pytest.mark.parametrize("change", [
    dict(logits_dtype=2), dict(logits_dtype=-1), dict(target_logits=None), dict(tokens=None), dict(parents=None),
    dict(cu_nodes=None), dict(path=None), dict(out_tokens=None), dict(accepted=None), dict(uniforms=None), dict(noise=None),
    dict(target_stride=999), dict(draft_stride=999), dict(noise_stride=999), dict(vocab=0), dict(vocab=(1 << 30) + 1),
    dict(batch=0), dict(batch=(1 << 20) + 1), dict(total_nodes=-1), dict(max_nodes=-1), dict(max_nodes=1025),
    dict(path_stride=0), dict(target_logits=P + 1), dict(draft_logits=2 * Q + 1), dict(logits_dtype=1, target_logits=P + 2),
    dict(tokens=P + 2), dict(temperature=P + 1), dict(noise=P + 2), dict(path=3 * Q + 2), dict(accepted=5 * Q + 1),
    dict(status_dev=P + 1), dict(path=P), dict(out_tokens=P + 8), dict(accepted=P - 8), dict(out_tokens=3 * Q + 140),
    dict(accepted=4 * Q), dict(path=2 * Q + 4), dict(out_tokens=P + 199_996)])
def test_verify_refusals(change):
    assert call("mla_tree_verify", VERIFY, change) == INVALID
    assert binding.last_error()


def tree_plan(kv, seq=(900, 64), q=(29, 1), **options):
    opts = binding.PlanOptions(**options) if options else None
    return binding.plan(seq, q, 12, kv, 152, opts, tree=True)[0]


def run_args(plan, **change):
    good = dict(plan_dev=P, plan_host=plan.ctypes.data, plan_bytes=plan.nbytes, q=P, kv_cache=P, kv_scales=P, block_tokens=16,
                page_table=P, page_table_stride=15, num_pages=50, seq_lens=P, q_lens=P, tree_masks=P, mask_words=1,
                sm_scale=0.07, kv_scale=1.0, out=P, lse=P, workspace=P, workspace_bytes=1 << 40, status_dev=None, stream=None)
    return dict(good, **change)


@pytest.mark.parametrize("kv,change,code", [
    (1, dict(tree_masks=None), INVALID), (1, dict(tree_masks=P + 2), INVALID), (1, dict(mask_words=0), INVALID),
    (1, dict(block_tokens=3), UNSUPPORTED), (1, dict(kv_scales=P + 2), INVALID), (0, dict(), INVALID),
    (0, dict(kv_scales=None, q=None), INVALID), (0, dict(kv_scales=None, out=P + 8), INVALID),
    (0, dict(kv_scales=None, sm_scale=float("nan")), INVALID), (1, dict(kv_scales=None, kv_scale=0.0), INVALID),
    (0, dict(kv_scales=None, page_table_stride=14), INVALID), (0, dict(kv_scales=None, workspace=None), BUFFER),
    (0, dict(kv_scales=None, plan_bytes=16), PLAN)])
def test_run_refusals(kv, change, code):
    plan = tree_plan(kv, unit_pages=1)
    assert call("mla_decode_run_tree", run_args(plan), change) == code
    assert binding.last_error()


def test_run_refuses_masks_too_narrow_and_pair_plans():
    plan = tree_plan(0, seq=(900, 64), q=(33, 1))
    assert call("mla_decode_run_tree", run_args(plan, kv_scales=None), {}) == INVALID
    pair, _ = binding.plan([900], [8], 12, 0, 152, binding.PlanOptions(cta_pair=1))
    assert call("mla_decode_run_tree", run_args(pair, kv_scales=None), {}) == UNSUPPORTED


COMMIT = dict(kv_dtype=1, kv_cache=P, kv_scales=P, block_tokens=16, layers=3, page_table=P, page_table_stride=8, num_pages=50,
              seq_lens=P, cu_nodes=P, batch=4, path=P, path_stride=9, accepted=P, seq_lens_dst=Q, status_dev=None, stream=None)


@pytest.mark.parametrize("change,code", [
    (dict(kv_cache=None), INVALID), (dict(page_table=None), INVALID), (dict(seq_lens=None), INVALID),
    (dict(cu_nodes=None), INVALID), (dict(path=None), INVALID), (dict(accepted=None), INVALID),
    (dict(seq_lens_dst=None), INVALID), (dict(kv_cache=P + 8), INVALID), (dict(kv_scales=P + 2), INVALID),
    (dict(path=P + 1), INVALID), (dict(status_dev=P + 2), INVALID), (dict(kv_dtype=2), INVALID), (dict(kv_dtype=0), INVALID),
    (dict(batch=0), INVALID), (dict(layers=0), INVALID), (dict(layers=65536), INVALID), (dict(num_pages=0), INVALID),
    (dict(num_pages=1 << 26), INVALID), (dict(page_table_stride=0), INVALID), (dict(path_stride=0), INVALID),
    (dict(path_stride=1025), INVALID), (dict(block_tokens=0), UNSUPPORTED), (dict(block_tokens=48), UNSUPPORTED),
    (dict(seq_lens_dst=P), INVALID), (dict(seq_lens_dst=P + 12), INVALID), (dict(seq_lens=Q + 12), INVALID),
    (dict(accepted=Q - 12), INVALID), (dict(cu_nodes=Q - 16), INVALID), (dict(path=Q - 140), INVALID)])
def test_commit_refusals(change, code):
    assert call("mla_cache_commit", COMMIT, change) == code
    assert binding.last_error()


def test_tensors_off_the_gpu_are_refused():
    i = torch.zeros(4, dtype=torch.int32)
    for go in (lambda: tree.masks(i, i, i.view(4, 1)),
               lambda: tree.verify(torch.zeros(4, 8), i, i, i, i.view(2, 2), i.view(2, 2), i),
               lambda: cache.commit(torch.zeros((1, 64, 576), dtype=torch.bfloat16), i.view(1, 4), i, i, i.view(1, 4), i, i)):
        with pytest.raises(ValueError, match="CUDA"):
            go()


# ------------------------------------------------------------------------------- plans
@pytest.mark.parametrize("heads,seq,q", [(12, [4096], [29]), (12, [100, 64, 5000], [1, 64, 7]), (128, [700], [13]),
                                         (48, [16384, 9000, 300], [5, 16, 11]), (1, [65], [65]), (33, [5000], [96])])
@pytest.mark.parametrize("kv", [0, 1])
@pytest.mark.parametrize("cap", [0, 48, 128])
def test_tree_plan_covers_every_row_and_key_once(heads, seq, q, kv, cap):
    """Of the planner's choice, in tiles of 48 rows, in tiles of 128."""
    buf, ws = binding.plan(seq, q, heads, kv, 152, binding.PlanOptions(max_rows_per_cta=cap), tree=True)
    pl = read_plan(buf)
    wide = pl["header"]["reserved0"]
    assert wide == {0: wide, 48: 0, 128: 1}[cap]
    rows = np.zeros((sum(q) * heads, max(seq)), np.int32)
    for u in pl["units"]:
        assert u["kv_begin"] % 64 == 0 and 0 < u["nrows"] <= (128 if wide else 48)
        rows[u["qrow0"]:u["qrow0"] + u["nrows"], u["kv_begin"]:u["kv_end"]] += 1
        lo = pl["requests"][u["b"]]["tok0"] * heads
        assert lo <= u["qrow0"] and u["qrow0"] + u["nrows"] <= lo + u["q"] * heads
    at = 0
    for n, k in zip(seq, q):
        assert (rows[at * heads:(at + k) * heads, :n] == 1).all() and (rows[at * heads:(at + k) * heads, n:] == 0).all()
        at += k
    parts = np.zeros(pl["header"]["n_part_rows"], np.int32)
    for m in pl["merges"]:
        parts[m["part_row0"]:m["part_row0"] + m["nrows"] * m["n_splits"]] += 1
    assert (parts == 1).all() and (ws > 0) == (len(parts) > 0)


def test_a_prime_tree_is_cut_into_full_tiles():
    """29 tokens of 12 heads: 348 rows in 8 tiles of 48 or 3 of 128, where the fold rule would make 29 of 12."""
    def rows(cap, tree):
        return sorted(u["nrows"] for u in read_plan(binding.plan([8192], [29], 12, 0, 152, binding.PlanOptions(
            force_splits=1, max_rows_per_cta=cap), tree=tree)[0])["units"])
    assert rows(48, True) == [12] + [48] * 7 and rows(128, True) == [92, 128, 128] == rows(0, True)
    assert rows(0, False) == [12] * 29


def test_few_rows_and_short_contexts_stay_in_narrow_tiles():
    def wide(q, n, kv, tree=True):
        return read_plan(binding.plan([n], [q], 12, kv, 152, tree=tree)[0])["header"]["reserved0"]
    for kv in (0, 1):
        assert [wide(q, 131072, kv) for q in (1, 2, 4, 5, 8, 64)] == [0, 0, 0, 1, 1, 1]
        assert [wide(8, n, kv) for n in (64, 4096, 131072)] == [0, 0, 1]
        assert wide(64, 131072, kv, tree=False) == 0


def test_tree_plan_refusals():
    for options in (dict(force_fold=1), dict(cta_pair=1)):
        with pytest.raises(binding.MlaError) as e:
            tree_plan(0, **options)
        assert e.value.code == INVALID


# ------------------------------------------------------------------------------- the plain forms
@pytest.mark.parametrize("with_draft", [False, True])
def test_the_plain_walk_keeps_the_distribution(with_draft):
    """Siblings drawn from the draft's distribution (or fixed ones taken as certain): the first token
    that comes out is distributed as the target's. 20000 draws of 6 tokens: a frequency is off by
    at most 5 sigma <= 5 sqrt(0.25 / 20000) = 0.018."""
    g = np.random.default_rng(5)
    n, vocab = 20000, 6
    target, draft = g.normal(size=vocab) * 1.2, g.normal(size=vocab) * 1.2
    p, q = tref.softmax(target, 0.8), tref.softmax(draft, 0.8)
    count = np.zeros(vocab)
    for _ in range(n):
        kids = g.choice(vocab, size=3, p=q) if with_draft else np.array([4, 1, 3])
        tokens = np.concatenate([[0], kids])
        _, out, _ = tref.verify([target] * 4, [draft] * 4 if with_draft else None, tokens, [-1, 0, 0, 0], 0.8,
                                g.random(4), g.exponential(size=vocab), 4)
        count[out[0]] += 1
    assert np.abs(count / n - p).max() < 0.018


def test_words_of_a_hand_made_tree():
    w, d = tref.words([[-1, 0, 0, 1, -1, 4]], 1)
    assert w[:, 0].tolist() == [0b1, 0b11, 0b101, 0b1011, 0b10000, 0b110000] and d.tolist() == [0, 1, 1, 2, 0, 1]
