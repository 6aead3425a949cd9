"""Key weights after the decode of a tree: on the committed chain, with the accepted nodes' rows of q
and lse; refused with the lse of a run that took masks."""
import numpy as np
import pytest
import torch

from mla_speculative_verify_gb300 import cache
from mla_speculative_verify_gb300.decoder import VerifyDecoder
from tests import cache_reference as ref
from tests import tree_reference as tref
from tests.test_tree_ops_gpu import cu_of, dev, i32

pytestmark = pytest.mark.gpu

HEADS, LENS, NODES = 12, [300, 77, 130], [29, 13, 1]


def tree_run(kind, seed):
    """A decoded batch of trees, with the rows of one root-to-leaf path of each."""
    batch = ref.Batch(HEADS, LENS, NODES, kind, 0, seed=seed)
    r = np.random.default_rng(seed)
    trees = [tref.random_tree(r, n) for n in NODES]
    paths = [tref.lines(t)[-1] for t in trees]
    assert len(paths[0]) > 2 and paths[0] != list(range(len(paths[0])))
    masks = dev(tref.words(trees, 1)[0])
    d = VerifyDecoder(LENS, NODES, HEADS, "bf16" if kind == "bf16" else "fp8", tree=True)
    q, kv, table = batch.q.cuda(), batch.kv.cuda(), dev(batch.table)
    out = torch.empty((sum(NODES), HEADS, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((sum(NODES), HEADS), device="cuda")
    d.run(q, kv, table, out, lse, kv_scale=batch.kv_scale, tree_masks=masks)
    return batch, trees, paths, d, q, kv, table, out, lse


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_the_lse_of_a_tree_is_refused(kind):
    batch, trees, _, d, q, kv, table, out, lse = tree_run(kind, 1)
    w = torch.zeros((3, 320), device="cuda")
    with pytest.raises(ValueError, match="tree"):
        d.key_weights(q, kv, table, lse, w, kv_scale=batch.kv_scale)
    assert not w.any()
    d.run(q, kv, table, out, lse, kv_scale=batch.kv_scale)  # the same tokens as a chain
    d.key_weights(q, kv, table, lse, w, kv_scale=batch.kv_scale)
    want, bound = ref.weights(batch, lse.cpu().double().numpy(), 1.0, np.zeros((3, 320)))
    assert (np.abs(w.cpu().double().numpy() - want) <= bound).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_the_committed_chain_takes_the_rows_of_the_tree(kind):
    """After the commit an accepted node sees what it saw in the tree, so its lse holds, and no second decode is
    needed. A weight is off by its sum's bound, and by the lse's bound of each row relative to that row's weight."""
    batch, trees, paths, _, q, kv, table, _, lse = tree_run(kind, 2)
    acc = [len(p) for p in paths]
    path = torch.full((3, max(acc)), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p)
    new_lens, cu = i32([0] * 3), dev(cu_of(NODES))
    cache.commit(kv, table, i32(LENS), cu, path.cuda(), i32(acc), new_lens)
    rows = [int(cu_of(NODES)[b]) + i for b, p in enumerate(paths) for i in p]
    lens = new_lens.tolist()
    assert lens == [n - k + a for n, k, a in zip(LENS, NODES, acc)]
    chain = VerifyDecoder(lens, acc, HEADS, "bf16" if kind == "bf16" else "fp8")
    w = torch.zeros((3, 320), device="cuda")
    chain.key_weights(q[rows].contiguous(), kv, table, lse[rows].contiguous(), w, kv_scale=batch.kv_scale)
    torch.cuda.synchronize()
    batch.seq_lens, batch.q_lens = np.asarray(lens, np.int32), np.asarray(acc, np.int32)
    batch.kv, batch.q = kv.cpu(), q[rows].cpu()
    _, _, exact, lse_bound = ref.attend(batch)
    assert (np.abs(lse[rows].cpu().double().numpy() - exact) <= lse_bound).all()
    want, bound = ref.weights(batch, exact, 1.0, np.zeros((3, 320)))
    at = np.concatenate([[0], np.cumsum(acc)])
    for b in range(3):  # exp(x) - 1 <= 1.01 x for the bounds' sizes, below 0.01
        bound[b] += 1.01 * lse_bound[at[b]:at[b + 1]].max() * want[b]
    got = w.cpu().double().numpy()
    assert lse_bound.max() < 0.01 and (np.abs(got - want) <= bound).all()
    assert np.allclose(got.sum(1), np.asarray(acc) * HEADS, rtol=1e-4)
