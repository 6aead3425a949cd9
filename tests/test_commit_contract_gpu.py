"""Commit of accepted paths where something does not fit: rows on bad pages, requests that verification refused."""
import numpy as np
import pytest
import torch

from mla_speculative_verify_gb300 import binding, cache, tree
from tests.test_tree_ops_gpu import commit_case, dev, i32, run_commit

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [1, 4, 16, 64])
def test_a_block_whose_rows_lie_on_a_bad_page_keeps_its_scale(block):
    """No older row stays in the block and none of its new ones can be read: codes and scale stay."""
    first = 48 if block < 64 else 0  # the accepted rows' first place, at the start of a block
    lens, nodes = [first + 139], [140 if first else 139]
    path = [0] if first else []
    path += [85, 95]  # their rows lie on one page
    batch, kv, scales, _ = commit_case(lens, nodes, 3, "e4m3", block, seed=3)
    batch.table[0, 2 if first else 1] = batch.pages
    got, got_s, new_lens, status = run_commit(batch, kv, scales, lens, nodes, [path])
    assert status == binding.MLA_DEVICE_BAD_PAGE and new_lens == [lens[0] - nodes[0] + len(path)]
    assert torch.equal(got.cpu(), kv) and torch.equal(got_s.cpu(), scales)


def test_a_block_that_one_row_reaches_takes_its_scale():
    """Rows 48 and 49 are to come from 53 and, on a bad page, from 70: the first arrives with its scale, the second keeps its codes."""
    batch, kv, scales, _ = commit_case([87], [40], 2, "e4m3", 4, seed=4)
    page = int(batch.table[0, 0])
    scales[:, page, 12], scales[:, page, 13] = 2.0 ** -9, 2.0 ** -4
    batch.table[0, 1] = batch.pages
    got, got_s, new_lens, status = run_commit(batch, kv, scales, [87], [40], [[0, 6, 23]])
    assert status == binding.MLA_DEVICE_BAD_PAGE and new_lens == [50]
    want, want_s = kv.clone(), scales.clone()
    want[:, page, 48], want_s[:, page, 12] = kv[:, page, 53], 2.0 ** -4
    assert torch.equal(got.cpu(), want) and torch.equal(got_s.cpu(), want_s)


def test_a_request_that_verification_refused_is_kept():
    """Its accepted is 0 although it has nodes: commit leaves its rows and its length, certain root included."""
    lens, nodes = [100, 90, 80, 5], [7, 20, 6, 0]
    batch, kv, scales, _ = commit_case(lens, nodes, 2, "e4m3", 16, seed=9)
    total, vocab, width = sum(nodes), 50, 6
    g = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn((total, vocab), generator=g, device="cuda")
    parents = [p for n in nodes for p in range(-1, n - 1)]
    path, out, accepted = (torch.full(shape, 7, dtype=torch.int32, device="cuda") for shape in ((4, width), (4, width), (4,)))
    status, new_lens, cu = i32([0]), i32([9] * 4), dev(np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32))
    k, s = kv.cuda(), scales.cuda()
    tree.verify(logits, i32([0] * total), i32(parents), cu, path, out, accepted, max_nodes=10, status=status)  # 20 nodes do not fit
    torch.cuda.synchronize()
    assert int(status.item()) == binding.MLA_DEVICE_PLAN_MISMATCH
    acc = accepted.tolist()
    assert acc[1] == 0 and acc[3] == 0 and acc[0] > 0 and acc[2] > 0
    status.zero_()
    cache.commit(k, dev(batch.table), i32(lens), cu, path, accepted, new_lens, s, status)
    torch.cuda.synchronize()
    assert new_lens.tolist() == [93 + acc[0], 90, 74 + acc[2], 5]
    assert int(status.item()) == binding.MLA_DEVICE_PLAN_MISMATCH
    paths = [path[b, :a].tolist() for b, a in enumerate(acc)]
    paths[1] = [0]  # moves nothing
    only = run_commit(batch, kv, scales, lens, nodes, paths)
    assert torch.equal(k, only[0]) and torch.equal(s, only[1])
