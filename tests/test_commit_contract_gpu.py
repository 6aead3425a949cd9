"""Commit of accepted paths where something does not fit: rows on bad pages."""
import pytest
import torch

from mla_speculative_verify_gb300 import binding
from tests.test_tree_ops_gpu import commit_case, run_commit

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
