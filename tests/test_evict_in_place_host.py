"""Evictions whose outputs lie where their inputs do: what is refused before anything is launched."""
import pytest
import torch

from mla_speculative_verify_gb300 import binding

M = 1 << 30  # a device address; nothing is read through any of these
GOOD = dict(weights=M, weights_stride=1000, seq_lens=2 * M, batch=3, max_seq=900, budget=100, n_first=4, n_last=16,
            kv_dtype=binding.MLA_KV_BF16, kv_cache=3 * M, kv_scales=None, block_tokens=0, page_table=4 * M, page_table_stride=15,
            num_pages=60, kv_cache_dst=3 * M, kv_scales_dst=None, page_table_dst=6 * M, page_table_dst_stride=2, num_pages_dst=10,
            kept=7 * M, seq_lens_dst=8 * M, weights_dst=9 * M, weights_dst_stride=100, workspace=None, workspace_bytes=0,
            status_dev=None, stream=None)


def refused(**change):
    """The message of the refusal, or None where the arguments are in order (what comes then, with no
    GPU or one, is not looked at: only calls that are refused get this far on a GPU)."""
    rc = binding.load().mla_cache_evict(*dict(GOOD, **change).values())
    return binding.last_error() if rc == binding.MLA_ERR_INVALID_ARG else None


@pytest.mark.parametrize("change", [
    dict(weights_dst=M), dict(weights_dst=M + 4 * 899), dict(weights_dst=M + 4 * 1899), dict(weights_dst=M + 4 * 2899),
    dict(weights_dst=M + 4 * 950), dict(weights_dst=M - 4 * 99), dict(weights_dst=M - 4, weights_dst_stride=1000),
    dict(weights_dst=M + 4 * 901, weights_dst_stride=1000), dict(weights_dst=M + 4 * 900, weights_dst_stride=999)])
def test_weights_dst_over_weights(change):
    assert "weights_dst must not overlap" in refused(**change)


@pytest.mark.parametrize("shift", [-2, -1, 1, 2])
def test_lengths_that_overlap_shifted(shift):
    assert "seq_lens_dst must be" in refused(seq_lens_dst=2 * M + 4 * shift)


def test_one_page_table():
    assert "page_table_dst is page_table" in refused(page_table_dst=4 * M)


# (These calls would be launched if there were a GPU, on addresses that are none.)
@pytest.mark.skipif(torch.cuda.is_available(), reason="needs a machine without a GPU")
@pytest.mark.parametrize("change", [
    dict(), dict(seq_lens_dst=2 * M), dict(seq_lens_dst=2 * M + 12), dict(seq_lens_dst=2 * M - 12),
    dict(weights_dst=M + 4 * 2900), dict(weights_dst=M - 4 * 300), dict(weights_dst=None),
    dict(weights_dst=M + 4 * 900, weights_dst_stride=1000), dict(weights_dst=M - 4 * 100, weights_dst_stride=1000),
    dict(kv_cache_dst=5 * M, page_table_dst=4 * M)])
def test_what_is_not_refused(change):
    assert refused(**change) is None
