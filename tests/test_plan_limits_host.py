"""Plans at the ends of what the planner takes: no host memory left, counts that pass 32 bits."""
import subprocess
import sys

import pytest

from mla_speculative_verify_gb300 import binding
from tests.plan_reader import read_plan

OUT_OF_MEMORY = """
import resource
from mla_speculative_verify_gb300 import binding
tree = {tree}
binding.plan([4096], [4], 12, 0, 152, tree=tree)
used = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (used + (48 << 20),) * 2)
try:
    binding.plan([1 << 22], [1 << 20], 128, 0, 152, tree=tree)
except binding.MlaError as e:
    print("code", e.code)
binding.plan([4096], [4], 12, 0, 152, tree=tree)
"""


@pytest.mark.parametrize("tree", [False, True])
def test_a_plan_without_host_memory_is_an_error_code(tree):
    """Not an exception that leaves the C entry and ends the process."""
    r = subprocess.run([sys.executable, "-c", OUT_OF_MEMORY.format(tree=tree)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert r.stdout.split() == ["code", str(binding.MLA_ERR_MEMORY)]


@pytest.mark.parametrize("tree", [False, True])
def test_more_partial_rows_than_a_plan_counts_are_refused(tree):
    """2^25 rows in 64 pieces: 2^31 partial rows came out negative, with a workspace of 0 bytes."""
    def rows(splits):
        return binding.plan([1 << 20], [1 << 18], 128, 0, 152, binding.PlanOptions(force_splits=splits, max_rows_per_cta=128 if tree else 0),
                            tree=tree)
    with pytest.raises(binding.MlaError) as e:
        rows(64)
    assert e.value.code == binding.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("ctx", [(1 << 30) + 1, (1 << 31) - 64, (1 << 31) - 1])
def test_contexts_whose_key_counts_pass_32_bits_are_refused(ctx, tree):
    """The pages of 2^31 - 1 keys came out as 0 and its last key as negative."""
    for options in (None, binding.PlanOptions(force_splits=1)):
        with pytest.raises(binding.MlaError) as e:
            binding.plan([100, ctx], [1, 2], 12, 0, 152, options, tree=tree)
        assert e.value.code == binding.MLA_ERR_INVALID_ARG


@pytest.mark.parametrize("tree", [False, True])
def test_the_longest_context_is_planned(tree):
    units = read_plan(binding.plan([1 << 30], [3], 12, 1, 152, tree=tree)[0])["units"]
    spans = sorted((u["kv_begin"], u["kv_end"]) for u in units)
    assert spans[0][0] == 0 and spans[-1][1] == 1 << 30 and all(a[1] == b[0] for a, b in zip(spans, spans[1:]))
