"""Plans at the ends of what the planner takes: no host memory left."""
import subprocess
import sys

import pytest

from mla_speculative_verify_gb300 import binding

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
