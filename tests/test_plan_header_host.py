"""What a plan's header has to say of itself before a launch goes by it (caller-held bytes, also those of other builds)."""
import numpy as np
import pytest

from mla_speculative_verify_gb300 import binding
from tests.plan_reader import HEADER

AT = {name: i for i, name in enumerate(HEADER)}
WIDE, TREE = AT["reserved0"], AT["reserved1"]


def refused(buf, changes):
    buf = buf.copy()
    words = buf.view(np.int32)
    for at, value in changes.items():
        words[at] = value
    with pytest.raises(binding.MlaError) as e:
        binding.plan_info(buf)
    return e.value.code == binding.MLA_ERR_PLAN


def narrow(kv):
    return binding.plan([900, 64], [29, 1], 12, kv, 152, binding.PlanOptions(max_rows_per_cta=48), tree=True)[0]


def wide(kv):
    return binding.plan([900, 64], [29, 1], 12, kv, 152, binding.PlanOptions(max_rows_per_cta=128), tree=True)[0]


@pytest.mark.parametrize("version", [5, 0, -1])
def test_plans_of_builds_without_trees_are_refused(version):
    """Version 5 had no tiles of 128 rows and no fp32 partials; its build takes none of this one's plans either, whose
    version differs."""
    for buf in (binding.plan([900], [4], 12, 0, 152)[0], narrow(0), wide(1)):
        assert int(buf.view(np.int32)[AT["version"]]) > 5
        binding.plan_info(buf)
        assert refused(buf, {AT["version"]: version})


@pytest.mark.parametrize("kv", [0, 1])
def test_headers_that_contradict_themselves_are_refused(kv):
    assert refused(wide(kv), {TREE: 0})                # 128-row tiles with room for bf16 partials
    assert refused(wide(kv), {AT["cta_pair"]: 1})      # two kernels at once
    assert refused(wide(kv), {WIDE: 0})                # 128-row tiles for the 48-row kernel
    assert refused(wide(kv), {AT["rows_cap"]: 129})
    assert refused(narrow(kv), {AT["rows_cap"]: 49})
    assert refused(narrow(kv), {AT["rows_cap"]: 0})
    chain = binding.plan([900], [4], 12, kv, 152)[0]
    assert refused(chain, {AT["rows_cap"]: 96}) and refused(chain, {WIDE: 1}) and refused(chain, {TREE: 2})


def test_a_pair_plan_belongs_to_a_bf16_cache():
    pair = binding.plan([900], [8], 12, 0, 152, binding.PlanOptions(cta_pair=1))[0]
    words = pair.view(np.int32)
    assert words[AT["cta_pair"]] == 1 and 48 < words[AT["rows_cap"]] <= 96
    binding.plan_info(pair)
    assert refused(pair, {AT["kv_dtype"]: 1}) and refused(pair, {AT["rows_cap"]: 97})
    assert refused(pair, {TREE: 1})
