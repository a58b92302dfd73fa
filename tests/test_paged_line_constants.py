"""The CPU models of paged attention use the kernel's own numbers."""

import os
import re

from exact_tiled_attention_19_gb300.build_lib import CSRC
from tests import test_paged_line_model, test_paged_protocol_model


def source():
    with open(os.path.join(CSRC, "attn_paged_kernel.cuh")) as f:
        return f.read()


def test_the_line_model_has_the_kernels_unit_cost():
    assert int(re.search(r"constexpr int kUnitCost = (\d+);", source()).group(1)) == test_paged_line_model.UNIT_COST


def test_the_protocol_model_has_the_kernels_stages_and_warps():
    text = source()
    stages = int(re.search(r"static constexpr int STAGES = (\d+) \* GROUPS;", text).group(1))
    warps = int(re.search(r"static constexpr int CONSUMER_WARPS = (\d+) \* GROUPS", text).group(1))
    assert warps == 4
    assert {(s, g) for _, s, g in test_paged_protocol_model.CASES} == {(stages, 1), (2 * stages, 2)}
