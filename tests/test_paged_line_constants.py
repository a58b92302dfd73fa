"""The CPU models of paged attention use the kernel's own numbers, and sizes that
no test can run are shown by the source."""

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


def test_the_appends_check_of_offsets_counts_threads_in_64_bits():
    """2^30 tokens of one head of 32 (keys and values) make 2^24 blocks of 256
    threads: a stride of 2^32, which is 0 in 32 bits and would never end."""
    with open(os.path.join(CSRC, "attn_rope.cu")) as f:
        text = f.read()
    threads = int(re.search(r"constexpr int kThreads = (\d+);", text).group(1))
    rows_a_block = threads // (32 // 16)
    assert 2 * 2 ** 30 // rows_a_block * threads == 2 ** 32
    loop = re.search(r"for \((.*); s < num_seqs; s \+= (.*)\) \{", text)
    assert loop.group(1).startswith("int64_t s = (int64_t)blockIdx.x") and loop.group(2).startswith("(int64_t)gridDim.x")
