"""CPU tests that the helpers' constants of the 4-bit cache are the library's."""

from exact_tiled_attention_19_gb300 import binding as B


def test_slot_bytes():
    for D, slot in B._Q4_SLOT_BYTES.items():
        for page in (8, 64, 4096):
            assert B.attn_paged_q4_block_bytes(page, D) == page * slot
    assert sorted(B._Q4_SLOT_BYTES) == [D for D in range(1, 300) if B.attn_paged_q4_block_bytes(8, D)]


def test_sequences_without_a_workspace():
    most = B._TABLES_NO_SCRATCH
    assert B.attn_paged_tables_workspace_size(most) == 0 < B.attn_paged_tables_workspace_size(most + 1)
