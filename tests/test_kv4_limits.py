"""Numbers at the ends of their ranges: calls that the host refuses before a pointer is followed (no GPU is needed)."""

import pytest

from speculative_decoding_tree_parent_gb300 import binding as B

from test_kv4_refusals import UNSUP, _attn, lib  # noqa: F401

MOST = 2 ** 31 - 1


@pytest.mark.parametrize("prefix", [MOST, MOST - 100, MOST - 1023])
def test_attention_refuses_prefixes_whose_blocks_it_cannot_count(lib, prefix):
    assert _attn(lib, max_prefix=prefix, max_pages=1 << 27) == UNSUP
    assert B.spec_workspace_size(B.SPEC_OP_ATTN_KV4, 1, 64, 64, 32, 8, 128, prefix, 0) == 0


def test_attention_counts_the_longest_prefix_it_takes():
    need = B.spec_workspace_size(B.SPEC_OP_ATTN_KV4, 1, 64, 64, 32, 8, 128, MOST - 1024, 0)
    assert need == B.spec_workspace_size(B.SPEC_OP_ATTN_KV4, 1, 64, 64, 32, 8, 128, 1 << 20, 0) > 0
