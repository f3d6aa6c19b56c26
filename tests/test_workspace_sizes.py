"""Workspace sizes of sizes that a call refuses are 0, as the header says, and asking does not end
the process (each question is put to a process of its own). No GPU is used."""

import subprocess
import sys

import pytest

ROOT = __file__.rsplit("/tests/", 1)[0]


def ask(op, *sizes):
    code = (f"from speculative_decoding_tree_parent_gb300 import binding as B\n"
            f"print(B.spec_workspace_size(B.{op}, *{sizes}))")
    out = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=120)
    return out.returncode, out.stdout.strip()


#                          batch, total, max_nodes, hq, hkv, d, max_prefix, vocab
@pytest.mark.parametrize("sizes", [
    (1, 64, 64, 1032, 8, 128, 4096, 0), (1, 64, 64, 129, 1, 128, 0, 0), (1, 64, 64, 1 << 20, 1, 128, 4096, 0),
    (1, 64, 1025, 32, 8, 128, 4096, 0), (1, 64, 64, 32, 8, 128, -1, 0), (70000, 64, 1, 8, 8, 128, 64, 0)])
def test_sizes_that_the_page_scale_attention_refuses(sizes):
    assert ask("SPEC_OP_ATTN_KV8P", *sizes) == (0, "0")


def test_the_largest_group_is_answered():
    code, out = ask("SPEC_OP_ATTN_KV8P", 1, 64, 64, 128, 1, 128, 1 << 20, 0)
    assert code == 0 and int(out) > 0
