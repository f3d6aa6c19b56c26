"""The check of the free stack's height before a resize (csrc/page_stack.cuh), compiled for the host:
heights near the ends of 32 bits, where a 32-bit sum with the returned pages wraps (n_free INT_MAX and
one page returned gave INT_MIN, which passed for a stack within the pool). No GPU is used."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_tree_parent_gb300", "csrc")


def test_the_stack_check_against_64_bits(tmp_path):
    from speculative_decoding_tree_parent_gb300 import build

    nvcc = build.nvcc()
    if not nvcc or not (os.path.exists(nvcc) or shutil.which(nvcc)):
        pytest.skip("nvcc not available")
    exe = tmp_path / "page_stack_host_check"
    subprocess.check_call([nvcc, "-std=c++17", "-O2", "-I", CSRC, os.path.join(ROOT, "tests", "page_stack_host_check.cu"),
                           "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert out.returncode == 0 and out.stdout.startswith("ok "), out.stdout


def test_both_kernels_use_it():
    with open(os.path.join(CSRC, "page_table.cu")) as fh:
        src = fh.read()
    assert src.count("page_stack_holds(") == 2 and "<= p.num_pages;" not in src
