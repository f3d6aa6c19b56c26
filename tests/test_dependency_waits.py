"""Rules of the kernels launched with programmatic stream serialization, read from the sources (no GPU
is used). Such a kernel may start while the one before it runs, so

- only the kernels that the header names may signal early: a later kernel may read the pool, the page
  tables and the tree's inputs before its wait where the caller allows it, and whatever writes those
  must have ended by then."""

import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_tree_parent_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as fh:
        return re.sub(r"//[^\n]*", "", fh.read())


def kernels():
    """{kernel name: (parameter list, body)} of every __global__ function."""
    out = {}
    for f in sorted(os.listdir(CSRC)):
        if not f.endswith(".cu"):
            continue
        src = source(f)
        for m in re.finditer(r"__global__\s+void\b", src):
            at = src.index("{", m.end())
            head = src[m.end():at]
            name = re.findall(r"(\w+)\s*\(", re.sub(r"__\w+__\s*\([^()]*(\([^()]*\))?[^()]*\)", "", head))[0]
            depth, i = 1, at + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(src[i], 0)
                i += 1
            out[name] = (head, src[at:i])
    return out


KERNELS = kernels()


def test_the_sources_are_understood():
    assert {"attn_tc_kernel", "attn_tc_merge_kernel", "attn_kv8p_kernel", "kv_commit_kernel", "kv_commit_kv8p_kernel",
            "page_table_kernel", "page_count_kernel", "qk_norm_rope_kernel", "accept_greedy_kernel",
            "accept_greedy_lazy_kernel", "accept_walk_kernel", "tree_mask_kernel"} <= set(KERNELS)


# who signals early, and the condition it does so under (None: always)
EARLY = {"tree_mask_kernel": None, "attn_tc_kernel": None, "attn_tc_merge_kernel": None, "attn_kv8p_kernel": None,
         "attn_kv8p_merge_kernel": None, "accept_greedy_kernel": "ca.k_tree == nullptr",
         "page_table_kernel": "gridDim.x > 1"}


def test_who_signals_early():
    for name, (_, body) in KERNELS.items():
        calls = re.findall(r"(if \([^;{}]*\)\s*)?\bpdl_trigger\(\);", body)
        if name not in EARLY:
            assert not calls, name
        else:
            cond = EARLY[name]
            assert len(calls) == 1, name
            assert calls[0].strip() == ("" if cond is None else f"if ({cond})"), (name, calls)
    # the page table's second kernel waits before it does anything, and ends the early start there
    body = KERNELS["page_count_kernel"][1]
    assert body.index("pdl_wait()") < body.index("ld(")


# launched in plain stream order (<<< >>>): they start when every kernel before them has ended
PLAIN = {"tree_mask_kernel", "attn_simt_kernel", "attn_combine_kernel"}
# the conditions under which a kernel may put its first wait off: the caller's early reads, and the
# commit that the acceptance launches behind itself
DEFERRED = {"if (!p.early)", "if (!p.early_reads)", "if (!early)", "if (!behind_accept)"}
LOAD = re.compile(r"\b(?:__ld\w+|ld)\(|prefetch\.global")


def waiting():
    return sorted(n for n in KERNELS if n not in PLAIN)


def test_kernels_in_plain_stream_order():
    for name in PLAIN:
        assert "pdl_wait" not in KERNELS[name][1]
        for f in os.listdir(CSRC):
            assert not re.search(r"launch_pdl\(\s*" + name, source(f)) if f.endswith(".cu") else True


@pytest.mark.parametrize("name", waiting())
def test_nothing_is_read_before_the_wait(name):
    body = KERNELS[name][1]
    at = body.find("pdl_wait();")
    assert at >= 0, "never waits"
    first = LOAD.search(body)
    assert first is None or at < first.start()
    cond = re.search(r"(if \([^;{}]*\))\s*$", body[:at])
    assert cond is None or cond.group(1) in DEFERRED


@pytest.mark.parametrize("name", ["attn_tc_kernel", "attn_kv8p_kernel", "attn_tc_merge_kernel"])
def test_a_grid_without_rows_still_waits(name):
    """With early reads every CTA of a batch of empty trees leaves at its sizes: the first one has to
    wait all the same, or the grid ends before its predecessor, and the next kernel's wait with it."""
    body = KERNELS[name][1]
    assert re.search(r"if \((\([^;{}]*\) == 0|idx == 0)\) pdl_wait\(\);", body)


@pytest.mark.parametrize("name", waiting())
def test_loads_are_plain(name):
    """__ldg and const __restrict__ promise that a value does not change while the kernel runs, which
    lets a load be moved ahead of the wait: not for what the kernel before may write."""
    head, body = KERNELS[name]
    assert "__ldg" not in body and "__restrict__" not in head


def test_loads_in_the_functions_they_call_are_plain():
    for f in os.listdir(CSRC):
        src = source(f)
        if "pdl_wait()" in src and f != "common.cuh":
            assert "__ldg" not in src and "__restrict__" not in src, f
    # (the one function of the shared header that uses it serves kernels in plain stream order)
    users = [f for f in os.listdir(CSRC) if re.search(r"\bseq_of_row\(", source(f)) and f != "common.cuh"]
    assert "__ldg" not in re.sub(r"int seq_of_row\(.*?\n}", "", source("common.cuh"), flags=re.S)
    assert all("pdl_wait()" not in source(f) for f in users)


@pytest.mark.parametrize("name", ["attn_tc_kernel", "attn_kv8p_kernel"])
def test_errors_are_reported_after_the_wait(name):
    """With early reads the attention runs ahead of its wait, and the status word is something that
    it writes."""
    body = KERNELS[name][1]
    assert not re.search(r"\breport\(", body) and "report_waited(p.status, SPEC_ERR_PAGE)" in body
