"""Node ranges (qo_indptr) of the 4-bit attention that do not rise or leave the rows: each sequence is judged by its own numbers,
those out of range are reported, the others are written."""

import numpy as np
import pytest
import torch

from speculative_decoding_tree_parent_gb300 import binding as B

import kv4_cases as C
from test_gpu_kv4_attention import check

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

t = lambda a, dt=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dt)


def test_attention_over_ranges_that_fall():
    """The second sequence of three ends before it begins; the third stands before the first."""
    c = C.case([50, 60], [3, 4], 8, 2, seed=41)
    d = C.device(c)
    ws = torch.zeros(B.spec_workspace_size(B.SPEC_OP_ATTN_KV4, 3, c.T, d.max_nodes, c.hq, c.hkv, C.D, d.max_prefix, 0),
                     dtype=torch.uint8, device="cuda")
    B.spec_tree_verify_attn_kv4(d.q, d.pool, t(c.table[[1, 0, 0]]), t(c.prefix[[1, 0, 0]]), d.max_prefix, d.kt, d.vt, d.mask,
                                t(np.array([3, 7, 0, 3], np.int32)), d.max_nodes, d.out, kv_scale=d.kv_scale, lse=d.lse, ws=ws,
                                dev_status=d.status)
    torch.cuda.synchronize()
    assert int(d.status.item()) == -9
    check(c, d)


def test_attention_over_an_empty_range_past_the_rows():
    c = C.case([50], [3], 8, 2, seed=42)
    d = C.device(c)
    d.qo, d.prefix, d.table = t(np.array([0, 3, 9, 9], np.int32)), t(c.prefix[[0, 0, 0]]), t(c.table[[0, 0, 0]])
    ws = torch.zeros(B.spec_workspace_size(B.SPEC_OP_ATTN_KV4, 3, c.T, d.max_nodes, c.hq, c.hkv, C.D, d.max_prefix, 0),
                     dtype=torch.uint8, device="cuda")
    B.spec_tree_verify_attn_kv4(d.q, d.pool, d.table, d.prefix, d.max_prefix, d.kt, d.vt, d.mask, d.qo, d.max_nodes, d.out,
                                kv_scale=d.kv_scale, lse=d.lse, ws=ws, dev_status=d.status)
    torch.cuda.synchronize()
    assert int(d.status.item()) == -9
    check(c, d)
