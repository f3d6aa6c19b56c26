"""The tensor-core attention with a tree that passes the row tiles of max_nodes but not its 64-bit
mask word: SPEC_ERR_CAPACITY, the sequence's rows left, nothing written past the workspace, the other
sequences right. (Without the refusal such a call writes out of range: 64 / 8 heads and max_nodes 40
give 3 row tiles, 2 a CTA, so a tree of 60 nodes gives the last CTA a fourth tile, the next sequence
and head's first or one past the workspace.)"""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_parent_gb300 import binding as B
from speculative_decoding_tree_parent_gb300 import workloads as W
from speculative_decoding_tree_parent_gb300.step import DeviceBatch

import attn_tolerance as AT

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

MAX_NODES, FITS, GUARD = 40, 48, 1 << 20   # 3 tiles of 16 nodes


@pytest.mark.parametrize("form", ["mask", "parents", "fp8"])
@pytest.mark.parametrize("prefix", [2048, 64])      # with and without split keys
def test_a_tree_past_the_row_tiles(form, prefix):
    inp = W.generate(W.spec(3, batch=10, prefix=(prefix // 2, prefix), nodes=(38, 62), hq=64, hkv=8, vocab=64,
                            tree="chain", max_depth=64, agree_prob=0.5), seed=prefix)
    sizes = np.diff(inp.qo_indptr)
    assert sizes.max() > FITS and sizes.min() <= FITS and inp.mask_words == 1
    db = DeviceBatch(inp, kv_fp8=form == "fp8")
    db.build_mask()                         # one word a row, as for max_nodes
    need = B.spec_workspace_size(B.SPEC_OP_ATTN, db.B, db.T, MAX_NODES, inp.hq, inp.hkv, inp.d, db.max_prefix)
    buf = torch.full((max(need, 256) + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    ws = buf[:max(need, 256)]
    db.out.fill_(7)
    a = (db.page_table, db.prefix_len, db.max_prefix, db.k_tree, db.v_tree)
    b = (db.qo, MAX_NODES, db.out, db.lse, ws, 0.0, db.status)
    if form == "mask":
        B.spec_tree_verify_attn(db.q, db.k_pool, db.v_pool, *a, db.mask, *b)
    elif form == "parents":
        B.spec_tree_verify_attn_parents(db.q, db.k_pool, db.v_pool, *a, db.parent, *b)
    else:
        B.spec_tree_verify_attn_kv8(db.q, db.k_pool, db.v_pool, db.kv_scale, *a, db.mask, *b)
    torch.cuda.synchronize()
    assert db.device_status() == -4
    assert (buf[max(need, 256):] == 0x5A).all()
    rng = np.random.default_rng(1)
    rows = []
    for s, n in enumerate(sizes):
        lo, hi = int(inp.qo_indptr[s]), int(inp.qo_indptr[s + 1])
        if n > FITS:
            assert (db.out[lo:hi] == 7).all()
        else:
            rows += [(lo + int(rng.integers(0, n)), int(rng.integers(0, inp.hq))) for _ in range(6)] + [(hi - 1, 63)]
    mask, _ = oracle.ancestor_mask_batch(inp.parent, inp.qo_indptr, inp.max_nodes)
    kw = dict(pools=db.kv_codes[:2], kv_scale=db.kv_codes[2]) if form == "fp8" else {}
    ref, _, A = AT.reference(inp, mask, rows, **kw)
    got = np.stack([db.out[t, h].double().cpu().numpy() for t, h in rows])
    AT.check(got, ref, A, form)
