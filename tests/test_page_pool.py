"""The page-scaled pool that a batch is built with: scales are powers of two that hold the
page's values, codes are within half a step of them."""

import numpy as np
import pytest

import oracle
from speculative_decoding_tree_parent_gb300 import workloads as W
from speculative_decoding_tree_parent_gb300.step import DeviceBatch


def test_page_pool_holds_the_values():
    inp = W.generate_index(3, batch=2, hq=4, hkv=2, vocab=64, prefix=(20, 70), tree="random", nodes=(5, 5), max_depth=3)
    k, v, scale = W.fp8_page_pool(inp)
    assert scale.shape == (inp.num_pages, inp.hkv, 2) and np.array_equal(np.exp2(np.log2(scale).round()), scale)
    for which, (codes, pool) in enumerate(((k, inp.k_pool), (v, inp.v_pool))):
        x = np.asarray(pool, np.float64)
        s = scale[:, :, which, None, None].astype(np.float64)
        assert (np.abs(x) <= 448 * s).all()
        # e4m3: half a step is 2^-4 of the value, or 2^-10 of the scale below its smallest normal
        err = np.abs(oracle.kv8p_values(codes, scale, which) - x)
        assert (err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s)).all()


def test_device_batch_refuses_other_forms():
    with pytest.raises(ValueError, match="page"):
        DeviceBatch(None, kv_fp8="row")
