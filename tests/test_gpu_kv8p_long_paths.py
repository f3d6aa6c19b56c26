"""The commit with page scales of paths longer than a draft tree (prompt chunks): every row
arrives, whatever the path's capacity. Codes, scales and lengths equal the oracle's."""

import numpy as np
import pytest
import torch

from test_gpu_kv8p_commit import call, check, put, setup

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("rows,prefix,cap,ps", [
    (1025, 0, 1025, 16), (1041, 0, 1043, 16), (1041, 7, 4096, 16), (2000, 16, 2048, 16), (2048, 5, 2048, 16),
    (8192, 3, 8192, 16), (2048, 33, 2050, 1), (3000, 63, 3000, 64), (40, 9, 20000, 16)])
def test_every_row_of_a_long_path(rows, prefix, cap, ps):
    c = setup([prefix, 40, prefix + 1], [rows - 1, 2, 17], 2, 64, ps, cap=cap, seed=rows)
    t = put(c)
    call(t)
    torch.cuda.synchronize()
    assert int(t["status"].item()) == 0
    check(c, t)


def test_a_long_path_past_its_capacity_is_left():
    """accept_len at path_cap: refused, with nothing of the sequence written."""
    c = setup([5], [1500], 2, seed=1, cap=1600)
    t = put(c)
    t["path"] = t["path"][:, :1500].contiguous()
    call(t)
    torch.cuda.synchronize()
    assert int(t["status"].item()) == -9 and int(t["seq"][0].item()) == -7
    assert np.array_equal(t["k"].cpu().numpy(), c["k"]) and np.array_equal(t["v"].cpu().numpy(), c["v"])
    assert np.array_equal(t["scale"].cpu().numpy(), c["scale"])


def test_rows_past_the_tree_tensors_are_refused():
    """A sequence whose node range ends behind the last row of k_tree and v_tree."""
    c = setup([5, 9], [3, 2], 2, seed=2)
    t = put(c)
    t["qo"][2] += 7
    call(t)
    torch.cuda.synchronize()
    assert int(t["status"].item()) == -9
    assert int(t["seq"][0].item()) == 9 and int(t["seq"][1].item()) == -7
