"""A free stack whose height is out of range, up to the ends of 32 bits: nothing moves (the check
itself is tested on the host, tests/test_page_stack_host.py)."""

import numpy as np
import pytest
import torch

from test_gpu_rope_pages import pages_case, pages_run

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


@pytest.mark.parametrize("tokens", [20, 4000])     # one CTA, several
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("n", [2 ** 31 - 1, 2 ** 31 - 4, -2 ** 31, -1, 2001])
def test_a_height_out_of_range_moves_nothing(n, in_place, tokens):
    c = pages_case(8, 300, 2000, 16, seed=5, tokens=tokens)
    c["held"][0] += 1                                # at least one page comes back
    c["lens"][0], c["n"] = 0, n
    table, held, free, n_out, slots = pages_run(c, True, in_place, status=-4)
    assert np.array_equal(table.cpu().numpy(), c["table"]) and np.array_equal(held.cpu().numpy(), c["held"])
    assert np.array_equal(free.cpu().numpy(), c["free"]) and n_out == n
