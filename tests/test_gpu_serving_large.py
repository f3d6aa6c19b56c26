"""The serving operators at the sizes where they divide their work another way: attention CTAs
with two row tiles (and, among them, sequences with one), runs of nodes per CTA in the norm and
rotation, several KV heads per CTA in the commit, many CTAs in the page tables. Cases, bounds and
checks are those of the operators' own tests."""

import numpy as np
import pytest
import torch

import serving_cases as S
import test_gpu_kv8p_attention as A
import test_gpu_kv8p_commit as C
import test_gpu_rope_pages as R

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 200, 255, 256, 257, 320, 511, 513, 600]


@pytest.mark.parametrize("hq,hkv,sizes", [
    (16, 4, [1, 70, 33, 32, 64, 65, 2, 31]),      # 32 nodes a tile: one to three tiles
    (64, 8, [40, 16, 17, 1, 15, 33, 5, 64]),      # 16 nodes a tile: up to four
    (24, 4, [43, 21, 22, 1, 20, 44, 5, 63])])     # groups of 6: 21 nodes, rows left over
def test_two_row_tiles_of_a_cta(hq, hkv, sizes):
    n = 40 if hkv == 4 else 24
    c = S.case([EDGES[(3 * i + 1) % len(EDGES)] for i in range(n)], [sizes[i % len(sizes)] for i in range(n)], hq, hkv,
               seed=hq + n)
    A.check(c, A.run(c))


def test_two_row_tiles_give_the_same_bits_again():
    c = S.case([600, 64, 333] * 14, [40, 64, 9] * 14, 16, 4, seed=8)
    one, two = A.run(c), A.run(c)
    assert torch.equal(one.out, two.out) and torch.equal(one.lse, two.lse)


@pytest.mark.parametrize("value", [np.inf, np.nan])
def test_masked_values_with_two_row_tiles(value):
    """Infinities and NaN in the K and V of a node reach the rows that see it and no others."""
    c = S.case([130] * 42, [40] * 42, 16, 4, seed=9)
    clean = A.run(c)
    c.kt[c.qo[:-1] + 39] = value          # the last node of each tree: only its own row sees it
    c.vt[c.qo[:-1] + 39] = value
    d = A.run(c)
    keep = np.setdiff1d(np.arange(int(c.qo[-1])), c.qo[:-1] + 39)
    sees = c.mask[keep, 39]
    assert not sees.any()
    assert torch.equal(d.out[keep], clean.out[keep]) and torch.equal(d.lse[keep], clean.lse[keep])


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("sizes,hq,hkv,d,rot", [
    ([400, 1, 0, 599, 77], 24, 4, 64, 32), ([1] * 700 + [0, 31], 8, 2, 128, 128), ([1500], 3, 1, 80, 48),
    ([333] * 3, 70, 5, 96, 96)])
def test_rope_runs_of_nodes(sizes, hq, hkv, d, rot, dtype, interleaved):
    c = R.build(sizes, [7 * i % 50 for i in range(len(sizes))], hq, hkv, d, rot, dtype, True, seed=d, pad_rows=11, extra=32)
    R.check(c, R.run(c, interleaved), interleaved)


@pytest.mark.parametrize("pow2", [True, False])
@pytest.mark.parametrize("hkv", [5, 8])
def test_commit_several_heads_of_a_cta(hkv, pow2):
    rng = np.random.default_rng(hkv)
    n = 40
    c = C.setup([int(x) for x in rng.integers(0, 40, n)], [int(x) for x in rng.integers(0, 20, n)] , hkv, cap=600, seed=hkv,
                pow2=pow2, grow=4.0)
    t = C.put(c)
    C.call(t)
    torch.cuda.synchronize()
    assert int(t["status"].item()) == 0
    C.check(c, t)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shrink", [False, True])
def test_pages_of_many_ctas(shrink, in_place):
    c = R.pages_case(300, 70, 30000, 16, seed=4, tokens=300, length=700)
    got = R.pages_run(c, shrink, in_place, pad_rows=5)
    assert not R.pages_check(c, got, shrink, pad_rows=5)
