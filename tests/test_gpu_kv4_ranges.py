"""Row ranges (qo_indptr) of the 4-bit cache's reading back that do not rise or leave the rows: each sequence is judged by its
own numbers, those out of range are reported, the others are written."""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_parent_gb300 import binding as B

import kv4_cases as C

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

t = lambda a, dt=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dt)


def read(qo, first, total, hkv=2, pages=50):
    """(k, v, status, wanted k, v with NaN where no sequence writes); all sequences have the same page table."""
    rng = np.random.default_rng(len(qo) + total)
    pool = C.pool(rng, pages, hkv)
    table = np.tile(rng.permutation(pages).astype(np.int32), (len(qo) - 1, 1))
    out = [torch.full((total, hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_kv_read_kv4(t(pool, torch.uint8), t(table), t(np.array(first, np.int32)), t(np.array(qo, np.int32)), *out,
                       dev_status=status)
    torch.cuda.synchronize()
    vals = [oracle.kv4_values(pool, None, w) for w in range(2)]
    want = [np.full((total, hkv, 128), 7.0) for _ in range(2)]
    for b in range(len(qo) - 1):
        if 0 <= qo[b] <= qo[b + 1] <= total and 0 <= first[b] <= 2 ** 31 - 1 - (qo[b + 1] - qo[b]):
            for i in range(qo[b + 1] - qo[b]):
                s = first[b] + i
                for w in range(2):
                    want[w][qo[b] + i] = vals[w][table[b, s // 16], :, s % 16]
    return [x.double().cpu().numpy() for x in out], int(status.item()), want


@pytest.mark.parametrize("qo,first,total", [
    ([-20, 5], [0], 40), ([100, 120], [0], 50), ([0, 64, 16, 48], [0, 3, 16], 64),       # (rows 16 .. 47 twice, the same values)
    ([0, 30, 90, 100, 100], [5, 0, 0, 0], 60), ([-5, 16, 40, 40], [0, 9, -1], 48), ([40, 72, 8, 40], [100, 0, 33], 72),
    ([0, 17, 17, 3], [31, 0, 0], 17), ([0, 20, -2 ** 31, 2 ** 31 - 1], [0, 0, 0], 20), ([0, 10, 20], [2 ** 31 - 1, 5], 20)])
def test_read_of_ranges_that_are_wrong(qo, first, total):
    got, status, want = read(qo, first, total)
    assert status == -9
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


def test_read_of_more_rows_than_there_are():
    """Ranges that rise and fall hold the same rows again and again: more pages than a batch of rising ranges has."""
    qo = [0, 640] * 21
    got, status, want = read(qo, [0] * (len(qo) - 1), 640)
    assert status == -9
    for g, w in zip(got, want):
        assert np.array_equal(g, w)


@pytest.mark.parametrize("batch", [1, 255, 256, 257, 700])
def test_read_of_many_sequences(batch):
    rng = np.random.default_rng(batch)
    counts = rng.integers(0, 4, batch) * rng.integers(0, 12, batch)
    counts[-1] = 5
    qo = np.concatenate([[0], np.cumsum(counts)])
    got, status, want = read([int(x) for x in qo], [int(x) for x in rng.integers(0, 700, batch)], int(qo[-1]) + 3, hkv=1)
    assert status == 0
    for g, w in zip(got, want):
        assert np.array_equal(g, w)
