"""The attention over page scales with a tree past max_nodes, within the same 64-bit mask word: the
sequence's rows are left, the error is reported, the other sequences are as they were and nothing
is written past the workspace. (Without the refusal such a call writes out of range: 10 sequences,
64 / 8 heads, max_nodes 40 give 3 row tiles, 2 a CTA, so a tree of 60 nodes gives the last CTA a
fourth tile, the next sequence's first or one past the workspace.)"""

import numpy as np
import pytest
import torch

from speculative_decoding_tree_parent_gb300 import binding as B

import serving_cases as S
from test_gpu_kv8p_attention import LSE_TOL, tol

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

GUARD = 1 << 20


def call(d, hkv, max_nodes, max_prefix):
    need = B.spec_workspace_size(B.SPEC_OP_ATTN_KV8P, d.prefix.numel(), d.q.shape[0], max_nodes, d.q.shape[1], hkv, 128,
                                 max_prefix, 0)
    buf = torch.full((max(need, 256) + GUARD,), 0x5A, dtype=torch.uint8, device="cuda")
    B.spec_tree_verify_attn_kv8p(d.q, d.k, d.v, d.scale, d.table, d.prefix, max_prefix, d.kt, d.vt, d.mask, d.qo,
                                 max_nodes, d.out, lse=d.lse, ws=buf[:max(need, 256)], dev_status=d.status)
    torch.cuda.synchronize()
    return need, buf[max(need, 256):]


@pytest.mark.parametrize("max_nodes,size,hq,hkv,batch,longest", [
    (40, 60, 64, 8, 10, 2048),    # two tiles a CTA, an odd count of them, split keys
    (40, 41, 64, 8, 10, 2048),    # within the last tile's rows
    (65, 100, 64, 8, 2, 512), (5, 6, 8, 8, 1, 300), (16, 17, 32, 4, 40, 96), (100, 101, 12, 4, 3, 640)])
@pytest.mark.parametrize("which", [0, -1])
def test_a_tree_past_max_nodes_leaves_its_sequence(max_nodes, size, hq, hkv, batch, longest, which):
    sizes = [max(1, max_nodes - 3 * i) for i in range(batch)]
    sizes[which] = size
    prefixes = [max(0, longest - 7 * i) for i in range(batch)]
    c = S.case(prefixes, sizes, hq, hkv, seed=size)
    words = -(-max_nodes // 64)
    assert words == -(-size // 64) == c.mask.shape[1] // 64 + (c.mask.shape[1] % 64 > 0)
    d = S.device(c)
    need, guard = call(d, hkv, max_nodes, longest)
    assert int(d.status.item()) == -4
    assert (guard == 0x5A).all()
    lo, hi = int(c.qo[which - 1 if which < 0 else which]), int(c.qo[which] if which < 0 else c.qo[which + 1])
    assert hi - lo == size
    assert (d.out[lo:hi] == 7).all() and (d.lse[lo:hi] == 7).all()
    rows = [t for t in range(c.T) if not lo <= t < hi]
    if not rows:
        return
    rng = np.random.default_rng(size)
    picks = [(int(rng.choice(rows)), int(rng.integers(0, hq))) for _ in range(60)]
    ref, lse, A = S.reference(c, picks)
    got = np.stack([d.out[t, h].double().cpu().numpy() for t, h in picks])
    gl = np.array([float(d.lse[t, h]) for t, h in picks])
    assert (np.abs(got - ref) <= tol(ref, A)).all() and np.abs(gl - lse).max() <= LSE_TOL


@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("longest", [64, 2048])
def test_a_batch_of_empty_trees(longest, early):
    """Rows behind the last sequence only: left as they were, and the calls behind it run as ever."""
    c = S.case([longest, 5], [0, 0], 16, 4, seed=3, pad_rows=6)
    d = S.device(c)
    with B.early_reads(early):
        for _ in range(3):
            call(d, 4, 4, longest)
    assert int(d.status.item()) == 0
    assert (d.out == 7).all() and (d.lse == 7).all()
