"""The attention over an E4M3 cache with page scales, against the fp64 oracle.

Bound of an output element, with p_k the exact softmax weights, A = sum_k p_k |v_k| and o the
exact output (half a step of a rounding: fp16 2^-11, bf16 2^-8 of the value):
- a key's weight is rounded to fp16 once (prefix), or to two bf16 terms (tree, 2^-16), before
  it meets V, while the row sum adds the unrounded ones: at most 2^-11 A. (Weights more than
  2^25 below the row's largest are fp16 subnormals; each is off by at most 2^-36 of the
  largest, together below 2^-20 A at these lengths.)
- q is split into two E4M3 terms: a row's elements within 2^10 of its largest are exact, the
  others off by at most 2^-18 of the largest. K's codes enter as they are. So a score s moves
  by at most 2^-18 max|q| sum|k| scale for them plus fp32 accumulation, 2^-20 sum|q_i k_i|
  scale; with N(0, 1) q and codes that is below 2^-13 in these tests, and a weight moves by as
  much of itself, numerator and row sum alike: 2^-12 A at most.
- partial sums stay fp32; the output is rounded to bf16: 2^-8 |o|.
So |gpu - oracle| <= 2^-10 A + 2^-8 |o|, and |lse - oracle| <= 2^-12.
"""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_parent_gb300 import binding as B

import serving_cases as S

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

LSE_TOL = 2.0 ** -12


def tol(ref, A):
    return 2.0 ** -10 * A + 2.0 ** -8 * np.abs(ref) + 1e-9


def workspace(d, hkv):
    n = B.spec_workspace_size(B.SPEC_OP_ATTN_KV8P, d.prefix.numel(), d.q.shape[0], d.max_nodes, d.q.shape[1], hkv, 128,
                              d.max_prefix, 0)
    return torch.full((max(n, 256),), 0xFF, dtype=torch.uint8, device="cuda")    # (fp32 NaN everywhere)


def call(d, ws=None, stream=None, lse=True, **kw):
    ws = workspace(d, d.k.shape[1]) if ws is None else ws
    B.spec_tree_verify_attn_kv8p(d.q, d.k, d.v, d.scale, d.table, d.prefix, d.max_prefix, d.kt, d.vt, d.mask, d.qo,
                                 d.max_nodes, d.out, lse=d.lse if lse else None, ws=ws, dev_status=d.status,
                                 stream=stream, **kw)
    return ws


def run(c, status=0, **kw):
    d = S.device(c)
    d.ws = call(d, **kw)
    torch.cuda.synchronize()
    assert int(d.status.item()) == status
    return d


def check(c, d, rows=None):
    ref, lse, A = S.reference(c, rows)
    n = int(c.qo[-1])
    got, gl = d.out[:n].double().cpu().numpy(), d.lse[:n].double().cpu().numpy()
    if rows is not None:
        got, gl = np.stack([got[t, h] for t, h in rows]), np.array([gl[t, h] for t, h in rows])
    assert np.isfinite(got).all()
    over = np.abs(got - ref) - tol(ref, A)
    assert over.max() <= 0, (float(over.max()), float(np.abs(got - ref).max()))
    assert np.abs(gl - lse).max() <= LSE_TOL
    return ref, A


LENGTHS = [
    # prefixes, tree sizes, hq, hkv
    ([0], [1], 8, 8), ([1], [1], 32, 8), ([15, 16, 17], [1, 1, 1], 8, 2), ([127, 128, 129, 0], [1, 1, 1, 1], 32, 8),
    ([255, 256, 257], [2, 63, 64], 4, 1), ([31, 1], [65, 1], 16, 4), ([1000], [64], 32, 8), ([517], [130], 8, 1),
    ([0, 0], [200, 3], 8, 8), ([2049, 64, 640], [33, 31, 129], 64, 8), ([777], [1], 128, 1), ([300, 5], [7, 64], 16, 1),
    ([4096], [64], 32, 8), ([90], [1024], 2, 1), ([4099, 13], [128, 100], 16, 2),
]


@pytest.mark.parametrize("prefixes,sizes,hq,hkv", LENGTHS)
def test_lengths(prefixes, sizes, hq, hkv):
    c = S.case(prefixes, sizes, hq, hkv, seed=len(prefixes) + sum(sizes))
    check(c, run(c))


@pytest.mark.parametrize("group", [1, 2, 3, 5, 6, 7, 12, 24, 40, 96, 128])
def test_group_sizes(group):
    c = S.case([160, 37], [9, 21], 2 * group, 2, seed=group)
    check(c, run(c))


@pytest.mark.parametrize("nodes", [1, 64])
def test_many_sequences(nodes):
    """More work items than SMs, unequal lengths."""
    rng = np.random.default_rng(nodes)
    n = 40
    prefixes = [int(x) for x in rng.integers(0, 700, n)]
    c = S.case(prefixes, [int(x) for x in rng.integers(1, nodes + 1, n)], 32, 8, seed=9)
    rows = [(int(rng.integers(0, c.T)), int(rng.integers(0, 32))) for _ in range(200)]
    check(c, run(c), rows)


def test_long_prefix():
    c = S.case([20011], [128], 16, 2, seed=3, q_scale=2.0, spread=0.5)
    rows = [(t, h) for t in (0, 63, 64, 127) for h in (0, 7, 8, 15)]
    check(c, run(c), rows)


def test_a_wrong_share_of_the_prefix_is_seen():
    """The bound rejects a zeroed output and one without the last eighth of the prefix."""
    c = S.case([1000], [64], 32, 8, seed=1)
    ref, A = check(c, run(c))
    assert (np.abs(ref) > tol(ref, A)).any()
    c.prefix = np.array([875], np.int32)
    short, _, _ = S.reference(c)
    assert (np.abs(short - ref) > tol(ref, A)).any()


def test_sequences_without_nodes_and_rows_behind_the_last():
    c = S.case([40, 100, 64], [5, 0, 3], 16, 4, seed=2, pad_rows=6)
    d = run(c)
    check(c, d)
    n = int(c.qo[-1])
    assert (d.out[n:] == 7).all() and (d.lse[n:] == 7).all()


def test_rows_that_see_nothing():
    """Mask rows of zeros: over an empty prefix the output is 0 and lse -inf; over a prefix the
    row attends to the prefix alone."""
    c = S.case([0, 50], [6, 6], 8, 2, seed=4)
    c.mask[[1, 4, 8]] = False
    d = run(c)
    out, lse = d.out.double().cpu().numpy(), d.lse.double().cpu().numpy()
    for t in (1, 4):
        assert (out[t] == 0).all() and np.isneginf(lse[t]).all()
    ref, rl, A = S.reference(c, [(t, h) for t in (0, 2, 8, 11) for h in range(8)])
    got = np.stack([out[t, h] for t in (0, 2, 8, 11) for h in range(8)])
    assert (np.abs(got - ref) <= tol(ref, A)).all()


@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
def test_what_a_row_may_not_see_does_not_reach_it(value):
    """Node 3's K and V, and the next sequence's, hold infinities or NaN: rows whose mask
    leaves node 3 out are as without it. (The case's cache rows past the prefix are NaN codes.)"""
    c = S.case([100, 30], [20, 9], 16, 4, seed=5)
    clean = run(c).out.clone()
    c.kt[3], c.vt[3] = value, value
    c.kt[20:], c.vt[20:] = value, value
    d = run(c)
    unseen = [t for t in range(20) if not c.mask[t, 3]]
    assert 5 < len(unseen) < 20
    assert torch.equal(d.out[unseen], clean[unseen])
    seen = [t for t in range(20) if c.mask[t, 3]]
    assert not torch.isfinite(d.out[seen].float()).all()


@pytest.mark.parametrize("which", ["k", "v"])
def test_a_nan_code_in_the_prefix_is_seen(which):
    c = S.case([64], [3], 4, 1, seed=6)
    getattr(c, which)[c.table[0, 2], 0, 5, 17] = 0x7F
    d = run(c)
    hit = d.out[:, :, 17] if which == "v" else d.out[:, :, 0]
    assert torch.isnan(hit.float()).all()


def test_scales_far_apart_and_zero_pages():
    """Page scales from 2^-50 (a page of zeros) to 2^10, with a row sum that has to count the
    zero page's keys in full."""
    c = S.case([160], [4], 8, 2, seed=7)
    c.scale[c.table[0, 3]] = 2.0 ** -50
    c.k[c.table[0, 3]] = 0
    c.v[c.table[0, 3]] = 0
    c.scale[c.table[0, 5], :, 1] = 2.0 ** 10
    check(c, run(c))
    c.v[c.table[0, 5]] = 0       # only small values are left beside a large scale
    check(c, run(c))


def test_scales_outside_the_range_are_read_clamped():
    c = S.case([48], [2], 4, 1, seed=8)
    c.scale[c.table[0, 1], :, 1] = [0.0]
    d = run(c)
    c.scale[c.table[0, 1], :, 1] = 2.0 ** -50
    check(c, d)


@pytest.mark.parametrize("gap", [8.0, 14.0, 17.0])
def test_a_key_that_takes_nearly_all_weight(gap):
    """The first key's score lies `gap` above the others and its value is zero, so the output
    is the other keys' small share: it has to keep its precision."""
    c = S.case([1500], [1], 4, 1, seed=11, spread=0.0)
    c.q[:] = S.bf16(c.q * 0.25)
    dec = lambda code: oracle.e4m3_decode(code)
    page = c.table[0, 0]
    c.q[:, :, 0] = 4.0
    c.k[:, :, :, 0] = 0
    s = c.scale[page, 0, 0]
    want = gap * np.sqrt(128.0) / 4.0 / s
    c.k[page, 0, 0, :] = 0
    c.scale[page, 0, 0] = np.float32(s * max(1.0, want / 400.0))
    c.k[page, 0, 0, 0] = oracle.e4m3_encode(np.float32(gap * np.sqrt(128.0) / 4.0 / c.scale[page, 0, 0]))
    assert dec(c.k[page, 0, 0, 0]) > 0
    c.v[page, 0, 0, :] = 0
    c.kt[:, :, 0] = 0
    check(c, run(c))


def test_q_of_every_size():
    """Rows of q far apart in size, elements of a row far apart, and a row of zeros."""
    c = S.case([100], [6], 4, 1, seed=12)
    rng = np.random.default_rng(0)
    c.q[0] *= 2.0 ** -100
    c.q[1] *= 2.0 ** -8
    c.q[2] = 0
    c.q[3] = S.bf16(c.q[3] * 2.0 ** rng.uniform(-20, 0, c.q[3].shape))
    c.q[4, :, 1:] *= 2.0 ** -9
    check(c, run(c))


def test_bad_page_reads_as_zeros_and_is_reported():
    c = S.case([80, 20], [3, 2], 8, 2, seed=13)
    c.table[0, 2] = c.pages
    d = run(c, status=-3)
    c.k = np.concatenate([c.k, np.zeros_like(c.k[:1])])
    c.v = np.concatenate([c.v, np.zeros_like(c.v[:1])])
    c.scale = np.concatenate([c.scale, np.ones_like(c.scale[:1])])
    check(c, d)


def test_a_prefix_past_its_row_leaves_the_sequence():
    c = S.case([48, 20], [3, 2], 8, 2, seed=14)
    d = S.device(c)
    d.prefix[0] = 16 * c.table.shape[1] + 1
    call(d)
    torch.cuda.synchronize()
    assert int(d.status.item()) == -4
    assert (d.out[:3] == 7).all() and not (d.out[3:] == 7).all()


def test_sm_scale_and_no_lse():
    c = S.case([70], [5], 8, 2, seed=15)
    d = run(c, sm_scale=0.05, lse=False)
    c.q = c.q * np.float32(0.05 * np.sqrt(128.0))
    ref, _, A = S.reference(c)
    got = d.out.double().cpu().numpy()
    assert (np.abs(got - ref) <= tol(ref, A) + 2.0 ** -20 * A).all()
    assert (d.lse == 7).all()


def test_same_bits_again_on_another_stream_and_in_a_graph():
    """The same call twice, on another stream, and captured in two graphs that share one
    workspace, replayed in turn: the same bits."""
    c, c2 = S.case([1000, 40], [64, 9], 32, 8, seed=16), S.case([333], [17], 32, 8, seed=17)
    d, d2 = run(c), run(c2)
    want, want2 = d.out.clone(), d2.out.clone()
    side = torch.cuda.Stream()
    ws = d.ws if d.ws.numel() >= d2.ws.numel() else d2.ws
    graphs = []
    for x in (d, d2):
        x.out.zero_()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call(x, ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(x, ws)
        graphs.append(g)
    assert torch.equal(d.out, want) and torch.equal(d2.out, want2)
    for _ in range(3):
        for g, x, w in zip(graphs, (d, d2), (want, want2)):
            x.out.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(x.out, w)


def test_two_calls_at_once():
    """Two calls in flight on two streams, each with its workspace."""
    cs = [S.case([900], [64], 32, 8, seed=18), S.case([1200, 7], [1, 30], 32, 8, seed=19)]
    ds = [S.device(c) for c in cs]
    ws = [workspace(d, 8) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    for _ in range(5):
        for d, w, s in zip(ds, ws, streams):
            call(d, w, stream=s)
    torch.cuda.synchronize()
    for c, d in zip(cs, ds):
        check(c, d)


def test_early_reads_give_the_same_bits():
    c = S.case([700], [64], 32, 8, seed=20)
    want = run(c).out
    with B.early_reads(True):
        assert torch.equal(run(c).out, want)
