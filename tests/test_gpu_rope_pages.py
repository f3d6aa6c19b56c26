"""Norm + rotation and the page-table resize against the oracle.

Rotation bound, per element: fp32 throughout, one rounding to the output's type. Before it an
element carries at most: the norm's factor (sum of d squares, a mean, rsqrtf with 2 ulp, two
products: below (d / 2 + 8) 2^-24 of itself), and in a pair three roundings of the larger of
its terms. So |gpu - oracle| <= half a step of the output type * |y| + (d / 2 + 12) 2^-24 *
(|u| + |v|), u and v the pair's normed inputs.
"""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_parent_gb300 import binding as B
from speculative_decoding_tree_parent_gb300 import workloads as W

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


def table(reach, rot):
    ang = np.arange(reach)[:, None] * 10000.0 ** (-np.arange(rot // 2) / (rot // 2))[None]
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def build(sizes, prefixes, hq, hkv, d, rot, dtype, norm, seed, pad_rows=0, extra=0):
    rng = np.random.default_rng(seed)
    qo = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    T = int(qo[-1]) + pad_rows
    heads = hq + 2 * hkv
    rnd = W.round_to_bf16 if dtype == torch.bfloat16 else (lambda x: x)
    x = rnd((rng.standard_normal((T, heads * d + extra)) * 3).astype(np.float32))
    depth = np.concatenate([[0 if i == 0 else int(rng.integers(1, i + 1)) for i in range(n)] for n in sizes if n]
                           + [[0] * pad_rows]).astype(np.int32)
    w = [rnd((1 + 0.3 * rng.standard_normal(d)).astype(np.float32)) if norm else None for _ in range(2)]
    tab = table(max(prefixes) + max(sizes) + 1, rot) if rot else None
    return dict(x=x, qo=qo, prefix=np.array(prefixes, np.int32), depth=depth, w=w, tab=tab, T=T, hq=hq, hkv=hkv, d=d,
                dtype=dtype, rot=rot)


def views(c):
    x = torch.from_numpy(c["x"]).to("cuda", c["dtype"])
    n, d = c["hq"] * c["d"], c["d"]
    m = c["hkv"] * d
    part = lambda lo, h: x[:, lo:lo + h * d].unflatten(1, (h, d))
    return x, part(0, c["hq"]), part(n, c["hkv"]), part(n + m, c["hkv"])


def run(c, interleaved, use_depth=True, with_v=True, status=0):
    t = lambda a, dt: None if a is None else torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dt)
    _, q, k, v = views(c)
    new = lambda h: torch.full((c["T"], h, c["d"]), 9.0, dtype=c["dtype"], device="cuda")
    out = new(c["hq"]), new(c["hkv"]), new(c["hkv"])
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_qk_norm_rope(q, k, v if with_v else None, t(c["tab"], torch.float32), t(c["prefix"], torch.int32),
                        t(c["qo"], torch.int32), out[0], out[1], out[2] if with_v else None,
                        depth=t(c["depth"], torch.int32) if use_depth else None, q_weight=t(c["w"][0], c["dtype"]),
                        k_weight=t(c["w"][1], c["dtype"]), eps=1e-5, interleaved=interleaved, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return out


def positions(c, use_depth=True):
    pos = np.zeros(int(c["qo"][-1]), np.int64)
    for b in range(len(c["prefix"])):
        lo, hi = c["qo"][b], c["qo"][b + 1]
        pos[lo:hi] = c["prefix"][b] + (c["depth"][lo:hi] if use_depth else np.arange(hi - lo))
    return pos


def check(c, out, interleaved, use_depth=True, with_v=True):
    n = int(c["qo"][-1])
    x = c["x"][:n, :(c["hq"] + 2 * c["hkv"]) * c["d"]].reshape(n, -1, c["d"])
    q, k, v = x[:, :c["hq"]], x[:, c["hq"]:c["hq"] + c["hkv"]], x[:, c["hq"] + c["hkv"]:]
    pos = positions(c, use_depth)
    want = oracle.qk_norm_rope(q, k, v, c["w"][0], c["w"][1], 1e-5, c["tab"], pos, interleaved)
    flat = oracle.qk_norm_rope(q, k, v, c["w"][0], c["w"][1], 1e-5, None, pos, interleaved)   # normed, not turned
    half = torch.finfo(c["dtype"]).eps / 2
    for got, ref, y in zip(out[:2], want[:2], flat[:2]):
        mag = np.abs(y).copy()
        r = c["rot"]
        if r:
            one, two = (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else (np.arange(r // 2), np.arange(r // 2, r))
            both = mag[..., one] + mag[..., two]
            mag[..., one], mag[..., two] = both, both
        err = np.abs(got[:n].double().cpu().numpy() - ref)
        assert (err <= half * np.abs(ref) + (c["d"] / 2 + 12) * 2.0 ** -24 * mag).all()
    if with_v:
        assert np.array_equal(out[2][:n].float().cpu().numpy(), v)
    for o in out:
        assert (o[n:] == 9).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sizes,prefixes,hq,hkv,d,rot,dtype,norm", [
    ([1], [0], 1, 1, 16, 16, torch.float32, True), ([64], [4096], 32, 8, 128, 128, torch.bfloat16, True),
    ([1, 1, 1], [5, 0, 777], 64, 8, 128, 64, torch.bfloat16, True), ([3, 0, 7], [1, 2, 3], 6, 2, 96, 96, torch.float32, True),
    ([33, 2], [100, 9], 5, 1, 80, 32, torch.bfloat16, False), ([9], [30], 8, 8, 64, 0, torch.bfloat16, True),
    ([4], [11], 16, 4, 256, 256, torch.float32, False), ([5], [70], 3, 1, 512, 512, torch.bfloat16, True),
    ([2], [8], 40, 40, 192, 64, torch.bfloat16, True), ([130] * 40, list(range(40)), 8, 2, 64, 64, torch.bfloat16, True)])
def test_rope(sizes, prefixes, hq, hkv, d, rot, dtype, norm, interleaved):
    c = build(sizes, prefixes, hq, hkv, d, rot, dtype, norm, seed=d + len(sizes), pad_rows=3, extra=16)
    check(c, run(c, interleaved), interleaved)


def test_rope_without_depth_or_values():
    c = build([17, 4], [40, 0], 8, 2, 128, 128, torch.bfloat16, True, seed=1)
    out = run(c, False, use_depth=False, with_v=False)
    check(c, out, False, use_depth=False, with_v=False)
    assert (out[2] == 9).all()


def test_rope_far_positions():
    c = build([3], [131071 - 8], 4, 2, 64, 64, torch.float32, True, seed=2)
    check(c, run(c, False), False)


def test_rope_in_place():
    """Outputs may be the inputs themselves where the rows are as far apart."""
    c = build([21, 9], [7, 300], 8, 2, 128, 128, torch.bfloat16, True, seed=3)
    want = run(c, True)
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dt)
    _, q, k, v = (x if x.dim() == 2 else x.contiguous() for x in views(c))
    B.spec_qk_norm_rope(q, k, v, t(c["tab"], torch.float32), t(c["prefix"], torch.int32), t(c["qo"], torch.int32), q, k,
                        v, depth=t(c["depth"], torch.int32), q_weight=t(c["w"][0], c["dtype"]),
                        k_weight=t(c["w"][1], c["dtype"]), eps=1e-5, interleaved=True)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((q, k, v), want))


@pytest.mark.parametrize("fault", ["far", "depth", "prefix"])
def test_rope_leaves_bad_nodes(fault):
    c = build([5, 6], [10, 20], 4, 2, 64, 64, torch.bfloat16, True, seed=4)
    good = run(c, False)
    if fault == "far":
        c["depth"][7] = c["tab"].shape[0]
        bad = [7]
    elif fault == "depth":
        c["depth"][7] = -1
        bad = [7]
    else:
        c["prefix"][1] = -3
        bad = list(range(5, 11))
    out = run(c, False, status=-9)
    keep = [t for t in range(11) if t not in bad]
    for a, b in zip(out, good):
        assert (a[bad] == 9).all() and torch.equal(a[keep], b[keep])


def test_rope_nan_stays_in_its_head():
    c = build([4], [3], 4, 2, 128, 128, torch.bfloat16, True, seed=5)
    good = run(c, False)
    c["x"][2, 128 + 5] = np.nan        # node 2, query head 1
    out = run(c, False)
    assert torch.isnan(out[0][2, 1].float()).all()
    out[0][2, 1] = good[0][2, 1]
    assert all(torch.equal(a, b) for a, b in zip(out, good))


# ---------------------------------------------------------------------------- page tables

def pages_case(B_, most, total, ps, seed, tokens=20, length=100, need_room=True):
    rng = np.random.default_rng(seed)
    qo = np.concatenate([[0], np.cumsum(rng.integers(0, tokens, B_))]).astype(np.int32)
    lens = rng.integers(0, length, B_).astype(np.int32)
    need = -(-(lens + np.diff(qo)) // ps)
    held = np.clip(need + rng.integers(-3, 4, B_), 0, most).astype(np.int32)
    ids = rng.permutation(total)
    table, at = np.full((B_, most), -1, np.int32), 0
    for b in range(B_):
        table[b, :held[b]] = ids[at:at + held[b]]
        at += held[b]
    assert at <= total
    free = np.full(total, -5, np.int32)
    free[:total - at] = ids[at:]
    return dict(qo=qo, lens=lens, held=held, table=table, free=free, n=total - at, ps=ps)


def pages_run(c, shrink, in_place=False, status=0, pad_rows=0, slots=True):
    t = lambda a, dt=torch.int32: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dt)
    held, n = t(c["held"]), t(np.array([c["n"]]))
    table, free = t(c["table"]), t(c["free"])
    ho, no = (held, n) if in_place else (torch.full_like(held, -9), torch.full_like(n, -9))
    sm = torch.full((int(c["qo"][-1]) + pad_rows,), -77, dtype=torch.int64, device="cuda") if slots else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    B.spec_page_table_resize(t(c["lens"]), t(c["qo"]), held, table, free, n, ho, no, slot_map=sm, page_size=c["ps"],
                             shrink=shrink, dev_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    return table, ho, free, int(no.item()), sm


def pages_check(c, got, shrink, pad_rows=0):
    want = oracle.page_table_resize(c["lens"], c["qo"], c["held"], c["table"], c["free"], c["n"], c["ps"], shrink)
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert np.array_equal(got[2].cpu().numpy(), want[2])
    assert got[3] == want[3]
    if got[4] is not None:
        n = int(c["qo"][-1])
        assert np.array_equal(got[4][:n].cpu().numpy(), want[4]) and (got[4][n:] == -77).all()
    return want[5]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("shrink", [False, True])
@pytest.mark.parametrize("B_,most,total,ps,tokens,length", [
    (1, 4, 20, 16, 1, 30), (1, 40, 50, 16, 400, 100), (7, 20, 200, 16, 20, 100), (33, 9, 400, 4, 9, 20),
    (600, 20, 9000, 16, 40, 150), (4096, 12, 40000, 16, 3, 100), (64, 300, 30000, 16, 4000, 100), (513, 6, 3000, 1, 2, 3)])
def test_resize(B_, most, total, ps, tokens, length, shrink, in_place):
    c = pages_case(B_, most, total, ps, seed=B_ + ps, tokens=tokens, length=length)
    err = pages_check(c, pages_run(c, shrink, in_place, pad_rows=5), shrink)
    assert not err


def test_resize_without_slots():
    c = pages_case(9, 20, 300, 16, seed=1)
    pages_check(c, pages_run(c, True, slots=False), True)


@pytest.mark.parametrize("left", [0, 1, 5, 17])
def test_too_few_free_pages(left):
    c = pages_case(12, 20, 300, 16, seed=2)
    c["held"] = np.maximum(c["held"] - 2, 0).astype(np.int32)      # everyone asks (pages held twice nowhere)
    c["n"] = left
    asked = int(np.maximum(-(-(c["lens"] + np.diff(c["qo"])) // 16) - c["held"], 0).sum())
    got = pages_run(c, False, status=-4 if asked > left else 0)
    assert pages_check(c, got, False) == ({"capacity"} if asked > left else set())


def test_rows_too_short_and_bad_lengths():
    c = pages_case(8, 20, 300, 16, seed=3)
    c["lens"][2] = 20 * 16 + 1
    got = pages_run(c, True, status=-4)
    assert pages_check(c, got, True) == {"capacity"}
    c = pages_case(8, 20, 300, 16, seed=4)
    c["lens"][5] = -2
    got = pages_run(c, True, status=-9)
    assert pages_check(c, got, True) == {"index"}


def test_a_stack_out_of_range_moves_nothing():
    c = pages_case(8, 20, 300, 16, seed=5)
    for n in (-1, 301):
        c["n"] = n
        table, held, free, n_out, slots = pages_run(c, True, status=-4)
        assert np.array_equal(table.cpu().numpy(), c["table"]) and np.array_equal(held.cpu().numpy(), c["held"])
        assert np.array_equal(free.cpu().numpy(), c["free"]) and n_out == n


def test_finished_sequences_feed_the_others():
    """An empty stack: what two finished sequences give back is granted in the same call."""
    c = dict(qo=np.array([0, 0, 40, 40, 72], np.int32), lens=np.array([0, 8, 0, 16], np.int32),
             held=np.array([3, 1, 2, 1], np.int32), table=np.full((4, 4), -1, np.int32), free=np.full(7, -1, np.int32),
             n=0, ps=16)
    c["table"][0, :3], c["table"][1, 0], c["table"][2, :2], c["table"][3, 0] = [0, 1, 2], 3, [4, 5], 6
    got = pages_run(c, True)
    assert not pages_check(c, got, True)
    assert got[3] == 1
