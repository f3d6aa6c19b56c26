"""The commit into an E4M3 cache with page scales: codes and scales equal the oracle's, every
other byte is as it was."""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_parent_gb300 import binding as B
from speculative_decoding_tree_parent_gb300 import workloads as W

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


def setup(prefixes, accepts, hkv, d=128, ps=16, cap=None, seed=0, pow2=True, grow=0.0):
    rng = np.random.default_rng(seed)
    cap = cap or max(accepts) + 2
    sizes = [a + 1 + int(rng.integers(0, 4)) for a in accepts]
    qo = np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)
    need = [(p + a) // ps + 1 for p, a in zip(prefixes, accepts)]
    ids = rng.permutation(sum(need) + 3)
    table, at = np.full((len(need), max(need)), -1, np.int32), 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    path = np.full((len(sizes), cap), -1, np.int32)
    for b, a in enumerate(accepts):
        path[b, 0] = 0
        path[b, 1:a + 1] = 1 + np.sort(rng.permutation(sizes[b] - 1)[:a])
    codes = lambda: rng.integers(0, 127, (len(ids), hkv, ps, d)).astype(np.uint8) | (
        rng.integers(0, 2, (len(ids), hkv, ps, d)).astype(np.uint8) << 7)
    scale = (2.0 ** rng.integers(-12, -6, (len(ids), hkv, 2))).astype(np.float32)
    if not pow2:
        scale *= rng.uniform(1, 2, scale.shape).astype(np.float32)
    rows = lambda: W.round_to_bf16((rng.standard_normal((qo[-1], hkv, d)) * 2.0 ** rng.uniform(-2, grow, (qo[-1], hkv, 1))
                                    ).astype(np.float32))
    return dict(k=codes(), v=codes(), scale=scale, table=table, prefix=np.array(prefixes, np.int32), kt=rows(), vt=rows(),
                path=path, accept=np.array(accepts, np.int32), qo=qo)


def put(c):
    t = lambda n, dt: torch.from_numpy(np.ascontiguousarray(c[n])).to("cuda", dt)
    d = {n: t(n, torch.int32) for n in ("table", "prefix", "path", "accept", "qo")}
    d.update({n: t(n, torch.uint8) for n in ("k", "v")})
    d.update({n: t(n, torch.bfloat16) for n in ("kt", "vt")})
    d["scale"] = t("scale", torch.float32)
    d["seq"] = torch.full((len(c["accept"]),), -7, dtype=torch.int32, device="cuda")
    d["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    return d


def call(d):
    B.spec_kv_commit_kv8p(d["kt"], d["vt"], d["path"], d["accept"], d["qo"], d["table"], d["prefix"], d["k"], d["v"],
                          d["scale"], seq_len_out=d["seq"], dev_status=d["status"])


def check(c, d):
    k, v, s, n = oracle.kv8p_commit(c["k"], c["v"], c["scale"], c["table"], c["prefix"], c["kt"], c["vt"], c["path"],
                                    c["accept"], c["qo"])
    assert np.array_equal(d["scale"].cpu().numpy(), s, equal_nan=True)
    assert np.array_equal(d["k"].cpu().numpy(), k)
    assert np.array_equal(d["v"].cpu().numpy(), v)
    assert np.array_equal(d["seq"].cpu().numpy(), n)


@pytest.mark.parametrize("prefixes,accepts,hkv,d,ps", [
    ([0], [0], 1, 128, 16), ([15], [0], 8, 128, 16), ([16, 17, 31], [3, 15, 1], 2, 128, 16), ([5], [40], 8, 128, 16),
    ([4105] * 3, [3, 0, 8], 8, 128, 16), ([100, 3], [511, 17], 2, 128, 16), ([7, 30], [9, 2], 3, 64, 16),
    ([1, 63], [70, 1], 2, 64, 32), ([9], [5], 2, 256, 16), ([13], [12], 1, 16, 1), ([20], [9], 2, 48, 8),
    ([33], [70], 2, 80, 64)])
@pytest.mark.parametrize("pow2", [True, False])
def test_commit(prefixes, accepts, hkv, d, ps, pow2):
    c = setup(prefixes, accepts, hkv, d, ps, seed=len(accepts) + d, pow2=pow2, grow=4.0)
    t = put(c)
    call(t)
    torch.cuda.synchronize()
    assert int(t["status"].item()) == 0
    check(c, t)


def test_commit_again_gives_the_same_bytes():
    c = setup([21, 64], [6, 33], 4, seed=3)
    t = put(c)
    call(t)
    call(t)
    torch.cuda.synchronize()
    check(c, t)


def test_a_page_filled_over_many_steps():
    """Row after row into one page, each larger than the last and then smaller ones: the scale
    only rises, and the values stay within a half step of what was written."""
    c = setup([0], [0], 2, seed=4)
    c["scale"][:] = np.nan       # a page without older rows does not read its scale
    t = put(c)
    rng = np.random.default_rng(5)
    rows, last = [], 0.0
    for i in range(16):
        x = W.round_to_bf16((rng.standard_normal(c["kt"].shape) * 4.0 ** min(i, 9)).astype(np.float32))
        c["kt"], c["vt"], c["prefix"] = x, -x, np.array([i], np.int32)
        u = put(c)
        u["k"], u["v"], u["scale"] = t["k"], t["v"], t["scale"]
        call(u)
        torch.cuda.synchronize()
        assert int(u["status"].item()) == 0
        check(c, u)
        c["k"], c["v"], c["scale"] = (u[n].cpu().numpy() for n in ("k", "v", "scale"))
        t, now = u, c["scale"][c["table"][0, 0], :, 0]
        assert (now >= last).all()
        last = now
        rows.append(x[0])
    page = c["table"][0, 0]
    got = oracle.kv8p_values(c["k"], c["scale"], 0)[page].transpose(1, 0, 2)
    want = np.stack(rows).astype(np.float64)
    step = last[None, :, None].astype(np.float64) * 2.0 ** -9
    # each rewriting of a row can add half a subnormal step; a normal value is rounded once
    assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -4 + 10 * step).all()


def test_infinities_nan_and_zeros():
    c = setup([3, 48], [4, 2], 2, seed=6)
    c["kt"][0, 0, 5], c["kt"][1, 1, 7], c["vt"][2, 0, 9] = np.inf, -np.inf, np.nan
    c["kt"][int(c["qo"][1]):], c["vt"][int(c["qo"][1]):] = 0, 0
    t = put(c)
    call(t)
    torch.cuda.synchronize()
    assert int(t["status"].item()) == 0
    check(c, t)


@pytest.mark.parametrize("fault,code", [("page", -3), ("node", -9), ("root", -9), ("len", -9), ("cap", -4), ("neg", -9)])
def test_a_sequence_with_an_error_is_left(fault, code):
    c = setup([14, 30, 5], [20, 3, 2], 4, seed=7)
    t = put(c)
    if fault == "page":
        t["table"][0, 2] = c["k"].shape[0]
    elif fault == "node":
        t["path"][0, 19] = int(c["qo"][1])
    elif fault == "root":
        t["path"][0, 0] = 1
    elif fault == "len":
        t["accept"][0] = c["path"].shape[1]
    elif fault == "cap":
        t["prefix"][0] = 16 * c["table"].shape[1] - 1
    else:
        t["prefix"][0] = -1
    call(t)
    torch.cuda.synchronize()
    assert int(t["status"].item()) == code
    assert int(t["seq"][0].item()) == -7
    one = {n: (c[n][1:] if n in ("table", "prefix", "path", "accept") else c[n]) for n in c}
    one["qo"] = c["qo"][1:]
    k, v, s, _ = oracle.kv8p_commit(one["k"], one["v"], one["scale"], one["table"], one["prefix"], one["kt"], one["vt"],
                                    one["path"], one["accept"], one["qo"])
    assert np.array_equal(t["k"].cpu().numpy(), k) and np.array_equal(t["v"].cpu().numpy(), v)
    assert np.array_equal(t["scale"].cpu().numpy(), s)
