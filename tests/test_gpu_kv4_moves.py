"""The 4-bit attention where a row's largest score keeps rising from block to block, so that its shift is moved and what was
summed before is scaled down, again and again; and captured calls over a pool that holds NaN behind every prefix."""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_parent_gb300 import binding as B

import kv4_cases as C
import serving_cases as S
from test_gpu_kv4_attention import attend, check, workspace

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

KEYS, NODES, SHIFT, LIMIT = 128, 32, 5.0, 15.0     # a block of the prefix, of the tree; where a move puts the largest, and when


def rising(prefix, nodes, G, hkv, batch, order, seed):
    """Every sequence over the same pages. A token's scores are about 16 * scale / 8 (in powers of two): 16 for most, while one token
    of a block stands 12 and more above all before it (order 1), or above all behind it (-1); the tree's nodes stand 16
    higher every 32 of them."""
    c = C.case([prefix], [nodes], G * hkv, hkv, seed)
    rng = np.random.default_rng(seed + 1)
    sign = rng.choice([-1.0, 1.0], (hkv, 128))
    code = rng.choice([1, 2, 2, 3], (c.pages, hkv, 16, 128)) + np.where(sign[:, None] < 0, 8, 0)
    scale = np.full((c.pages, hkv, 16, 8), 0x50, np.uint8)                # 8
    blocks = -(-prefix // KEYS)
    peaks = [0x56, 0x5A, 0x5D, 0x60, 0x62, 0x64, 0x65, 0x66]              # 14, 20, 26, 32, 40, 48, 52, 56
    for k in range(blocks):
        at = k if order > 0 else blocks - 1 - k
        if at == 0:
            continue
        lp = min(8 * k + int(rng.integers(8)), (prefix - 1) // 16)
        scale[c.table[0, lp], :, int(rng.integers(min(16, prefix - 16 * lp)))] = peaks[at - 1]
    _, vs = oracle.kv4_codes(c.pool, 1)
    vc, _ = oracle.kv4_codes(c.pool, 1)
    c.pool = oracle.kv4_record(code.astype(np.uint8), scale, vc, vs)
    if prefix % 16:
        rec = c.pool[c.table[0, prefix // 16]]
        C.put_nan_scales(rec, range(prefix % 16, 16))
        c.pool[c.table[0, prefix // 16]] = rec
    c.kv_scale = np.stack([np.full(hkv, 0.125), c.kv_scale[1]]).astype(np.float32)
    T = batch * nodes
    c.q = S.bf16(np.repeat(sign, G, 0) + 0.05 * rng.standard_normal((T, G * hkv, 128)))
    step = (np.arange(nodes) // NODES + 7.0) if order > 0 else (1.0 - np.arange(nodes) // NODES * 0.25)
    c.kt = S.bf16(np.tile(step, batch)[:, None, None] * (sign + 0.05 * rng.standard_normal((T, hkv, 128))))
    c.vt = S.bf16(rng.standard_normal((T, hkv, 128)))
    c.sizes, c.T = [nodes] * batch, T
    c.qo = np.arange(batch + 1, dtype=np.int32) * nodes
    c.mask = np.tile(c.mask, (batch, 1))
    c.table, c.prefix = np.tile(c.table, (batch, 1)), np.full(batch, prefix, np.int32)
    return c


def scores(c, b):
    """Scores of a sequence's rows in powers of two, [head][node][prefix, then tree], and the values [head][key], in 64 bits."""
    G, P, n = c.hq // c.hkv, int(c.prefix[b]), c.sizes[b]
    lo, hi = int(c.qo[b]), int(c.qo[b + 1])
    if not hasattr(c, "cached"):                            # (the same pages for all)
        pages = c.table[0, :-(-P // 16)]
        c.cached = [np.nan_to_num(oracle.kv4_values(c.pool[pages], c.kv_scale, w)).swapaxes(1, 2).reshape(-1, c.hkv, 128)[:P]
                    for w in range(2)]
    k, v = (np.concatenate([x, y[lo:hi].astype(np.float64)]).repeat(G, 1).swapaxes(0, 1) for x, y in zip(c.cached, (c.kt, c.vt)))
    y = c.q[lo:hi].astype(np.float64).swapaxes(0, 1) @ k.swapaxes(1, 2) / 128 ** 0.5 / np.log(2)
    see = np.concatenate([np.ones((n, P), bool), c.mask[lo:hi, :n]], 1)
    return np.where(see[None], y, -np.inf), v


def moves(c, max_prefix, ctas):
    """How often each row [batch][head][node] is moved after a run's first block, by the rule of the kernel: the list of all tiles'
    blocks is cut into equal shares, a tile of at most 64 rows gives its blocks to two slots in turn."""
    G, nodes = c.hq // c.hkv, c.sizes[0]
    R = next(r for r in (16, 32, 64, 128) if nodes * G <= r or r == 128)
    cost, per, dual = {16: 4, 32: 6}.get(R, 8), R // G, R == 128
    P = int(c.prefix[0])
    cuts = [(k * KEYS, min(P, (k + 1) * KEYS)) for k in range(-(-P // KEYS))]
    cuts += [(P + k * NODES, P + min(nodes, (k + 1) * NODES)) for k in range(-(-nodes // NODES))]
    tiles, unit = -(-nodes // per), len(cuts) + cost
    total = len(c.sizes) * c.hkv * tiles * unit
    ctas = min(ctas, len(c.sizes) * c.hkv * tiles * (-(-max_prefix // KEYS) + -(-c.mask.shape[1] // NODES) + cost))
    tops = [np.stack([scores(c, b)[0][:, :, lo:hi].max(-1, initial=-np.inf) for lo, hi in cuts]) for b in range(len(c.sizes))]
    count = np.zeros((len(c.sizes), c.hq, nodes), int)
    each, more = divmod(total, ctas)
    for cta in range(ctas):
        at, end = each * cta + min(cta, more), each * (cta + 1) + min(cta + 1, more)
        i = 0                                               # the CTA's block
        while at < end:
            t, j0 = divmod(at, unit)
            b, t = divmod(t, c.hkv * tiles)
            g, t = divmod(t, tiles)
            nb = min(len(cuts) - j0, end - at)
            if nb > 0:
                rows = (slice(g * G, (g + 1) * G), slice(t * per, (t + 1) * per))
                for slot in range(1 if dual else 2):
                    off = None
                    for k in range(0 if dual else (i ^ slot) & 1, nb, 1 if dual else 2):
                        top = tops[b][j0 + k][rows]
                        first = off is None
                        off = np.full(top.shape, np.nan) if first else off
                        with np.errstate(invalid="ignore"):
                            new = np.isnan(off) & (top > -np.inf)
                            move = ~np.isnan(off) & (top + off > LIMIT)
                        off = np.where(new | move, SHIFT - top, off)
                        count[b][rows] += move
                i += nb
                at += nb
            else:
                at += min(unit - j0, end - at)
    return count


SHAPES = {   # rows of a tile: nodes, group, batch
    "rows of 16": (4, 4, 90), "rows of 32": (8, 4, 90), "rows of 64": (16, 4, 90), "rows of 128": (32, 4, 70),
    "rows of 64, two tree blocks": (40, 1, 90), "rows of 128, three tree blocks": (80, 1, 70), "two tiles": (50, 4, 30)}


@pytest.mark.parametrize("name", SHAPES)
def test_rows_that_are_moved_again_and_again(name):
    nodes, G, batch = SHAPES[name]
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for order in (1, -1):
        c = rising(900, nodes, G, 2, batch, order, seed=nodes + G)
        d = C.device(c)
        count = moves(c, d.max_prefix, sms)
        if order > 0:
            assert (count >= 1).mean() > 0.5 and (count >= 2).any(), count
        else:
            assert (count == 0).mean() > 0.5
        attend(c, d)
        assert int(d.status.item()) == 0
        out, lse = d.out.double().cpu().numpy(), d.lse.double().cpu().numpy()
        for b in range(batch):
            y, v = scores(c, b)
            top = y.max(-1, keepdims=True)
            w = np.exp2(y - top)
            L = w.sum(-1, keepdims=True)
            w /= L
            ref, A = (w @ v).swapaxes(0, 1), (w @ np.abs(v)).swapaxes(0, 1)
            got = out[c.qo[b]:c.qo[b + 1]]
            err, tol = np.abs(got - ref), C.tolerance(ref, A, y.shape[-1], np.abs(v).max())
            assert (err <= tol).all(), (order, b, (err - tol).max())
            want = ((top + np.log2(L)) * np.log(2))[..., 0].T
            assert np.abs(lse[c.qo[b]:c.qo[b + 1]] - want).max() <= C.LSE_TOL


@pytest.mark.parametrize("prefix", [0, 40])
def test_many_tiles_of_one_block(prefix):
    """Tiles whose only block leaves a slot without work, between tiles of two and three."""
    rng = np.random.default_rng(prefix)
    prefixes = [int(rng.choice([0, prefix, prefix, 130, 260])) for _ in range(120)]
    c = C.case(prefixes, [1] * 120, 16, 16, seed=51, pad_rows=1)
    d = C.device(c)
    attend(c, d)
    assert int(d.status.item()) == 0
    check(c, d)


def test_a_captured_call_over_a_pool_with_nan_behind_the_prefixes():
    """One graph over the largest sizes, replayed with other lengths; what a page holds past a prefix has NaN scales, and
    so has every page that the sequence's prefix does not reach."""
    big = C.case([900, 700, 300], [40, 30, 30], 8, 2, seed=20)
    d = C.device(big)
    ws = workspace(big, d)
    attend(big, d, ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.spec_tree_verify_attn_kv4(d.q, d.pool, d.table, d.prefix, d.max_prefix, d.kt, d.vt, d.mask, d.qo, d.max_nodes,
                                    d.out, kv_scale=d.kv_scale, lse=d.lse, ws=ws, dev_status=d.status)
    for seed, prefixes, sizes in ((21, [900, 0, 17], [40, 1, 40]), (22, [5, 650, 299], [1, 40, 30]), (23, [0, 0, 0], [33, 33, 1]),
                                  (24, [127, 129, 241], [2, 3, 4])):
        c = C.case(prefixes, sizes, 8, 2, seed=seed)
        n, m = int(c.qo[-1]), c.mask.shape[1]
        mask = np.zeros((big.T, 40), bool)
        mask[:n, :m] = c.mask
        pool = C.pool(np.random.default_rng(seed), big.pages, 2)
        for b, p in enumerate(prefixes):
            for lp in range(p // 16, big.table.shape[1]):
                if big.table[b, lp] >= 0:
                    rec = pool[big.table[b, lp]]
                    C.put_nan_scales(rec, range(p % 16 if lp == p // 16 else 0, 16))
                    pool[big.table[b, lp]] = rec
        for t, a in ((d.prefix, c.prefix), (d.qo, c.qo), (d.mask, S.words(mask)), (d.pool, pool)):
            t.copy_(torch.from_numpy(a))
        d.out.fill_(7), d.lse.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        full = C.SimpleNamespace(**vars(big))
        full.prefix, full.qo, full.mask, full.sizes, full.pool = c.prefix, c.qo, mask, sizes, pool
        check(full, d)
        assert int(d.status.item()) == 0


@pytest.mark.parametrize("nodes", [4, 20, 200])
def test_large_values_in_the_tree(nodes):
    """Values of 2^98 beside a head's V scale of 1, 2^90 beside one of 2^-4: products summed over 1024 nodes would stay finite."""
    c = C.case([40, 0], [nodes, 3], 8, 2, seed=61)
    c.kv_scale[1] = [1.0, 2.0 ** -4]
    c.vt[:, 0] *= np.float32(2.0 ** 96)
    c.vt[:, 1] *= np.float32(2.0 ** 90)
    assert np.abs(c.vt[:, 0]).max() < 2.0 ** 99 and np.abs(c.vt[:, 1]).max() < 2.0 ** 95
    d = C.device(c)
    attend(c, d)
    assert int(d.status.item()) == 0
    check(c, d)
