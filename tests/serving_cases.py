"""Inputs of the serving operators' tests: paged E4M3 caches with page scales, trees with
their ancestor bits, and the oracle's attention over them. Inputs only, no arithmetic of the
operators themselves."""

from types import SimpleNamespace

import numpy as np
import torch

import oracle
from speculative_decoding_tree_parent_gb300 import workloads as W

PS, D = 16, 128


def bf16(x):
    return W.round_to_bf16(np.asarray(x, np.float32))


def trees(sizes, rng, reach=8):
    """Random parents of each size and their ancestor rows (bool [T, max]) and bit words."""
    parent, qo = [], [0]
    for n in sizes:
        parent += [-1 if i == 0 else int(rng.integers(max(0, i - reach), i)) for i in range(n)]
        qo.append(qo[-1] + n)
    T, most = qo[-1], max(1, max(sizes))
    mask = np.zeros((T, most), bool)
    for b, n in enumerate(sizes):
        for i in range(n):
            t = qo[b] + i
            if i:
                mask[t] = mask[qo[b] + parent[t]]
            mask[t, i] = True
    return np.array(parent, np.int32), np.array(qo, np.int32), mask


def words(mask):
    return oracle.pack_mask_words(mask, -(-mask.shape[1] // 64)).view(np.int64)


def case(prefixes, sizes, hq, hkv, seed, q_scale=1.0, spread=2.0, extra_pages=3, pad_rows=0):
    """A batch over shuffled pages; every page and head has a scale of its own (not a power of
    two), 2^+-spread apart; the pages' rows past a prefix hold codes too, NaN among them."""
    rng = np.random.default_rng(seed)
    parent, qo, mask = trees(sizes, rng)
    T = int(qo[-1]) + pad_rows
    mask = np.concatenate([mask, np.zeros((pad_rows, mask.shape[1]), bool)])
    need = [-(-p // PS) for p in prefixes]
    pages = sum(need) + extra_pages
    ids = rng.permutation(pages)
    table = np.full((len(sizes), max(1, max(need))), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    # finite codes drawn from rounded normals (every exponent appears), then the scales
    codes = [oracle.e4m3_encode(rng.standard_normal((pages, hkv, PS, D)) * 100.0) for _ in range(2)]
    scale = (2.0 ** rng.uniform(-spread, spread, (pages, hkv, 2)) / 100.0).astype(np.float32)
    for b, p in enumerate(prefixes):    # what lies past a prefix holds nothing
        if p % PS:
            for c in codes:
                c[table[b, p // PS], :, p % PS:] = 0x7F
    g = lambda *s: bf16(rng.standard_normal(s))
    return SimpleNamespace(prefix=np.array(prefixes, np.int32), sizes=sizes, hq=hq, hkv=hkv, parent=parent, qo=qo,
                           mask=mask, table=table, pages=pages, k=codes[0], v=codes[1], scale=scale,
                           q=g(T, hq, D) * np.float32(q_scale), kt=g(T, hkv, D), vt=g(T, hkv, D), T=T)


def device(c, stream=None):
    t = lambda a, dt: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dt)
    return SimpleNamespace(
        q=t(c.q, torch.bfloat16), kt=t(c.kt, torch.bfloat16), vt=t(c.vt, torch.bfloat16), k=t(c.k, torch.uint8),
        v=t(c.v, torch.uint8), scale=t(c.scale, torch.float32), table=t(c.table, torch.int32),
        prefix=t(c.prefix, torch.int32), qo=t(c.qo, torch.int32), mask=t(words(c.mask), torch.int64),
        out=torch.full((c.T, c.hq, D), 7.0, dtype=torch.bfloat16, device="cuda"),
        lse=torch.full((c.T, c.hq), 7.0, dtype=torch.float32, device="cuda"),
        status=torch.zeros(1, dtype=torch.int32, device="cuda"), max_prefix=int(c.prefix.max()),
        max_nodes=c.mask.shape[1])


def reference(c, rows=None):
    """(out, lse, A) in fp64; A: the same attention over |v|. rows: sampled (node, head)."""
    kv = oracle.kv8p_values(c.k, c.scale, 0), oracle.kv8p_values(c.v, c.scale, 1)
    kp, vp = np.nan_to_num(kv[0]), np.nan_to_num(kv[1])      # (NaN only past the prefixes)
    n = int(c.qo[-1])
    a = (c.q[:n], kp, vp, c.table, c.prefix, c.kt[:n], c.vt[:n], c.mask[:n], c.qo, c.hq, c.hkv)
    with np.errstate(invalid="ignore", divide="ignore"):
        if rows is None:
            out, lse = oracle.tree_verify_attention(*a)
            ab, _ = oracle.tree_verify_attention(*a[:2], np.abs(vp), *a[3:6], np.abs(c.vt[:n]), *a[7:])
        else:
            out, lse = oracle.tree_verify_attention_rows(rows, *a)
            ab, _ = oracle.tree_verify_attention_rows(rows, *a[:2], np.abs(vp), *a[3:6], np.abs(c.vt[:n]), *a[7:])
    return out, lse, ab
