"""Oracle: the operators around a verification step, in fp64 and plain loops.

kv8p_values        the values an E4M3 cache with a scale per (page, KV head) stands for
kv8p_commit        the accepted rows written into such a cache, its scales kept
qk_norm_rope       norm per head and rotation of queries and keys, values copied
page_table_resize  page-table rows grown and cut to the lengths, and the step's slot map

The scale of a page is the smallest power of two s in [2^-50, 2^50] with max|x| <= 448 s over
the finite elements written to it, never below what its older rows have; older codes are
rewritten for a larger scale.
"""

import numpy as np

from .fp8 import e4m3_decode, e4m3_encode

SCALE_EXP = 50


def read_scale(s):
    """A stored page scale as every call reads it: clamped to [2^-50, 2^50], NaN as 2^-50."""
    s = np.asarray(s, np.float64)
    return np.clip(np.where(np.isnan(s), 0.0, s), 2.0 ** -SCALE_EXP, 2.0 ** SCALE_EXP)


def kv8p_values(codes, kv_scale, which):
    """codes [pages][hkv][ps][d] -> float64 values; which: 0 the K scales, 1 the V scales."""
    return e4m3_decode(codes) * read_scale(kv_scale)[:, :, which, None, None]


def _encode(x):
    """e4m3_encode of values that may hold infinities (saturated) and NaN (kept)."""
    x = np.asarray(x, np.float64)
    nan = np.isnan(x)
    return np.where(nan, 0x7F, e4m3_encode(np.where(nan, 0.0, np.clip(x, -448.0, 448.0)))).astype(np.uint8)


def kv8p_commit(k_pool, v_pool, kv_scale, page_table, prefix_len, k_tree, v_tree, path, accept_len, qo_indptr):
    """Returns (k_pool, v_pool, kv_scale, seq_len); the inputs are not modified."""
    pools = [np.array(k_pool, copy=True), np.array(v_pool, copy=True)]
    scale = np.array(kv_scale, np.float32, copy=True)
    ps = pools[0].shape[2]
    B = len(qo_indptr) - 1
    seq_len = np.zeros(B, np.int32)
    for b in range(B):
        P, L = int(prefix_len[b]), int(accept_len[b])
        seq_len[b] = P + L + 1
        for lp in range(P // ps, (P + L) // ps + 1):
            page = int(page_table[b][lp])
            slots = range(max(P, lp * ps), min(P + L + 1, (lp + 1) * ps))
            rows = [int(qo_indptr[b]) + int(path[b][s - P]) for s in slots]
            r0 = slots[0] - lp * ps
            for w, tree in enumerate((k_tree, v_tree)):
                x = np.asarray(tree, np.float64)[rows]                      # [rows, hkv, d]
                for g in range(x.shape[1]):
                    fin = np.abs(x[:, g][np.isfinite(x[:, g])])
                    top = fin.max() if fin.size else 0.0
                    e = -SCALE_EXP
                    while e < SCALE_EXP and top > 448.0 * 2.0 ** e:
                        e += 1
                    s = 2.0 ** e
                    if r0 > 0:
                        was = float(read_scale(scale[page, g, w]))
                        s = max(s, was)
                        if s != was:
                            old = e4m3_decode(pools[w][page, g, :r0])
                            # the product in fp32, as the value is formed from code and scale
                            pools[w][page, g, :r0] = _encode((old * was).astype(np.float32).astype(np.float64) / s)
                    with np.errstate(invalid="ignore"):
                        q = x[:, g].astype(np.float32) / np.float32(s)
                    pools[w][page, g, r0:r0 + len(rows)] = _encode(q.astype(np.float64))
                    scale[page, g, w] = s
    return pools[0], pools[1], scale, seq_len


def qk_norm_rope(q, k, v, q_weight, k_weight, eps, cos_sin, positions, interleaved):
    """q [T,Hq,D], k, v [T,Hkv,D] -> (q, k, v) in float64 at the given positions [T]."""
    out = []
    rot = 0 if cos_sin is None else cos_sin.shape[1]
    for x, w in ((q, q_weight), (k, k_weight)):
        y = np.asarray(x, np.float64).copy()
        if w is not None:
            y = y / np.sqrt((y ** 2).mean(-1, keepdims=True) + eps) * np.asarray(w, np.float64)
        for t in range(y.shape[0]):
            for i in range(rot // 2):
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
                c, s = float(cos_sin[positions[t], i]), float(cos_sin[positions[t], rot // 2 + i])
                u, z = y[t, :, a].copy(), y[t, :, b].copy()
                y[t, :, a], y[t, :, b] = u * c - z * s, z * c + u * s
        out.append(y)
    return out[0], out[1], np.asarray(v, np.float64).copy()


def page_table_resize(seq_len, qo_indptr, held, page_table, free_pages, n_free, page_size, shrink):
    """One sequence after the other: (page_table, held, free_pages, n_free, slots, errors)."""
    table, free = np.array(page_table, copy=True), [int(x) for x in free_pages[:n_free]]
    held = [int(x) for x in held]
    out_free, errors, bad = np.array(free_pages, copy=True), set(), set()
    B, most = table.shape
    need = []
    for b in range(B):
        n = int(qo_indptr[b + 1]) - int(qo_indptr[b])
        want = -(-(int(seq_len[b]) + n) // page_size)
        if seq_len[b] < 0 or n < 0 or not 0 <= held[b] <= most:
            errors.add("index")
            bad.add(b)
            want = held[b]
        elif want > most:
            errors.add("capacity")
            want = held[b]
        need.append(want)
    for b in range(B):                       # returned pages first
        if shrink and need[b] < held[b]:
            free += [int(x) for x in table[b, need[b]:held[b]]]
            held[b] = need[b]
    full = False
    for b in range(B):                       # then the grants, in order
        if need[b] > held[b]:
            if full or need[b] - held[b] > len(free):
                full = True
                errors.add("capacity")
                continue
            while held[b] < need[b]:
                table[b, held[b]] = free.pop()
                held[b] += 1
    for i in range(n_free, len(free)):       # places below the old height keep what they hold
        out_free[i] = free[i]
    slots = np.full(int(qo_indptr[-1]), -1, np.int64)
    for b in range(B):
        for i in range(int(qo_indptr[b + 1]) - int(qo_indptr[b])):
            at = int(seq_len[b]) + i
            if b not in bad and at // page_size < held[b]:
                slots[int(qo_indptr[b]) + i] = int(table[b, at // page_size]) * page_size + at % page_size
    return table, np.array(held, np.int32), out_free, len(free), slots, errors
