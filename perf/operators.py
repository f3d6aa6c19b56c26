"""What the serving-side operators of the verification library cost, case by case.

Four operators that one step of tree speculative decoding runs around its mask, attention and
acceptance: the norm and rotation of queries and keys, the attention over an 8-bit paged cache
with a scale per (page, KV head), the commit that writes such a cache, and the page table that
grows with the lengths on the device. `listed` and `draw` give sizes, `prepare` the inputs a
program holds, `run` one pass (the plain torch form, or the library's calls where `own` is
true), `work` the bytes and operations of a pass, `exact` the outputs in 64 bits.
"""

import math

import numpy as np
import torch

own = False

PAGE = 16     # tokens in a page
DIM = 128     # head dim of the attention and of the cache
F8_MAX = 448.0
SCALE_LO, SCALE_HI = -50, 50    # page scales: powers of two in [2^-50, 2^50]


def listed():
    return [
        # one token of one sequence over a short context: a chat turn's decode step, latency only
        {"name": "attn_decode_1", "op": "attn", "batch": 1, "nodes": 1, "nodes_min": 1, "prefix_min": 517,
         "prefix": 517, "hq": 32, "hkv": 8},
        # the benchmark's single-sequence verification: 64-node tree over a 4096-token prefix
        {"name": "attn_tree_1", "op": "attn", "batch": 1, "nodes": 64, "nodes_min": 64, "prefix_min": 4096,
         "prefix": 4096, "hq": 32, "hkv": 8},
        # plain decoding of a full batch beside the speculating one: one token each, ragged prefixes
        {"name": "attn_decode_128", "op": "attn", "batch": 128, "nodes": 1, "nodes_min": 1, "prefix_min": 256,
         "prefix": 8190, "hq": 64, "hkv": 8},
        # the benchmark's batched verification: 64-node trees, prefixes of 512 to 8192 tokens
        {"name": "attn_tree_32", "op": "attn", "batch": 32, "nodes": 64, "nodes_min": 64, "prefix_min": 512,
         "prefix": 8192, "hq": 32, "hkv": 8},
        # long context, large heads: eight 32K prefixes with 128-node trees (64 query heads)
        {"name": "attn_tree_long", "op": "attn", "batch": 8, "nodes": 128, "nodes_min": 101, "prefix_min": 32768,
         "prefix": 32768, "hq": 64, "hkv": 8},
        # the accepted path of one sequence: four tokens that end inside a page
        {"name": "commit_1", "op": "commit", "batch": 1, "path": 9, "accept_min": 3, "accept": 3, "prefix": 4105,
         "hkv": 8},
        # prompt chunks written by the same call: 32 sequences of about 500 tokens
        {"name": "commit_chunk", "op": "commit", "batch": 32, "path": 512, "accept_min": 391, "accept": 511,
         "prefix": 1003, "hkv": 8},
        # the tree's 64 nodes after the projection of one sequence
        {"name": "rope_tree", "op": "rope", "batch": 1, "nodes": 64, "hq": 32, "hkv": 8, "d": 128, "rot": 128,
         "prefix": 4096, "dtype": "bf16", "norm": True, "interleaved": False},
        # a chunk of prompt tokens: ragged sequences, large heads, adjacent pairs rotated over half the head
        {"name": "rope_chunk", "op": "rope", "batch": 13, "nodes": 1021, "hq": 64, "hkv": 8, "d": 128, "rot": 64,
         "prefix": 30011, "dtype": "bf16", "norm": True, "interleaved": True},
        # the step's growth of a running batch: a few new pages and the slots of 64 nodes each
        {"name": "pages_step", "op": "pages", "batch": 32, "tokens_min": 64, "tokens": 64, "len": 8000,
         "held": "step", "shrink": False},
        # tables built from nothing for a batch of prompts, and the slots of every token
        {"name": "pages_build", "op": "pages", "batch": 192, "tokens_min": 63, "tokens": 8191, "len": 0,
         "held": "none", "shrink": True},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "commit", "rope", "pages"])
    if op == "attn":
        batch = _log_int(rng, 1, 64)
        nodes = rng.choice([1, 1, 3, 17, 33, 64, 65, 100, 128])
        prefix = _log_int(rng, 1, 32768)
        hkv = rng.choice([1, 2, 4, 8])
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
        while batch * nodes * hq * (prefix + nodes) > 1 << 30 or batch * prefix * hkv > 1 << 21:
            batch, prefix = max(1, batch // 2), max(1, prefix * 2 // 3)
        return {"op": "attn", "batch": batch, "nodes": nodes, "nodes_min": max(1, nodes - nodes // 3),
                "prefix_min": rng.choice([0, prefix // 3, prefix]), "prefix": prefix, "hq": hq, "hkv": hkv}
    if op == "commit":
        accept = _log_int(rng, 1, 511)
        return {"op": "commit", "batch": _log_int(rng, 1, 64), "path": accept + rng.randint(1, 9),
                "accept_min": rng.randint(0, accept), "accept": accept, "prefix": rng.randint(0, 4100),
                "hkv": rng.choice([1, 2, 4, 8])}
    if op == "rope":
        d = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([d, d, d // 2 // 16 * 16])
        hkv = rng.choice([1, 2, 4, 8])
        return {"op": "rope", "batch": _log_int(rng, 1, 16), "nodes": _log_int(rng, 1, 511), "hq": hkv * rng.choice([1, 3, 4, 8]),
                "hkv": hkv, "d": d, "rot": rot, "prefix": _log_int(rng, 1, 32000), "dtype": rng.choice(["bf16", "bf16", "f32"]),
                "norm": rng.random() < 0.7, "interleaved": rng.random() < 0.4}
    tokens = _log_int(rng, 1, 4099)
    return {"op": "pages", "batch": _log_int(rng, 1, 256), "tokens_min": rng.randint(0, tokens), "tokens": tokens,
            "len": rng.randint(0, 4099), "held": rng.choice(["step", "none", "more"]), "shrink": rng.random() < 0.5}


def _spread(lo, hi, n):
    """n whole numbers between lo and hi, both among them where n > 1 (the last is hi)."""
    v = np.arange(n) * 0.6180339887498949 % 1.0
    out = np.floor(lo + v * (hi - lo + 1)).astype(np.int64)
    out[-1] = hi
    return np.clip(out, lo, hi)


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _indptr(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int64)


def _trees(counts, rng):
    """A random tree of each size: parents, depths and ancestor bits (64 nodes a word)."""
    words = (int(counts.max()) + 63) // 64
    parent = np.full(int(counts.sum()), -1, np.int64)
    depth = np.zeros_like(parent)
    bits = np.zeros((len(parent), words), np.uint64)
    at = 0
    for n in counts:
        for i in range(int(n)):
            p = -1 if i == 0 else int(rng.integers(max(0, i - 12), i))
            parent[at + i] = p
            if i:
                depth[at + i] = depth[at + p] + 1
                bits[at + i] = bits[at + p]
            bits[at + i, i >> 6] |= np.uint64(1 << (i & 63))
        at += int(n)
    return parent, depth, bits.view(np.int64)


def _f8_pool(gen, pages, hkv, spread):
    """Random pages as E4M3 codes with a scale per (page, head): codes [pages][hkv][16][128]
    for keys and for values, scales [pages][hkv][2]."""
    codes = [torch.empty((pages, hkv, PAGE, DIM), dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = torch.empty((pages, hkv, 2), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (hkv * PAGE * DIM))
    for lo in range(0, pages, step):
        n = min(step, pages - lo)
        for w in range(2):
            x = torch.randn((n, hkv, PAGE, DIM), generator=gen, device="cuda")
            x *= torch.exp2((torch.rand((n, hkv, 1, 1), generator=gen, device="cuda") * 2 - 1) * spread)
            s = x.abs().amax((2, 3)) / F8_MAX
            codes[w][lo:lo + n] = (x / s[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            scale[lo:lo + n, :, w] = s
    return codes[0], codes[1], scale


def _sizes(case):
    """The lengths of a case's sequences, from the case alone."""
    n = case["batch"]
    if case["op"] == "attn":
        return _spread(case["nodes_min"], case["nodes"], n), _spread(case["prefix_min"], case["prefix"], n)[::-1].copy()
    if case["op"] == "commit":
        return _spread(case["accept_min"], case["accept"], n), np.maximum(0, case["prefix"] - 5 * np.arange(n) % 61)
    if case["op"] == "rope":
        return _spread((case["nodes"] + 1) // 2, case["nodes"], n), _spread(case["prefix"] // 2, case["prefix"], n)
    return _spread(case["tokens_min"], case["tokens"], n), _spread(case["len"] // 2, case["len"], n)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return {"attn": _prepare_attn, "commit": _prepare_commit, "rope": _prepare_rope, "pages": _prepare_pages}[case["op"]](
        case, rng, gen)


def _tables(rng, need, spare=0):
    """Page ids of each sequence in a shuffled pool, and the number of pages."""
    total = int(need.sum()) + spare
    ids = rng.permutation(total)
    table = np.full((len(need), max(1, int(need.max()))), -1, np.int64)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += int(n)
    return table, max(1, total), ids[at:]


def _prepare_attn(case, rng, gen):
    counts, prefix = _sizes(case)
    T, hq, hkv = int(counts.sum()), case["hq"], case["hkv"]
    table, pages, _ = _tables(rng, (prefix + PAGE - 1) // PAGE)
    kp, vp, scale = _f8_pool(gen, pages, hkv, 1.0)
    _, _, bits = _trees(counts, rng)
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda").to(torch.bfloat16)
    return {"op": "attn", "q": randn(T, hq, DIM), "k_tree": randn(T, hkv, DIM), "v_tree": randn(T, hkv, DIM),
            "k_pool": kp, "v_pool": vp, "scale": scale, "table": _i32(table), "prefix": _i32(prefix),
            "max_prefix": int(prefix.max()), "mask": torch.from_numpy(bits).cuda(), "qo": _i32(_indptr(counts)),
            "max_nodes": int(counts.max()), "out": torch.zeros((T, hq, DIM), dtype=torch.bfloat16, device="cuda"),
            "lse": torch.zeros((T, hq), dtype=torch.float32, device="cuda")}


def _prepare_commit(case, rng, gen):
    accept, prefix = _sizes(case)
    B, hkv, cap = case["batch"], case["hkv"], case["path"]
    counts = accept + 3          # the path leaves three nodes of each tree out
    table, pages, _ = _tables(rng, (prefix + accept + PAGE) // PAGE, 5)
    kp, vp, scale = _f8_pool(gen, pages, hkv, 1.0)
    scale = torch.exp2(torch.ceil(torch.log2(scale)))     # as this cache's writer leaves them
    path = np.full((B, cap), -1, np.int64)
    for b in range(B):
        path[b, 1:accept[b] + 1] = 1 + np.sort(rng.permutation(int(counts[b]) - 1)[:accept[b]])
        path[b, 0] = 0
    T = int(counts.sum())
    rows = lambda: (torch.randn((T, hkv, DIM), generator=gen, device="cuda")
                    * torch.exp2(torch.rand((T, hkv, 1), generator=gen, device="cuda") * 4 - 2)).to(torch.bfloat16)
    return {"op": "commit", "k_tree": rows(), "v_tree": rows(), "path": _i32(path), "accept": _i32(accept),
            "qo": _i32(_indptr(counts)), "table": _i32(table), "prefix": _i32(prefix), "k_pool": kp, "v_pool": vp,
            "scale": scale, "seq_len": torch.zeros(B, dtype=torch.int32, device="cuda")}


def _prepare_rope(case, rng, gen):
    counts, prefix = _sizes(case)
    T, hq, hkv, d, rot = int(counts.sum()), case["hq"], case["hkv"], case["d"], case["rot"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    heads = hq + 2 * hkv
    qkv = (torch.randn((T, heads * d), generator=gen, device="cuda") * 3).to(dt)   # the fused projection's rows
    depth = np.concatenate([np.sort(rng.integers(0, n, n)) for n in counts])       # tree depths, the root's first
    reach = case["prefix"] + case["nodes"] + 1
    inv = 500000.0 ** (-np.arange(rot // 2) / max(1, rot // 2))
    ang = np.arange(reach)[:, None] * inv[None, :]
    table = torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)).cuda()
    w = lambda: (1 + 0.2 * torch.randn(d, generator=gen, device="cuda")).to(dt)
    new = lambda h: torch.zeros((T, h, d), dtype=dt, device="cuda")
    return {"op": "rope", "qkv": qkv, "hq": hq, "hkv": hkv, "d": d, "rot": rot, "table": table, "prefix": _i32(prefix),
            "depth": _i32(depth), "qo": _i32(_indptr(counts)), "qw": w() if case["norm"] else None,
            "kw": w() if case["norm"] else None, "interleaved": case["interleaved"], "eps": 1e-6,
            "out": (new(hq), new(hkv), new(hkv))}


def _held(case, counts, lens):
    need = (lens + counts + PAGE - 1) // PAGE
    if case["held"] == "none":
        return np.zeros_like(need), need
    if case["held"] == "step":        # what the tokens before this step filled
        return (lens + PAGE - 1) // PAGE, need
    return np.maximum(0, need + np.arange(len(need)) % 7 - 2), need     # some rows hold more, some less


def _prepare_pages(case, rng, gen):
    counts, lens = _sizes(case)
    held, need = _held(case, counts, lens)
    most = int(max(held.max(), need.max())) + 2
    table, _, left = _tables(rng, held, int(np.maximum(need - held, 0).sum()) + 7)
    full = np.full((case["batch"], most), -1, np.int64)
    full[:, :table.shape[1]] = table[:, :most]
    total = int(held.sum()) + len(left)
    free = np.full(total, -1, np.int64)
    free[:len(left)] = left
    return {"op": "pages", "len": _i32(lens), "qo": _i32(_indptr(counts)), "held": _i32(held), "table": _i32(full),
            "free": _i32(free), "n_free": _i32([len(left)]), "held_out": torch.zeros(case["batch"], dtype=torch.int32, device="cuda"),
            "n_free_out": torch.zeros(1, dtype=torch.int32, device="cuda"), "shrink": case["shrink"],
            "slots": torch.full((int(counts.sum()),), -1, dtype=torch.int64, device="cuda")}


# ---------------------------------------------------------------------------- one pass

def run(state):
    if own:
        return _OWN[state["op"]](state)
    return _PLAIN[state["op"]](state)


def _owner(qo, T):
    """The sequence of each of T rows."""
    return torch.searchsorted(qo[1:], torch.arange(T, dtype=qo.dtype, device=qo.device), right=True)


def _plain_attn(s):
    T, hq, d = s["q"].shape
    hkv = s["k_tree"].shape[1]
    B, N, G = s["prefix"].numel(), s["max_nodes"], hq // hkv
    pages = (s["max_prefix"] + PAGE - 1) // PAGE
    first, count = s["qo"][:-1].long(), (s["qo"][1:] - s["qo"][:-1]).long()
    at = torch.arange(N, device="cuda")
    real = at[None, :] < count[:, None]                                    # [B, N] nodes of each sequence
    rows = torch.where(real, first[:, None] + at[None, :], 0)
    # queries of a KV head: [B, hkv, N * G, d]
    q = s["q"][rows].float().view(B, N, hkv, G, d).permute(0, 2, 1, 3, 4).reshape(B, hkv, N * G, d)
    ids = s["table"][:, :pages].long().clamp_min(0)
    deq = lambda pool, w: (pool[ids].view(torch.float8_e4m3fn).float() * s["scale"][ids][..., w][..., None, None]
                           ).permute(0, 2, 1, 3, 4).reshape(B, hkv, pages * PAGE, d)
    tree = lambda x: x[rows].float().permute(0, 2, 1, 3)                   # [B, hkv, N, d]
    k = torch.cat([deq(s["k_pool"], 0), tree(s["k_tree"])], 2)
    score = (q @ k.transpose(2, 3)) * (d ** -0.5)
    del k
    seen = (s["mask"][rows][..., None] >> torch.arange(64, device="cuda") & 1).bool().view(B, N, -1)[..., :N]
    pre = torch.arange(pages * PAGE, device="cuda")[None, :] < s["prefix"][:, None]
    allow = torch.cat([pre[:, None, :].expand(B, N, -1), seen], 2)         # [B, N, keys]
    score = score.view(B, hkv, N, G, -1).masked_fill_(~allow[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True).clamp_min(-3e38)
    p = score.sub_(top).exp_()
    total = p.sum(-1)
    v = torch.cat([deq(s["v_pool"], 1), tree(s["v_tree"])], 2)
    o = (p.view(B, hkv, N * G, -1) @ v).view(B, hkv, N, G, d)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    lse = torch.log(total) + top[..., 0]
    b, i = _owner(s["qo"], T), torch.arange(T, device="cuda")
    i = i - first[b]
    return o[b, :, i].reshape(T, hq, d).to(torch.bfloat16), lse[b, :, i].reshape(T, hq)


def _plain_commit(s):
    B, cap = s["path"].shape
    T, hkv, d = s["k_tree"].shape
    P, L = s["prefix"].long(), s["accept"].long()
    np_ = (cap + PAGE - 2) // PAGE + 1                                      # pages a path can touch
    lp = P[:, None] // PAGE + torch.arange(np_, device="cuda")              # [B, np]
    slot = lp[..., None] * PAGE + torch.arange(PAGE, device="cuda")         # [B, np, 16]
    new = (slot >= P[:, None, None]) & (slot <= (P + L)[:, None, None])
    old = slot < P[:, None, None]
    touched = new.any(-1)
    page = torch.where(touched, s["table"].long().gather(1, lp.clamp_max(s["table"].shape[1] - 1)), 0)
    node = s["path"].long().gather(1, (slot - P[:, None, None]).clamp(0, cap - 1).view(B, -1)).view(slot.shape)
    row = torch.where(new, s["qo"][:-1].long()[:, None, None] + node, 0)
    for w, (src, pool) in enumerate(((s["k_tree"], s["k_pool"]), (s["v_tree"], s["v_pool"]))):
        x = src[row].float().permute(0, 1, 3, 2, 4)                         # [B, np, hkv, 16, d]
        keep = old[:, :, None, :, None]
        put = new[:, :, None, :, None]
        top = torch.where(put, x.abs(), 0.0).amax((3, 4))
        want = torch.exp2(torch.ceil(torch.log2((top / F8_MAX).clamp_min(2.0 ** SCALE_LO))).clamp(SCALE_LO, SCALE_HI))
        was = s["scale"][page][..., w]
        now = torch.where(old.any(-1)[..., None], torch.maximum(was, want), want)
        code = pool[page]
        have = code.view(torch.float8_e4m3fn).float() * was[..., None, None]
        val = torch.where(put, x, have) / now[..., None, None]
        val = val.clamp(-F8_MAX, F8_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
        hit = touched.nonzero(as_tuple=True)
        pool[page[hit]] = torch.where(put | keep, val, code)[hit]
        s["scale"][page[hit], :, w] = now[hit]
    s["seq_len"].copy_(P + L + 1)
    return s["k_pool"].view(torch.float8_e4m3fn), s["v_pool"].view(torch.float8_e4m3fn), s["scale"], s["seq_len"]


def _plain_rope(s):
    T, d, rot, hq, hkv = s["qkv"].shape[0], s["d"], s["rot"], s["hq"], s["hkv"]
    b = _owner(s["qo"], T)
    at = (s["prefix"][b] + s["depth"]).long()
    c, n = s["table"][at][:, None, :rot // 2], s["table"][at][:, None, rot // 2:]
    x = s["qkv"].view(T, hq + 2 * hkv, d)
    done = []
    for part, w in ((x[:, :hq], s["qw"]), (x[:, hq:hq + hkv], s["kw"])):
        y = part.float()
        if w is not None:
            y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + s["eps"]) * w.float()
        r = y[..., :rot]
        u, v = (r[..., 0::2], r[..., 1::2]) if s["interleaved"] else (r[..., :rot // 2], r[..., rot // 2:])
        u, v = u * c - v * n, v * c + u * n
        r = torch.stack([u, v], -1).flatten(-2) if s["interleaved"] else torch.cat([u, v], -1)
        done.append(torch.cat([r, y[..., rot:]], -1).to(part.dtype))
    return done[0], done[1], x[:, hq + hkv:].clone()


def _plain_pages(s):
    B, most = s["table"].shape
    total = s["free"].numel()
    lens, held, n0 = s["len"].long(), s["held"].long(), s["n_free"].long()
    count = (s["qo"][1:] - s["qo"][:-1]).long()
    need = (lens + count + PAGE - 1) // PAGE
    fits = need <= most
    grow = torch.where(fits, (need - held).clamp_min(0), 0)
    back = torch.where(fits, (held - need).clamp_min(0), 0) if s["shrink"] else torch.zeros_like(held)
    col = torch.arange(most, device="cuda")
    # returned pages go on the stack in order; grants come off its top
    start = n0 + back.cumsum(0) - back
    returned = (col[None, :] >= need[:, None]) & (col[None, :] < (need + back)[:, None])
    stack = torch.cat([s["free"], s["free"].new_zeros(1)])
    to = torch.where(returned, start[:, None] + col - need[:, None], total)
    stack.index_put_((to,), s["table"])
    n1 = n0 + back.sum()
    upto = grow.cumsum(0)
    ok = upto <= n1
    take = (n1 - 1 - (upto - grow))[:, None] - (col - held[:, None])
    given = (col[None, :] >= held[:, None]) & (col[None, :] < (held + grow)[:, None]) & ok[:, None]
    table = torch.where(given, stack[take.clamp(0, total - 1)], s["table"])
    now = torch.where(ok, held + grow, held) - back
    n2 = n1 - torch.where(ok, grow, 0).sum()
    place = torch.arange(total, device="cuda")
    free = torch.where((place >= n0) & (place < n2), stack[:total], s["free"])
    T = s["slots"].numel()
    b = _owner(s["qo"], T)
    pos = lens[b] + torch.arange(T, device="cuda") - s["qo"][b]
    lp = pos // PAGE
    slot = torch.where(lp < now[b], table[b, lp.clamp_max(most - 1)].long() * PAGE + pos % PAGE, -1)
    return table, now.to(torch.int32), free, n2.to(torch.int32), slot


_PLAIN = {"attn": _plain_attn, "commit": _plain_commit, "rope": _plain_rope, "pages": _plain_pages}


def _lib():
    from speculative_decoding_tree_parent_gb300 import binding
    return binding


def _own_attn(s):
    B = _lib()
    if "ws" not in s:
        T, hq, d = s["q"].shape
        n = B.spec_workspace_size(B.SPEC_OP_ATTN_KV8P, s["prefix"].numel(), T, s["max_nodes"], hq, s["k_tree"].shape[1],
                                  d, s["max_prefix"], 0)
        s["ws"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    B.spec_tree_verify_attn_kv8p(s["q"], s["k_pool"], s["v_pool"], s["scale"], s["table"], s["prefix"], s["max_prefix"],
                                 s["k_tree"], s["v_tree"], s["mask"], s["qo"], s["max_nodes"], s["out"], lse=s["lse"],
                                 ws=s["ws"])
    return s["out"], s["lse"]


def _own_commit(s):
    _lib().spec_kv_commit_kv8p(s["k_tree"], s["v_tree"], s["path"], s["accept"], s["qo"], s["table"], s["prefix"],
                               s["k_pool"], s["v_pool"], s["scale"], seq_len_out=s["seq_len"])
    return s["k_pool"].view(torch.float8_e4m3fn), s["v_pool"].view(torch.float8_e4m3fn), s["scale"], s["seq_len"]


def _own_rope(s):
    T, d, hq, hkv = s["qkv"].shape[0], s["d"], s["hq"], s["hkv"]
    x = s["qkv"].view(T, hq + 2 * hkv, d)
    q, k, v = s["out"]
    _lib().spec_qk_norm_rope(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], s["table"], s["prefix"], s["qo"], q, k, v,
                             depth=s["depth"], q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"],
                             interleaved=s["interleaved"])
    return q, k, v


def _own_pages(s):
    _lib().spec_page_table_resize(s["len"], s["qo"], s["held"], s["table"], s["free"], s["n_free"], s["held_out"],
                                  s["n_free_out"], slot_map=s["slots"], page_size=PAGE, shrink=s["shrink"])
    return s["table"], s["held_out"], s["free"], s["n_free_out"], s["slots"]


_OWN = {"attn": _own_attn, "commit": _own_commit, "rope": _own_rope, "pages": _own_pages}


# ---------------------------------------------------------------------------- what a pass costs

def work(case):
    a, b = _sizes(case)
    n, T = case["batch"], int(a.sum())
    if case["op"] == "attn":
        hq, hkv = case["hq"], case["hkv"]
        pages = int(((b + PAGE - 1) // PAGE).sum())
        words = (int(a.max()) + 63) // 64
        return {"bytes": int(b.sum()) * hkv * DIM * 2 + pages * (hkv * 8 + 4) + T * (hq + hkv) * DIM * 4 + T * hq * 4
                + T * words * 8 + n * 8, "flops": int(4 * hq * DIM * (a * (b + 1)).sum())}
    if case["op"] == "commit":
        rows = int((a + 1).sum()) * case["hkv"] * DIM * 2
        first = np.where(b % PAGE > 0, b % PAGE, 0).sum() * case["hkv"] * DIM * 2     # older codes of the first page
        pages = int(((b + a) // PAGE - b // PAGE + 1).sum())
        return {"bytes": int(rows * 3 + first + pages * (case["hkv"] * 8 + 4) + T * 4 + n * 16), "flops": rows * 3}
    if case["op"] == "rope":
        e = 2 if case["dtype"] == "bf16" else 4
        heads = case["hq"] + 2 * case["hkv"]
        return {"bytes": T * (2 * heads * case["d"] * e + case["rot"] * 4 + 4), "flops": T * heads * case["d"] * 7}
    held, need = _held(case, a, b)
    grow = int(np.maximum(need - held, 0).sum())
    pages = int(((b + a + PAGE - 1) // PAGE - b // PAGE).sum())     # entries that the slots are read from
    return {"bytes": T * 8 + grow * 8 + (pages - min(pages, grow)) * 4 + n * 16, "flops": T * 4}


# ---------------------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": _exact_attn, "commit": _exact_commit, "rope": _exact_rope, "pages": _exact_pages}[case["op"]](s)


def _exact_attn(s):
    T, hq, d = s["q"].shape
    hkv = s["k_tree"].shape[1]
    G = hq // hkv
    out = torch.zeros((T, hq, d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((T, hq), dtype=torch.float64, device="cuda")
    qo, prefix = s["qo"].tolist(), s["prefix"].tolist()
    value = torch.arange(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn).double()
    for b, P in enumerate(prefix):
        lo, hi = qo[b], qo[b + 1]
        ids = s["table"][b, :(P + PAGE - 1) // PAGE].long()
        shift = torch.arange(hi - lo, device="cuda")
        see = (s["mask"][lo:hi][:, shift // 64] >> (shift % 64)) & 1
        for g in range(hkv):
            kk = torch.cat([(value[s["k_pool"][ids, g].long()] * s["scale"][ids, g, 0].double()[:, None, None])
                            .reshape(-1, d)[:P], s["k_tree"][lo:hi, g].double()])
            vv = torch.cat([(value[s["v_pool"][ids, g].long()] * s["scale"][ids, g, 1].double()[:, None, None])
                            .reshape(-1, d)[:P], s["v_tree"][lo:hi, g].double()])
            x = torch.einsum("nhd,kd->nhk", s["q"][lo:hi, g * G:(g + 1) * G].double(), kk) / math.sqrt(d)
            x[:, :, P:][(see == 0)[:, None, :].expand(-1, G, -1)] = -math.inf
            z = torch.logsumexp(x, -1)
            out[lo:hi, g * G:(g + 1) * G] = torch.einsum("nhk,kd->nhd", torch.exp(x - z[..., None]), vv)
            lse[lo:hi, g * G:(g + 1) * G] = z
    return out, lse


_CODES = np.array([(-1) ** (c >> 7) * ((c & 7) * 2.0 ** -9 if c >> 3 & 15 == 0 else (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10))
                   for c in range(127)])    # the values of the codes 0 .. 126, rising


def _nearest(x):
    """The E4M3 value nearest to each |x|, ties to the even code, with x's sign."""
    a = np.minimum(np.abs(x), F8_MAX)
    hi = np.clip(np.searchsorted(_CODES, a), 1, 126)
    below, above = a - _CODES[hi - 1], _CODES[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.copysign(np.where(up, _CODES[hi], _CODES[hi - 1]), x)


def _exact_commit(s):
    c = {k: v.float().cpu().double().numpy() if v.dtype == torch.bfloat16 else v.cpu().numpy()
         for k, v in s.items() if isinstance(v, torch.Tensor)}
    pools = [s[n].view(torch.float8_e4m3fn).float().cpu().double().numpy() for n in ("k_pool", "v_pool")]
    scale = c["scale"].astype(np.float64)
    for b, (P, L) in enumerate(zip(c["prefix"], c["accept"])):
        rows = c["qo"][b] + c["path"][b, :L + 1]
        for lp in range(P // PAGE, (P + L) // PAGE + 1):
            page = c["table"][b, lp]
            lo, hi = max(P, lp * PAGE), min(P + L + 1, lp * PAGE + PAGE)
            for w, (src, pool) in enumerate(((c["k_tree"], pools[0]), (c["v_tree"], pools[1]))):
                x = src[rows[lo - P:hi - P]]                                # [new rows, hkv, d]
                for g in range(x.shape[1]):
                    top = np.abs(x[:, g]).max()
                    e = SCALE_LO
                    while e < SCALE_HI and top > F8_MAX * 2.0 ** e:
                        e += 1
                    now, r = 2.0 ** e, lo % PAGE
                    if r:
                        now = max(now, scale[page, g, w])
                        pool[page, g, :r] = _nearest(pool[page, g, :r] * scale[page, g, w] / now)
                    pool[page, g, r:r + hi - lo] = _nearest(x[:, g] / now)
                    scale[page, g, w] = now
    return pools[0], pools[1], scale, None


def _exact_rope(s):
    T, d, rot, hq, hkv = s["qkv"].shape[0], s["d"], s["rot"], s["hq"], s["hkv"]
    x = s["qkv"].double().view(T, hq + 2 * hkv, d)
    qo, half = s["qo"].tolist(), rot // 2
    place = torch.cat([s["prefix"][b].long() + s["depth"][lo:hi].long() for b, (lo, hi) in enumerate(zip(qo, qo[1:]))])
    turn = torch.complex(s["table"][place, :half].double(), s["table"][place, half:].double())[:, None]
    got = []
    for part, w in ((x[:, :hq], s["qw"]), (x[:, hq:hq + hkv], s["kw"])):
        y = part.clone()
        if w is not None:
            y *= (part.pow(2).sum(-1, keepdim=True) / d + s["eps"]).pow(-0.5)
            y *= w.double()
        i = torch.arange(half, device="cuda")
        one, two = (2 * i, 2 * i + 1) if s["interleaved"] else (i, i + half)
        z = torch.complex(y[..., one], y[..., two]) * turn
        y[..., one], y[..., two] = z.real, z.imag
        got.append(y)
    return got[0], got[1], x[:, hq + hkv:].clone()


def _exact_pages(s):
    return None          # whole numbers only: the outputs have to be equal
