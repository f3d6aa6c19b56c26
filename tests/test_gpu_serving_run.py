"""The serving operators as they are used together: prompts written page by page, then steps of
page-table growth, norm + rotation, mask, attention, acceptance and commit, eager and replayed
from one captured graph with other trees. Every stage is checked against the oracle's form of it,
given what the stages before wrote (so codes, scales, tables, paths and lengths are equal, and
only the two stages in floating point have bounds: those of their own tests)."""

from types import SimpleNamespace

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_parent_gb300 import binding as B
from speculative_decoding_tree_parent_gb300 import workloads as W
from speculative_decoding_tree_parent_gb300.step import DeviceBatch

import serving_cases as S

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BATCH, HQ, HKV, D, PS = 4, 8, 2, 128, 16
TOTAL, NODES, CAP, VOCAB = 100, 40, 9, 48    # nodes of a step (the mask call's contract) and of a tree; path places; tokens
LONGEST, PAGES, MOST = 400, 120, 30          # longest prefix; pool pages; pages of a row
EPS = 1e-5


class Run:
    """Device buffers of a fixed shape, their host copies, and the step's calls."""

    def __init__(self, seed):
        self.rng = np.random.default_rng(seed)
        z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt, device="cuda")
        T = TOTAL
        self.T = T
        self.qkv = z(T, (HQ + 2 * HKV) * D, dt=torch.bfloat16)
        self.w = [torch.from_numpy(S.bf16(self.rng.uniform(0.5, 1.5, D))).to("cuda", torch.bfloat16) for _ in range(2)]
        ang = np.arange(LONGEST + NODES)[:, None] * 10000.0 ** (-np.arange(D // 2) / (D / 2))
        self.tab = np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)
        self.cos_sin = torch.from_numpy(self.tab).cuda()
        self.parent, self.tokens, self.qo = z(T), z(T), z(BATCH + 1)
        self.logits = z(T, VOCAB, dt=torch.float32)
        self.mask, self.depth = z(T, 1, dt=torch.int64), z(T)
        bf = lambda h: z(T, h, D, dt=torch.bfloat16)
        self.q, self.k, self.v, self.out = bf(HQ), bf(HKV), bf(HKV), bf(HQ)
        self.lse = z(T, HQ, dt=torch.float32)
        self.path, self.out_tokens, self.acc = z(BATCH, CAP), z(BATCH, CAP), z(BATCH)
        self.prefix, self.nxt, self.held = z(BATCH), z(BATCH), z(BATCH)
        self.table = torch.full((BATCH, MOST), -1, dtype=torch.int32, device="cuda")
        self.free = torch.from_numpy(self.rng.permutation(PAGES).astype(np.int32)).cuda()
        self.n_free = torch.tensor([PAGES], dtype=torch.int32, device="cuda")
        self.slots = z(T, dt=torch.int64)
        self.kp, self.vp = (z(PAGES, HKV, PS, D, dt=torch.uint8) for _ in range(2))
        self.scale = torch.ones((PAGES, HKV, 2), dtype=torch.float32, device="cuda")
        self.status = z(1)
        ws = lambda op, *a: torch.zeros(max(256, B.spec_workspace_size(op, BATCH, T, NODES, *a)), dtype=torch.uint8,
                                        device="cuda")
        self.attn_ws = ws(B.SPEC_OP_ATTN_KV8P, HQ, HKV, D, LONGEST, 0)
        self.acc_ws = ws(B.SPEC_OP_ACCEPT, 0, 0, 0, 0, VOCAB)

    def rope(self, qkv, qo, q, k, v, depth):
        x = qkv.view(qkv.shape[0], HQ + 2 * HKV, D)
        B.spec_qk_norm_rope(x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], self.cos_sin, self.prefix, qo, q, k, v,
                            depth=depth, q_weight=self.w[0], k_weight=self.w[1], eps=EPS, dev_status=self.status)

    def resize(self, qo, slots):
        B.spec_page_table_resize(self.prefix, qo, self.held, self.table, self.free, self.n_free, self.held, self.n_free,
                                 slot_map=slots, page_size=PS, shrink=True, dev_status=self.status)

    def prompts(self, lengths):
        """The prompts' rows, committed as chains."""
        qo = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
        T = int(qo[-1])
        qkv = torch.from_numpy(S.bf16(self.rng.standard_normal((T, (HQ + 2 * HKV) * D)))).to("cuda", torch.bfloat16)
        q, k, v = (torch.empty((T, h, D), dtype=torch.bfloat16, device="cuda") for h in (HQ, HKV, HKV))
        path = torch.arange(max(lengths), dtype=torch.int32, device="cuda").repeat(BATCH, 1)
        acc = torch.tensor([n - 1 for n in lengths], dtype=torch.int32, device="cuda")
        dqo = torch.from_numpy(qo).cuda()
        host = self.state()
        slots = torch.zeros(T, dtype=torch.int64, device="cuda")
        self.resize(dqo, slots)
        self.rope(qkv, dqo, q, k, v, None)
        B.spec_kv_commit_kv8p(k, v, path, acc, dqo, self.table, self.prefix, self.kp, self.vp, self.scale,
                              seq_len_out=self.nxt, dev_status=self.status)
        self.prefix.copy_(self.nxt)
        pos = np.concatenate([np.arange(n) for n in lengths])
        self.check_pages(host, qo, slots)
        self.check_rope(qkv, T, pos, q, k, v)
        self.check_commit(host, qo, k, v, path.cpu().numpy(), acc.cpu().numpy())

    def draw(self, sizes):
        """A step's inputs, into the buffers that the captured calls read."""
        rng = self.rng
        parent, qo, mask = S.trees(sizes, rng)
        n = int(qo[-1])
        tokens = rng.integers(0, VOCAB, n).astype(np.int32)
        logits = rng.standard_normal((n, VOCAB)).astype(np.float32)
        for b in range(BATCH):                    # most nodes agree with one child, so that paths are taken
            for i in range(1, sizes[b]):
                if rng.random() < 0.8:
                    logits[qo[b] + parent[qo[b] + i], tokens[qo[b] + i]] += 6.0
        x = S.bf16(rng.standard_normal((self.T, (HQ + 2 * HKV) * D)))
        self.qkv.copy_(torch.from_numpy(x))
        self.parent[:n].copy_(torch.from_numpy(parent))
        self.tokens[:n].copy_(torch.from_numpy(tokens))
        self.logits[:n].copy_(torch.from_numpy(logits))
        self.qo.copy_(torch.from_numpy(qo))
        self.host = SimpleNamespace(parent=parent, qo=qo, mask=mask, tokens=tokens, logits=logits, n=n)

    def calls(self):
        self.resize(self.qo, self.slots)
        B.spec_build_tree_mask(self.parent, self.qo, NODES, self.mask, self.depth, self.status)
        self.rope(self.qkv, self.qo, self.q, self.k, self.v, self.depth)
        B.spec_tree_verify_attn_kv8p(self.q, self.kp, self.vp, self.scale, self.table, self.prefix, LONGEST, self.k,
                                     self.v, self.mask, self.qo, NODES, self.out, lse=self.lse, ws=self.attn_ws,
                                     dev_status=self.status)
        B.spec_accept(B.SPEC_GREEDY, self.parent, self.tokens, self.logits, self.qo, NODES, self.acc, self.path,
                      self.out_tokens, self.acc_ws, dev_status=self.status)
        B.spec_kv_commit_kv8p(self.k, self.v, self.path, self.acc, self.qo, self.table, self.prefix, self.kp, self.vp,
                              self.scale, seq_len_out=self.nxt, dev_status=self.status)
        self.prefix.copy_(self.nxt)

    # --- the oracle's side ---------------------------------------------------------------
    def state(self):
        torch.cuda.synchronize()
        h = lambda t: t.cpu().numpy().copy()
        return SimpleNamespace(prefix=h(self.prefix), held=h(self.held), table=h(self.table), free=h(self.free),
                               n_free=int(self.n_free.item()), k=h(self.kp), v=h(self.vp), scale=h(self.scale))

    def check_pages(self, before, qo, slots):
        table, held, free, n_free, want, errors = oracle.page_table_resize(
            before.prefix, qo, before.held, before.table, before.free, before.n_free, PS, True)
        torch.cuda.synchronize()
        assert not errors and int(self.status.item()) == 0
        assert np.array_equal(self.held.cpu().numpy(), held) and int(self.n_free.item()) == n_free
        assert np.array_equal(self.free.cpu().numpy()[:n_free], free[:n_free])
        got = self.table.cpu().numpy()
        for b in range(BATCH):
            assert np.array_equal(got[b, :held[b]], table[b, :held[b]])
        assert np.array_equal(slots.cpu().numpy()[:len(want)], want)

    def check_rope(self, qkv, n, pos, q, k, v):
        x = qkv.float().cpu().numpy().reshape(-1, HQ + 2 * HKV, D)[:n]
        w = [t.float().cpu().numpy() for t in self.w]
        a = (x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], *w, EPS)
        want, flat = oracle.qk_norm_rope(*a, self.tab, pos, False), oracle.qk_norm_rope(*a, None, pos, False)
        for got, ref, y in zip((q, k), want, flat):
            mag = np.abs(y).copy()
            both = mag[..., :D // 2] + mag[..., D // 2:]
            mag[..., :D // 2], mag[..., D // 2:] = both, both
            err = np.abs(got[:n].double().cpu().numpy() - ref)
            assert (err <= 2.0 ** -8 * np.abs(ref) + (D / 2 + 12) * 2.0 ** -24 * mag).all()
        assert np.array_equal(v[:n].float().cpu().numpy(), a[2])

    def check_commit(self, before, qo, k, v, path, acc):
        n = int(qo[-1])
        f = lambda t: t[:n].float().cpu().numpy()
        kp, vp, scale, seq = oracle.kv8p_commit(before.k, before.v, before.scale, self.table.cpu().numpy(),
                                                before.prefix, f(k), f(v), path, acc, qo)
        after = self.state()
        assert np.array_equal(after.prefix, seq) and np.array_equal(after.scale, scale)
        assert np.array_equal(after.k, kp) and np.array_equal(after.v, vp)

    def check_step(self, before):
        torch.cuda.synchronize()
        assert int(self.status.item()) == 0
        h, n = self.host, self.host.n
        self.check_pages(before, h.qo, self.slots)
        assert np.array_equal(self.mask[:n].cpu().numpy(), S.words(h.mask))
        depth = h.mask.sum(1) - 1
        assert np.array_equal(self.depth[:n].cpu().numpy(), depth)
        pos = np.concatenate([before.prefix[b] + depth[h.qo[b]:h.qo[b + 1]] for b in range(BATCH)])
        self.check_rope(self.qkv, n, pos, self.q, self.k, self.v)
        f = lambda t: t[:n].float().cpu().numpy()
        c = SimpleNamespace(k=before.k, v=before.v, scale=before.scale, qo=h.qo, q=f(self.q), kt=f(self.k), vt=f(self.v),
                            table=self.table.cpu().numpy(), prefix=before.prefix, mask=h.mask, hq=HQ, hkv=HKV)
        ref, lse, A = S.reference(c)
        err = np.abs(self.out[:n].double().cpu().numpy() - ref)
        assert (err <= 2.0 ** -10 * A + 2.0 ** -8 * np.abs(ref) + 1e-9).all()
        assert np.abs(self.lse[:n].double().cpu().numpy() - lse).max() <= 2.0 ** -12
        a = oracle.greedy_accept(h.parent, h.tokens, h.logits, h.qo, CAP)
        acc, path, toks = a.accept_len, a.path, a.out_tokens
        assert np.array_equal(self.acc.cpu().numpy(), acc)
        got, gt = self.path.cpu().numpy(), self.out_tokens.cpu().numpy()
        for b in range(BATCH):
            assert np.array_equal(got[b, :acc[b] + 1], path[b, :acc[b] + 1])
            assert np.array_equal(gt[b, :acc[b] + 1], toks[b, :acc[b] + 1])
        self.check_commit(before, h.qo, self.k, self.v, got, acc)
        return int(acc.sum())


def test_steps_together_eager_and_captured():
    r = Run(5)
    r.prompts([1, 5, 120, 250])
    taken = 0
    r.draw([7, 13, 40, 40])
    before = r.state()
    r.calls()
    taken += r.check_step(before)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r.calls()
    for sizes in ([40, 40, 19, 1], [25, 25, 25, 25], [1, 39, 20, 40]):
        r.draw(sizes)
        before = r.state()
        graph.replay()
        taken += r.check_step(before)
    assert taken > 0                                        # paths beyond the root were committed


def batch(**kw):
    return W.generate_index(3, batch=3, hq=8, hkv=2, vocab=512, prefix=(90, 300), tree="random", nodes=(24, 24),
                            max_depth=5, agree_prob=0.8, extra_pages=12, **kw)


@pytest.mark.parametrize("fused", [False, True])
def test_device_batch_with_page_scales(fused):
    inp = batch()
    db = DeviceBatch(inp, kv_fp8="page")
    kc, vc, sc = db.kv_codes
    launches = db.step(fused=fused)
    torch.cuda.synchronize()
    assert db.device_status() == 0 and launches == db.launches_per_step(fused=fused)
    mask = oracle.ancestor_mask_batch(inp.parent, inp.qo_indptr)[0]
    c = SimpleNamespace(k=kc, v=vc, scale=sc, qo=inp.qo_indptr, q=inp.q, kt=inp.k_tree, vt=inp.v_tree,
                        table=inp.page_table, prefix=inp.prefix_len, mask=mask, hq=inp.hq, hkv=inp.hkv)
    ref, lse, A = S.reference(c)
    err = np.abs(db.out.double().cpu().numpy() - ref)
    assert (err <= 2.0 ** -10 * A + 2.0 ** -8 * np.abs(ref) + 1e-9).all()
    a = oracle.greedy_accept(inp.parent, inp.draft_tokens, inp.target_logits, inp.qo_indptr, inp.path_cap)
    acc, path = a.accept_len, a.path
    assert np.array_equal(db.accept_len.cpu().numpy(), acc)
    kp, vp, scale, seq = oracle.kv8p_commit(kc, vc, sc, inp.page_table, inp.prefix_len, inp.k_tree, inp.v_tree, path, acc,
                                            inp.qo_indptr)
    assert np.array_equal(db.k_pool.cpu().numpy(), kp) and np.array_equal(db.v_pool.cpu().numpy(), vp)
    assert np.array_equal(db.kv_scale.cpu().numpy(), scale) and np.array_equal(db.seq_len.cpu().numpy(), seq)
