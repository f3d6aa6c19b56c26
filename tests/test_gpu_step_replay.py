"""Whole steps captured once and replayed with other trees, logits, lengths and pages, every kernel
starting while the one before it runs: each result has the bits of the same calls made one at a time,
each waited for. The page tables of a step are written by the resize in front of it (on the device,
from the lengths); accepted paths, codes and pages are compared with the oracle as well."""

import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_tree_parent_gb300 import binding as B
from speculative_decoding_tree_parent_gb300 import workloads as W
from speculative_decoding_tree_parent_gb300.step import DeviceBatch

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BATCH, NODES, CAP, REPLAYS = 6, 24, 8, 6
FED = ("parent", "tokens", "q", "k_tree", "v_tree", "target_logits", "prefix_len", "draft_logits", "uniforms")
READ = ("mask", "depth", "out", "lse", "accept_len", "path", "out_tokens", "seq_len", "k_pool", "v_pool", "page_table")


def inputs(seed, mode):
    return W.generate(W.spec(3, batch=BATCH, hq=16, hkv=2, vocab=640, prefix=(90, 900), tree="random",
                             nodes=(NODES, NODES), max_depth=5, agree_prob=0.8, extra_pages=200, modes=(mode,),
                             draft_noise=0.5 if mode == "stochastic" else None), seed=seed)


class Step:
    """A step with its page tables, over one set of device buffers."""

    def __init__(self, inp, kv, mode, fused, early):
        self.db, self.fused, self.mode, self.early = DeviceBatch(inp, mode=mode, kv_fp8=kv), fused, mode, early
        db = self.db
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        db.path, db.out_tokens = z(BATCH, CAP), z(BATCH, CAP)
        db.max_prefix = 900
        op = B.SPEC_OP_ATTN_KV8P if kv == "page" else B.SPEC_OP_ATTN
        need = B.spec_workspace_size(op, BATCH, db.T, db.max_nodes, inp.hq, inp.hkv, inp.d, 900, 0)
        db.attn_ws = torch.zeros(max(need, 256), dtype=torch.uint8, device="cuda")
        self.pages = db.k_pool.shape[0]
        most = (900 + NODES) // 16 + 1
        self.stack, self.free, self.n_free = z(self.pages), z(self.pages), z(1)
        self.held, self.slots = z(BATCH), torch.zeros(db.T, dtype=torch.int64, device="cuda")
        db.page_table = z(BATCH, most)

    def feed(self, inp, seed):
        rng = np.random.default_rng(seed)
        self.stack.copy_(torch.from_numpy(rng.permutation(self.pages).astype(np.int32)))
        other = DeviceBatch(inp, mode=self.mode)
        for n in FED:
            if getattr(self.db, n) is not None:
                getattr(self.db, n).copy_(getattr(other, n))
        torch.cuda.synchronize()

    def calls(self, sync=lambda: None):
        db = self.db
        self.free.copy_(self.stack)
        self.n_free.fill_(self.pages)
        self.held.zero_()
        db.page_table.fill_(-1)
        sync()
        B.spec_page_table_resize(db.prefix_len, db.qo, self.held, db.page_table, self.free, self.n_free, self.held,
                                 self.n_free, slot_map=self.slots, page_size=16, dev_status=db.status)
        sync()
        db.build_mask()
        sync()
        db.attention()
        sync()
        with B.early_reads(self.early):       # (the kernel before, the attention, writes none of its inputs)
            if self.fused:
                db.accept_commit()
            else:
                db.accept()
                sync()
                db.commit()
        sync()

    def results(self):
        torch.cuda.synchronize()
        assert int(self.db.status.item()) == 0
        names = READ + (("kv_scale",) if self.db.kv_page else ())
        return {n: getattr(self.db, n).clone() for n in names}


@pytest.mark.parametrize("kv,mode,fused,early", [
    (False, "greedy", False, False), (False, "greedy", True, False), (False, "greedy", True, True),
    (False, "stochastic", False, False), (False, "stochastic", True, False), (True, "greedy", False, False),
    (True, "stochastic", False, False), ("page", "greedy", False, False)])
def test_replays_equal_calls_made_one_at_a_time(kv, mode, fused, early):
    first = inputs(100, mode)
    a, b = Step(first, kv, mode, fused, early), Step(first, kv, mode, fused, early)
    a.feed(first, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        a.calls()
    lengths = set()
    for i in range(REPLAYS):
        inp = inputs(100 + i, mode)
        a.feed(inp, i)
        b.feed(inp, i)
        before = [t.clone() for t in (b.db.k_pool, b.db.v_pool)]
        graph.replay()
        got = a.results()
        b.calls(torch.cuda.synchronize)
        want = b.results()
        for n in want:
            assert torch.equal(got[n], want[n]), (n, i)
        lengths |= set(want["accept_len"].tolist())
        if mode == "greedy":
            acc = oracle.greedy_accept(inp.parent, inp.draft_tokens, inp.target_logits, inp.qo_indptr, CAP)
            assert np.array_equal(got["accept_len"].cpu().numpy(), acc.accept_len)
        if kv is False:                       # the committed rows, and nothing else
            table, path, acc = (got[n].cpu().numpy() for n in ("page_table", "path", "accept_len"))
            for n, tree, old in zip(("k_pool", "v_pool"), (inp.k_tree, inp.v_tree), before):
                new = old.float().cpu().numpy()
                for s in range(BATCH):
                    for k in range(int(acc[s]) + 1):
                        at = int(inp.prefix_len[s]) + k
                        new[table[s, at // 16], :, at % 16] = tree[int(inp.qo_indptr[s]) + path[s, k]]
                assert np.array_equal(got[n].float().cpu().numpy(), new)
    assert max(lengths) > 0
