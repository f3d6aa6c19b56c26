"""Shapes and types that the binding of the serving operators compares before it calls the library: a
pool of another head dim, an output too small and the like are refused, not read or written out of
range. Stand-ins with a device tensor's surface are passed and the library is replaced, so nothing is
launched. No GPU is used."""

import pytest
import torch

from speculative_decoding_tree_parent_gb300 import binding as B

T, HQ, HKV, D, PAGES, SEQS, MOST, CAP = 6, 8, 2, 128, 5, 3, 4, 9


class Stand:
    """What the binding asks of a contiguous device tensor."""

    is_cuda = True

    def __init__(self, *shape, dt=torch.bfloat16):
        self.t, self.shape, self.dtype = torch.empty(shape, dtype=dt, device="meta"), torch.Size(shape), dt

    def numel(self):
        return self.t.numel()

    def stride(self):
        return self.t.stride()

    def is_contiguous(self):
        return True

    def element_size(self):
        return self.t.element_size()

    def data_ptr(self):
        return 4096

    def long(self):
        return Stand(*self.shape, dt=torch.int64)


class Reached(Exception):
    pass


@pytest.fixture(autouse=True)
def no_library(monkeypatch):
    def reached(*a):
        raise Reached
    names = [n for n in B.EXPORTS]
    lib = type("Lib", (), {n: staticmethod(reached) for n in names})
    monkeypatch.setattr(B, "load", lambda *a: lib)
    monkeypatch.setattr(B, "_lib", lib)
    monkeypatch.setattr(B, "_stream", lambda s: None)


def z(*s, dt=torch.bfloat16):
    return Stand(*s, dt=dt)


def i(*s):
    return z(*s, dt=torch.int32)


def attn(**kw):
    a = dict(q=z(T, HQ, D), k_pool=z(PAGES, HKV, 16, D, dt=torch.uint8), v_pool=z(PAGES, HKV, 16, D, dt=torch.uint8),
             kv_scale=z(PAGES, HKV, 2, dt=torch.float32), page_table=i(SEQS, MOST), prefix_len=i(SEQS), max_prefix=64,
             k_tree=z(T, HKV, D), v_tree=z(T, HKV, D), mask=z(T, 1, dt=torch.int64), qo_indptr=i(SEQS + 1), max_nodes=4,
             out=z(T, HQ, D), lse=z(T, HQ, dt=torch.float32))
    a.update(kw)
    return B.spec_tree_verify_attn_kv8p(**a)


def commit(**kw):
    a = dict(k_tree=z(T, HKV, D), v_tree=z(T, HKV, D), path=i(SEQS, CAP), accept_len=i(SEQS), qo_indptr=i(SEQS + 1),
             page_table=i(SEQS, MOST), prefix_len=i(SEQS), k_pool=z(PAGES, HKV, 16, D, dt=torch.uint8),
             v_pool=z(PAGES, HKV, 16, D, dt=torch.uint8), kv_scale=z(PAGES, HKV, 2, dt=torch.float32), seq_len_out=i(SEQS))
    a.update(kw)
    return B.spec_kv_commit_kv8p(**a)


def rope(**kw):
    a = dict(q=z(T, HQ, D), k=z(T, HKV, D), v=z(T, HKV, D), cos_sin=z(50, D, dt=torch.float32), prefix_len=i(SEQS),
             qo_indptr=i(SEQS + 1), q_out=z(T, HQ, D), k_out=z(T, HKV, D), v_out=z(T, HKV, D), depth=i(T), q_weight=z(D),
             k_weight=z(D))
    a.update(kw)
    return B.spec_qk_norm_rope(**a)


def pages(**kw):
    a = dict(seq_len=i(SEQS), qo_indptr=i(SEQS + 1), held=i(SEQS), page_table=i(SEQS, MOST), free_pages=i(PAGES),
             n_free=i(1), held_out=i(SEQS), n_free_out=i(1), slot_map=z(T, dt=torch.int64))
    a.update(kw)
    return B.spec_page_table_resize(**a)


@pytest.mark.parametrize("call", [attn, commit, rope, pages])
def test_matching_shapes_reach_the_library(call):
    with pytest.raises(Reached):
        call()


def test_larger_buffers_are_fine():
    """Arrays with room to spare, as a serving loop keeps them."""
    for call, kw in ((attn, dict(page_table=i(SEQS + 2, MOST), lse=z(T + 4, HQ, dt=torch.float32), prefix_len=i(SEQS + 2))),
                     (commit, dict(path=i(SEQS + 2, CAP), accept_len=i(SEQS + 1))), (rope, dict(depth=i(T + 3))),
                     (pages, dict(held=i(SEQS + 4), slot_map=z(T + 9, dt=torch.int64)))):
        with pytest.raises(Reached):
            call(**kw)


def pool(*s):
    return dict(k_pool=z(*s, dt=torch.uint8), v_pool=z(*s, dt=torch.uint8), kv_scale=z(s[0], s[1], 2, dt=torch.float32))


@pytest.mark.parametrize("call", [attn, commit])
@pytest.mark.parametrize("kw,match", [
    (pool(PAGES, HKV, 16, 64), "pools"), (dict(kv_scale=z(PAGES, HKV, dt=torch.float32)), "kv_scale"),
    (dict(page_table=i(SEQS - 1, MOST)), "page_table"), (dict(page_table=i(SEQS, MOST).long()), "page_table"),
    (dict(prefix_len=i(SEQS - 1)), "prefix_len"), (dict(prefix_len=i(SEQS).long()), "prefix_len"),
    (dict(v_tree=z(T, HKV, D - 1)), "v_tree"), (dict(dev_status=z(1, dt=torch.int64)), "dev_status")])
def test_shapes_of_both_cache_calls(call, kw, match):
    with pytest.raises(ValueError, match=match):
        call(**kw)


@pytest.mark.parametrize("call,kw,match", [
    (commit, pool(PAGES, HKV + 1, 16, D), "pools"), (commit, dict(v_tree=z(T - 1, HKV, D)), "v_tree"),
    (commit, dict(path=i(SEQS - 1, CAP)), "path"), (commit, dict(accept_len=i(SEQS - 1)), "accept_len"),
    (commit, dict(seq_len_out=i(SEQS - 1)), "seq_len_out"), (commit, dict(qo_indptr=i(SEQS + 1).long()), "qo_indptr"),
    (attn, pool(PAGES, HKV + 1, 16, D), "pools"), (attn, dict(k_tree=z(T - 1, HKV, D)), "k_tree"),
    (attn, dict(mask=z(T - 1, 1, dt=torch.int64)), "mask"), (attn, dict(max_nodes=65), "mask"),
    (attn, dict(out=z(T, HQ - 1, D)), "out"), (attn, dict(lse=z(T, HQ - 1, dt=torch.float32)), "lse"),
    (attn, dict(lse=z(T, HQ)), "lse"),
    (rope, dict(q_out=z(T, HQ, D - 16)), "q_out"), (rope, dict(k_out=z(T - 1, HKV, D)), "k_out"),
    (rope, dict(v_out=z(T, 1, D)), "v_out"), (rope, dict(q_weight=z(D - 1)), "q_weight"), (rope, dict(depth=i(T - 1)), "depth"),
    (rope, dict(k=z(T - 1, HKV, D)), "k"), (rope, dict(k=z(T, HKV, D - 16)), "k"), (rope, dict(v=z(T, HKV + 1, D)), "v"),
    (rope, dict(prefix_len=i(SEQS - 1)), "prefix_len"), (rope, dict(depth=i(T).long()), "depth"),
    (pages, dict(held=i(SEQS - 1)), "held"), (pages, dict(held_out=i(SEQS - 1)), "held_out"),
    (pages, dict(page_table=i(SEQS - 1, MOST)), "page_table"), (pages, dict(n_free=i(0)), "n_free"),
    (pages, dict(seq_len=i(SEQS - 1)), "seq_len")])
def test_shapes(call, kw, match):
    with pytest.raises(ValueError, match=match):
        call(**kw)
