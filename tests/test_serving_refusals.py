"""Host checks of the serving operators: each call returns at its check, so no pointer is
followed and no GPU is needed."""

import ctypes

import pytest
import torch

from speculative_decoding_tree_parent_gb300 import binding as B
from speculative_decoding_tree_parent_gb300 import build

OK, ODD = ctypes.c_void_p(4096), ctypes.c_void_p(4098)
ARG, WS, UNSUP = -1, -5, -6


@pytest.fixture(scope="module")
def lib():
    return B.load(build.build())


def _attn(lib, **kw):
    a = dict(q=OK, k=OK, v=OK, s=OK, num_pages=300, ps=16, pt=OK, max_pages=300, pl=OK, max_prefix=4096, kt=OK, vt=OK,
             mask=OK, qo=OK, batch=1, T=64, N=64, hq=32, hkv=8, d=128, scale=0.0, out=OK, lse=None, ws=OK,
             bytes=1 << 40, status=None, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.spec_tree_verify_attn_kv8p(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), ARG), (dict(T=-1), ARG), (dict(N=0), ARG), (dict(N=1025), ARG), (dict(max_prefix=-1), ARG),
    (dict(hq=30), ARG), (dict(hkv=0), ARG), (dict(d=64), UNSUP), (dict(ps=32), UNSUP), (dict(hq=1032, hkv=8), UNSUP),
    (dict(batch=8192), UNSUP), (dict(q=None), ARG), (dict(mask=None), ARG), (dict(out=None), ARG), (dict(s=None), ARG),
    (dict(k=None), ARG), (dict(pt=None), ARG), (dict(max_pages=255), ARG), (dict(q=ODD), ARG), (dict(vt=ODD), ARG),
    (dict(v=ODD), ARG), (dict(s=ODD), ARG), (dict(num_pages=0), ARG)])
def test_attention_refuses(lib, kw, code):
    assert _attn(lib, **kw) == code


def test_attention_workspace_and_no_work(lib):
    need = B.spec_workspace_size(B.SPEC_OP_ATTN_KV8P, 1, 64, 64, 32, 8, 128, 4096, 0)
    if need:
        assert _attn(lib, ws=None) == WS and _attn(lib, bytes=need - 1) == WS and _attn(lib, ws=ODD) == WS
    assert _attn(lib, batch=0) == 0 and _attn(lib, T=0) == 0
    assert B.spec_workspace_size(B.SPEC_OP_ATTN_KV8P, 1, 64, 64, 32, 8, 64, 4096, 0) == 0
    assert B.spec_workspace_size(B.SPEC_OP_ATTN_KV8P, 1, 64, 64, 30, 8, 128, 4096, 0) == 0


def _commit(lib, **kw):
    a = dict(kt=OK, vt=OK, path=OK, cap=9, acc=OK, qo=OK, pt=OK, max_pages=4, num_pages=4, ps=16, pl=OK, seq=None,
             k=OK, v=OK, s=OK, batch=1, T=4, hkv=8, d=128, status=None, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.spec_kv_commit_kv8p(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(cap=0), ARG), (dict(batch=-1), ARG), (dict(d=24), UNSUP), (dict(ps=128), UNSUP), (dict(d=528), UNSUP),
    (dict(s=None), ARG), (dict(path=None), ARG), (dict(k=ODD), ARG), (dict(kt=ODD), ARG), (dict(hkv=70000), UNSUP),
    (dict(batch=0), 0)])
def test_commit_refuses(lib, kw, code):
    assert _commit(lib, **kw) == code


def _rope(lib, **kw):
    a = dict(dtype=1, q=OK, qs=4096, k=OK, ks=1024, v=OK, vs=1024, qw=OK, kw=OK, eps=1e-6, tab=OK, max_pos=100, rot=128,
             inter=0, pl=OK, depth=OK, qo=OK, batch=1, T=4, hq=32, hkv=8, d=128, qo_=OK, ko=OK, vo=OK, status=None,
             stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.spec_qk_norm_rope(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), UNSUP), (dict(batch=-1), ARG), (dict(hq=0), ARG), (dict(d=72), UNSUP), (dict(d=528, rot=16), UNSUP),
    (dict(rot=136), UNSUP), (dict(rot=144), UNSUP), (dict(rot=8), UNSUP), (dict(rot=-16), ARG), (dict(eps=-1.0), ARG),
    (dict(eps=float("nan")), ARG), (dict(vo=None), ARG), (dict(v=None), ARG), (dict(qs=4095), ARG), (dict(qs=4100), ARG),
    (dict(ks=1000), ARG), (dict(vs=512), ARG), (dict(tab=None), ARG), (dict(max_pos=0), ARG), (dict(pl=None), ARG),
    (dict(q=ODD), ARG), (dict(vo=ODD), ARG), (dict(qw=ODD), ARG), (dict(tab=ODD), ARG), (dict(hq=5000, qs=640000), UNSUP),
    (dict(batch=0), 0), (dict(T=0), 0)])
def test_rope_refuses(lib, kw, code):
    assert _rope(lib, **kw) == code


def _pages(lib, **kw):
    a = dict(seq=OK, qo=OK, held=OK, pt=OK, max_pages=8, free=OK, num_pages=64, n=OK, ps=16, shrink=0, batch=4, T=8,
             held_out=OK, n_out=OK, slots=OK, status=None, stream=None)
    assert not set(kw) - set(a)
    a.update(kw)
    return lib.spec_page_table_resize(*a.values())


@pytest.mark.parametrize("kw,code", [
    (dict(batch=-1), ARG), (dict(T=-1), ARG), (dict(max_pages=0), ARG), (dict(num_pages=0), ARG), (dict(ps=0), ARG),
    (dict(batch=4097), UNSUP), (dict(batch=4096, max_pages=1 << 20), UNSUP), (dict(seq=None), ARG),
    (dict(held=None), ARG), (dict(n_out=None), ARG), (dict(free=None), ARG), (dict(batch=0), 0)])
def test_resize_refuses(lib, kw, code):
    assert _pages(lib, **kw) == code


def test_binding_refuses_wrong_tensors():
    """Types, shapes and places that the binding checks before the library is called."""
    z = lambda *s, dt=torch.bfloat16: torch.zeros(s, dtype=dt)
    i = lambda *s: torch.zeros(s, dtype=torch.int32)
    with pytest.raises(ValueError):    # pools are codes
        B.spec_kv_commit_kv8p(z(4, 8, 128), z(4, 8, 128), i(1, 9), i(1), i(2), i(1, 4), i(1), z(4, 8, 16, 128),
                              z(4, 8, 16, 128), z(4, 8, 2, dt=torch.float32))
    u = z(4, 8, 16, 128, dt=torch.uint8)
    with pytest.raises(ValueError):    # the scale array of the per-head calls
        B.spec_kv_commit_kv8p(z(4, 8, 128), z(4, 8, 128), i(1, 9), i(1), i(2), i(1, 4), i(1), u, u,
                              z(2, 8, dt=torch.float32))
    with pytest.raises(ValueError):    # host tensors
        B.spec_tree_verify_attn_kv8p(z(4, 32, 128), u, u, z(4, 8, 2, dt=torch.float32), i(1, 4), i(1), 16, z(4, 8, 128),
                                     z(4, 8, 128), z(4, 1, dt=torch.int64), i(2), 4, z(4, 32, 128))
    with pytest.raises(ValueError):
        B.spec_page_table_resize(i(1), i(2), i(1).long(), i(1, 4), i(4), i(1), i(1), i(1))
    with pytest.raises(ValueError):
        B.spec_qk_norm_rope(z(4, 32, 128), z(4, 8, 128), None, None, i(1), i(2), z(4, 32, 128), z(4, 8, 128), None,
                            q_weight=z(128, dt=torch.float32))
