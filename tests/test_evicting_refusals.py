"""Refusals of the weight sums' and the evicting cache's calls (no GPU needed): every bad
argument is answered on the host, before any launch, with its status and a text."""
import ctypes

import numpy as np
import pytest
import torch

from tile_routed_mixed_causal_b200 import _lib as L
from tile_routed_mixed_causal_b200 import api
from tile_routed_mixed_causal_b200 import build as tra_build

OK, INVALID, UNSUPPORTED, BUFFER = 0, 1, 2, 3
PTR = 1 << 20       # aligned stand-in for a device address; never used
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    tra_build.build()
    return L.load()


def _shape(lengths=(130, 64), Hq=8, Hkv=2, d=128):
    cu = np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)
    return L.Shape(cu, Hq, Hkv, d, device=None)


def _cache(**kw):
    f = dict(B=2, Hq=8, Hkv=2, d=128, cap=6, n_pool=24)
    f |= {n: PTR for n in L.PagedCache.NAMES}
    return L._PagedCache(**(f | kw))


# ------------------------------------------------------------------------ weight sums
def _sums(lib, shape=None, **kw):
    shape = shape or _shape()
    a = dict(q=PTR, k=PTR, n=0, scale=0.1, lse=PTR, given=0, w=PTR, status=PTR) | kw
    return lib.attention_weight_sums(shape.c, a["q"], a["k"], a["n"], a["scale"], a["lse"], a["given"], a["w"],
                                     a["status"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(lse=None), INVALID), (dict(w=None), INVALID),
    (dict(status=None), INVALID), (dict(q=PTR + 2), INVALID), (dict(k=PTR + 8), INVALID),
    (dict(lse=PTR + 4), INVALID), (dict(w=PTR + 4), INVALID), (dict(n=-1), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
])
def test_weight_sums_refusals(lib, kw, code):
    assert _sums(lib, **kw) == code
    assert lib.tra_last_error()


@pytest.mark.parametrize("shape,code", [
    (dict(Hq=6, Hkv=4), INVALID), (dict(d=96), UNSUPPORTED), (dict(lengths=(64, -1)), INVALID),
])
def test_weight_sums_shapes(lib, shape, code):
    assert _sums(lib, _shape(**shape)) == code


def test_weight_sums_of_nothing(lib):
    assert _sums(lib, _shape(lengths=(0, 0))) == OK     # nothing to launch


# ------------------------------------------------------------------------ cache
BAD_CACHES = [
    (dict(B=0), INVALID), (dict(Hq=0), INVALID), (dict(Hkv=0), INVALID), (dict(Hkv=3), INVALID),
    (dict(Hq=18, Hkv=2), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(cap=0), INVALID), (dict(n_pool=0), INVALID),
    (dict(cap=1 << 24), UNSUPPORTED), (dict(n_pool=1 << 25), UNSUPPORTED), (dict(B=65536), UNSUPPORTED),
    (dict(Hq=264, Hkv=264), UNSUPPORTED),
]
BAD_POINTERS = [(dict([(n, None)]), INVALID) for n in L.PagedCache.NAMES] + \
               [(dict([(n, PTR + 8)]), INVALID) for n in L.PagedCache.NAMES]


def _calls(lib, cache, ws=PTR, nws=BIG, status=PTR):
    c = ctypes.byref(cache)
    shape = _shape()
    yield lib.paged_cache_fill(c, shape.c, PTR, PTR, PTR, 2, 0, ws, nws, status, None)
    yield lib.paged_attention_decode(c, PTR, PTR, PTR, 0.1, PTR, None, None, ws, nws, status, None)
    yield lib.paged_cache_evict(c, 2, 0, None, None, None, None, ws, nws, status, None)


@pytest.mark.parametrize("kw,code", BAD_CACHES + BAD_POINTERS, ids=str)
def test_bad_caches(lib, kw, code):
    for status in _calls(lib, _cache(**kw)):
        assert status == code
        assert lib.tra_last_error()


@pytest.mark.parametrize("kw,code", BAD_CACHES, ids=str)
def test_bad_caches_have_no_workspace(lib, kw, code):
    assert lib.tra_paged_workspace_bytes(ctypes.byref(_cache(**kw))) == 0


def test_workspace(lib):
    need = lib.tra_paged_workspace_bytes(ctypes.byref(_cache()))
    assert need > 0
    assert lib.tra_paged_workspace_bytes(ctypes.byref(_cache(cap=60, n_pool=240))) > need
    # sizes that pass 32 bits
    assert lib.tra_paged_workspace_bytes(ctypes.byref(_cache(B=64, Hq=64, Hkv=8, cap=4096))) > 1 << 32
    for kw, code in ((dict(ws=None), INVALID), (dict(ws=PTR + 8), INVALID), (dict(status=None), INVALID),
                     (dict(nws=need - 1), BUFFER), (dict(nws=0), BUFFER)):
        for status in _calls(lib, _cache(), **kw):
            assert status == code


def test_null_cache(lib):
    assert lib.tra_paged_workspace_bytes(None) == 0
    assert lib.paged_cache_evict(None, 2, 0, None, None, None, None, PTR, BIG, PTR, None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(k=PTR + 8), INVALID), (dict(v=PTR + 2), INVALID),
    (dict(w=PTR + 2), INVALID), (dict(keep=0), INVALID), (dict(keep=7), INVALID), (dict(recent=-1), INVALID),
    (dict(shape=dict(Hq=16)), INVALID), (dict(shape=dict(Hkv=4)), INVALID), (dict(shape=dict(d=64)), INVALID),
    (dict(shape=dict(lengths=(64,))), INVALID),
])
def test_fill_refusals(lib, kw, code):
    a = dict(shape={}, k=PTR, v=PTR, w=None, keep=2, recent=0) | kw
    s = _shape(**a["shape"])
    assert lib.paged_cache_fill(ctypes.byref(_cache()), s.c, a["k"], a["v"], a["w"], a["keep"], a["recent"], PTR, BIG,
                                PTR, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
    (dict(q=PTR + 8), INVALID), (dict(k=PTR + 4), INVALID), (dict(v=PTR + 2), INVALID), (dict(out=PTR + 8), INVALID),
    (dict(so=PTR + 4), INVALID), (dict(wo=PTR + 4), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=float("nan")), INVALID),
])
def test_decode_refusals(lib, kw, code):
    a = dict(q=PTR, k=PTR, v=PTR, out=PTR, so=None, wo=None, scale=0.1) | kw
    assert lib.paged_attention_decode(ctypes.byref(_cache()), a["q"], a["k"], a["v"], a["scale"], a["out"], a["so"],
                                      a["wo"], PTR, BIG, PTR, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(keep=0), INVALID), (dict(keep=7), INVALID), (dict(recent=-1), INVALID), (dict(so=PTR + 4096), INVALID),
    (dict(to=PTR + 4096), INVALID), (dict(so=PTR + 4096, to=PTR + 4096, wo=PTR + 4096), INVALID),
    (dict(so=PTR + 4096, to=PTR + 4096, wo=PTR + 4096, po=PTR), INVALID),   # pos in place, the others not
    (dict(so=PTR + 4, to=PTR + 4096, wo=PTR + 4096, po=PTR + 4096), INVALID),
])
def test_evict_refusals(lib, kw, code):
    a = dict(keep=2, recent=0, so=None, to=None, wo=None, po=None) | kw
    assert lib.paged_cache_evict(ctypes.byref(_cache()), a["keep"], a["recent"], a["so"], a["to"], a["wo"], a["po"], PTR,
                                 BIG, PTR, None) == code


# ------------------------------------------------------------------------ Python side
def test_tensors_have_to_be_on_a_gpu():
    s = _shape(lengths=(64,))
    q, k = torch.zeros(64, 8, 128, dtype=torch.bfloat16), torch.zeros(64, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(L.TraError):
        L.attention_weight_sums(s, q, k, torch.zeros(64, 2), torch.zeros(8, 64), softmax_scale=0.1)
    with pytest.raises(L.TraError):
        api.prompt_importance(s, q, k)


def test_cache_arrays_are_checked(lib):
    c = L.PagedCache(1, 4, 2, 64, 3, device="cpu")     # allocation and checks need no GPU
    assert c.n_pool == 6 and int(c["state"][0, 0]) == -1
    assert sorted(c["table"].flatten().tolist()) == list(range(6))
    for n in L.PagedCache.NAMES:
        bad = dict(c.t)
        bad[n] = bad[n].double()
        with pytest.raises(L.TraError, match=n):
            L.PagedCache(1, 4, 2, 64, 3, tensors=bad)
        if n != "k8":       # (the number of pages is taken from k8)
            bad[n] = c.t[n][..., :-1]
            with pytest.raises(L.TraError, match=n):
                L.PagedCache(1, 4, 2, 64, 3, tensors=bad)
    with pytest.raises(L.TraError):
        L.PagedCache(1, 18, 2, 64, 3, device="cpu")    # nine query heads per KV head
    with pytest.raises(L.TraError):
        L.PagedCache(0, 4, 2, 64, 3, device="cpu")
    with pytest.raises(L.TraError):
        L.paged_cache_evict(c, keep=1)                 # not on a GPU


@pytest.mark.parametrize("keep,limit", [(0, 4), (4, 4), (5, 4)])
def test_plan_sizes(keep, limit):
    with pytest.raises(ValueError):
        api.EvictingDecodePlan(_shape(), keep, limit, device="cpu")


def test_plan_needs_a_prompt_first(lib):
    plan = api.EvictingDecodePlan(_shape(), 2, 4, device="cpu")
    with pytest.raises(RuntimeError, match="prefill"):
        plan.step(None, None, None, None)
